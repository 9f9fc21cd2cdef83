"""One attention layer of the verify pass for a batch of requests.

    python -m quantized_speculative_verify_gb300.verify_batch [--requests 8] [--shared 4096] [--steps 5]

Requests that start with the same long prompt are forks of one sequence of a
paged cache: its pages are held once, and the attention reads them once for all
requests.  Each request verifies a draft tree of its own and uses a low-rank
adapter of its own beside the shared quantized projections.  A step is

    pages_extend        room for every request's tree (shared last pages are copied)
    add_norm_quant      residual + RMS norm + rotation + int8, the operand of q, k, v
    hq_verify_gemm      the fused q, k, v (and gate) projection of all requests' rows
    lora_apply          each request's adapter, added in place to q, k and v
    rope_write          q and k rotated by their positions, k and v into the pages
    prefix_attention    all trees over the shared prefix and their own positions
    gated_norm_quant    the attention's output gate, rotation and int8
    hq_verify_gemm, lora_apply   the o projection
    greedy_tokens       each request's rules on its rows' logits, and their greedy tokens
    tree_accept_batch   the accepted paths; the requests' histories grow by them
    pages_compact       the accepted paths' keys and values, the rest given up

(without rotary positions pages_write takes the place of rope_write, without a
gate hq_rotate_quant_act that of gated_norm_quant).  Everything runs on the
current stream without a host synchronization, so a step can be captured in a
CUDA graph.  Weights and activations here are synthetic.
"""
from __future__ import annotations

import argparse
import math

import torch

from . import hq, synth


class BatchLayer:
    """A layer's packed projections, norm weight and adapters, with the buffers
    for up to `rows` tree nodes (at most HQ_MAX_M) of a batch.  freqs: radians a
    position of the heads' pairs (rope_freqs), None: no rotary positions; layout,
    gain, q_norm and k_norm (fp32 [dim], with eps), as rope_write takes them, go
    with them (frequencies of kind "yarn" with a gain of 0.1 ln(factor) + 1); gate:
    the attention's output is gated by the sigmoid of a projection of its own."""

    def __init__(self, hidden: int, heads: int, kv_heads: int, dim: int, rows: int, adapters: int, rank: int, seed: int = 0,
                 group: int = 64, fmt: str = "w4", device="cuda", freqs=None, gate: bool = False, layout: str = "half",
                 gain: float = 1.0, q_norm=None, k_norm=None, eps: float = 1e-6):
        if freqs is None and (gain != 1.0 or q_norm is not None or k_norm is not None):
            raise ValueError("BatchLayer: gain, q_norm and k_norm go with the rotary positions (freqs)")
        self.hidden, self.heads, self.kv_heads, self.dim, self.rows = hidden, heads, kv_heads, dim, rows
        q, kv = heads * dim, kv_heads * dim
        signs = hq.hq_make_signs(seed, hidden), hq.hq_make_signs(seed + 1, q)

        def w(n, k, i):
            return synth.weights(n, k, seed=seed * 100 + i, device=device)
        parts = [w(q, hidden, 0), w(kv, hidden, 1), w(kv, hidden, 2)] + ([w(q, hidden, 4)] if gate else [])
        self.qkv = hq.pack_fused(parts, group, fmt, signs[0])
        self.o = hq.pack_layer(w(hidden, q, 3), group, fmt, signs[1])
        g = torch.Generator(device=device).manual_seed(seed)
        self.norm = 1.0 + 0.1 * torch.randn(hidden, generator=g, device=device)

        def adapter(k, n):
            a = torch.randn((adapters, rank, k), generator=g, device=device) / math.sqrt(k)
            b = torch.randn((adapters, n, rank), generator=g, device=device) / math.sqrt(rank)
            return a.half(), (0.02 * b).half()
        self.adapters = {"q": adapter(hidden, q), "k": adapter(hidden, kv), "v": adapter(hidden, kv), "o": adapter(q, hidden)}
        self.scale = torch.ones(adapters, device=device)
        self.turns = None if freqs is None else hq.rope_turns(freqs, device)
        self.rope = dict(layout=layout, gain=gain, q_weight=q_norm, k_weight=k_norm, eps=eps)
        self.gated = torch.empty((rows, q), dtype=torch.float16, device=device) if gate else None
        self.Y = torch.empty((rows, self.qkv.layer.N), device=device)
        self.out = torch.empty((rows, hidden), device=device)
        self.h = torch.empty((rows, hidden), dtype=torch.float16, device=device)
        self.q16 = torch.empty((rows, heads, dim), dtype=torch.float16, device=device)
        self.att = torch.empty((rows, heads, dim), device=device)
        self.ws_gemm = torch.zeros(max(hq.hq_workspace_bytes(l.desc, rows) for l in (self.qkv.layer, self.o)),
                                   dtype=torch.uint8, device=device)
        self.ws_lora = torch.empty(hq.hq_lora_workspace_bytes(rows, rank), dtype=torch.uint8, device=device)
        self.ws_attn = torch.zeros(hq.hq_prefix_attention_workspace_bytes(1, rows, rows, heads, kv_heads, dim),
                                   dtype=torch.uint8, device=device)

    def step(self, cache: hq.PagedCache, planes, x, residual, seqs, starts, add, parent, ids, max_rows: int, shared: int,
             max_len: int, flags: int = hq.HQ_LAUNCH_DEFAULT) -> torch.Tensor:
        """The layer's output [rows][hidden] (the next x) for the trees whose
        rows are starts[b] .. starts[b + 1]; residual is updated in place, the
        cache's sequences grow by add.  ids: each row's adapter (-1: none)."""
        M = x.shape[0]
        layer = self.qkv.layer
        hq.pages_extend(cache, seqs, add)
        _, _, qop, sx = hq.act_buffers(layer.desc, M, x.device, int8_codes=False)
        h, Y, out = self.h[:M], self.Y[:M], self.out[:M]
        hq.add_norm_quant(layer.desc, x, residual, self.norm, layer.signs, 1e-5, residual_out=residual, h=h, qop=qop, sx=sx)
        hq.hq_verify_gemm(layer.desc, layer.blob, qop, sx, M, Y, None, self.ws_gemm, flags)
        q, k, v = self.qkv.split(Y)[:3]
        for part, y in (("q", q), ("k", k), ("v", v)):
            A, B = self.adapters[part]
            hq.lora_apply(h, A, B, ids, None, self.scale, base=y, Y=y, workspace=self.ws_lora)
        q, k, v = (t.unflatten(1, (-1, self.dim)) for t in (q, k, v))
        q16, att = self.q16[:M], self.att[:M]
        if self.turns is None:
            hq.pages_write(cache, planes[0], planes[1], k, v, starts, max_rows, seqs=seqs)
            q16.copy_(q)
        else:
            hq.rope_write(cache, planes[0], planes[1], q, k, v, self.turns, starts, max_rows, parent=parent, seqs=seqs, out=q16,
                          **self.rope)
        hq.prefix_attention(cache, planes[0], planes[1], q16, starts, max_rows, shared, max_len, 1.0 / math.sqrt(self.dim),
                            parent=parent, seqs=seqs, out=att, workspace=self.ws_attn)
        flat = att.view(M, self.heads * self.dim)
        _, _, qop, sx = hq.act_buffers(self.o.desc, M, x.device, int8_codes=False)
        if self.gated is None:
            hq.hq_rotate_quant_act(self.o.desc, flat, M, self.o.signs, None, None, qop, sx)
        else:
            gated = self.gated[:M]
            hq.gated_norm_quant(self.o.desc, flat, self.qkv.split(Y)[3], None, self.o.signs, self.dim, "sigmoid", h=gated, qop=qop,
                                sx=sx)
            flat = gated
        hq.hq_verify_gemm(self.o.desc, self.o.blob, qop, sx, M, out, None, self.ws_gemm, flags)
        A, B = self.adapters["o"]
        hq.lora_apply(flat, A, B, ids, None, self.scale, base=out, Y=out, workspace=self.ws_lora)
        return out


def prefill(cache: hq.PagedCache, planes, slot: int, n: int, seed: int) -> None:
    """Fills sequence `slot` with n synthetic positions (a prompt's keys and values)."""
    dev = cache.pool.device
    seqs, add = (torch.tensor([i], dtype=torch.int32, device=dev) for i in (slot, n))
    hq.pages_extend(cache, seqs, add)
    g = torch.Generator(device=dev).manual_seed(seed)
    kv = torch.randn((2, n, cache.heads, cache.dim), generator=g, device=dev)
    hq.pages_write(cache, planes[0], planes[1], kv[0], kv[1], None, n, seqs=seqs)


class Head:
    """The final norm, the LM head and the requests' rules on its logits, for up
    to `rows` tree nodes of a batch."""

    def __init__(self, hidden: int, vocab: int, rows: int, requests: int, cap: int, seed: int = 0, group: int = 64, fmt: str = "w4",
                 device="cuda"):
        self.layer = hq.pack_layer(synth.weights(vocab, hidden, seed=seed * 100 + 9, device=device), group, fmt,
                                   hq.hq_make_signs(seed + 2, hidden))
        self.norm = torch.ones(hidden, device=device)
        self.logits = torch.empty((rows, vocab), device=device)
        self.ws_gemm = torch.zeros(hq.hq_workspace_bytes(self.layer.desc, rows), dtype=torch.uint8, device=device)
        self.ws_greedy = torch.zeros(hq.hq_greedy_tokens_workspace_bytes(rows), dtype=torch.uint8, device=device)
        ints = dict(dtype=torch.int32, device=device)
        self.history = hq.History(torch.zeros((requests, cap), **ints), torch.zeros(requests, **ints))
        self.rules = hq.LogitRules(requests, *(torch.full((requests,), p, device=device) for p in (1.1, 0.2, 0.1)))

    def accept(self, x, residual, starts, parent, tokens, max_rows: int, flags: int = hq.HQ_LAUNCH_DEFAULT):
        """The accepted path, their number and the bonus token of each request's
        tree (request b's history is slot b), which its history grows by."""
        M, layer = x.shape[0], self.layer
        _, _, qop, sx = hq.act_buffers(layer.desc, M, x.device, int8_codes=False)
        logits = self.logits[:M]
        hq.add_norm_quant(layer.desc, x, residual, self.norm, layer.signs, 1e-5, residual_out=residual, qop=qop, sx=sx)
        hq.hq_verify_gemm(layer.desc, layer.blob, qop, sx, M, logits, None, self.ws_gemm, flags)
        greedy = hq.greedy_tokens(logits, starts, max_rows, parent, tokens, history=self.history, rules=self.rules,
                                  workspace=self.ws_greedy)
        return hq.tree_accept_batch(greedy, parent, tokens, starts, max_rows, history=self.history)


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--nodes", type=int, default=16, help="tree nodes per request; requests x nodes at most 128")
    p.add_argument("--shared", type=int, default=4096, help="positions of the shared prompt")
    p.add_argument("--steps", type=int, default=5)
    p.add_argument("--vocab", type=int, default=32000)
    a = p.parse_args()
    B, m, cfg = a.requests, a.nodes, synth.DECODER_9B
    if B * m > hq.HQ_MAX_M:
        p.error(f"requests x nodes must be at most {hq.HQ_MAX_M}")
    dev, D, M = "cuda", hq.HQ_ATTN_HEAD_DIM, B * m
    heads, kv_heads, ps = cfg["hidden"] // D, cfg["kv"] // D, 64
    factor = 4.0
    freqs, gain = hq.rope_freqs(D, kind="yarn", factor=factor, original=8192), 0.1 * math.log(factor) + 1.0
    layer = BatchLayer(cfg["hidden"], heads, kv_heads, D, M, adapters=B, rank=16, freqs=freqs, gain=gain, gate=True)
    head = Head(cfg["hidden"], a.vocab, M, B, (a.steps + 1) * m)
    max_pages = -(-(a.shared + (a.steps + 1) * m) // ps)
    cache = hq.PagedCache.empty(2, max_pages + B * (a.steps * m // ps + 3), kv_heads, ps, D, B + 1, max_pages)
    prefill(cache, (0, 1), 0, a.shared, seed=1)

    def ints(v):
        return torch.tensor(list(v), dtype=torch.int32, device=dev)
    seqs = ints(range(1, B + 1))
    hq.pages_fork(cache, ints([0] * B), seqs)
    starts, add, ids = ints(range(0, M + 1, m)), ints([m] * B), ints([b for b in range(B) for _ in range(m)])
    g = torch.Generator().manual_seed(3)
    parent = ints([0 if i == 0 else max(0, i - 1 - int(torch.randint(0, 3, (1,), generator=g))) for _ in range(B) for i in range(m)])
    tokens = torch.randint(0, a.vocab, (M,), generator=g).to(dev, torch.int32)
    # each tree's root is its request's newest token, the last of its history
    head.history.tokens[:, 0] = tokens[::m]
    head.history.lens.fill_(1)
    x, residual = torch.randn((M, cfg["hidden"]), device=dev), torch.randn((M, cfg["hidden"]), device=dev).bfloat16()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(a.steps):
        base = cache.lens[1:].clone()  # each tree's root goes here
        begin.record()
        out = layer.step(cache, (0, 1), x, residual, seqs, starts, add, parent, ids, m, a.shared, a.shared + (a.steps + 1) * m)
        path, n, bonus = head.accept(out, residual, starts, parent, tokens, m)
        hq.pages_compact(cache, seqs, base, path, n)
        end.record()
        # the next trees, drafted from what the model said of these
        tokens = torch.where(torch.rand(M, device=dev) < 0.5, bonus.repeat_interleave(m), tokens)
        tokens[::m] = bonus
        torch.cuda.synchronize()
        print(f"step {step}: {M} rows, lengths {cache.lens[1:].tolist()}, {int((cache.ref > 0).sum())} pages held, "
              f"{begin.elapsed_time(end) * 1e3:.0f} us")
    print("said:", head.history.tokens[0, :int(head.history.lens[0])].tolist())
    if hq.pages_status(cache) != hq.HQ_OK or hq.hq_workspace_status(layer.ws_attn) != hq.HQ_OK or \
            hq.history_status(head.history) != hq.HQ_OK:
        raise SystemExit("a page operation, the attention or the acceptance reported an error")


if __name__ == "__main__":
    main()
