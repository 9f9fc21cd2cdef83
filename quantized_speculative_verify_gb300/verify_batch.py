"""One attention layer of the verify pass for a batch of requests.

    python -m quantized_speculative_verify_gb300.verify_batch [--requests 8] [--shared 4096] [--steps 5]

Requests that start with the same long prompt are forks of one sequence of a
paged cache: its pages are held once, and the attention reads them once for all
requests.  Each request verifies a draft tree of its own and uses a low-rank
adapter of its own beside the shared quantized projections.  A step is

    pages_extend        room for every request's tree (shared last pages are copied)
    add_norm_quant      residual + RMS norm + rotation + int8, the operand of q, k, v
    hq_verify_gemm      the fused q, k, v projection of all requests' rows
    lora_apply          each request's adapter, added in place to q, k and v
    pages_write         the trees' keys and values into the pages
    prefix_attention    all trees over the shared prefix and their own positions
    hq_rotate_quant_act, hq_verify_gemm, lora_apply   the o projection
    pages_compact       (after acceptance) the accepted path, the rest given up

Everything runs on the current stream without a host synchronization, so a step
can be captured in a CUDA graph.  Weights and activations here are synthetic.
"""
from __future__ import annotations

import argparse
import math

import torch

from . import hq, synth


class BatchLayer:
    """A layer's packed projections, norm weight and adapters, with the buffers
    for up to `rows` tree nodes (at most HQ_MAX_M) of a batch."""

    def __init__(self, hidden: int, heads: int, kv_heads: int, dim: int, rows: int, adapters: int, rank: int, seed: int = 0,
                 group: int = 64, fmt: str = "w4", device="cuda"):
        self.hidden, self.heads, self.kv_heads, self.dim, self.rows = hidden, heads, kv_heads, dim, rows
        q, kv = heads * dim, kv_heads * dim
        signs = hq.hq_make_signs(seed, hidden), hq.hq_make_signs(seed + 1, q)

        def w(n, k, i):
            return synth.weights(n, k, seed=seed * 100 + i, device=device)
        self.qkv = hq.pack_fused([w(q, hidden, 0), w(kv, hidden, 1), w(kv, hidden, 2)], group, fmt, signs[0])
        self.o = hq.pack_layer(w(hidden, q, 3), group, fmt, signs[1])
        g = torch.Generator(device=device).manual_seed(seed)
        self.norm = 1.0 + 0.1 * torch.randn(hidden, generator=g, device=device)

        def adapter(k, n):
            a = torch.randn((adapters, rank, k), generator=g, device=device) / math.sqrt(k)
            b = torch.randn((adapters, n, rank), generator=g, device=device) / math.sqrt(rank)
            return a.half(), (0.02 * b).half()
        self.adapters = {"q": adapter(hidden, q), "k": adapter(hidden, kv), "v": adapter(hidden, kv), "o": adapter(q, hidden)}
        self.scale = torch.ones(adapters, device=device)
        self.Y = torch.empty((rows, q + 2 * kv), device=device)
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
        q, k, v = self.qkv.split(Y)
        for part, y in (("q", q), ("k", k), ("v", v)):
            A, B = self.adapters[part]
            hq.lora_apply(h, A, B, ids, None, self.scale, base=y, Y=y, workspace=self.ws_lora)
        heads = (self.kv_heads, self.dim)
        hq.pages_write(cache, planes[0], planes[1], k.unflatten(1, heads), v.unflatten(1, heads), starts, max_rows, seqs=seqs)
        q16, att = self.q16[:M], self.att[:M]
        q16.copy_(q.unflatten(1, (self.heads, self.dim)))
        hq.prefix_attention(cache, planes[0], planes[1], q16, starts, max_rows, shared, max_len, 1.0 / math.sqrt(self.dim),
                            parent=parent, seqs=seqs, out=att, workspace=self.ws_attn)
        flat = att.view(M, self.heads * self.dim)
        _, _, qop, sx = hq.act_buffers(self.o.desc, M, x.device, int8_codes=False)
        hq.hq_rotate_quant_act(self.o.desc, flat, M, self.o.signs, None, None, qop, sx)
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


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--nodes", type=int, default=16, help="tree nodes per request; requests x nodes at most 128")
    p.add_argument("--shared", type=int, default=4096, help="positions of the shared prompt")
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args()
    B, m, cfg = a.requests, a.nodes, synth.DECODER_9B
    if B * m > hq.HQ_MAX_M:
        p.error(f"requests x nodes must be at most {hq.HQ_MAX_M}")
    dev, D, M = "cuda", hq.HQ_ATTN_HEAD_DIM, B * m
    heads, kv_heads, ps = cfg["hidden"] // D, cfg["kv"] // D, 64
    layer = BatchLayer(cfg["hidden"], heads, kv_heads, D, M, adapters=B, rank=16)
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
    x, residual = torch.randn((M, cfg["hidden"]), device=dev), torch.randn((M, cfg["hidden"]), device=dev).bfloat16()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(a.steps):
        base = cache.lens[1:].clone()  # each tree's root goes here
        begin.record()
        layer.step(cache, (0, 1), x, residual, seqs, starts, add, parent, ids, m, a.shared, a.shared + (a.steps + 1) * m)
        end.record()
        # stands in for hq_tree_accept: the root, nodes 1 and 2 of every tree
        hq.pages_compact(cache, seqs, base, ints([1, 2]).repeat(B, 1), ints([2] * B))
        torch.cuda.synchronize()
        print(f"step {step}: {M} rows, lengths {cache.lens[1:].tolist()}, {int((cache.ref > 0).sum())} pages held, "
              f"{begin.elapsed_time(end) * 1e3:.0f} us")
    if hq.pages_status(cache) != hq.HQ_OK or hq.hq_workspace_status(layer.ws_attn) != hq.HQ_OK:
        raise SystemExit("a page operation or the attention reported an error")


if __name__ == "__main__":
    main()
