"""The calls between a batch's layers together, as a server runs them: a layer
with rotary positions and an output gate, the LM head, rules on the logits,
acceptance, and the cache cut back to the accepted path, step after step.

Tolerances.  A batch against its requests alone: as in the test of the layer
without these calls (the same kernels see the same rows; the attention's cut and
codes at rounding borders differ), 2^-7 of the output's norm.  Keys in the cache:
the rotary bound of the rows that were projected.
"""
import numpy as np
import pytest
import torch

from quantized_speculative_verify_gb300 import hq, verify_batch
from quantized_speculative_verify_gb300.verify_batch import BatchLayer, Head, prefill
from test_gpu_gate import check as check_codes
from test_gpu_gate import value
from test_gpu_greedy import accept
from test_gpu_rope import close, expected

pytestmark = pytest.mark.gpu
DEV = "cuda"
HIDDEN, HEADS, KV, D, PS, V = 512, 8, 2, 64, 16, 700


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def fresh(seqs, shared):
    cache = hq.PagedCache.empty(2, 200, KV, PS, D, seqs, 40)
    prefill(cache, (0, 1), 0, shared, seed=5)
    hq.pages_fork(cache, ints([0] * (seqs - 1)), ints(range(1, seqs)))
    return cache


def make(M, requests):
    freqs = hq.rope_freqs(48, kind="bands", factor=4.0, original=100.0)
    return (BatchLayer(HIDDEN, HEADS, KV, D, M, adapters=3, rank=8, seed=2, freqs=freqs, gate=True),
            Head(HIDDEN, V, M, requests, 60, seed=3))


@pytest.mark.parametrize("shared", [100, 530])
def test_steps_of_a_batch_give_each_request_what_it_gets_alone(shared):
    rows, flags = [5, 1, 9], hq.HQ_LAUNCH_DETERMINISTIC
    B, M = len(rows), sum(rows)
    starts, parent = [0, 5, 6, 15], [0, 0, 0, 1, 2, 0, 0, 0, 1, 1, 3, 0, 5, 5, 2]
    ids = [2] * 5 + [-1] + [0] * 9
    layer, head = make(M, B)
    cache = fresh(B + 1, shared)
    alone = [(make(M, 1), fresh(2, shared)) for _ in range(B)]
    g = torch.Generator(device=DEV).manual_seed(1)
    accepted = 0
    for _ in range(3):
        x = torch.randn((M, HIDDEN), generator=g, device=DEV)
        res = torch.randn((M, HIDDEN), generator=g, device=DEV).bfloat16()
        base, r_all = cache.lens[1:].clone(), res.clone()
        out = layer.step(cache, (0, 1), x, r_all, ints([1, 2, 3]), ints(starts), ints(rows), ints(parent), ints(ids), 9, shared, 600,
                         flags).clone()
        # what the model says after each node, without drafts: the drafts of half the nodes are that
        said = hq.greedy_tokens(logits_of(head, out, r_all.clone(), flags), ints(starts), 9, ints(parent)).tolist()
        tokens = [said[starts[b] + parent[starts[b] + i]] if i % 3 else 7 * i for b, m in enumerate(rows) for i in range(m)]
        before = head.history.lens.tolist()
        path, n, bonus = head.accept(out, r_all, ints(starts), ints(parent), ints(tokens), 9, flags)
        # the keys of every node hold the position of its depth
        q, k, v = (t.unflatten(1, (-1, D)) for t in layer.qkv.split(layer.Y[:M])[:3])
        turns = layer.turns.cpu().numpy().view(np.uint64).tolist()
        for b, m in enumerate(rows):
            lo, depth = starts[b], [0] * m
            for i in range(1, m):
                depth[i] = depth[parent[lo + i]] + 1
            at = [int(base[b]) + i for i in range(m)]
            page = [int(cache.table[b + 1, p // PS]) for p in at]
            want, lim = expected(k[lo:lo + m], [int(base[b]) + d for d in depth], turns, "half", 1.0, None, 0.0)
            close(cache.pool[0, page, :, [p % PS for p in at]], want, lim)
        hq.pages_compact(cache, ints([1, 2, 3]), base, path, n)
        # accepted keys moved to the places of their positions
        for b, m in enumerate(rows):
            lo, p = starts[b], path[b, :int(n[b])].tolist()
            accepted += len(p)
            at = [int(base[b])] + [int(base[b]) + 1 + d for d in range(len(p))]
            assert int(cache.lens[b + 1]) == at[-1] + 1
            page = [int(cache.table[b + 1, a // PS]) for a in at]
            want, lim = expected(k[[lo] + [lo + i for i in p]], at, turns, "half", 1.0, None, 0.0)
            close(cache.pool[0, page, :, [a % PS for a in at]], want, lim)
        assert head.history.lens.tolist() == [h + int(a) + 1 for h, a in zip(before, n)]
        for b in range(B):
            lo, hi = starts[b], starts[b + 1]
            (one_layer, one_head), c = alone[b]
            r_one, root = res[lo:hi].clone(), c.lens[1:].clone()
            one = one_layer.step(c, (0, 1), x[lo:hi].contiguous(), r_one, ints([1]), ints([0, hi - lo]), ints([hi - lo]),
                                 ints(parent[lo:hi]), ints(ids[lo:hi]), hi - lo, shared, 600, flags)
            assert float((one - out[lo:hi]).norm()) <= 2.0 ** -7 * float(out[lo:hi].norm())
            # acceptance of the batch's own outputs, so that codes at rounding borders decide nothing
            p1, n1, b1 = one_head.accept(out[lo:hi].contiguous(), r_one, ints([0, hi - lo]), ints(parent[lo:hi]), ints(tokens[lo:hi]),
                                         hi - lo, flags)
            hq.pages_compact(c, ints([1]), root, path[b:b + 1, :hi - lo].contiguous(), n[b:b + 1])
            assert int(n1[0]) == int(n[b]) and int(b1[0]) == int(bonus[b]) and p1[0].tolist() == path[b, :hi - lo].tolist()
            assert torch.equal(one_head.history.tokens[0], head.history.tokens[b])
            assert int(c.lens[1]) == int(cache.lens[b + 1])
    assert accepted > 0
    for c in [cache] + [c for _, c in alone]:
        assert hq.pages_status(c) == hq.HQ_OK
    assert hq.history_status(head.history) == hq.HQ_OK and hq.hq_workspace_status(layer.ws_attn) == hq.HQ_OK


def logits_of(head, x, residual, flags):
    M, layer = x.shape[0], head.layer
    _, _, qop, sx = hq.act_buffers(layer.desc, M, x.device, int8_codes=False)
    hq.add_norm_quant(layer.desc, x, residual, head.norm, layer.signs, 1e-5, residual_out=residual, qop=qop, sx=sx)
    logits = torch.empty((M, V), device=DEV)
    hq.hq_verify_gemm(layer.desc, layer.blob, qop, sx, M, logits, None, head.ws_gemm, flags)
    return logits


def test_a_step_replayed_from_a_graph_goes_on_like_eager_steps():
    """The whole step is captured once: lengths, histories and paths are read on the device."""
    rows, M = [4, 6], 10
    starts, parent, add = ints([0, 4, 10]), ints([0, 0, 1, 1, 0, 0, 1, 2, 3, 0]), ints(rows)
    g = torch.Generator(device=DEV).manual_seed(4)
    x, res = torch.randn((M, HIDDEN), generator=g, device=DEV), torch.randn((M, HIDDEN), generator=g, device=DEV).bfloat16()
    tokens = torch.randint(0, V, (M,), generator=g, device=DEV).to(torch.int32)
    seen = []
    for captured in (False, True):
        layer, head = make(M, 2)
        cache, r, base = fresh(3, 70), res.clone(), torch.zeros(2, dtype=torch.int32, device=DEV)
        ids, seqs = ints([0] * M), ints([1, 2])

        def step():
            base.copy_(cache.lens[1:])
            out = layer.step(cache, (0, 1), x, r, seqs, starts, add, parent, ids, 6, 70, 600, hq.HQ_LAUNCH_DETERMINISTIC)
            path, n, _ = head.accept(out, r, starts, parent, tokens, 6, hq.HQ_LAUNCH_DETERMINISTIC)
            hq.pages_compact(cache, seqs, base, path, n)
        if captured:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step()
            torch.cuda.current_stream().wait_stream(s)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for _ in range(3):
                graph.replay()
        else:
            for _ in range(4):
                step()
        torch.cuda.synchronize()
        assert hq.pages_status(cache) == hq.HQ_OK and hq.history_status(head.history) == hq.HQ_OK
        used = [cache.pool[:, cache.table[b, :-(-int(cache.lens[b]) // PS)].long()].transpose(2, 3).reshape(2, -1, KV, D)[:, :int(cache.lens[b])]
                for b in (1, 2)]
        seen.append((cache.lens.tolist(), head.history.tokens.tolist(), head.history.lens.tolist(), used, r.clone()))
    assert seen[0][:3] == seen[1][:3] and min(seen[0][2]) >= 4
    assert all(torch.equal(a, b) for a, b in zip(seen[0][3], seen[1][3])) and torch.equal(seen[0][4], seen[1][4])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_a_layer_rotates_as_its_model_does(layout):
    """Gain, layout and the weights of q's and k's norms reach the rotation: queries and keys are the formula's."""
    rows, shared, gain, eps = [5, 3], 90, 0.1 * np.log(4.0) + 1.0, 1e-5
    M, starts, parent = sum(rows), [0, 5, 8], [0, 0, 0, 1, 2, 0, 0, 1]
    g = torch.Generator(device=DEV).manual_seed(21)
    qw, kw = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    freqs = hq.rope_freqs(48, kind="yarn", factor=4.0, original=100.0)
    layer = BatchLayer(HIDDEN, HEADS, KV, D, M, adapters=3, rank=8, seed=2, freqs=freqs, gain=gain, layout=layout, q_norm=qw, k_norm=kw,
                       eps=eps, gate=True)
    cache = fresh(3, shared)
    x, r = torch.randn((M, HIDDEN), generator=g, device=DEV), torch.randn((M, HIDDEN), generator=g, device=DEV).bfloat16()
    layer.step(cache, (0, 1), x, r, ints([1, 2]), ints(starts), ints(rows), ints(parent), ints([0] * M), 5, shared, 200)
    q, k, _ = (t.unflatten(1, (-1, D)) for t in layer.qkv.split(layer.Y[:M])[:3])
    turns = layer.turns.cpu().numpy().view(np.uint64).tolist()
    gain, eps = float(np.float32(gain)), float(np.float32(eps))
    for b, m in enumerate(rows):
        lo, depth = starts[b], [0] * m
        for i in range(1, m):
            depth[i] = depth[parent[lo + i]] + 1
        pos = [shared + d for d in depth]
        close(layer.q16[lo:lo + m], *expected(q[lo:lo + m], pos, turns, layout, gain, qw, eps))
        at = [shared + i for i in range(m)]
        page = [int(cache.table[b + 1, p // PS]) for p in at]
        close(cache.pool[0, page, :, [p % PS for p in at]], *expected(k[lo:lo + m], pos, turns, layout, gain, kw, eps))
    assert hq.pages_status(cache) == hq.HQ_OK


def test_the_command_drafts_from_the_newest_tokens(monkeypatch):
    """Every tree's root is the last token of its request's history."""
    seen, greedy = [], hq.greedy_tokens

    def spy(logits, starts, max_rows, parent, tokens, **kw):
        h, roots = kw["history"], tokens[starts[:-1].long()]
        assert h.lens.tolist() == [max(1, n) for n in h.lens.tolist()]
        assert torch.equal(h.tokens.gather(1, h.lens.long().unsqueeze(1) - 1)[:, 0], roots)
        seen.append(roots.tolist())
        return greedy(logits, starts, max_rows, parent, tokens, **kw)
    monkeypatch.setattr(verify_batch.hq, "greedy_tokens", spy)
    monkeypatch.setattr(verify_batch.synth, "DECODER_9B", dict(verify_batch.synth.DECODER_9B, hidden=512, kv=256))
    monkeypatch.setattr("sys.argv", ["verify_batch", "--requests", "3", "--nodes", "5", "--shared", "100", "--steps", "3", "--vocab", "700"])
    verify_batch.main()
    assert len(seen) == 3 and seen[0] != seen[1]


def test_the_delta_rule_layer_behind_its_gate():
    """delta_tree, the gated norm per head, the output projection: the operand holds the codes of the formula."""
    M, H, DD = 16, 4, hq.HQ_DELTA_HEAD_DIM
    K = H * DD
    g = torch.Generator(device=DEV).manual_seed(6)
    state = 0.3 * torch.randn((H, DD, DD), generator=g, device=DEV)
    q, k, v = (torch.randn((M, H, DD), generator=g, device=DEV) for _ in range(3))
    k = k / k.norm(dim=2, keepdim=True)
    alpha, beta = torch.rand((M, H), generator=g, device=DEV), torch.rand((M, H), generator=g, device=DEV)
    parent = ints([max(0, i - 1 - i % 3) for i in range(M)])
    out = hq.delta_tree(state, q, k, v, alpha, beta, parent).view(M, K)
    gate, w = torch.randn((M, K), generator=g, device=DEV).bfloat16(), 1.0 + 0.2 * torch.randn(DD, generator=g, device=DEV)
    signs = hq.hq_make_signs(8, K)
    layer = hq.pack_layer(0.05 * torch.randn((256, K), generator=g, device=DEV), 64, "w4", signs)
    qx, _, qop, sx = hq.act_buffers(layer.desc, M, DEV)
    hq.gated_norm_quant(layer.desc, out, gate, w, layer.signs, DD, "silu", 1e-6, qx=qx, qop=qop, sx=sx)
    check_codes(value(out, gate, w, DD, "silu", 1e-6), signs, None, qx, sx)
    ws = torch.zeros(hq.hq_workspace_q8_bytes(layer.desc, M), dtype=torch.uint8, device=DEV)
    Y, Y8 = torch.empty((M, 256), device=DEV), torch.empty((M, 256), device=DEV)
    hq.hq_verify_gemm(layer.desc, layer.blob, qop, sx, M, Y, None, ws, hq.HQ_LAUNCH_EXACT_ORDER)
    hq.hq_verify_gemm_q8(layer.desc, layer.blob, qx, sx, None, M, Y8, None, ws, hq.HQ_LAUNCH_EXACT_ORDER)
    assert torch.equal(Y, Y8)


def test_greedy_tokens_feed_an_acceptance_that_agrees_with_the_formula():
    M, g = 12, torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn((M, V), generator=g, device=DEV)
    parent = [0, 0, 1, 1, 2, 4, 5, 0, 7, 8, 9, 10]
    greedy = hq.greedy_tokens(x, None, M, ints(parent))
    tokens = [0] + [int(greedy[parent[i]]) for i in range(1, M)]
    path, n, bonus = hq.tree_accept_batch(greedy, ints(parent), ints(tokens), None, M)
    want = accept(greedy.tolist(), parent, tokens)
    assert path[0, :want[1]].tolist() == want[0] and int(n[0]) == want[1] > 0 and int(bonus[0]) == want[2]
