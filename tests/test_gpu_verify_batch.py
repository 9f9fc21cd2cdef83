"""A layer step for a batch of requests, its operators together: every request
gets from the batch what it gets alone, step after step, and the cache ends as
if each had been decoded by itself.

Tolerance.  The same kernels see the same rows; only the attention's cut into
parts differs (probabilities rounded to fp16 relative to another maximum: 2^-11
of the largest value each), and a code of the int8 quantization may move by one
step where its input lies at a rounding border: sx <= max|x'| / 127 of a row,
times the largest weight row, over a few codes.  The outputs are compared
through the norm of the difference: 2^-7 of the output's.
"""
import pytest
import torch

from quantized_speculative_verify_gb300 import hq
from quantized_speculative_verify_gb300.verify_batch import BatchLayer, prefill

pytestmark = pytest.mark.gpu
DEV = "cuda"
HIDDEN, HEADS, KV, D, PS = 512, 8, 2, 64, 16


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def fresh(seqs, shared):
    cache = hq.PagedCache.empty(2, 200, KV, PS, D, seqs, 40)
    prefill(cache, (0, 1), 0, shared, seed=5)
    return cache


def positions(cache, s):
    n = int(cache.lens[s])
    t = cache.table[s, :-(-n // PS)].long()
    return cache.pool[:, t].transpose(2, 3).reshape(2, -1, KV, D)[:, :n]


@pytest.mark.parametrize("shared,flags", [(100, hq.HQ_LAUNCH_DETERMINISTIC), (530, hq.HQ_LAUNCH_DETERMINISTIC)])
def test_a_batch_gives_each_request_what_it_gets_alone(shared, flags):
    rows = [5, 1, 9]
    B, M = len(rows), sum(rows)
    layer = BatchLayer(HIDDEN, HEADS, KV, D, M, adapters=3, rank=8, seed=2)
    alone = BatchLayer(HIDDEN, HEADS, KV, D, M, adapters=3, rank=8, seed=2)
    starts = [0, 5, 6, 15]
    parent = [0, 0, 0, 1, 2, 0, 0, 0, 1, 1, 3, 0, 5, 5, 2]
    ids = [2] * 5 + [-1] + [0] * 9
    keeps = [[[1, 3], [], [2]], [[2], [], [1, 4, 7]]]
    cache = fresh(B + 1, shared)
    hq.pages_fork(cache, ints([0] * B), ints([1, 2, 3]))
    caches = []
    for b in range(B):
        c = fresh(2, shared)
        hq.pages_fork(c, ints([0]), ints([1]))
        caches.append(c)
    g = torch.Generator(device=DEV).manual_seed(1)
    for keep in keeps:
        x = torch.randn((M, HIDDEN), generator=g, device=DEV)
        res = torch.randn((M, HIDDEN), generator=g, device=DEV).bfloat16()
        base = cache.lens[1:].clone()
        r_all = res.clone()
        out = layer.step(cache, (0, 1), x, r_all, ints([1, 2, 3]), ints(starts), ints(rows), ints(parent), ints(ids), 9,
                         shared, 600, flags).clone()
        pad = torch.full((B, 3), -1, dtype=torch.int32)
        for b, k in enumerate(keep):
            pad[b, :len(k)] = torch.tensor(k, dtype=torch.int32)
        hq.pages_compact(cache, ints([1, 2, 3]), base, pad.to(DEV), ints([len(k) for k in keep]))
        for b in range(B):
            lo, hi = starts[b], starts[b + 1]
            r_one, c = res[lo:hi].clone(), caches[b]
            root = c.lens[1:].clone()
            one = alone.step(c, (0, 1), x[lo:hi].contiguous(), r_one, ints([1]), ints([0, hi - lo]), ints([hi - lo]),
                             ints(parent[lo:hi]), ints(ids[lo:hi]), hi - lo, shared, 600, flags)
            hq.pages_compact(c, ints([1]), root, ints(keep[b] + [-1]).unsqueeze(0), ints([len(keep[b])]))
            assert torch.equal(r_one, r_all[lo:hi])
            assert float((one - out[lo:hi]).norm()) <= 2.0 ** -7 * float(out[lo:hi].norm())
            p, q = positions(cache, b + 1).float(), positions(c, 1).float()
            assert p.shape == q.shape
            assert float((p - q).norm()) <= 2.0 ** -10 * float(q.norm())
    assert torch.equal(positions(cache, 0), positions(caches[0], 0))  # the prompt itself is as it was
    for c in [cache] + caches:
        assert hq.pages_status(c) == hq.HQ_OK
    assert hq.hq_workspace_status(layer.ws_attn) == hq.HQ_OK and hq.hq_workspace_status(layer.ws_gemm) == hq.HQ_OK
