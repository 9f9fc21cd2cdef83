"""Attention of a batch over the paged cache with a shared prefix, against a
plain computation in 64 bits.

Tolerance, with w the exact weights of a row (largest 1), L their sum and
A = sum w |v| / L:
  - the probabilities are rounded to the cache's type: eps / 2 relative each,
    eps / 2 * A; in fp16 those below 2^-14 by at most 2^-25 of a part's largest:
    2^-25 * sum |v| / L;
  - a score is a sum of D exact products, at most 2^-21 * scale * sum |q| |k|
    off, and so is the maximum it is compared with: 4 times that relative in a
    weight over its sum;
  - fp32 sums of up to a few thousand terms in tiles, and their merge: 2^-16 A;
  - the output's own rounding.
"""
import math

import numpy as np
import pytest
import torch

from guard import Guarded
from quantized_speculative_verify_gb300 import hq

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


class Batch:
    """A cache whose sequences (slots in any order) share their first positions, and queries on it."""

    def __init__(self, lens, rows, shared, Hq, Hkv, D, ps, dtype, seed=0, tree=True, slots=None, fill=None, spare=3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.lens, self.rows, self.shared, self.Hq, self.Hkv, self.D, self.ps, self.dtype = lens, rows, shared, Hq, Hkv, D, ps, dtype
        self.slots = list(range(B)) if slots is None else slots
        n_seqs = max(self.slots) + 2
        whole = shared // ps
        need = [-(-n // ps) for n in lens]
        pages = whole + sum(max(0, n - whole) for n in need) + spare
        max_pages = max(need) + 1
        order = rng.permutation(pages).tolist()
        pool = torch.randn((3, pages, Hkv, ps, D), generator=g, device=DEV).to(dtype)
        if fill is not None:  # whatever no sequence holds
            pool_fill = torch.full_like(pool, fill)
        table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32)
        pre = [order.pop() for _ in range(whole)]
        used = torch.zeros((pages, ps), dtype=torch.bool)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            mine = pre + [order.pop() for _ in range(need[b] - whole)]
            table[self.slots[b], :need[b]] = torch.tensor(mine, dtype=torch.int32)
            for i, p in enumerate(mine):
                used[p, :min(ps, n - i * ps)] = True
        live = [b for b in range(B) if lens[b]]
        if shared % ps and live:
            src = int(table[self.slots[live[0]], whole])
            for b in live[1:]:
                pool[:, int(table[self.slots[b], whole]), :, :shared % ps] = pool[:, src, :, :shared % ps]
        if fill is not None:
            pool = torch.where(used.to(DEV).view(1, pages, 1, ps, 1), pool, pool_fill)
        ln = torch.zeros(n_seqs, dtype=torch.int32)
        for b, n in enumerate(lens):
            ln[self.slots[b]] = n
        self.cache = hq.PagedCache(pool, torch.ones(pages, dtype=torch.int32, device=DEV), table.to(DEV), ln.to(DEV))
        self.starts = [0] + np.cumsum(rows).tolist()
        R = self.starts[-1]
        self.q = (1.5 * torch.randn((R, Hq, D), generator=g, device=DEV)).to(dtype)
        self.parent = [0] * R
        for b, m in enumerate(rows):
            for i in range(1, m):
                self.parent[self.starts[b] + i] = int(rng.integers(max(0, i - 3), i)) if tree else i - 1
        self.tree, self.scale = tree, 1.0 / math.sqrt(D)

    def run(self, out_type=None, flags=0, workspace=None, max_len=None, **kw):
        out = Guarded(tuple(self.q.shape), out_type or self.dtype, DEV, fill=float("nan"))
        B = len(self.lens)
        n = hq.hq_prefix_attention_workspace_bytes(B, self.starts[-1], max(self.rows), self.Hq, self.Hkv, self.D)
        ws = Guarded((n,), torch.uint8, DEV, fill=0) if workspace is None else workspace
        a = dict(starts=ints(self.starts), max_rows=max(self.rows), shared=self.shared, max_len=max_len or max(self.lens),
                 scale=self.scale, parent=ints(self.parent) if self.tree else None, seqs=ints(self.slots))
        a.update(kw)
        hq.prefix_attention(self.cache, 2, 1, self.q, out=out.t, workspace=ws.t, flags=flags, **a)
        self.status = hq.hq_workspace_status(ws.t)
        out.check()
        ws.check()
        return out.t

    def visible(self, b, i):
        n, m = self.lens[b], self.rows[b]
        seen, j = list(range(n - m)), i
        while True:
            seen.append(n - m + j)
            if j == 0:
                return seen
            j = self.parent[self.starts[b] + j]

    def check(self, out, rows=None):
        eps, eps_o = torch.finfo(self.dtype).eps, torch.finfo(out.dtype).eps
        G = self.Hq // self.Hkv
        worst = 0.0
        for b, n in enumerate(self.lens):
            r0, m = self.starts[b], self.rows[b]
            if n == 0:
                assert not out[r0:r0 + m].any()
                continue
            if rows is not None and not any(r[0] == b for r in rows):
                continue
            t = self.cache.table[self.slots[b], :-(-n // self.ps)].long()
            assert 0 <= int(t.min()) and int(t.max()) < self.cache.c.n_pages
            K, V = (self.cache.pool[p, t].double().transpose(0, 1).reshape(self.Hkv, -1, self.D)[:, :n] for p in (2, 1))
            for i in range(m):
                if rows is not None and (b, i) not in rows:
                    continue
                seen = torch.tensor(self.visible(b, i), device=DEV)
                q = self.q[r0 + i].double().view(self.Hkv, G, self.D)
                k, v = K[:, seen], V[:, seen]
                x = q @ k.transpose(1, 2) * self.scale
                w = torch.exp(x - x.amax(2, keepdim=True))
                L = w.sum(2, keepdim=True)
                ref = w @ v / L
                A = w @ v.abs() / L
                ds = 2.0 ** -21 * self.scale * float((q.abs() @ k.abs().transpose(1, 2)).max())
                lim = A * (eps / 2 + 4 * ds + 2.0 ** -16) + eps_o / 2 * ref.abs() + 2.0 ** -25
                if self.dtype == F16:
                    lim = lim + 2.0 ** -25 * v.abs().sum(1, keepdim=True) / L
                err = (out[r0 + i].double().view(self.Hkv, G, self.D) - ref).abs()
                assert bool((err <= lim).all()), f"sequence {b} row {i}: {float((err - lim).max()):.3e}"
                worst = max(worst, float((err / lim).max()))
        return worst


def spread(n, lo, hi, seed):
    return np.random.default_rng(seed).integers(lo, hi + 1, n).tolist()


CASES = [  # batch, most rows, shared, own positions up to, Hq, Hkv, D, page, type, out, tree
    (1, 1, 0, 0, 1, 1, 64, 16, F16, F16, False),
    (1, 1, 0, 1, 8, 2, 128, 16, BF16, F32, False),
    (4, 1, 1000, 200, 32, 8, 128, 16, F16, F16, False),
    (3, 16, 63, 64, 8, 2, 64, 32, BF16, BF16, True),
    (5, 7, 64, 3, 5, 1, 128, 64, F16, F32, True),
    (9, 3, 65, 130, 6, 2, 128, 16, BF16, BF16, True),
    (2, 128, 129, 60, 4, 4, 64, 128, F16, F16, True),
    (7, 31, 300, 500, 16, 2, 128, 256, F16, F16, True),
    (40, 1, 2048, 70, 64, 1, 128, 64, BF16, BF16, False),
    (130, 2, 640, 33, 8, 8, 64, 16, F16, F16, True),
    (33, 16, 1111, 90, 10, 2, 128, 32, F16, F16, True),
    (6, 5, 0, 700, 12, 4, 128, 16, F16, F16, True),
    (2, 100, 0, 30, 24, 3, 64, 32, BF16, F32, False),
    (3, 4, 9000, 17, 96, 1, 128, 128, F16, F16, True),
    (16, 16, 4097, 0, 32, 8, 128, 16, BF16, BF16, True),
]


@pytest.mark.parametrize("B,m,shared,own,Hq,Hkv,D,ps,dtype,out,tree", CASES)
def test_prefix_attention_matches_64_bits(B, m, shared, own, Hq, Hkv, D, ps, dtype, out, tree):
    rows = [m] + spread(B - 1, 1, m, B)
    lens = [shared + own + m] + [shared + x + r for x, r in zip(spread(B - 1, 0, own, B + 1), rows[1:])]
    t = Batch(lens, rows, shared, Hq, Hkv, D, ps, dtype, seed=B + m, tree=tree,
              slots=np.random.default_rng(B).permutation(B + 2)[:B].tolist())
    got = t.run(out)
    assert t.status == hq.HQ_OK
    t.check(got)
    assert torch.equal(got, t.run(out, flags=hq.HQ_LAUNCH_PDL))  # bit for bit
    # a later, larger bound on the lengths changes the cut, not the result
    again = t.run(out, max_len=min(t.cache.c.max_pages * ps, max(lens) + ps))
    t.check(again)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_shared_positions_need_not_be_declared(dtype):
    """Any `shared` up to the common prefix gives the same attention."""
    t = Batch([500, 431, 460], [3, 9, 1], 420, 8, 2, 128, 32, dtype, seed=2)
    for shared in (420, 419, 256, 64, 63, 1, 0):
        got = t.run(shared=shared)
        assert t.status == hq.HQ_OK
        t.check(got)


def test_without_starts_and_without_seqs():
    t = Batch([70, 90, 80], [2, 2, 2], 60, 8, 2, 128, 16, F16, seed=3)
    got = t.run(starts=None, seqs=None)
    assert t.status == hq.HQ_OK
    t.check(got)


def test_rows_with_strides():
    t = Batch([200, 150], [5, 4], 100, 6, 2, 64, 16, BF16, seed=4)
    wide = torch.zeros((9, 6 * 64 + 16), dtype=BF16, device=DEV)
    wide[:, :384] = t.q.reshape(9, 384)
    t.q = wide[:, :384].unflatten(1, (6, 64))
    assert t.q.stride(0) == 400
    outw = torch.full((9, 392), 3.0, device=DEV)
    ws = torch.zeros(hq.hq_prefix_attention_workspace_bytes(2, 9, 5, 6, 2, 64), dtype=torch.uint8, device=DEV)
    out = outw[:, :384].unflatten(1, (6, 64))
    hq.prefix_attention(t.cache, 2, 1, t.q, ints(t.starts), 5, 100, 200, t.scale, parent=ints(t.parent), seqs=ints(t.slots),
                        out=out, workspace=ws)
    t.check(out)
    assert bool((outw[:, 384:] == 3.0).all())


def test_empty_sequences_and_unclaimed_rows_are_zero():
    t = Batch([0, 90, 0, 75], [2, 3, 1, 2], 64, 8, 2, 128, 16, F16, seed=5)
    got = t.run()
    assert t.status == hq.HQ_OK
    t.check(got)  # the first sequence is empty: the prefix is read through the second
    # all empty
    e = Batch([0, 0], [1, 2], 0, 4, 2, 64, 16, F16, seed=6)
    assert not e.run(max_len=16).any() and e.status == hq.HQ_OK
    # rows before, between and after the sequences' (the rest keep theirs)
    u = Batch([80, 70], [3, 2], 32, 8, 2, 128, 16, F16, seed=7)
    R = u.starts[-1]
    q = torch.randn((R + 4, 8, 128), device=DEV).half()
    q[2:2 + R] = u.q
    out = torch.full_like(q, 5.0)
    parent = [0, 0] + u.parent + [0, 0]
    hq.prefix_attention(u.cache, 2, 1, q, ints([s + 2 for s in u.starts]), 3, 32, 80, u.scale, parent=ints(parent),
                        seqs=ints(u.slots), out=out)
    u.check(out[2:2 + R])
    assert not out[:2].any() and not out[2 + R:].any()


def test_lengths_that_contradict_the_call_give_zero_rows_and_an_error():
    t = Batch([90, 66, 300], [2, 3, 1], 64, 8, 2, 128, 16, F16, seed=8)
    got = t.run(max_len=200)  # the third is longer; the second has 63 old positions, fewer than the 64 shared
    assert t.status == hq.HQ_ERR_INVALID_ARG
    assert not got[2:].any()
    t.check(got, rows={(0, 0), (0, 1)})
    got = t.run(seqs=ints([0, 99, -1]))
    assert t.status == hq.HQ_ERR_INVALID_ARG and not got[2:].any()
    t.check(got, rows={(0, 0), (0, 1)})
    # starts that are not ascending, or point outside
    got = t.run(starts=ints([0, 2, -1, 99]))
    t.check(got, rows={(0, 0), (0, 1)})
    t.run(starts=ints([4, 2 ** 31 - 1, -2 ** 31, 3]))


def test_bad_pages_read_as_zeros_and_report():
    t = Batch([150, 190], [2, 2], 0, 8, 2, 128, 16, F16, seed=9)
    for bad in (-1, 10 ** 6, t.cache.c.n_pages, -2 ** 31):
        was = int(t.cache.table[0, 3])
        t.cache.table[0, 3] = bad
        got = t.run()
        assert t.status == hq.HQ_ERR_INVALID_ARG
        t.cache.table[0, 3] = was
        t.check(got, rows={(1, 0), (1, 1)})
        zero = t.cache.pool[:, was].clone()
        t.cache.pool[:, was] = 0
        t.check(got)
        t.cache.pool[:, was] = zero
        t.check(t.run())
        assert t.status == hq.HQ_OK


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), 65504.0])
@pytest.mark.parametrize("dtype,ps,shared", [(F16, 16, 70), (BF16, 128, 200)])
def test_what_no_row_sees_does_not_matter(fill, dtype, ps, shared):
    """Free pages and the rows past a sequence's end hold anything."""
    t = Batch([shared + 31, shared + 5, 0, shared + 90], [4, 5, 2, 1], shared, 8, 2, 128, ps, dtype, seed=10, fill=fill)
    got = t.run()
    assert t.status == hq.HQ_OK and bool(torch.isfinite(got.float()).all())
    t.check(got)


def test_nonfinite_branches_reach_only_their_own_rows():
    t = Batch([120, 100], [9, 3], 64, 8, 2, 128, 16, F16, seed=11)
    t.parent[:9] = [0, 0, 0, 1, 1, 2, 3, 5, 5]
    for node, plane, x in ((1, 1, float("nan")), (5, 1, float("inf")), (2, 2, float("nan"))):
        s = Batch([120, 100], [9, 3], 64, 8, 2, 128, 16, F16, seed=11)
        s.parent = t.parent
        pos = 120 - 9 + node
        s.cache.pool[plane, int(s.cache.table[0, pos // 16]), 1, pos % 16, 7] = x
        got = s.run()
        hit = [i for i in range(9) if pos in s.visible(0, i)]
        free = {(0, i) for i in range(9) if i not in hit} | {(1, i) for i in range(3)}
        assert 0 < len(hit) < 9
        s.check(got, rows=free)
        for i in hit:
            assert not torch.isfinite(got[i, 4:]).all() and bool(torch.isfinite(got[i, :4]).all())


def test_peaked_and_flat_scores():
    t = Batch([700, 650], [4, 4], 600, 8, 2, 128, 16, BF16, seed=12)
    for scale in (1.0, 0.0, -0.3):
        t.scale = scale
        if scale > 0.5:
            t.q *= 2
        t_abs = t.scale
        got = t.run()
        t.scale = t_abs
        assert bool(torch.isfinite(got.float()).all())
        if scale <= 0:
            s, t.scale = t.scale, abs(t.scale)  # the bound takes the size of the scale
            q = t.q
            t.q = torch.where(torch.tensor(s < 0, device=DEV), -q, q) if s else q * 0
            t.check(got)
            t.q, t.scale = q, s
        else:
            t.check(got)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes a plane, and of more than 2^31 elements in all."""
    pages, Hkv, ps, D = 70000, 2, 128, 128
    pool = torch.zeros((2, pages, Hkv, ps, D), dtype=F16, device=DEV)
    assert pool[0].numel() * 2 > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(1)
    use = [69999, 3, 65536, 40000]
    pool[:, use] = torch.randn((2, 4, Hkv, ps, D), generator=g, device=DEV).half()
    cache = hq.PagedCache(pool, torch.zeros(pages, dtype=torch.int32, device=DEV),
                          torch.tensor([use + [-1]], dtype=torch.int32, device=DEV), ints([400]))
    q = torch.randn((1, 4, D), generator=g, device=DEV).half()
    got = hq.prefix_attention(cache, 0, 1, q, None, 1, 200, 400, 0.09).double()
    k, v = (pool[p, use].transpose(0, 1).reshape(Hkv, 512, D)[:, :400].double() for p in (0, 1))
    w = torch.softmax(q.double().view(Hkv, 2, D) @ k.transpose(1, 2) * 0.09, 2)
    assert float((got.view(Hkv, 2, D) - w @ v).abs().max()) <= 2.0 ** -10
    # the page operations reach the far pages too
    hq.pages_copy(cache, ints([69999]), ints([69998]))
    assert torch.equal(pool[:, 69998], pool[:, 69999])
    x = torch.randn((1, Hkv, D), generator=g, device=DEV)
    cache.lens.fill_(1)
    hq.pages_write(cache, 1, 0, x, -x, None, 1)
    assert torch.equal(pool[1, 69999, :, 0], x[0].half()) and torch.equal(pool[0, 69999, :, 0], -x[0].half())
    assert hq.pages_status(cache) == hq.HQ_OK


def test_agrees_with_the_tree_attention_of_one_sequence():
    """The contiguous cache's operator on the same positions."""
    M, Hq, Hkv, L = 16, 32, 8, 300
    t = Batch([L + M], [M], 0, Hq, Hkv, 128, 16, F16, seed=13)
    pages = t.cache.table[0, :-(-(L + M) // 16)].long()
    k, v = (t.cache.pool[p, pages].transpose(0, 1).reshape(Hkv, -1, 128)[:, :L + M].contiguous() for p in (2, 1))
    ref = hq.tree_attention(t.q, k, v, L, ints(t.parent), t.scale)
    got = t.run(F32)
    assert float((got - ref).abs().max()) <= 2 * (2.0 ** -11 + 1e-4) * float(v.abs().max())


def test_on_a_side_stream_and_in_a_graph():
    """A captured step follows the lengths and tables on the device."""
    t = Batch([150, 140, 170], [1, 1, 1], 128, 8, 2, 128, 16, F16, seed=14, tree=False)
    out = torch.empty_like(t.q)
    ws = torch.zeros(hq.hq_prefix_attention_workspace_bytes(3, 3, 1, 8, 2, 128), dtype=torch.uint8, device=DEV)
    seqs, q = ints(t.slots), t.q
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        hq.prefix_attention(t.cache, 2, 1, q, None, 1, 128, 176, t.scale, seqs=seqs, out=out, workspace=ws)
    st.synchronize()
    t.check(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hq.prefix_attention(t.cache, 2, 1, q, None, 1, 128, 176, t.scale, seqs=seqs, out=out, workspace=ws)
    t.lens = [129, 143, 0]
    t.cache.lens[:3] = ints(t.lens)
    q.copy_(torch.randn(q.shape, device=DEV).half())
    g.replay()
    torch.cuda.synchronize()
    assert hq.hq_workspace_status(ws) == hq.HQ_OK
    t.check(out)


MANY_ROWS = [  # batch, most rows, shared, own positions up to, Hq, Hkv, D, page, type: rows enough for the tensor-memory kernel
    (20, 1, 700, 40, 32, 8, 128, 16, F16), (32, 1, 512, 9, 8, 2, 128, 64, BF16), (65, 1, 640, 0, 2, 2, 64, 32, F16),
    (33, 1, 4096, 20, 12, 3, 64, 128, BF16), (13, 9, 900, 5, 8, 8, 128, 256, F16), (3, 128, 1300, 200, 8, 8, 128, 16, BF16),
    (5, 100, 515, 7, 6, 2, 64, 16, F16), (70, 2, 2049, 64, 40, 8, 128, 32, F16), (24, 16, 6000, 30, 32, 4, 128, 64, BF16),
]


@pytest.mark.parametrize("B,m,shared,own,Hq,Hkv,D,ps,dtype", MANY_ROWS)
def test_many_rows_match_64_bits(B, m, shared, own, Hq, Hkv, D, ps, dtype):
    rows = [m] + spread(B - 1, 1, m, B)
    lens = [shared + own + m] + [shared + x + r for x, r in zip(spread(B - 1, 0, own, B + 1), rows[1:])]
    t = Batch(lens, rows, shared, Hq, Hkv, D, ps, dtype, seed=B + m)
    got = t.run()
    assert t.status == hq.HQ_OK
    t.check(got)
    assert torch.equal(got, t.run(flags=hq.HQ_LAUNCH_PDL))
    t.check(t.run(shared=shared // 2 + 1))


@pytest.mark.parametrize("B,rising", [(20, True), (20, False), (80, True), (80, False)])
def test_scores_that_rise_or_fall_along_the_prefix(B, rising):
    """The running maximum moves at every tile, by a little and by a lot."""
    t = Batch([1500 + b % 7 for b in range(B)], [1] * B, 1400, 8, 2, 128, 16, F16, seed=B)
    pages = t.cache.table[0, :1400 // 16].long()
    ramp = torch.linspace(0.0, 6.0, len(pages), device=DEV)
    ramp = ramp if rising else ramp.flip(0)
    t.cache.pool[2, pages] = (t.cache.pool[2, pages].float() * ramp.view(-1, 1, 1, 1)).half()
    got = t.run()
    assert t.status == hq.HQ_OK
    t.check(got)


def test_nan_in_the_prefix_reaches_every_row_of_its_head():
    for B in (20, 80):
        t = Batch([800] * B, [1] * B, 700, 8, 2, 128, 16, BF16, seed=B)
        t.cache.pool[1, int(t.cache.table[0, 20]), 1, 3, 5] = float("nan")
        got = t.run()
        assert bool(torch.isnan(got[:, 4:, 5]).all()) and bool(torch.isfinite(got[:, :4].float()).all())
        assert bool(torch.isfinite(got[:, 4:, :5].float()).all())


def test_a_negative_scale_with_many_rows():
    t = Batch([900 + b for b in range(70)], [1] * 70, 800, 8, 2, 128, 32, F16, seed=3)
    t.scale = -0.1
    got = t.run()
    t.q, t.scale = -t.q, 0.1
    t.check(got)


def test_inactive_sequences_among_many_rows():
    lens = [0 if b % 5 == 0 else 700 + b for b in range(60)]
    t = Batch(lens, [2] * 60, 600, 8, 2, 128, 16, F16, seed=4)
    got = t.run()
    assert t.status == hq.HQ_OK
    t.check(got)
    t.cache.lens.zero_()  # none left: the prefix has no table to be read through
    assert not t.run(max_len=700).any() and t.status == hq.HQ_OK


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 65504.0])
@pytest.mark.parametrize("dtype,D,ps,shared,B", [(F16, 128, 16, 70, 3), (BF16, 64, 128, 700, 20), (F16, 128, 64, 1000, 9)])
def test_what_no_row_sees_does_not_matter_to_large_trees(fill, dtype, D, ps, shared, B):
    rows = [60] + spread(B - 1, 1, 60, 1)
    lens = [shared + n + m for n, m in zip(spread(B, 0, 300, 2), rows)]
    t = Batch(lens, rows, shared, 8, 2, D, ps, dtype, seed=10, fill=fill)
    got = t.run()
    assert t.status == hq.HQ_OK and bool(torch.isfinite(got.float()).all())
    t.check(got)


@pytest.mark.parametrize("dtype,m,Hq", [(F16, 100, 8), (BF16, 40, 2), (F16, 128, 2), (BF16, 13, 16)])
def test_nonfinite_branches_of_large_trees_reach_only_their_own_rows(dtype, m, Hq):
    rng = np.random.default_rng(m)
    for node, plane, x in ((1, 1, float("nan")), (m // 2, 1, float("inf")), (3, 2, float("nan")), (m - 1, 1, float("-inf"))):
        s = Batch([600 + m, 600], [m, 3], 560 if m % 2 else 100, Hq, 2, 128, 32, dtype, seed=m)
        pos = 600 + node
        s.cache.pool[plane, int(s.cache.table[0, pos // 32]), 1, pos % 32, 7] = x
        got = s.run()
        hit = [i for i in range(m) if pos in s.visible(0, i)]
        free = {(0, i) for i in range(m) if i not in hit} | {(1, i) for i in range(3)}
        assert hit and s.status == hq.HQ_OK
        h = Hq // 2
        s.check(got, rows=set(list(free)[:40]))
        assert bool(torch.isfinite(got[:, :h].float()).all())
        out = torch.tensor([i not in hit for i in range(m)], device=DEV)
        assert bool(torch.isfinite(got[:m][out].float()).all())
        for i in hit:
            assert not torch.isfinite(got[i, h:, 7]).any()
            if plane == 1:
                assert bool(torch.isfinite(got[i, h:, :7].float()).all())


@pytest.mark.parametrize("B,m,shared,own,Hq,Hkv,D,ps,dtype", [
    (1, 33, 0, 0, 4, 4, 128, 16, F16), (2, 128, 0, 900, 8, 2, 128, 64, BF16), (50, 9, 600, 260, 8, 2, 64, 16, F16),
    (4, 128, 2000, 5, 64, 2, 128, 128, BF16), (6, 40, 511, 128, 5, 5, 128, 32, F16), (3, 17, 512, 127, 16, 8, 64, 256, BF16),
])
def test_large_trees_match_64_bits(B, m, shared, own, Hq, Hkv, D, ps, dtype):
    rows = [m] + spread(B - 1, 1, m, B)
    lens = [shared + own + m] + [shared + x + r for x, r in zip(spread(B - 1, 0, own, B + 1), rows[1:])]
    for tree in (True, False):
        t = Batch(lens, rows, shared, Hq, Hkv, D, ps, dtype, seed=B + m, tree=tree)
        got = t.run()
        assert t.status == hq.HQ_OK
        t.check(got)
        assert torch.equal(got, t.run())


@pytest.mark.parametrize("B,m,shared,own,Hq,Hkv,D,ps,dtype", [
    (1, 16, 2000, 300, 2, 2, 128, 16, F16), (1, 17, 2000, 300, 2, 2, 128, 16, F16), (1, 5, 5000, 0, 8, 2, 64, 128, BF16),
    (8, 1, 128, 50, 8, 2, 128, 64, BF16), (9, 1, 128, 50, 8, 2, 128, 64, BF16), (9, 1, 127, 50, 8, 2, 128, 64, BF16),
    (33, 1, 129, 0, 1, 1, 64, 16, F16), (32, 1, 129, 300, 1, 1, 64, 16, F16), (2, 8, 100, 900, 4, 1, 128, 32, F16),
    (2, 4, 900, 900, 4, 1, 128, 32, F16), (2, 17, 130, 700, 1, 1, 64, 32, BF16), (128, 1, 3000, 1000, 8, 2, 128, 64, BF16),
    (48, 16, 1234, 700, 8, 2, 128, 32, F16), (70, 1, 0, 1500, 8, 2, 128, 16, F16), (20, 6, 256, 1, 16, 4, 64, 16, BF16),
])
def test_sizes_where_another_kernel_takes_over(B, m, shared, own, Hq, Hkv, D, ps, dtype):
    rows = [m] + spread(B - 1, 1, m, B)
    lens = [shared + own + m] + [shared + x + r for x, r in zip(spread(B - 1, 0, own, B + 1), rows[1:])]
    t = Batch(lens, rows, shared, Hq, Hkv, D, ps, dtype, seed=B + m + shared)
    got = t.run().clone()
    assert t.status == hq.HQ_OK
    t.check(got)
    ws = Guarded((hq.hq_prefix_attention_workspace_bytes(B, t.starts[-1], m, Hq, Hkv, D),), torch.uint8, DEV, fill=0)
    for flags in (0, hq.HQ_LAUNCH_PDL, hq.HQ_LAUNCH_PDL):  # one workspace, calls on each other's heels
        assert torch.equal(got, t.run(flags=flags, workspace=ws))
    assert t.status == hq.HQ_OK


def test_a_batch_of_no_sequences_claims_no_row():
    t = Batch([80], [3], 32, 8, 2, 128, 16, F16, seed=7)
    for stream in (None, torch.cuda.Stream()):
        out = torch.full_like(t.q, 5.0)
        torch.cuda.synchronize()
        got = hq.prefix_attention(t.cache, 2, 1, t.q, ints([0]), 3, 32, 80, t.scale, out=out, stream=stream)
        torch.cuda.synchronize()
        assert got is out and not out.any()
    assert not hq.prefix_attention(t.cache, 2, 1, t.q, ints([0]), 3, 32, 80, t.scale).any()


@pytest.mark.parametrize("B,m", [(2, 2), (60, 1), (2, 40)])
def test_errors_reach_the_cache_without_a_workspace(B, m):
    t = Batch([300 + b % 5 for b in range(B)], [m] * B, 200, 8, 2, 128, 16, F16, seed=9)

    def run(**kw):
        a = dict(shared=200, max_len=320, parent=ints(t.parent), seqs=ints(t.slots))
        a.update(kw)
        return hq.prefix_attention(t.cache, 2, 1, t.q, ints(t.starts), m, scale=t.scale, **a)
    t.check(run())
    assert hq.pages_status(t.cache) == hq.HQ_OK
    run(max_len=300)  # some sequences are longer
    assert hq.pages_status(t.cache) == hq.HQ_ERR_INVALID_ARG and hq.pages_status(t.cache) == hq.HQ_OK
    for at in (3, 15):  # among the shared positions, among the own ones
        was = int(t.cache.table[0, at])
        t.cache.table[0, at] = -1
        run()
        assert hq.pages_status(t.cache) == hq.HQ_ERR_INVALID_ARG
        t.cache.table[0, at] = was
        t.check(run())
        assert hq.pages_status(t.cache) == hq.HQ_OK


@pytest.mark.parametrize("B,m,Hq,Hkv,D,sink", [
    (3, 1, 8, 2, 128, 0), (3, 1, 8, 2, 64, 3000), (2, 7, 8, 8, 64, 5), (40, 1, 8, 2, 128, 0), (64, 2, 4, 1, 64, 2999), (1, 40, 2, 2, 128, 1),
    (1, 100, 4, 2, 64, 17)])
@pytest.mark.parametrize("below", [18.3, 20.6])
def test_a_flat_tail_far_below_one_key(B, m, Hq, Hkv, D, sink, below):
    """One key outweighs each of thousands of others by 2^below: in fp16 their
    probabilities keep its precision (no term for subnormal ones here).

    K holds `k` in dimension 0 of the one key and 0 elsewhere, q 1 there, so the
    scores are exact: scale * k and 0.  V is 0 at the one key and 1 elsewhere:
    the output is the tail's share, N w / (1 + N w) with w = 2^-below up to the
    rounding of scale * log2(e) (2^-23 relative of `below`).  Each probability is
    off by 2^-11 at most, all alike; the fp32 output by its sums."""
    shared = 3500
    t = Batch([shared + 20 + m] * B, [m] * B, shared, Hq, Hkv, D, 16, F16, seed=1, tree=False)
    t.cache.pool[2] = 0
    t.cache.pool[1] = 1
    for b in range(B):
        page = int(t.cache.table[t.slots[b], sink // 16])
        t.cache.pool[2, page, :, sink % 16, 0] = 4.0
        t.cache.pool[1, page, :, sink % 16] = 0
    t.q.zero_()
    t.q[:, :, 0] = 1.0
    t.scale = below * math.log(2.0) / 4.0
    got = t.run(F32).double()
    assert t.status == hq.HQ_OK
    for b in range(B):
        for i in range(m):
            n = shared + 20 + i  # the others that the row sees
            w = 2.0 ** -below
            ref = n * w / (1.0 + n * w)
            err = float((got[t.starts[b] + i] - ref).abs().max())
            assert err <= ref * (2.0 ** -11 + 2.0 ** -16 + 4 * below * 2.0 ** -23), f"{err / ref:.2e}"
