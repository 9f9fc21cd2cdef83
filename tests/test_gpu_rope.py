"""Rotary positions on the way into the paged cache, against a plain
computation in 64 bits with exact angles.

Angles.  turns is an integer, so the exact angle of position p is p * turns mod
2^64 turns of 2^-64.  The kernel keeps 32 of the 64 bits (2^-32 turns, 2^-29
radians), rounds them to a float in units of half a turn (at most 2^-25 of pi,
2^-23.3 radians) and takes sine and cosine (2 units in the last place, 2^-23):
each is off by at most 2^-22, with the product by gain (2^-24 relative).  A
rotated element is u c - v s: two products and a sum more, so it is within
(2^-22 + 3 * 2^-24) * (|u| + |v|) * |gain| < 2^-21 * (|u| + |v|) * |gain|.
A normed head: 8 + 5 terms of the sum of squares (13 * 2^-24, half of it in the
root), rsqrt 2^-22, three roundings: less than 2^-20 relative in u and v.  The
result is rounded once: eps / 2, or half the smallest subnormal.
"""
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


class Rows:
    """A cache whose sequences (in any slots) have been grown by their new rows, and those rows' q, k and v."""

    def __init__(self, before, rows, Hq, Hkv, D, ps, in_type, dtype, seed=0, slots=None, tree=False, pad=0, gap=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(rows)
        self.before, self.rows, self.Hq, self.Hkv, self.D, self.ps, self.dtype, self.in_type = before, rows, Hq, Hkv, D, ps, dtype, in_type
        self.slots = list(range(B)) if slots is None else slots
        lens = [n + m for n, m in zip(before, rows)]
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + 3
        order = rng.permutation(pages).tolist()
        n_seqs = max(self.slots) + 2
        table = torch.full((n_seqs, max(need) + 1), -1, dtype=torch.int32)
        ln = torch.zeros(n_seqs, dtype=torch.int32)
        for b in range(B):
            table[self.slots[b], :need[b]] = torch.tensor([order.pop() for _ in range(need[b])], dtype=torch.int32)
            ln[self.slots[b]] = lens[b]
        pool = torch.randn((3, pages, Hkv, ps, D), generator=g, device=DEV).to(dtype)
        self.cache = hq.PagedCache(pool, torch.ones(pages, dtype=torch.int32, device=DEV), table.to(DEV), ln.to(DEV))
        self.old = pool.clone()
        self.starts = [0] + np.cumsum(rows).tolist()
        R = self.starts[-1] + gap  # rows that no sequence claims
        cols = (Hq + 2 * Hkv) * D
        y = torch.randn((R, cols + pad), generator=g, device=DEV).to(in_type)
        self.q, self.k, self.v = (t.unflatten(1, (-1, D)) for t in y[:, :cols].split([Hq * D, Hkv * D, Hkv * D], 1))
        self.parent = [0] * R
        for b, m in enumerate(rows):
            for i in range(1, m):
                self.parent[self.starts[b] + i] = int(rng.integers(max(0, i - 3), i)) if tree else i - 1
        self.tree = tree

    def place(self, b, i):
        p = self.before[b] + i
        return int(self.cache.table[self.slots[b], p // self.ps]), p % self.ps

    def positions(self):
        """(row, page, slot in it, rotary position) of every row."""
        table = self.cache.table.cpu().numpy()
        out = []
        for b, m in enumerate(self.rows):
            depth = [0] * m
            for i in range(m):
                p = self.parent[self.starts[b] + i]
                depth[i] = depth[p] + 1 if i and 0 <= p < i else 0
                at = self.before[b] + i
                out.append((self.starts[b] + i, int(table[self.slots[b], at // self.ps]), at % self.ps, self.before[b] + depth[i]))
        return out


def expected(x, pos, turns, layout, gain, weight, eps):
    """The rotated heads x [rows][heads][D] in 64 bits, and how far they may be off before the last rounding."""
    D, half = x.shape[2], len(turns)
    y = x.double().cpu().numpy()
    lose = 0.0
    if weight is not None:
        ms = (y * y).mean(2, keepdims=True) + eps
        y = np.where(ms > 0, y / np.sqrt(np.where(ms > 0, ms, 1.0)), 0.0) * weight.double().cpu().numpy()
        lose = 2.0 ** -20
    a = np.array([[(int(p) * int(t)) % (1 << 64) for t in turns] for p in pos], dtype=object)
    a = np.array([[float(int(v) - (1 << 64) if v >= 1 << 63 else int(v)) for v in r] for r in a]).reshape(len(pos), half)
    a = (a / 2.0 ** 64 * 2.0 * np.pi)[:, None, :]
    c, s = np.cos(a) * gain, np.sin(a) * gain
    if layout == "half":
        u, v = y[:, :, :half].copy(), y[:, :, half:2 * half].copy()
    else:
        u, v = y[:, :, 0:2 * half:2].copy(), y[:, :, 1:2 * half:2].copy()
    lim = lose * np.abs(y)
    size = (2.0 ** -21 + lose) * abs(gain) * (np.abs(u) + np.abs(v))
    ru, rv = u * c - v * s, v * c + u * s
    if layout == "half":
        y[:, :, :half], y[:, :, half:2 * half] = ru, rv
        lim[:, :, :half], lim[:, :, half:2 * half] = size, size
    else:
        y[:, :, 0:2 * half:2], y[:, :, 1:2 * half:2] = ru, rv
        lim[:, :, 0:2 * half:2], lim[:, :, 1:2 * half:2] = size, size
    return y, lim


def close(got, y, lim):
    f = torch.finfo(got.dtype)
    off = np.abs(got.double().cpu().numpy() - y)
    bound = lim + (np.abs(y) + lim) * (f.eps / 2) + f.smallest_normal * f.eps / 2
    assert np.all(off <= bound), f"worst {np.max(off / bound)} of the bound"


def check(r, out, turns, layout="half", gain=1.0, qw=None, kw=None, eps=1e-6, pos=None):
    at = r.positions()
    row = [a[0] for a in at]
    p = [a[3] for a in at] if pos is None else [int(pos[i]) for i in row]
    t = turns.cpu().numpy().view(np.uint64).tolist()
    close(out[row], *expected(r.q[row], p, t, layout, gain, qw, eps))
    page, slot = [a[1] for a in at], [a[2] for a in at]
    close(r.cache.pool[0, page, :, slot], *expected(r.k[row], p, t, layout, gain, kw, eps))
    assert torch.equal(r.cache.pool[1, page, :, slot], r.v[row].to(r.dtype))
    # and nothing else has changed
    pool = r.cache.pool.clone()
    for x in range(2):
        pool[x, page, :, slot] = r.old[x, page, :, slot]
    assert torch.equal(pool.view(torch.int16), r.old.view(torch.int16))
    assert hq.pages_status(r.cache) == hq.HQ_OK


CASES = [  # before, rows, Hq, Hkv, D, rot, layout, page size, in, cache, tree, norm
    ([5], [1], 4, 1, 64, 64, "half", 16, F32, F16, False, False),
    ([0], [1], 1, 1, 64, 16, "interleaved", 16, F16, F16, False, True),
    ([100, 3, 77], [16, 1, 9], 32, 8, 128, 128, "half", 16, F32, BF16, True, False),
    ([100, 3, 77], [16, 1, 9], 8, 8, 128, 96, "interleaved", 64, F32, F16, True, True),
    ([15, 16, 17, 0], [1, 1, 1, 1], 5, 5, 128, 32, "half", 16, BF16, BF16, False, True),
    ([1000], [128], 16, 2, 64, 48, "half", 32, F16, F16, True, False),
    ([0, 31], [70, 33], 6, 3, 256, 256, "interleaved", 32, F32, F16, False, False),
    ([0, 200], [300, 5], 3, 1, 256, 144, "half", 128, BF16, BF16, False, True),
    ([9, 0, 0, 4], [0, 17, 0, 2], 40, 10, 128, 112, "half", 256, F32, BF16, True, False),
    ([7], [3], 70, 1, 64, 64, "half", 16, F32, F16, False, False),
]


@pytest.mark.parametrize("before,rows,Hq,Hkv,D,rot,layout,ps,it,dt,tree,norm", CASES)
def test_rope_matches_64_bits(before, rows, Hq, Hkv, D, rot, layout, ps, it, dt, tree, norm):
    slots = [2 * b + 1 for b in range(len(rows))][::-1]
    r = Rows(before, rows, Hq, Hkv, D, ps, it, dt, seed=D + rot + Hq, slots=slots, tree=tree, pad=8, gap=2)
    turns = hq.rope_turns(hq.rope_freqs(rot, 10000.0, "yarn", 8.0, 64.0), DEV)
    w = [1.0 + 0.3 * torch.randn(D, device=DEV) for _ in range(2)] if norm else [None, None]
    out = Guarded(tuple(r.q.shape), dt, DEV, fill=7.0)
    hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), max(rows), layout, gain=1.2, q_weight=w[0], k_weight=w[1],
                  parent=ints(r.parent) if tree else None, seqs=ints(slots), out=out.t)
    torch.cuda.synchronize()
    out.check()
    assert bool((out.t[r.starts[-1]:] == 7.0).all())  # rows that no sequence claims
    check(r, out.t, turns, layout, 1.2, w[0], w[1])


@pytest.mark.parametrize("only", ["q", "k"])
def test_one_of_the_two_weights(only):
    r = Rows([10], [4], 4, 2, 64, 16, F32, F16, seed=3)
    turns, w = hq.rope_turns(hq.rope_freqs(64), DEV), torch.rand(64, device=DEV) + 0.5
    qw, kw = (w, None) if only == "q" else (None, w)
    out = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 4, q_weight=qw, k_weight=kw)
    check(r, out, turns, qw=qw, kw=kw)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_given_positions(layout):
    r = Rows([3], [9], 2, 1, 128, 16, F32, F16, seed=4)
    pos = [0, 1, -1, 131071, 2 ** 24 + 1, 2 ** 30 - 1, 2 ** 31 - 1, -2 ** 31, 123456789]
    turns = hq.rope_turns(hq.rope_freqs(128), DEV)
    out = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 9, layout, positions=ints(pos))
    check(r, out, turns, layout, pos=pos)


def test_position_zero_is_the_plain_write():
    r = Rows([3, 40], [9, 2], 4, 2, 128, 16, F32, F16, seed=5)
    turns = hq.rope_turns(hq.rope_freqs(128), DEV)
    out = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 9, positions=torch.zeros(11, dtype=torch.int32, device=DEV))
    plain = Rows([3, 40], [9, 2], 4, 2, 128, 16, F32, F16, seed=5)
    hq.pages_write(plain.cache, 0, 1, plain.k, plain.v, ints(plain.starts), 9)
    assert torch.equal(out, r.q.half())
    assert torch.equal(r.cache.pool, plain.cache.pool)


@pytest.mark.parametrize("B", [1, 31, 32, 33, 200, 1500])
def test_many_sequences_some_without_rows(B):
    rng = np.random.default_rng(B)
    rows = rng.integers(0, 3, B).tolist()
    rows[-1] = 1
    before = rng.integers(0, 40, B).tolist()
    r = Rows(before, rows, 1, 1, 64, 16, F16, F16, seed=B)
    turns = hq.rope_turns(hq.rope_freqs(16), DEV)
    out = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), max(max(rows), 1))
    check(r, out, turns)


@pytest.mark.parametrize("it,dt,layout,norm", [(BF16, BF16, "half", False), (F32, F16, "interleaved", True), (F16, F16, "half", True),
                                                (F32, BF16, "half", False)])
def test_prompts_of_many_rows(it, dt, layout, norm):
    """Enough rows for the kernel that takes few threads a row."""
    rows, before = [1500, 3, 0, 1400], [0, 40, 0, 17]
    r = Rows(before, rows, 3, 1, 64, 64, it, dt, seed=17, pad=8, gap=1)
    turns, w = hq.rope_turns(hq.rope_freqs(48), DEV), torch.rand(64, device=DEV) + 0.5 if norm else None
    out = Guarded(tuple(r.q.shape), dt, DEV, fill=7.0)
    hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 1500, layout, q_weight=w, k_weight=w, out=out.t)
    torch.cuda.synchronize()
    out.check()
    assert bool((out.t[-1] == 7.0).all())
    check(r, out.t, turns, layout, qw=w, kw=w)


def test_equal_rows_without_starts_and_rows_past_max_rows():
    r = Rows([5, 6, 7], [4, 4, 4], 2, 1, 64, 16, F32, F16, seed=8)
    turns = hq.rope_turns(hq.rope_freqs(64), DEV)
    out = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, None, 4)
    check(r, out, turns)
    # a sequence's rows past max_rows are not its newest ones: left as they were
    r = Rows([5, 6], [4, 2], 2, 1, 64, 16, F32, F16, seed=9)
    r.cache.lens[0] -= 1  # three rows of it count
    out = torch.full((6, 2, 64), 7.0, dtype=F16, device=DEV)
    hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 3, out=out)
    assert bool((out[3] == 7.0).all()) and not bool((out[2] == 7.0).any()) and not bool((out[4:] == 7.0).all())


def test_a_buffer_that_the_call_makes_is_zero_without_sequences():
    r = Rows([5], [4], 2, 1, 64, 16, F32, F16, seed=18, gap=2)
    turns = hq.rope_turns(hq.rope_freqs(64), DEV)
    assert not bool(hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints([0]), 4).any())
    out = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 4)
    assert not bool(out[4:].any())
    check(r, out, turns)


def test_parents_that_are_none_end_the_walk():
    r = Rows([10], [6], 2, 1, 64, 16, F32, F16, seed=10)
    r.parent = [5, 0, 7, 2, -3, 4]  # the walks end at 0, 2 and 4
    turns = hq.rope_turns(hq.rope_freqs(64), DEV)
    out = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 6, parent=ints(r.parent))
    check(r, out, turns)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_q_in_place(layout):
    r = Rows([30], [40], 5, 1, 128, 16, BF16, BF16, seed=11, tree=True, pad=64)
    turns = hq.rope_turns(hq.rope_freqs(96), DEV)
    q = r.q.clone()
    got = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 40, layout, parent=ints(r.parent), out=r.q)
    assert got is r.q
    r.q = q
    check(r, got, turns, layout)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_infinities_and_nan_stay_in_their_pair_or_element(layout):
    r = Rows([4], [3], 2, 1, 64, 16, F32, F16, seed=12)
    q, k, v = r.q.clone(), r.k.clone(), r.v.clone()
    q[0, 0, 40], q[1, 1, 63], q[2, 0, 2], k[1, 0, 50], v[0, 0, 0] = float("nan"), float("inf"), float("nan"), -float("inf"), float("nan")
    turns = hq.rope_turns(hq.rope_freqs(32), DEV)
    out = hq.rope_write(r.cache, 0, 1, q, k, v, turns, ints(r.starts), 3, layout)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 0, 40] = want[1, 1, 63] = True
    pair = [2, 18] if layout == "half" else [2, 3]
    want[2, 0, pair] = True
    assert torch.equal(bad, want)
    page, slot = zip(*[r.place(0, i) for i in range(3)])
    assert (~torch.isfinite(r.cache.pool[0, list(page), :, list(slot)])).nonzero().tolist() == [[1, 0, 50]]
    assert (~torch.isfinite(r.cache.pool[1, list(page), :, list(slot)])).nonzero().tolist() == [[0, 0, 0]]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_norm_of_heads_of_any_size(D, eps):
    sizes = [0.0, 1e-44, 1e-38, 1e-30, 1e-20, 1e-12, 1.0, 1e10, 1e19, 1e25, 3e37]
    r = Rows([4], [len(sizes)], 2, 1, D, 16, F32, BF16, seed=13)
    scale = torch.tensor(sizes, device=DEV).view(-1, 1, 1)
    r.q, r.k = r.q.double().clamp(-5, 5).mul(scale).float(), r.k.double().clamp(-5, 5).mul(scale).float()
    turns, w = hq.rope_turns(hq.rope_freqs(D), DEV), torch.rand(D, device=DEV) + 0.5
    out = hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), len(sizes), q_weight=w, k_weight=w, eps=eps)
    check(r, out, turns, qw=w, kw=w, eps=float(np.float32(eps)))


def test_bad_places_are_skipped_and_reported():
    turns = hq.rope_turns(hq.rope_freqs(64), DEV)

    def run(change, seqs=None):
        r = Rows([20, 3, 9], [2, 2, 2], 2, 1, 64, 16, F32, F16, seed=14)
        change(r)
        out = torch.full((6, 2, 64), 7.0, dtype=F16, device=DEV)
        hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, ints(r.starts), 2, seqs=seqs, out=out)
        assert hq.pages_status(r.cache) == hq.HQ_ERR_INVALID_ARG
        assert hq.pages_status(r.cache) == hq.HQ_OK
        return r, [not bool((out[2 * b:2 * b + 2] == 7.0).all()) for b in range(3)], out
    assert run(lambda r: r.cache.lens[1:2].fill_(1))[1] == [True, True, True]  # one row of it has no place
    r, _, out = run(lambda r: r.cache.lens[1:2].fill_(1))
    assert bool((out[2] == 7.0).all())
    assert run(lambda r: r.cache.lens[1:2].fill_(-5))[1] == [True, False, True]
    assert run(lambda r: r.cache.lens[1:2].fill_(1 << 30))[1] == [True, False, True]
    assert run(lambda r: None, seqs=ints([0, 77, 2]))[1] == [True, False, True]
    assert run(lambda r: None, seqs=ints([0, -1, 2]))[1] == [True, False, True]
    for page in (-1, 1 << 20):
        r, wrote, _ = run(lambda r: r.cache.table[1].fill_(page))
        assert wrote == [True, True, True]  # q does not need the page
        at = [r.place(b, i) for b in (0, 2) for i in range(2)]
        pool = r.cache.pool.clone()
        for x in range(2):
            pool[x, [a[0] for a in at], :, [a[1] for a in at]] = r.old[x, [a[0] for a in at], :, [a[1] for a in at]]
        assert torch.equal(pool, r.old)


@pytest.mark.parametrize("starts", [[0, 4, 2, 6], [-3, 2, 4, 6], [0, 9, 9, 9], [5, 3, 1, 0], [7, 7, 7, 7]])
def test_starts_that_are_not_ascending_stay_in_bounds(starts):
    r = Rows([20, 3, 9], [2, 2, 2], 2, 1, 64, 16, F32, F16, seed=15)
    out = Guarded((6, 2, 64), F16, DEV, fill=7.0)
    hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, hq.rope_turns(hq.rope_freqs(64), DEV), ints(starts), 4, out=out.t)
    torch.cuda.synchronize()
    out.check()
    hq.pages_status(r.cache)
    assert torch.equal(r.cache.pool[2], r.old[2])


def test_a_captured_write_follows_its_inputs_and_streams():
    r = Rows([20, 3], [2, 3], 4, 2, 128, 16, F32, F16, seed=16, tree=True)
    turns, starts, parent = hq.rope_turns(hq.rope_freqs(128), DEV), ints(r.starts), ints(r.parent)
    out = torch.empty((5, 4, 128), dtype=F16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda **k: hq.rope_write(r.cache, 0, 1, r.q, r.k, r.v, turns, starts, 3, parent=parent, out=out, **k)  # noqa: E731
    call(stream=s)  # a stream that is not the current one
    s.synchronize()
    check(r, out, turns)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(flags=hq.HQ_LAUNCH_PDL)
    r.cache.pool.copy_(r.old)
    r.cache.lens[0] += 6
    r.before = [26, 3]
    graph.replay()
    torch.cuda.synchronize()
    check(r, out, turns)


def test_pages_and_rows_past_32_bits():
    """A pool of over 4 GB a plane, and input rows over 2^31 elements apart."""
    D, Hkv, ps, pages = 128, 8, 256, 9000  # 4.7 GB a plane
    pool = torch.empty((2, pages, Hkv, ps, D), dtype=BF16, device=DEV)
    table = torch.tensor([[pages - 1, pages - 2], [0, 1]], dtype=torch.int32, device=DEV)
    cache = hq.PagedCache(pool, torch.ones(pages, dtype=torch.int32, device=DEV), table, ints([300, 2]))
    wide = torch.empty(2 ** 31 + 64 * D, dtype=BF16, device=DEV)
    ld, R = 2 ** 30, 3
    parts = [wide.as_strided((R, h, D), (ld, D, 1), o * D) for o, h in ((0, 4), (4, Hkv), (4 + Hkv, Hkv))]
    g = torch.Generator(device=DEV).manual_seed(1)
    for t in parts:
        t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    turns = hq.rope_turns(hq.rope_freqs(D), DEV)
    out = hq.rope_write(cache, 0, 1, *parts, turns, ints([0, 1, 3]), 2)
    t = turns.cpu().numpy().view(np.uint64).tolist()
    pos = [299, 0, 1]
    close(out, *expected(parts[0], pos, t, "half", 1.0, None, 0.0))
    for i, (page, slot) in enumerate([(pages - 2, 299 - ps), (0, 0), (0, 1)]):
        close(pool[0, page, :, slot].unsqueeze(0), *expected(parts[1][i:i + 1], pos[i:i + 1], t, "half", 1.0, None, 0.0))
        assert torch.equal(pool[1, page, :, slot], parts[2][i])
    assert hq.pages_status(cache) == hq.HQ_OK
