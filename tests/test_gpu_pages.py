"""The page operations of the paged cache against a plain model: tables,
counts, lengths and every byte of the pool, exactly."""
import numpy as np
import pytest
import torch

from page_model import Bad, Full, PageModel
from quantized_speculative_verify_gb300 import hq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def keep_rows(keep, width=None):
    width = max([1] + [len(k) for k in keep if k is not None]) if width is None else width
    rows = torch.full((len(keep), width), -7, dtype=torch.int32)
    for i, k in enumerate(keep):
        if k:
            rows[i, :len(k)] = torch.tensor(k, dtype=torch.int32)
    return rows.to(DEV), ints([-1 if k is None else len(k) for k in keep])


class Pair:
    """The model and the GPU's cache, always compared whole."""

    def __init__(self, planes=2, pages=64, heads=2, ps=16, dim=64, seqs=8, max_pages=12, seed=0, flags=0):
        self.m = PageModel(planes, pages, heads, ps, dim, seqs, max_pages, seed)
        # planes further apart than they are large
        room = torch.zeros((planes, pages + 1, heads, ps, dim), dtype=torch.float16, device=DEV)
        room[:, :pages] = torch.from_numpy(self.m.pool.view(np.float16)).to(DEV)
        self.room = room
        self.guard = room[:, pages].clone()
        self.c = hq.PagedCache(room[:, :pages], torch.zeros(pages, dtype=torch.int32, device=DEV),
                               torch.full((seqs, max_pages), -1, dtype=torch.int32, device=DEV),
                               torch.zeros(seqs, dtype=torch.int32, device=DEV))
        self.flags = flags

    def check(self, status=hq.HQ_OK):
        assert hq.pages_status(self.c) == status
        assert self.c.ref.tolist() == self.m.ref
        assert self.c.table.tolist() == self.m.table
        assert self.c.lens.tolist() == self.m.len
        assert np.array_equal(self.c.pool.cpu().numpy().view(np.uint16), self.m.pool)
        assert torch.equal(self.room[:, -1], self.guard)

    def do(self, name, *args):
        """The operation on both; the GPU reports what the model raises."""
        want = hq.HQ_OK
        try:
            getattr(self.m, name)(*args)
        except Bad:
            want = hq.HQ_ERR_INVALID_ARG
        except Full:
            want = hq.HQ_ERR_NO_PAGES
        if name == "compact":
            keep, n = keep_rows(args[2])
            hq.pages_compact(self.c, ints(args[0]), ints(args[1]), keep, n, flags=self.flags)
        elif name == "write":
            kp, vp, seqs, starts, k, v = args
            f = [torch.from_numpy(x.view(np.float16)).to(DEV) for x in (k, v)]
            hq.pages_write(self.c, kp, vp, f[0], f[1], ints(starts), max([1] + [b - a for a, b in zip(starts, starts[1:])]),
                           seqs=ints(seqs), flags=self.flags)
        else:
            getattr(hq, "pages_" + name)(self.c, *[ints(a) for a in args], flags=self.flags)
        self.check(want)
        return want

    def rows(self, n, seed):
        rng = np.random.default_rng(seed)
        return (rng.integers(0, 2 ** 15, (n, self.m.pool.shape[2], self.m.pool.shape[4])).astype(np.uint16) & 0x7BFF)


def test_grow_fork_write_compact_free():
    p = Pair()
    p.do("extend", [0, 3], [37, 0])
    p.do("write", 0, 1, [0], [0, 37], p.rows(37, 1), p.rows(37, 2))
    p.do("fork", [0, 0], [1, 5])
    p.do("extend", [5, 1, 0], [4, 20, 1])        # three holders of the last page: each takes a copy
    p.do("write", 1, 0, [1, 5], [0, 20, 24], p.rows(24, 3), p.rows(24, 4))
    p.do("compact", [1, 5], [37, 37], [[3, 7, 19], [1]])   # rows 38.. kept: some move, some do not
    p.do("compact", [0], [-1], [list(range(2, 39, 2))])    # drops every other position: the shared pages are replaced
    p.do("free", [1])
    p.do("free", [1, 0, 5])                      # an empty slot among them
    assert p.m.ref == [0] * 64


def test_list_order_decides_which_pages_are_handed_out():
    p = Pair(pages=10, max_pages=6)
    p.do("extend", [4, 2], [17, 33])
    assert p.m.table[4][:2] == [0, 1] and p.m.table[2][:3] == [2, 3, 4]
    p.do("free", [4])
    p.do("extend", [2, 1], [48, 1])
    assert p.m.table[2][3:6] == [0, 1, 5] and p.m.table[1][0] == 6


def test_too_few_pages_changes_nothing():
    p = Pair(pages=5, max_pages=12)
    p.do("extend", [0], [30])
    p.do("fork", [0, 0], [1, 2])
    assert p.do("extend", [3, 4], [33, 16]) == hq.HQ_ERR_NO_PAGES
    assert p.do("extend", [3], [48]) == hq.HQ_OK
    assert p.do("extend", [1], [1]) == hq.HQ_ERR_NO_PAGES          # no page for the copy
    assert p.do("compact", [1], [-1], [[2, 5]]) == hq.HQ_ERR_NO_PAGES
    assert p.do("compact", [1], [3], [[]]) == hq.HQ_OK             # cutting off needs none


def test_bad_entries_change_nothing():
    p = Pair()
    p.do("extend", [0, 1], [40, 5])
    E = hq.HQ_ERR_INVALID_ARG
    assert p.do("extend", [0, 0], [1, 1]) == E
    assert p.do("extend", [8], [1]) == E and p.do("extend", [-1], [1]) == E
    assert p.do("extend", [2, 1], [1, -1]) == E
    assert p.do("extend", [2], [12 * 16 + 1]) == E
    assert p.do("extend", [2, 1], [1, 12 * 16 - 4]) == E
    assert p.do("fork", [0], [1]) == E                # not an empty slot
    assert p.do("fork", [0, 3], [3, 4]) == E          # a source that is a destination
    assert p.do("fork", [0, 0], [3, 3]) == E
    assert p.do("fork", [8], [3]) == E and p.do("fork", [0], [99]) == E
    assert p.do("free", [0, 0]) == E and p.do("free", [1, 8]) == E
    for b, k in ((0, [0]), (0, [2, 2]), (0, [3, 2]), (0, [40]), (38, [1, 2]), (-2, [1]), (40, []), (0, list(range(1, 41)))):
        assert p.do("compact", [1, 0], [2, b], [[1], k]) == E, (b, k)
    assert p.do("compact", [0, 0], [0, 0], [[1], [1]]) == E
    # an entry that is left out is not looked at
    assert p.do("compact", [0, 1], [99, 1], [None, [1, 3]]) == hq.HQ_OK


@pytest.mark.parametrize("ps,heads,dim,planes", [(16, 1, 8, 1), (32, 3, 64, 2), (64, 2, 128, 4), (128, 1, 72, 3), (256, 2, 64, 1)])
def test_random_operations(ps, heads, dim, planes):
    rng = np.random.default_rng(ps + dim)
    p = Pair(planes=planes, pages=40, heads=heads, ps=ps, dim=dim, seqs=9, max_pages=8, seed=ps, flags=hq.HQ_LAUNCH_PDL)
    seen = set()
    for step in range(60):
        op = rng.choice(["fork", "extend", "extend", "compact", "compact", "free", "write"])
        seqs = rng.permutation(9)[: rng.integers(1, 5)].tolist()
        if op == "fork":
            empty = [s for s in range(9) if p.m.len[s] == 0]
            if not empty:
                continue
            dst = empty[: rng.integers(1, len(empty) + 1)]
            r = p.do("fork", [int(s) for s in rng.choice([s for s in range(9) if s not in dst] or [0], len(dst))], dst)
        elif op == "extend":
            r = p.do("extend", seqs, [int(x) for x in rng.integers(0, 3 * ps, len(seqs))])
        elif op == "free":
            r = p.do("free", seqs[:1])
        elif op == "compact":
            live = [s for s in seqs if p.m.len[s]]
            if not live:
                continue
            base = [int(rng.integers(-1, p.m.len[s])) for s in live]
            keep = []
            for s, b in zip(live, base):
                room = p.m.len[s] - 1 - b
                n = int(rng.integers(0, room + 1))
                keep.append(sorted(int(x) + 1 for x in rng.permutation(room)[:n]) if rng.random() < 0.9 else None)
            r = p.do("compact", live, base, keep)
        else:
            live = [s for s in seqs if p.m.len[s]]
            n = [min(p.m.len[s], int(rng.integers(0, 20))) for s in live]
            # only pages of its own may be written
            n = [x if all(p.m.ref[p.m.table[s][q // ps]] == 1 for q in range(p.m.len[s] - x, p.m.len[s])) else 0
                 for s, x in zip(live, n)]
            starts = [0] + np.cumsum(n).astype(int).tolist()
            if starts[-1] == 0:
                continue
            r = p.do("write", 0, planes - 1, live, starts, p.rows(starts[-1], step), p.rows(starts[-1], step + 1)) \
                if planes > 1 else hq.HQ_OK
        seen.add((op, r))
    assert len(seen) >= 4


def test_many_sequences_and_long_lists():
    """1024 entries in one list; more pages than one pass of the scan; long kept lists."""
    p = Pair(planes=1, pages=6000, heads=1, ps=16, dim=8, seqs=1100, max_pages=300)
    p.do("extend", list(range(1000, 0, -1)), [(i * 7) % 90 for i in range(1000)])
    p.do("extend", [1050], [4700])
    p.do("fork", [1050, 1050], [1060, 1070])
    p.do("compact", [1060, 1050, 7], [5, -1, 0], [list(range(1, 2000, 2)), list(range(1, 4600)), []])
    p.do("compact", [1070], [1000], [list(range(1, 3000)) + [3100, 3200]])
    p.do("free", [s for s in range(1024)])


def test_rows_move_down_in_place_in_long_sequences():
    """A sequence that owns its pages: every row is read before it is overwritten."""
    p = Pair(planes=2, pages=80, heads=2, ps=32, dim=64, seqs=2, max_pages=80)
    p.do("extend", [1], [2500])
    p.do("compact", [1], [10], [list(range(2, 2489))])      # every row moves down by one
    p.do("compact", [1], [99], [list(range(1, 2400, 3))])


def test_pages_copy_and_bad_pairs():
    p = Pair(planes=3, pages=20, heads=2, ps=32, dim=128)
    p.do("copy", [0, 5, 7], [9, 2, 19])
    was = p.c.pool.clone()
    hq.pages_copy(p.c, ints([20, 1, -1]), ints([3, 25, 4]))
    assert hq.pages_status(p.c) == hq.HQ_ERR_INVALID_ARG and torch.equal(p.c.pool, was)
    assert hq.pages_status(p.c) == hq.HQ_OK


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_write_rounds_fp32_and_skips_what_is_not_there(dtype):
    c = hq.PagedCache.empty(2, 12, 3, 16, 64, 4, 4, dtype=dtype)
    hq.pages_extend(c, ints([0, 1, 2]), ints([20, 3, 16]))
    wide = torch.randn((10, 3 * 64 + 8), device=DEV)
    k, v = wide[:, :192].unflatten(1, (3, 64)), torch.randn((10, 3, 64), device=DEV).to(torch.float32)
    assert k.stride(0) == 200
    # sequence 1 has 3 positions and gets 4 rows: the first has no place; sequence 3 is empty
    hq.pages_write(c, 1, 0, k, v, ints([0, 4, 8, 9, 10]), 4)
    assert hq.pages_status(c) == hq.HQ_ERR_INVALID_ARG
    t, exp = c.table.tolist(), torch.zeros_like(c.pool)
    place = [(0, 16 + i, i) for i in range(4)] + [(1, i - 1, 4 + i) for i in range(1, 4)] + [(2, 15, 8)]
    for s, pos, r in place:
        exp[1, t[s][pos // 16], :, pos % 16] = k[r].to(dtype)
        exp[0, t[s][pos // 16], :, pos % 16] = v[r].to(dtype)
    assert torch.equal(c.pool, exp)
    # sequences outside the cache, and starts that are not ascending
    hq.pages_write(c, 0, 1, k, v, ints([0, 2, 4]), 2, seqs=ints([4, -1]))
    assert hq.pages_status(c) == hq.HQ_ERR_INVALID_ARG
    hq.pages_write(c, 0, 1, k, v, ints([5, 2, -3, 99]), 4, seqs=ints([0, 1, 2]))
    assert torch.equal(c.pool, exp) and hq.pages_status(c) == hq.HQ_OK
    # one row each, without starts
    hq.pages_write(c, 0, 1, k[:3].contiguous().to(dtype), v[:3].to(dtype), None, 1)
    assert hq.pages_status(c) == hq.HQ_OK
    assert torch.equal(c.pool[0, t[1][0], :, 2], k[1].to(dtype)) and torch.equal(c.pool[1, t[2][0], :, 15], v[2].to(dtype))


def test_corrupt_table_entries_stay_harmless():
    """Entries outside the pool inside a sequence's length are skipped by every operation."""
    p = Pair(pages=16)
    p.do("extend", [0, 1], [70, 70])
    for bad in (-5, 16, 2 ** 31 - 1, -2 ** 31):
        q = Pair(pages=16)
        q.do("extend", [0, 1], [70, 70])
        q.c.table[0, 1] = bad
        q.c.table[0, 4] = bad
        hq.pages_fork(q.c, ints([0]), ints([2]))
        hq.pages_extend(q.c, ints([2, 0]), ints([3, 1]))
        keep, n = keep_rows([list(range(2, 60))])
        hq.pages_compact(q.c, ints([0]), ints([0]), keep, n)
        hq.pages_free(q.c, ints([0, 2]))
        assert hq.pages_status(q.c) == hq.HQ_OK
        assert q.c.table[1].tolist() == q.m.table[1] and q.c.lens.tolist()[:3] == [0, 70, 0]
        own = [x for x in q.m.table[1] if x >= 0]
        assert all(int(q.c.ref[x]) == 1 for x in own)
        assert np.array_equal(q.c.pool[:, own].cpu().numpy().view(np.uint16), q.m.pool[:, own])
        assert torch.equal(q.room[:, -1], q.guard)


def test_one_verify_step_in_a_graph():
    """fork, extend, write and compact captured once, replayed on the cache's state."""
    p = Pair()
    p.do("extend", [0], [21])
    p.do("fork", [0], [1])
    seqs, add, base = ints([1]), ints([4]), ints([21])
    keep, n = keep_rows([[2, 3]])
    k = torch.randn((4, 2, 64), device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            hq.pages_extend(p.c, seqs, add, flags=hq.HQ_LAUNCH_PDL)
            hq.pages_write(p.c, 0, 1, k, k, None, 4, seqs=seqs, flags=hq.HQ_LAUNCH_PDL)
            hq.pages_compact(p.c, seqs, base, keep, n, flags=hq.HQ_LAUNCH_PDL)
    torch.cuda.synchronize()
    kh = k.half().cpu().numpy().view(np.uint16)
    for step in range(3):
        g.replay()
        torch.cuda.synchronize()
        p.m.extend([1], [4])
        p.m.write(0, 1, [1], [0, 4], kh, kh)
        p.m.compact([1], [21 + 3 * step], [[2, 3]])
        p.check()
        base += 3
        torch.cuda.synchronize()
