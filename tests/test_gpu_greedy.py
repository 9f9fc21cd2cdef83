"""Penalties, biases and masks on the logits with the greedy token of every row,
and the acceptance of a batch of trees.

The rules are fp32 operations that round once each, in a given order, so the
plain computation does the same in numpy's fp32 and every output has to be the
same bits (NaN as NaN).  An output in 16 bits is that value rounded.
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


def counters(ws, rows):
    """What calls leave in the workspace beside sorted histories: nothing (rows up to 256 have records of one size)."""
    one = hq.hq_greedy_tokens_workspace_bytes(1)
    return int(ws.view(-1)[:min(rows, 256) * one].view(-1, one)[:, :16].sum()) + int(ws[256 * one:].sum())


def path_of(parent, i):
    """Node i and its ancestors, without the root."""
    nodes = []
    while i > 0:
        nodes.append(i)
        if not 0 <= parent[i] < i:
            break
        i = parent[i]
    return nodes


class Request:
    """Everything about a batch in numpy, and its expected outputs."""

    def __init__(self, rows, V, seed=0, slots=None, n_slots=None, history=50, cap=None, dtype=F32, near=None):
        rng = np.random.default_rng(seed)
        self.rows, self.V, self.dtype = rows, V, dtype
        self.slots = list(range(len(rows))) if slots is None else slots
        self.n = n_slots or max(self.slots) + 1
        self.starts = [0] + np.cumsum(rows).tolist()
        R = self.starts[-1]
        near = min(V, near or max(1, V // 10))
        self.x = torch.from_numpy((3 * rng.standard_normal((R, V))).astype(np.float32)).to(dtype)
        cap = cap or history + 7
        self.text = rng.integers(0, near, (self.n, cap)).astype(np.int32)
        self.len = rng.integers(0, history + 1, self.n).astype(np.int32)
        self.prompt = (self.len * rng.uniform(0, 1.2, self.n)).astype(np.int32)
        self.draft = rng.integers(0, near, R).astype(np.int32)
        self.parent = np.zeros(R, dtype=np.int32)
        for b, m in enumerate(rows):
            for i in range(1, m):
                self.parent[self.starts[b] + i] = rng.integers(max(0, i - 3), i)
        self.rep = (1.0 + rng.uniform(0, 0.5, self.n)).astype(np.float32)
        self.pres, self.freq = (rng.uniform(-0.2, 0.8, self.n).astype(np.float32) for _ in range(2))
        self.bias = [[(int(rng.integers(0, V)), np.float32(4 * rng.standard_normal())) for _ in range(int(rng.integers(0, 40)))]
                     for _ in range(self.n)]
        words = (V + 31) // 32
        self.masks = rng.integers(0, 2 ** 32, (R + 1, words), dtype=np.uint64).astype(np.uint32)
        self.mask_ids = rng.integers(-1, R + 1, R).astype(np.int32)
        self.use = dict(rep=True, pres=True, freq=True, bias=True, mask=True, history=True, draft=True, prompt=True)

    def expect(self, b, i):
        """Adjusted logits and greedy token of row i of sequence b."""
        u, row, s, V = self.use, self.starts[b] + i, self.slots[b], self.V
        l = self.x[row].float().numpy().copy()
        there = 0 <= s < self.n
        n, seen = np.zeros(V, dtype=np.int64), np.zeros(V, dtype=bool)
        if u["history"] and there:
            k = int(np.clip(self.len[s], 0, self.text.shape[1]))
            t = self.text[s, :k]
            ok = (t >= 0) & (t < V)
            seen[t[ok]] = True
            late = ok & (np.arange(k) >= (self.prompt[s] if u["prompt"] else 0))
            np.add.at(n, t[late], 1)
        if u["draft"]:
            for j in path_of(self.parent[self.starts[b]:self.starts[b + 1]], i):
                t = self.draft[self.starts[b] + j]
                if 0 <= t < V:
                    seen[t] = True
                    n[t] += 1
        with np.errstate(all="ignore"):
            if u["rep"] and there:
                l = np.where(seen, np.where(l > 0, l / self.rep[s], l * self.rep[s]), l)
            if u["freq"] and there:
                l = np.where(n > 0, l - self.freq[s] * n.astype(np.float32), l)
            if u["pres"] and there:
                l = np.where(n > 0, l - self.pres[s], l)
            if u["bias"] and there:
                for t, v in dict(self.bias[s]).items():
                    if 0 <= t < V:
                        l[t] = l[t] + v
        assert l.dtype == np.float32
        allowed = np.ones(V, dtype=bool)
        m = self.mask_ids[row] if self.mask_ids is not None else row
        if u["mask"] and 0 <= m < self.masks.shape[0]:
            allowed = (self.masks[m][np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32) & 1).astype(bool)
        l = np.where(allowed, l, np.float32(-np.inf))
        where = np.flatnonzero(allowed)
        if not len(where):
            return l, -1
        nan = where[np.isnan(l[where])]
        return l, int(nan[0] if len(nan) else where[np.argmax(l[where])])

    def device(self):
        u = self.use
        d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        self.history = hq.History(d(self.text), d(self.len), d(self.prompt) if u["prompt"] else None) if u["history"] else None
        starts = np.cumsum([0] + [len(x) for x in self.bias]).astype(np.int32)
        toks = np.array([t for x in self.bias for t, _ in x], dtype=np.int32)
        vals = np.array([v for x in self.bias for _, v in x], dtype=np.float32)
        self.rules = hq.LogitRules(self.n, d(self.rep) if u["rep"] else None, d(self.pres) if u["pres"] else None,
                                   d(self.freq) if u["freq"] else None, (d(starts), d(toks), d(vals)) if u["bias"] else None,
                                   d(self.masks.view(np.int32)) if u["mask"] else None)
        return dict(starts=ints(self.starts), max_rows=max(max(self.rows), 1), parent=d(self.parent),
                    tokens=d(self.draft) if u["draft"] else None, seqs=ints(self.slots), history=self.history, rules=self.rules,
                    mask_ids=d(self.mask_ids) if self.mask_ids is not None else None)

    def run(self, out_type=None, pad=0, lead=0, opad=0, in_place=False):
        R, V = self.x.shape
        wide = torch.full((R * (V + pad) + lead,), 9.0, dtype=self.dtype, device=DEV)
        x = wide[lead:].view(R, V + pad)[:, :V]
        x.copy_(self.x)
        out = None
        if in_place:
            out = x
        elif out_type is not None:
            out = torch.full((R, V + opad), 7.0, dtype=out_type, device=DEV)[:, :V]
        greedy, ws = Guarded((R,), torch.int32, DEV, fill=-9), torch.zeros(hq.hq_greedy_tokens_workspace_bytes(R), dtype=torch.uint8, device=DEV)
        kw = self.device()
        hq.greedy_tokens(x, kw.pop("starts"), kw.pop("max_rows"), out=out, greedy=greedy.t, workspace=ws, **kw)
        torch.cuda.synchronize()
        greedy.check()
        assert counters(ws, R) == 0
        self.check(greedy.t, out)
        if pad:
            assert bool((wide[lead:].view(R, V + pad)[:, V:] == 9.0).all())

    def check(self, greedy, out):
        greedy = greedy.tolist()
        for b, m in enumerate(self.rows):
            for i in range(m):
                l, g = self.expect(b, i)
                assert greedy[self.starts[b] + i] == g, (b, i)
                if out is not None:
                    got, want = out[self.starts[b] + i].cpu(), torch.from_numpy(l).to(out.dtype)
                    assert torch.equal(torch.isnan(got), torch.isnan(want)), (b, i)
                    assert torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)]), (b, i)


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 32, 33, 127, 1000, 1023, 1024, 1025, 4099, 20000, 50257])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_every_rule_at_odd_vocabularies(V, dtype):
    Request([3, 1, 5], V, seed=V, slots=[2, 0, 4], n_slots=5, dtype=dtype).run(out_type=dtype)


@pytest.mark.parametrize("rows,V,history", [([1], 151552, 300), ([16] * 8, 12345, 2000), ([1] * 128, 9000, 100), ([128], 3001, 50),
                                            ([127, 0, 4, 0], 7777, 900), ([1], 16384 * 41 + 5, 40000), ([2] * 40, 70001, 20)])
def test_shapes(rows, V, history):
    r = Request(rows, V, seed=len(rows) + V, history=history)
    r.run()
    r.run(out_type=F32)


@pytest.mark.parametrize("off", ["rep", "pres", "freq", "bias", "mask", "history", "draft", "prompt"])
def test_without_one_of_the_rules(off):
    r = Request([4, 2], 3333, seed=5)
    r.use[off] = False
    r.run(out_type=F32)
    r = Request([4, 2], 3333, seed=6)
    for k in ("rep", "pres", "freq", "bias", "mask"):  # that rule alone
        r.use[k] = k == off
    r.run(out_type=F32)


def test_no_rules_is_the_greedy_token_of_tree_accept():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((20, 151553), generator=g, device=DEV)
    x[3, 77] = x[3, 100000] = 50.0
    x[4, 9], x[4, 5000] = float("nan"), float("inf")
    x[5] = -float("inf")
    x[6] = 0.0
    x[6, ::2] = -0.0
    got = hq.greedy_tokens(x, None, 1)
    parent = torch.zeros(20, dtype=torch.int32, device=DEV)
    want, _, _ = hq.tree_accept(x, parent, parent)
    assert torch.equal(got, want) and got[3:7].tolist() == [77, 9, 0, 0]


@pytest.mark.parametrize("dtype,out,pad,lead,opad", [(F32, F32, 1, 0, 0), (F32, F32, 3, 1, 2), (F16, F32, 5, 3, 1), (F16, F16, 2, 2, 0),
                                                      (BF16, BF16, 7, 1, 8), (BF16, F32, 0, 0, 4), (F32, None, 2, 3, 0), (F32, F32, 4, 0, 4)])
def test_strides_and_any_alignment(dtype, out, pad, lead, opad):
    Request([2, 5], 5003, seed=7, dtype=dtype).run(out_type=out, pad=pad, lead=lead, opad=opad)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_past_32_bits(dtype):
    r = Request([1, 2], 5000, seed=25, dtype=dtype)
    ld = 2 ** 30 + 3
    wide = torch.empty(2 * ld + 5000, dtype=dtype, device=DEV)
    x = wide.as_strided((3, 5000), (ld, 1))
    x.copy_(r.x)
    kw = r.device()
    greedy = hq.greedy_tokens(x, kw.pop("starts"), kw.pop("max_rows"), out=x, **kw)
    r.check(greedy, x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(dtype):
    Request([2, 5], 5003, seed=8, dtype=dtype).run(in_place=True)
    Request([2, 5], 5004, seed=8, dtype=dtype).run(in_place=True, pad=4)


def test_rows_whose_mask_leaves_nothing_or_little():
    r = Request([3, 3], 2049, seed=9)
    r.mask_ids = np.arange(6, dtype=np.int32)
    r.masks[0] = 0
    r.masks[1] = 0
    r.masks[1, 64] = 1  # the last token alone
    r.masks[2] = 0
    r.masks[2, 0] = 1
    r.masks[3] = 0xFFFFFFFF
    r.x[1, 2048] = -float("inf")  # allowed, and the only one
    r.run(out_type=F32)
    r = Request([3, 3], 2048, seed=9)
    r.mask_ids = None  # row r has mask r
    r.masks = r.masks[:4]  # rows 4 and 5 have none
    r.masks[3] = 0
    r.run(out_type=F32)


@pytest.mark.parametrize("V", [1500, 6001])
def test_nan_infinities_and_the_lowest_values(V):
    r = Request([4, 4], V, seed=10)
    low = torch.finfo(F32).min
    r.x[0, ::3], r.x[1, ::2], r.x[2, 5:] = float("nan"), float("inf"), -float("inf")
    r.x[3] = low
    r.x[4] = float("nan")
    r.x[5, V - 1] = float("nan")
    r.x[6] = -float("inf")
    r.rep[0] = 3.0
    r.run(out_type=F32)


def test_ties_go_to_the_lowest_token():
    r = Request([2, 2], 9000, seed=11)
    r.x = torch.round(r.x * 0.5).float()
    r.rep[:] = 2.0
    r.pres[:] = r.freq[:] = 1.0
    r.bias = [[(t, np.float32(round(float(v)))) for t, v in x] for x in r.bias]
    r.run(out_type=F32)


def test_a_chain_without_parents_and_tokens_without_a_history():
    r = Request([5, 1, 7], 900, seed=23)
    r.parent = np.array([max(0, i - 1) for m in r.rows for i in range(m)], dtype=np.int32)
    kw = r.device()
    kw["parent"] = None
    x = r.x.to(DEV)
    greedy = hq.greedy_tokens(x, kw.pop("starts"), kw.pop("max_rows"), **kw)
    r.check(greedy, None)
    r.use["history"] = r.use["mask"] = False  # drafted tokens alone
    kw = r.device()
    kw["parent"] = None
    r.check(hq.greedy_tokens(x, kw.pop("starts"), kw.pop("max_rows"), **kw), None)


def test_buffers_that_a_call_makes_say_nothing_of_rows_without_a_sequence():
    x = torch.randn((5, 300), device=DEV)
    assert hq.greedy_tokens(x, ints([0, 2]), 2)[2:].tolist() == [-1, -1, -1]
    assert hq.greedy_tokens(x, ints([0]), 1).tolist() == [-1] * 5


def test_more_biases_in_a_chunk_than_are_held_there():
    r = Request([2, 1], 3000, seed=24)
    rng = np.random.default_rng(3)
    r.bias[0] = [(int(t), np.float32(v)) for t, v in zip(rng.integers(0, 3000, 2500), rng.standard_normal(2500) * 4)]
    r.run(out_type=F32)


def test_tokens_outside_the_vocabulary_and_bad_lengths_and_slots():
    r = Request([4, 3, 2, 2, 2], 700, seed=12, slots=[0, 1, 2, 9, -1], n_slots=4, history=60)
    r.text[0, ::3], r.text[1, ::2] = -1, 700
    r.text[1, 1] = np.iinfo(np.int32).min
    r.draft[1], r.draft[5] = -5, 2 ** 31 - 1
    r.bias[0] += [(-1, np.float32(9)), (700, np.float32(9)), (2 ** 31 - 1, np.float32(9))]
    r.len[0], r.len[1], r.len[2] = 10 ** 6, -3, r.text.shape[1]
    r.prompt[2] = -4
    r.run(out_type=F32)


def test_of_a_token_biased_twice_the_last_entry_counts():
    r = Request([2], 5000, seed=13, n_slots=1)
    r.bias[0] = [(4000, np.float32(30)), (17, np.float32(1)), (4000, np.float32(-2)), (4000, np.float32(25)), (17, np.float32(3))] * 3
    r.mask_ids[:] = -1
    r.run(out_type=F32)


def test_bias_starts_that_do_not_fit_give_none():
    r = Request([1, 1, 1], 900, seed=14)
    r.use["mask"] = False
    kw = r.device()
    n = int(r.rules.bias[0][-1])
    for bad in ([0, -1, 3, n], [0, n + 1, n + 2, n], [0, 5, 2, n]):
        r.rules.bias[0].copy_(ints(bad))
        s = list(r.bias)
        flat = [e for x in s for e in x]
        r.bias = [flat[lo:hi] if 0 <= lo <= hi <= n else [] for lo, hi in zip(bad, bad[1:])]
        x = r.x.to(DEV)
        greedy = hq.greedy_tokens(x, kw["starts"], 1, **{k: v for k, v in kw.items() if k not in ("starts", "max_rows")})
        r.check(greedy, None)
        r.bias = s


@pytest.mark.parametrize("history", [1000, 16384, 20000, 40000])
def test_long_histories_of_many_requests(history):
    """Histories long enough to be sorted first, and longer than what is sorted; the workspace of the larger calls serves the smaller."""
    ws = torch.zeros(hq.hq_greedy_tokens_workspace_bytes(64), dtype=torch.uint8, device=DEV)
    for rows, V in (([1] * 64, 30011), ([3] * 5, 9000), ([1] * 64, 131073)):
        r = Request(rows, V, seed=history + V, history=history, near=V // 3, slots=[2 * b for b in range(len(rows))][::-1])
        r.len[::3] = min(history, r.text.shape[1])
        x, kw = r.x.to(DEV), r.device()
        greedy = hq.greedy_tokens(x, kw.pop("starts"), kw.pop("max_rows"), workspace=ws, **kw)
        r.check(greedy, None)
        assert counters(ws, 64) == 0


def test_rows_that_no_sequence_claims_are_left():
    r = Request([2, 3], 2000, seed=15)
    kw = r.device()
    x = torch.cat([r.x, r.x[:2]]).to(DEV)
    out, greedy = torch.full((7, 2000), 7.0, device=DEV), torch.full((7,), -9, dtype=torch.int32, device=DEV)
    pad = lambda t: torch.cat([t, t[:2]])  # noqa: E731
    hq.greedy_tokens(x, kw["starts"], 3, pad(kw["parent"]), pad(kw["tokens"]), kw["seqs"], r.history, r.rules, pad(kw["mask_ids"]),
                     out=out, greedy=greedy)
    r.check(greedy, out)
    assert greedy[5:].tolist() == [-9, -9] and bool((out[5:] == 7.0).all())
    # nor are those past max_rows
    greedy.fill_(-9)
    hq.greedy_tokens(x, kw["starts"], 2, pad(kw["parent"]), pad(kw["tokens"]), kw["seqs"], r.history, r.rules, pad(kw["mask_ids"]), greedy=greedy)
    assert int(greedy[4]) == -9 and int(greedy[3]) >= 0


@pytest.mark.parametrize("starts", [[0, 4, 2, 6], [-3, 2, 4, 6], [0, 9, 9, 9], [5, 3, 1, 0]])
def test_starts_that_are_not_ascending_leave_the_workspace_usable(starts):
    r = Request([2, 2, 2], 40000, seed=16)
    kw = r.device()
    x, ws = r.x.to(DEV), torch.zeros(hq.hq_greedy_tokens_workspace_bytes(6), dtype=torch.uint8, device=DEV)
    greedy = Guarded((6,), torch.int32, DEV, fill=-9)
    kw.pop("starts"), kw.pop("max_rows")
    hq.greedy_tokens(x, ints(starts), 4, greedy=greedy.t, workspace=ws, **kw)
    torch.cuda.synchronize()
    greedy.check()
    assert counters(ws, 6) == 0
    hq.greedy_tokens(x, ints(r.starts), 2, greedy=greedy.t, workspace=ws, **kw)
    r.check(greedy.t, None)


def test_a_captured_call_with_long_histories():
    """Two kernels: the histories sorted by token, then the logits."""
    rows, V, ws = [1] * 64, 60000, torch.zeros(hq.hq_greedy_tokens_workspace_bytes(64), dtype=torch.uint8, device=DEV)
    r = Request(rows, V, seed=21, history=15000, near=V)
    kw = r.device()
    starts, _ = kw.pop("starts"), kw.pop("max_rows")
    x, greedy = r.x.to(DEV), torch.empty(64, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hq.greedy_tokens(x, starts, 1, greedy=greedy, workspace=ws, stream=s, **kw)
    s.synchronize()
    r.check(greedy, None)
    for flags in (hq.HQ_LAUNCH_DEFAULT, hq.HQ_LAUNCH_PDL):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(2):  # the second sorts into what the first has read
                hq.greedy_tokens(x, starts, 1, greedy=greedy, workspace=ws, flags=flags, **kw)
        n = Request(rows, V, seed=22 + flags, history=15000, near=V)
        r.len, r.text = n.len, n.text
        r.history.lens.copy_(torch.from_numpy(n.len))
        r.history.tokens.copy_(torch.from_numpy(n.text))
        graph.replay()
        torch.cuda.synchronize()
        r.check(greedy, None)
        assert counters(ws, 64) == 0


def test_a_captured_call_follows_its_inputs_and_streams():
    r = Request([3, 4], 30000, seed=17)
    kw = r.device()
    starts, _ = kw.pop("starts"), kw.pop("max_rows")
    x, ws = r.x.to(DEV), torch.zeros(hq.hq_greedy_tokens_workspace_bytes(7), dtype=torch.uint8, device=DEV)
    out, greedy = torch.empty_like(x), torch.empty(7, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mine = hq.greedy_tokens(x, starts, 4, stream=s, **kw)  # buffers of its own on another stream
    s.synchronize()
    r.check(mine, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.greedy_tokens(x, starts, 4, out=out, greedy=greedy, workspace=ws, flags=hq.HQ_LAUNCH_PDL, **kw)
    for seed in (18, 19):
        n = Request([3, 4], 30000, seed=seed)
        r.x, r.len, r.text = n.x, n.len, n.text
        x.copy_(n.x)
        r.history.lens.copy_(torch.from_numpy(n.len))
        r.history.tokens.copy_(torch.from_numpy(n.text))
        graph.replay()
        torch.cuda.synchronize()
        r.check(greedy, out)


# --------------------------------------------------------------- acceptance ---
def accept(greedy, parent, tokens):
    """Accepted path, their number and the bonus token of one tree; None if it is none."""
    m = len(greedy)
    if m == 0 or any(not 0 <= parent[i] < i for i in range(1, m)):
        return None
    depth, valid = [0] * m, [True] * m
    for i in range(1, m):
        depth[i] = depth[parent[i]] + 1
        valid[i] = valid[parent[i]] and greedy[parent[i]] >= 0 and tokens[i] == greedy[parent[i]]
    best = max(range(m), key=lambda i: (depth[i] if valid[i] else -1, -i))
    path, i = [], best
    while i:
        path.append(i)
        i = parent[i]
    return path[::-1], depth[best], greedy[best]


class Trees:
    def __init__(self, rows, seed, chain=False, agree=0.8, cap=400):
        rng = np.random.default_rng(seed)
        self.rows, self.starts = rows, [0] + np.cumsum(rows).tolist()
        R = self.starts[-1]
        self.greedy, self.tokens = (rng.integers(0, 1000, R).astype(np.int32) for _ in range(2))
        self.parent = np.zeros(R, dtype=np.int32)
        for b, m in enumerate(rows):
            for i in range(1, m):
                p = i - 1 if chain else int(rng.integers(max(0, i - 4), i))
                self.parent[self.starts[b] + i] = p
                if rng.random() < agree:
                    self.greedy[self.starts[b] + p] = self.tokens[self.starts[b] + i]
        self.text = rng.integers(0, 1000, (len(rows) + 3, cap)).astype(np.int32)
        self.len = rng.integers(0, 200, len(rows) + 3).astype(np.int32)

    def expect(self, b):
        lo, hi = self.starts[b], self.starts[b + 1]
        return accept(self.greedy[lo:hi].tolist(), self.parent[lo:hi].tolist(), self.tokens[lo:hi].tolist())

    def run(self, slots=None, parent=True, history=True, max_rows=None, ld=None, **kw):
        d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        B, m = len(self.rows), max_rows or max(max(self.rows), 1)
        h = hq.History(d(self.text), d(self.len)) if history else None
        path = Guarded((B, ld or m), torch.int32, DEV, fill=-7)
        n, bonus = Guarded((B,), torch.int32, DEV, fill=-7), Guarded((B,), torch.int32, DEV, fill=-7)
        hq.tree_accept_batch(d(self.greedy), d(self.parent) if parent else None, d(self.tokens), ints(self.starts), m,
                             seqs=None if slots is None else ints(slots), history=h, path=path.t, n_accept=n.t, bonus=bonus.t, **kw)
        torch.cuda.synchronize()
        for t in (path, n, bonus):
            t.check()
        return path.t.tolist(), n.t.tolist(), bonus.t.tolist(), h

    def check(self, got, slots=None, m=None, skipped=()):
        path, n, bonus, h = got
        m = m or max(max(self.rows), 1)
        text, lens = self.text.copy(), self.len.copy()
        for b in range(len(self.rows)):
            e = self.expect(b)
            s = b if slots is None else slots[b]
            if e is None:
                assert (n[b], bonus[b]) == (-1, -1) and path[b][:m] == [-1] * m
                continue
            assert (path[b][:m], n[b], bonus[b]) == (e[0] + [-1] * (m - e[1]), e[1], e[2]), b
            assert path[b][m:] == [-7] * (len(path[b]) - m)
            if b in skipped or h is None:
                continue
            more = [self.tokens[self.starts[b] + i] for i in e[0]] + ([e[2]] if e[2] >= 0 else [])
            text[s, lens[s]:lens[s] + len(more)] = more
            lens[s] += len(more)
        if h is not None:
            assert np.array_equal(h.tokens.cpu().numpy(), text) and np.array_equal(h.lens.cpu().numpy(), lens)
            assert hq.history_status(h) == (hq.HQ_ERR_INVALID_ARG if skipped else hq.HQ_OK)
            assert hq.history_status(h) == hq.HQ_OK


@pytest.mark.parametrize("rows", [[1], [16], [2, 1, 3], [128], [127, 128, 1, 64, 33, 32, 31], [5, 0, 9, 0], list(range(60))])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("agree", [0.0, 0.8, 1.0])
def test_acceptance_of_a_batch(rows, chain, agree):
    t = Trees(rows, seed=len(rows) + sum(rows), chain=chain, agree=agree)
    t.check(t.run())
    t.check(t.run(parent=not chain, history=False))
    slots = (np.arange(len(rows))[::-1] + 2).tolist()
    t.check(t.run(slots=slots, ld=max(rows) + 5), slots=slots)


def test_acceptance_is_that_of_each_tree_alone():
    V, M = 300, 40
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((M, V), generator=g, device=DEV)
    greedy = hq.greedy_tokens(x, None, M)
    t = Trees([M], seed=4)
    t.greedy = greedy.cpu().numpy()
    for i in range(1, M):
        if i % 5:
            t.tokens[i] = t.greedy[t.parent[i]]
    path, n, bonus, _ = t.run(history=False)
    g1, p1, out = hq.tree_accept(x, torch.from_numpy(t.parent).to(DEV), torch.from_numpy(t.tokens).to(DEV))
    assert torch.equal(g1, greedy) and path[0] == p1.tolist() and [n[0], bonus[0]] == out.tolist() and n[0] > 0


def test_malformed_trees_and_negative_greedy_tokens():
    t = Trees([6, 6, 6, 6, 6], seed=5, agree=1.0)
    t.parent[6 * 1 + 3], t.parent[6 * 2 + 2], t.parent[6 * 3 + 5] = 3, -1, 100
    t.parent[0] = t.parent[24] = 77  # a root's is not read
    t.greedy[24:] = -1
    t.tokens[24:] = -1  # equal, and still not accepted
    t.check(t.run())


def test_histories_that_do_not_fit_stay_as_they_are():
    t = Trees([4, 4, 4, 4, 4], seed=6, agree=1.0, chain=True, cap=50)
    t.len[:] = 5
    t.len[0], t.len[1], t.len[2], t.len[3] = 50 - 4, 50 - 3, -1, 51
    t.check(t.run(), skipped=(1, 2, 3))
    slots = [1, 99, -2, 1, 4]  # a slot outside, and one listed twice
    t.len[:] = 5
    t.check(t.run(slots=slots), slots=slots, skipped=(1, 2, 3))


def test_a_batch_without_rows_and_without_sequences():
    t = Trees([0, 0], seed=7)
    path, n, bonus, h = t.run()
    assert n == bonus == [-1, -1] and path == [[-1], [-1]]
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    path, n, bonus = hq.tree_accept_batch(z, None, z, ints([0]), 4)
    assert path.shape == (0, 4) and n.shape == (0,)


@pytest.mark.parametrize("starts", [[0, 4, 2, 6], [-3, 2, 4, 6], [0, 9, 9, 9], [5, 3, 1, 0]])
def test_acceptance_with_starts_that_are_not_ascending_stays_in_bounds(starts):
    t = Trees([2, 2, 2], seed=8)
    t.starts = starts
    t.run(max_rows=4)


def test_captured_acceptance_grows_the_histories_each_time():
    t = Trees([5, 9], seed=9)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    greedy, parent, tokens, starts = d(t.greedy), d(t.parent), d(t.tokens), ints(t.starts)
    h = hq.History(d(t.text), d(t.len))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = hq.tree_accept_batch(greedy, parent, tokens, starts, 9, stream=s)
    s.synchronize()
    assert [got[1].tolist(), got[2].tolist()] == [[t.expect(b)[1] for b in range(2)], [t.expect(b)[2] for b in range(2)]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.tree_accept_batch(greedy, parent, tokens, starts, 9, history=h, flags=hq.HQ_LAUNCH_PDL)
    for k in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert h.lens[:2].tolist() == [int(t.len[b]) + k * (t.expect(b)[1] + 1) for b in range(2)]
    assert hq.history_status(h) == hq.HQ_OK
