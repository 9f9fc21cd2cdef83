"""Greedy tokens on each way through the kernel that a launch takes: one, two or
four rows of a sequence to a block, histories sorted by a kernel in front or not,
adjusted logits kept or not; and biases in any number.

Which way a call takes follows from its sizes; `way` states the rule again, so
that every case says what it is for.  Results are compared bit for bit with the
same rules in numpy's fp32.
"""
import numpy as np
import pytest
import torch

from quantized_speculative_verify_gb300 import hq
from test_gpu_greedy import BF16, DEV, F16, F32, Request, counters

pytestmark = pytest.mark.gpu


def way(rows, V, room):
    """Tokens of a chunk, rows of a block, and whether histories in rooms of `room` tokens are sorted."""
    B, m, sms = len(rows), max(rows), torch.cuda.get_device_properties(0).multi_processor_count
    chunk, group = 1024, 1
    while chunk < 4096 and B * m * -(-V // (2 * chunk)) >= 4 * sms:
        chunk *= 2
    chunks = -(-V // chunk)
    while group < 4 and group < m and B * -(-m // group) * chunks > 16 * sms:
        group *= 2
    return chunk, group, chunks < 64 and B <= 256 and 4 * min(room, 16384) * B * -(-m // group) * chunks > 12 << 20


WAYS = [  # rows, V, history, chunk, rows a block, sorted
    ([16, 9, 15, 2, 13, 16, 1, 7], 151551, 50, 4096, 2, False),   # groups of two and one, chunks that end early
    ([16, 9, 15, 2, 13, 16, 1, 7], 151551, 9000, 4096, 2, True),
    ([7, 6, 5, 4, 3, 2, 1, 0] * 8, 40963, 300, 4096, 4, False),   # groups of four, three, two and one; a last chunk of three
    ([7, 6, 5, 4, 3, 2, 1, 0] * 8, 40963, 3000, 4096, 4, True),
    ([1] * 128, 50257, 4000, 4096, 1, True),
    ([3, 1, 2] * 20, 30011, 17000, 4096, 1, True),                # more than what is sorted
]


@pytest.mark.parametrize("rows,V,history,chunk,group,sort", WAYS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_way_with_and_without_the_logits_kept(rows, V, history, chunk, group, sort, dtype):
    assert way(rows, V, history + 7) == (chunk, group, sort)
    r = Request(rows, V, seed=V + history, history=history, dtype=dtype, near=V // 3)
    r.len[::3] = history
    r.run()
    r.run(out_type=dtype, pad=V % 2, opad=1)  # rows of a block that start at other alignments
    r.run(in_place=True, lead=1, pad=5)


@pytest.mark.parametrize("rows,V,history,chunk,group,sort", WAYS[:4])
def test_groups_with_16_bit_logits_kept_in_fp32(rows, V, history, chunk, group, sort):
    assert way(rows, V, history + 7) == (chunk, group, sort)
    Request(rows, V, seed=V - history, history=history, dtype=F16, near=500).run(out_type=F32, lead=3, opad=2)


def test_groups_without_rules_or_with_masks_alone():
    rows, V = [16, 9, 15, 2, 13, 16, 1, 7], 151551
    for mask in (False, True):
        r = Request(rows, V, seed=31)
        r.use = dict.fromkeys(r.use, False)
        r.use["mask"] = mask
        r.run(out_type=F32, pad=1)


def test_groups_whose_rows_are_masked_out_or_not_finite():
    rows, V = [7, 6, 5, 4, 3, 2, 1, 0] * 8, 40963
    assert way(rows, V, 3007) == (4096, 4, True)
    r = Request(rows, V, seed=32, history=3000)
    R = r.starts[-1]
    r.mask_ids = np.arange(R, dtype=np.int32)
    r.masks[::5] = 0
    r.masks[1::5] = 0xFFFFFFFF
    r.x[2::7, ::9] = float("nan")
    r.x[3::7, 5::11] = float("inf")
    r.x[4::7] = -float("inf")
    r.x[6::7] = torch.finfo(F32).min
    r.run(out_type=F32)


@pytest.mark.parametrize("B,V,history,room,sort", [
    (1, 32000, 500, 131072, False),   # one request in a large room: 2 MB of what would be sorted
    (4, 32000, 16384, 131072, False),
    (64, 32000, 500, 131072, True),   # by the room
    (64, 32000, 500, 507, False),
    (64, 32000, 4000, 4000, True),
    (128, 258048, 300, 20000, True),  # 63 chunks
    (128, 258049, 300, 20000, False),
    (257, 20000, 300, 20000, False),
])
def test_which_calls_sort(B, V, history, room, sort):
    """The sorted histories stay in the workspace, so a call that does not sort leaves it as it was, all zeros."""
    assert way([1] * B, V, room)[2] == sort
    g = torch.Generator(device=DEV).manual_seed(B)
    tokens = torch.randint(0, V, (B, room), generator=g, device=DEV).to(torch.int32)
    lens = torch.full((B,), history, dtype=torch.int32, device=DEV)
    rules = hq.LogitRules(B, presence=torch.full((B,), 100.0, device=DEV))
    x = torch.randn((B, V), generator=g, device=DEV)
    ws = torch.zeros(hq.hq_greedy_tokens_workspace_bytes(B), dtype=torch.uint8, device=DEV)
    greedy = hq.greedy_tokens(x, None, 1, history=hq.History(tokens, lens), rules=rules, workspace=ws)
    said = torch.zeros((B, V), dtype=torch.bool, device=DEV).scatter_(1, tokens[:, :history].long(), True)
    assert torch.equal(greedy.long(), torch.where(said, x - 100.0, x).argmax(1))
    assert counters(ws, B) == 0 and bool(ws.any()) == sort


@pytest.mark.parametrize("V,n", [(3000, 128), (3000, 129), (3000, 300), (151552, 300), (151552, 5000), (20011, 40000), (151553, 151553)])
def test_many_biases(V, n):
    """Next to one another, spread, several to a token, one for every token; of a token listed again the last one counts."""
    r = Request([3, 1, 2], V, seed=n, n_slots=3)
    rng = np.random.default_rng(n)
    first = int(rng.integers(0, V - min(n, V) + 1))
    near = first + rng.permutation(min(n, V))
    r.bias[0] = [(int(t), np.float32(v)) for t, v in zip(near, rng.standard_normal(len(near)) * 4)]
    far = rng.integers(-2, V + 2, n)
    r.bias[1], r.bias[2] = [], [(int(t), np.float32(v)) for t, v in zip(far, rng.standard_normal(n) * 4)] if n > 129 else []
    r.run(out_type=F32)
    r.run()


def test_many_biases_in_groups():
    rows, V = [7, 6, 5, 4, 3, 2, 1, 0] * 8, 40963
    r = Request(rows, V, seed=35, history=3000)
    rng = np.random.default_rng(36)
    for s in range(0, 64, 9):
        r.bias[s] = [(int(t), np.float32(v)) for t, v in zip(rng.integers(0, V, 2000), rng.standard_normal(2000) * 4)]
        r.bias[s] += [(int(t), np.float32(v)) for t, v in zip(4096 + rng.integers(0, 300, 600), rng.standard_normal(600) * 4)]
    r.run(out_type=F32)
    assert way(rows, V, 3007) == (4096, 4, True)


def test_the_work_for_a_bias_does_not_grow_with_the_list():
    """A bias for every token of a large vocabulary: each block reads the list twice, a third of a millisecond.  A walk through
    the list for each token took 70."""
    V = 151552
    x = torch.randn((1, V), device=DEV)
    ints = dict(dtype=torch.int32, device=DEV)
    tokens, values = torch.randperm(V, device=DEV).to(torch.int32), torch.randn(V, device=DEV)
    rules = hq.LogitRules(1, bias=(torch.tensor([0, V], **ints), tokens, values))
    ws = torch.zeros(hq.hq_greedy_tokens_workspace_bytes(1), dtype=torch.uint8, device=DEV)
    greedy = torch.empty(1, **ints)
    want = x[0].clone()
    want[tokens.long()] += values
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        hq.greedy_tokens(x, None, 1, rules=rules, greedy=greedy, workspace=ws)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    assert int(greedy[0]) == int(want.argmax()) and counters(ws, 1) == 0
    assert min(times) < 1.0, times  # ms
