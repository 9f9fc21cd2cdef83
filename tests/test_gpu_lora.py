"""Low-rank adapters of many requests, against a plain computation in 64 bits.

Tolerance.  The products are exact and each sum is formed in fp32: t = A x adds
K products (per warp in steps of the tensor cores, then 64 partial sums), B t
adds 3 r.  A tensor-core step may truncate: one unit of 2^-23 of the largest
magnitude per step of 16.  With n = K / 16 / 64 + 6 + 64 additions in the
longest chain of t and 3 r / 16 + 8 in that of B t, the result is within
2^-22 * (n + 3 r / 16 + 8) of sum_j |B| sum_k |A| |x| times the scale, and the
last addition rounds once more.
"""
import pytest
import torch

from guard import Guarded
from quantized_speculative_verify_gb300 import hq

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def make(M, K, N, n, r, xt, wt, seed, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.nn.functional.pad(torch.randn((M, K), generator=g, device=DEV).to(xt), (0, pad))[:, :K]
    A = (torch.randn((n, r, K), generator=g, device=DEV) / K ** 0.5).to(wt)
    B = (torch.randn((n, N, r), generator=g, device=DEV) / r ** 0.5).to(wt)
    base = torch.randn((M, N), generator=g, device=DEV)
    scale = 0.5 + torch.rand(n, generator=g, device=DEV)
    return x, A, B, base, scale, g


def check(Y, x, A, B, ids, ranks, scale, base):
    n, r, K = A.shape
    for m, a in enumerate(ids.tolist()):
        b = base[m].double() if base is not None else torch.zeros(B.shape[1], dtype=torch.float64, device=DEV)
        if not 0 <= a < n:
            assert torch.equal(Y[m].double(), b)
            continue
        k = min(max(int(ranks[a]), 0), r) if ranks is not None else r
        s = float(scale[a].double()) if scale is not None else 1.0
        t = A[a, :k].double() @ x[m].double()
        d = s * (B[a, :, :k].double() @ t)
        mag = s * (B[a, :, :k].double().abs() @ (A[a, :k].double().abs() @ x[m].double().abs()))
        steps = K / 1024 + 70 + 3 * r / 16 + 8
        lim = 2.0 ** -22 * steps * mag + 2.0 ** -24 * (b + d).abs()
        err = (Y[m].double() - (b + d)).abs()
        assert bool((err <= lim).all()), f"row {m}: {float((err - lim).max())}"


CASES = [  # M, K, N, adapters, r, x, w
    (1, 8, 1, 1, 8, F32, F16), (1, 4096, 4096, 3, 16, F16, F16), (2, 40, 33, 2, 8, BF16, BF16),
    (7, 264, 1000, 4, 24, F32, BF16), (16, 4096, 513, 5, 64, BF16, BF16), (33, 1032, 257, 3, 40, F32, F16),
    (128, 512, 300, 2, 72, F16, F16), (128, 4096, 777, 1, 128, BF16, BF16), (100, 2048, 4096, 120, 32, F16, BF16),
    (19, 8192, 129, 6, 256, BF16, F16), (64, 12288, 64, 64, 8, F32, BF16), (5, 65536, 31, 2, 16, F16, F16),
]


@pytest.mark.parametrize("M,K,N,n,r,xt,wt", CASES)
def test_lora_matches_64_bits(M, K, N, n, r, xt, wt):
    x, A, B, base, scale, g = make(M, K, N, n, r, xt, wt, seed=M + K + N)
    ids = torch.randint(-1, n + 1, (M,), generator=g, device=DEV).to(torch.int32)  # -1 and n: none
    ranks = torch.randint(-2, r + 3, (n,), generator=g, device=DEV).to(torch.int32)
    Y = Guarded((M, N), F32, DEV, fill=float("nan"))
    hq.lora_apply(x, A, B, ids, ranks, scale, base=base, Y=Y.t)
    torch.cuda.synchronize()
    Y.check()
    check(Y.t, x, A, B, ids, ranks, scale, base)
    again = hq.lora_apply(x, A, B, ids, ranks, scale, base=base)
    assert torch.equal(again, Y.t)  # bit for bit
    # full ranks, no scale, no base
    Y = hq.lora_apply(x, A, B, ids)
    check(Y, x, A, B, ids, None, None, None)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 128])
def test_lora_rows_of_one_adapter_in_any_order(rows):
    M, K, N, r = 128, 256, 200, 16
    x, A, B, base, scale, g = make(M, K, N, 4, r, BF16, BF16, seed=rows)
    ids = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    ids[torch.randperm(M, generator=g, device=DEV)[:rows]] = 2
    Y = hq.lora_apply(x, A, B, ids, None, scale, base=base)
    check(Y, x, A, B, ids, None, scale, base)


def test_lora_in_place_on_columns_of_a_fused_output():
    """Beside one part of a fused projection: Y's rows are wider than N, not 16-byte aligned."""
    M, K, N, total = 21, 512, 333, 1001
    x, A, B, _, scale, g = make(M, K, N, 5, 8, F16, F16, seed=3, pad=40)
    assert x.stride(0) == K + 40
    full = torch.randn((M, total), generator=g, device=DEV)
    was = full.clone()
    ids = (torch.arange(M, device=DEV) % 6 - 1).to(torch.int32)
    part = full[:, 101:101 + N]
    ws = torch.empty(hq.hq_lora_workspace_bytes(M, 8), dtype=torch.uint8, device=DEV)
    hq.lora_apply(x, A, B, ids, None, scale, base=part, Y=part, workspace=ws, flags=hq.HQ_LAUNCH_PDL)
    check(part, x, A, B, ids, None, scale, was[:, 101:101 + N])
    assert torch.equal(full[:, :101], was[:, :101]) and torch.equal(full[:, 101 + N:], was[:, 101 + N:])


@pytest.mark.parametrize("wt", [F16, BF16])
def test_lora_does_not_touch_what_is_past_a_rank(wt):
    """NaN past the rank, in unused adapters and in other rows stays where it is."""
    M, K, N, r = 6, 128, 70, 24
    x, A, B, base, scale, g = make(M, K, N, 3, r, F32, wt, seed=4)
    ranks = torch.tensor([5, 0, 13], dtype=torch.int32, device=DEV)
    for a, k in enumerate(ranks.tolist()):
        A[a, k:] = float("nan")
        B[a, :, k:] = float("nan")
    ids = torch.tensor([0, 1, 2, -1, 2, 0], dtype=torch.int32, device=DEV)
    x[3] = float("nan")   # no adapter
    x[5] = float("inf")   # its own row only
    Y = hq.lora_apply(x, A, B, ids, ranks, scale, base=base)
    good = [0, 1, 2, 3, 4]
    check(Y[good], x[good], A, B, ids[good], ranks, scale, base[good])
    assert not torch.isfinite(Y[5]).any()


def test_lora_extremes_of_the_types():
    """Largest and subnormal values: the split terms hold them."""
    K, N, r = 32, 16, 8
    x = torch.zeros((2, K), device=DEV)
    x[0, 0], x[0, 1], x[1, 2] = 1.0 + 2.0 ** -23, -1.0, 3.0e-38
    A = torch.zeros((1, r, K), dtype=F16, device=DEV)
    A[0, 0, :3] = torch.tensor([2.0 ** -24, 2.0 ** -24, 1.0], device=DEV).to(F16)
    B = torch.zeros((1, N, r), dtype=F16, device=DEV)
    B[0, :, 0] = 65504.0
    Y = hq.lora_apply(x, A, B, torch.zeros(2, dtype=torch.int32, device=DEV))
    assert float(Y[0, 0]) == 65504.0 * 2.0 ** -47
    assert abs(float(Y[1, 0]) / (65504.0 * 3.0e-38) - 1) < 2.0 ** -7  # the last terms of 3e-38 are below bf16's range


def test_lora_on_a_side_stream_and_in_a_graph():
    M, K, N, r = 16, 1024, 700, 16
    x, A, B, base, scale, g = make(M, K, N, 4, r, F16, F16, seed=8)
    ids = (torch.arange(M, device=DEV) // 4).to(torch.int32)
    ws = torch.empty(hq.hq_lora_workspace_bytes(M, r), dtype=torch.uint8, device=DEV)
    Y = torch.empty((M, N), device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        hq.lora_apply(x, A, B, ids, None, scale, base=base, Y=Y, workspace=ws)
    st.synchronize()
    check(Y, x, A, B, ids, None, scale, base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.lora_apply(x, A, B, ids, None, scale, base=base, Y=Y, workspace=ws)
    ids.copy_((torch.arange(M, device=DEV) % 3).to(torch.int32))  # the graph follows the ids
    graph.replay()
    torch.cuda.synchronize()
    check(Y, x, A, B, ids, None, scale, base)


@pytest.mark.parametrize("step", [1, 256, 65536, 77777])
def test_lora_ids_from_a_large_pool(step):
    """Ids far apart, many of them in the same places of a hash table, twice and five times each."""
    M, K, N, r = 128, 32, 40, 8
    n = min(128 * step, 400000)
    x, A, B, base, scale, g = make(M, K, N, n, r, BF16, BF16, seed=step)
    pool = (torch.arange(128, device=DEV) * step) % n
    ids = pool[torch.randint(0, 64, (M,), generator=g, device=DEV)].to(torch.int32)
    ids[torch.randperm(M, generator=g, device=DEV)[:20]] = ids[0].clone()
    ids[5], ids[77] = -7, n  # none
    Y = hq.lora_apply(x, A, B, ids, None, scale, base=base)
    check(Y, x, A, B, ids, None, scale, base)


@pytest.mark.parametrize("wt", [F16, BF16])
def test_lora_does_not_touch_what_is_past_a_rank_with_many_rows(wt):
    M, K, N, r = 60, 96, 70, 136
    x, A, B, base, scale, g = make(M, K, N, 4, r, F32, wt, seed=14)
    ranks = torch.tensor([5, 0, 70, 131], dtype=torch.int32, device=DEV)
    for a, k in enumerate(ranks.tolist()):
        A[a, k:] = float("nan")
        B[a, :, k:] = float("nan")
    ids = (torch.arange(M, device=DEV) % 5 - 1).to(torch.int32)
    x[0] = float("nan")  # no adapter
    x[8] = float("inf")  # its own row only
    Y = hq.lora_apply(x, A, B, ids, ranks, scale, base=base)
    good = [i for i in range(M) if i != 8]
    check(Y[good], x[good], A, B, ids[good], ranks, scale, base[good])
    assert not torch.isfinite(Y[8]).any()


@pytest.mark.parametrize("rows", [1, 5])
def test_lora_scale_may_come_from_the_kernel_before(rows):
    """Only ids, ranks and the adapters are read early: the factors of a
    programmatic launch may be outputs of the launch before it."""
    M, K, N, n, r = 120, 4096, 9000, 24, 32
    x, A, B, base, _, g = make(M, K, N, n, r, BF16, BF16, seed=5)
    ids = ((torch.arange(M, device=DEV) // rows) % n).to(torch.int32)
    ws = [torch.empty(hq.hq_lora_workspace_bytes(M, r), dtype=torch.uint8, device=DEV) for _ in range(2)]
    factors = hq.lora_apply(x, A, B, ids, base=base)
    for at in (0, 8900):  # of the first row, the first and the last block's
        out = torch.zeros_like(factors)
        got = torch.empty_like(factors)
        scale = out[0, at:at + n]
        torch.cuda.synchronize()
        hq.lora_apply(x, A, B, ids, base=base, Y=out, workspace=ws[0])
        hq.lora_apply(x, A, B, ids, scale=scale, base=base, Y=got, workspace=ws[1], flags=hq.HQ_LAUNCH_PDL)
        torch.cuda.synchronize()
        assert torch.equal(out, factors)
        assert torch.equal(got, hq.lora_apply(x, A, B, ids, scale=factors[0, at:at + n].clone(), base=base))


def same_as_64_bits(Y, x, A, B, ids, ranks, base):
    """check() for rows with infinities: the same infinities and NaN, the finite rows in its bounds."""
    for m, a in enumerate(ids.tolist()):
        k = int(ranks[a])
        ref = base[m].double() + B[a, :, :k].double() @ (A[a, :k].double() @ x[m].double())
        got = Y[m].double()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"row {m}"
        assert torch.equal(torch.where(torch.isinf(ref), ref, 0.0 * base[m]), torch.where(torch.isinf(got), got, 0.0 * base[m])), f"row {m}"
        if torch.isfinite(ref).all():
            check(Y[m:m + 1], x[m:m + 1], A, B, ids[m:m + 1], ranks, None, base[m:m + 1])


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 20])
@pytest.mark.parametrize("xt,wt", [(F32, F16), (F32, BF16), (F16, BF16), (BF16, F16), (F16, F16)])
@pytest.mark.parametrize("where", ["x", "A", "B"])
def test_lora_infinities_do_not_depend_on_the_rows_of_an_adapter(rows, xt, wt, where):
    K, N, r = 520, 150, 8
    x, A, B, base, _, g = make(rows, K, N, 2, r, xt, wt, seed=rows)
    A[1] = torch.where(torch.randn((r, K), generator=g, device=DEV) > 0, 0.5, -0.25).to(wt)  # few significant bits
    A[0] = A[0] + torch.where(A[0] < 0, -0.01, 0.01).to(wt)  # no zeros
    B += torch.where(B < 0, -0.01, 0.01).to(wt)
    ranks = torch.tensor([1, 1], dtype=torch.int32, device=DEV)
    inf = float("inf")
    if where == "x":
        x[0, 77] = inf
        if rows > 1:
            x[rows // 2, 300] = -inf
    elif where == "A":
        x += torch.where(x < 0, -0.01, 0.01).to(xt)
        A[:, 0, 11] = inf
    else:
        B[:, 3, 0], B[:, 149, 0] = inf, -inf
    for a in (0, 1):
        ids = torch.full((rows,), a, dtype=torch.int32, device=DEV)
        Y = hq.lora_apply(x, A, B, ids, ranks, base=base)
        assert torch.isinf(Y[0]).any() and (where != "B" or torch.isfinite(Y[0]).any())
        same_as_64_bits(Y, x, A, B, ids, ranks, base)


@pytest.mark.parametrize("rows", [1, 3, 20])
@pytest.mark.parametrize("wt", [F16, BF16])
def test_lora_largest_finite_activations(rows, wt):
    """fp32 values that round past bf16's largest, as activations and as products A x."""
    K, N, r = 264, 70, 16
    x, A, B, base, _, g = make(rows, K, N, 1, r, F32, wt, seed=rows)
    top = torch.finfo(F32).max
    x[0, 5] = top
    A[0, :, 5] = torch.linspace(-1.0, 1.0, r, device=DEV).to(wt)
    A[0, 0] = 0
    A[0, 0, 5] = 1.0  # t = the largest value itself
    B *= 0.01
    ids, ranks = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.tensor([r], dtype=torch.int32, device=DEV)
    Y = hq.lora_apply(x, A, B, ids, base=base)
    assert bool(torch.isfinite(Y).all())
    check(Y, x, A, B, ids, ranks, None, base)


@pytest.mark.parametrize("wt", [F16, BF16])
def test_lora_infinities_in_place_among_several_adapters(wt):
    """Each block takes several groups of rows in turn; one in the middle holds the infinities."""
    M, K, N, n, r = 128, 256, 40000, 8, 24
    x, A, B, base, _, g = make(M, K, N, n, r, F32, wt, seed=3)
    ids = (torch.arange(M, device=DEV) // 16).to(torch.int32)
    ranks = torch.tensor([24, 17, 8, 1, 24, 0, 5, 24], dtype=torch.int32, device=DEV)
    B[3, ::1000, 0] = float("inf")
    x[50, 9] = float("-inf")  # of the same adapter
    x[70, 1] = float("nan")   # of the next
    Y = base.clone()
    hq.lora_apply(x, A, B, ids, ranks, base=Y, Y=Y)
    same_as_64_bits(Y, x, A, B, ids, ranks, base)
    assert torch.isinf(Y[50]).all() and torch.isinf(Y[49]).sum() == 40 and torch.isnan(Y).any(1).sum() == 1
