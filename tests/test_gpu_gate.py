"""The norm per head with its gate and int8 output, against a plain computation
in 64 bits.

Tolerances.  A normed head: 8 + 5 additions to the sum of squares (13 * 2^-24,
half of it in the root), rsqrt 2^-22, three roundings: 14 * 2^-24.  The gate:
exp 2^-22 (2 units in the last place), sum, quotient and two products: 9 *
2^-24.  y is within 2^-19 of its value, h with its own rounding (eps / 2) more.
The rotation of a 32-block is 5 additions, and the values that enter are 2^-19
off: |dz| <= 2^-18.5 * sum|y| / sqrt(32) over the block; a code is the rounding
of c = 127 z / max|z|, so |q - c| <= 1/2 + 127 * 2 |dz| / max|z| + 127 * 2^-22.
Below fp32's normal range a rounding is off by up to 2^-150 whatever the value:
x / rms, then times w, then times the gate, so the first one counts |w act(gate)|
times and the second |act(gate)| times: (1 + |a| + |w a|) * 2^-150, below 2^-144
for weights below 2.5 and gates below 16.
"""
import numpy as np
import pytest
import torch

from guard import Guarded
from quantized_speculative_verify_gb300 import hq
from test_gpu_norm import rotate64, signs_dev

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
REL = 2.0 ** -19


def make(M, K, D, xt, gt, seed, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn((M, K + pad), generator=g, device=DEV)).to(xt)[:, :K]
    gate = (2.0 * torch.randn((M, K + pad), generator=g, device=DEV)).to(gt)[:, :K] if gt else None
    return x, gate, 1.0 + 0.3 * torch.randn(D, generator=g, device=DEV), hq.hq_make_signs(seed, K)


def value(x, gate, w, D, act, eps):
    y = x.double().cpu().numpy()
    if w is not None:
        y = y.reshape(y.shape[0], -1, D)
        ms = (y * y).mean(2, keepdims=True) + float(np.float32(eps))
        y = np.where(ms > 0, y / np.sqrt(np.where(ms > 0, ms, 1.0)), 0.0) * w.double().cpu().numpy()
        y = y.reshape(x.shape)
    if gate is not None:
        z = gate.double().cpu().numpy()
        s = 1.0 / (1.0 + np.exp(-z))
        y = y * {"none": z, "sigmoid": s, "silu": z * s}[act]
    return y


def check(y, signs, h=None, qx=None, sx=None):
    if h is not None:
        f = torch.finfo(h.dtype)
        off = np.abs(h.double().cpu().numpy() - y)
        assert np.all(off <= (REL + f.eps / 2) * np.abs(y) + f.smallest_normal * f.eps + 2.0 ** -144), np.max(off / np.maximum(np.abs(y), 1e-30))
    if qx is not None:
        z = rotate64(y, signs)
        dz = 2.0 ** -18.5 * np.abs(y).reshape(y.shape[0], -1, 32).sum(2).max(1, keepdims=True) / np.sqrt(32.0)
        amax = np.abs(z).max(1, keepdims=True)
        safe = np.where(amax > 0, amax, 1.0)
        q = qx.cpu().numpy().astype(np.float64)
        off = np.abs(q - 127.0 * z / safe) - 0.5
        assert np.all(off <= 254.0 * dz / safe + 127 * 2.0 ** -22), np.max(off)
        assert np.all((np.abs(q).max(1) == 127) == (amax[:, 0] > 0))
        ref = (amax / 127.0)[:, 0]
        assert np.all(np.abs(sx.double().cpu().numpy() - ref) <= ref * 2.0 ** -22 + (dz / 127.0)[:, 0] + 2.0 ** -149)


CASES = [  # M, K, D, group, format, x, gate, h, act, norm
    (1, 64, 64, 32, "w4", F32, F32, F32, "silu", True), (1, 4096, 128, 64, "w4", F32, BF16, BF16, "silu", True),
    (3, 256, 256, 16, "w8", F16, F16, F16, "sigmoid", False), (16, 4096, 128, 64, "w4", F32, F32, F16, "sigmoid", True),
    (17, 1088, 64, 32, "w4", BF16, BF16, F32, "none", True), (32, 2048, 256, 16, "w4", F32, BF16, BF16, "silu", False),
    (33, 1024, 128, 64, "w4", F16, F32, F16, "silu", True), (64, 512, 64, 16, "w4", BF16, F32, BF16, "none", False),
    (65, 2048, 128, 128, "w8", BF16, BF16, BF16, "silu", True), (128, 8192, 128, 256, "w4", F32, F32, F32, "sigmoid", False),
    (5, 12288, 256, 128, "w4", F32, BF16, BF16, "silu", True), (2, 16384, 128, 64, "w8", F32, F16, F16, "silu", True),
    (2, 32768, 64, 256, "w4", BF16, BF16, BF16, "sigmoid", True), (1, 65536, 256, 64, "w4", F32, F32, F16, "silu", True),
    (3, 9984, 128, 32, "w4", F16, None, F16, "silu", True), (4, 4160, 64, 32, "w8", F32, None, F32, "none", False),
]


@pytest.mark.parametrize("M,K,D,G,fmt,xt,gt,ht,act,norm", CASES)
def test_gated_norm_matches_64_bits(M, K, D, G, fmt, xt, gt, ht, act, norm):
    x, gate, w, signs = make(M, K, D, xt, gt, seed=M + K, pad=8)
    w = w if norm else None
    d = hq.make_desc(K, 128, G, fmt)
    h = Guarded((M, K), ht, DEV)
    qx, sx, gs = Guarded((M, K), torch.int8, DEV), Guarded((M,), F32, DEV), Guarded((M, K // G), torch.int32, DEV)
    qop = Guarded((hq.hq_act_operand_bytes(d, M),), torch.uint8, DEV)
    hq.gated_norm_quant(d, x, gate, w, signs_dev(signs), D, act, 1e-5, h=h.t, qx=qx.t, gsum=gs.t, qop=qop.t, sx=sx.t)
    torch.cuda.synchronize()
    for t in (h, qx, sx, gs, qop):
        t.check()
    check(value(x, gate, w, D, act, 1e-5), signs, h.t, qx.t, sx.t)
    assert torch.equal(gs.t, qx.t.view(M, K // G, G).to(torch.int32).sum(2, dtype=torch.int32))
    # the operand holds these codes: the GEMM on it equals the GEMM on the codes, bit for bit
    layer = hq.pack_layer(0.02 * torch.randn((128, K), device=DEV), G, fmt, signs)
    ws = torch.zeros(hq.hq_workspace_q8_bytes(layer.desc, M), dtype=torch.uint8, device=DEV)
    Y, Y8 = (torch.empty((M, 128), device=DEV) for _ in range(2))
    hq.hq_verify_gemm(layer.desc, layer.blob, qop.t, sx.t, M, Y, None, ws, hq.HQ_LAUNCH_EXACT_ORDER)
    hq.hq_verify_gemm_q8(layer.desc, layer.blob, qx.t, sx.t, None, M, Y8, None, ws, hq.HQ_LAUNCH_EXACT_ORDER)
    torch.cuda.synchronize()
    assert torch.equal(Y, Y8)
    # h alone is another kernel's, and the codes alone leave it out
    h2, qx2, sx2 = torch.empty_like(h.t), torch.empty_like(qx.t), torch.empty_like(sx.t)
    hq.gated_norm_quant(d, x, gate, w, None, D, act, 1e-5, h=h2)
    hq.gated_norm_quant(d, x, gate, w, signs_dev(signs), D, act, 1e-5, qx=qx2, sx=sx2)
    assert torch.equal(h2, h.t) and torch.equal(qx2, qx.t) and torch.equal(sx2, sx.t)


@pytest.mark.parametrize("M,K,D,xt,gt,ht", [(1, 64, 64, F32, F32, BF16), (7, 192, 64, F16, F16, F16), (1000, 4096, 128, BF16, BF16, BF16),
                                            (3001, 1024, 256, F32, BF16, BF16), (257, 8192, 128, F32, F32, F32), (4000, 704, 64, BF16, F32, F16),
                                            (400, 8192, 128, F16, F16, F16), (500, 8192, 256, F32, BF16, BF16), (700, 2560, 64, F32, F16, F16),
                                            (1300, 4096, 64, F16, F16, F32), (333, 16384, 128, BF16, BF16, BF16), (400, 8192, 64, BF16, BF16, BF16)])
@pytest.mark.parametrize("codes", [False, True])
def test_many_rows(M, K, D, xt, gt, ht, codes):
    x, gate, w, signs = make(M, K, D, xt, gt, seed=M, pad=16)
    d = hq.make_desc(K, 128, 32, "w4")
    h = torch.full((M, K + 8), 7.0, dtype=ht, device=DEV)
    qx, sx = (Guarded((M, K), torch.int8, DEV), Guarded((M,), F32, DEV)) if codes else (None, None)
    gs = Guarded((M, K // 32), torch.int32, DEV) if codes else None
    hq.gated_norm_quant(d, x, gate, w, signs_dev(signs), D, "silu", 1e-6, h=h[:, :K], qx=qx and qx.t, gsum=gs and gs.t, sx=sx and sx.t)
    torch.cuda.synchronize()
    if codes:
        gs.check()
        assert torch.equal(gs.t, qx.t.view(M, K // 32, 32).to(torch.int32).sum(2, dtype=torch.int32))
    assert bool((h[:, K:] == 7.0).all())
    check(value(x, gate, w, D, "silu", 1e-6), signs, h[:, :K], qx and qx.t, sx and sx.t)
    for t in (qx, sx):
        if t is not None:
            t.check()


@pytest.mark.parametrize("over", ["x", "gate"])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("size", [1.0, 1e-36])
def test_h_in_place(over, codes, size):
    M, K, D = 50, 2048, 128
    x, gate, w, signs = make(M, K, D, BF16, BF16, seed=3)
    x, gate = (size * x.float()).to(BF16).contiguous(), gate.contiguous()
    d, y = hq.make_desc(K, 128, 32, "w4"), value(x, gate, None, D, "silu", 0.0)
    qx, sx = (torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)) if codes else (None, None)
    h = x if over == "x" else gate
    hq.gated_norm_quant(d, x, gate, None, signs_dev(signs), D, "silu", 1e-6, h=h, qx=qx, sx=sx)
    check(y, signs, h, qx, sx)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_heads_of_any_size(D, eps):
    sizes = [0.0, 1e-44, 1e-38, 1e-30, 1e-20, 1e-12, 1.0, 1e10, 1e19, 1e25, 3e37]
    K = D * len(sizes)
    x, gate, w, signs = make(3, K, D, F32, F32, seed=D)
    scale = torch.tensor(sizes, device=DEV).repeat_interleave(D)
    x = (x.double().clamp(-5, 5) * scale).float()
    h, qx, sx = torch.empty((3, K), device=DEV), torch.empty((3, K), dtype=torch.int8, device=DEV), torch.empty(3, device=DEV)
    hq.gated_norm_quant(hq.make_desc(K, 128, 32, "w4"), x, gate, w, signs_dev(signs), D, "silu", eps, h=h, qx=qx, sx=sx)
    check(value(x, gate, w, D, "silu", eps), signs, h, qx, sx)


def test_rows_of_any_size_among_many():
    """Rows whose codes are formed in other units, and rows that are not finite, between common ones of the same block."""
    M, K, D = 500, 8192, 128
    x, gate, w, signs = make(M, K, D, F32, BF16, seed=9)
    scale = torch.ones(M, device=DEV)
    scale[::7], scale[3::11], scale[5::13] = 1e-36, 1e30, 0.0
    x = (x.double().clamp(-4, 4) * scale.unsqueeze(1)).float()
    bad = list(range(6, M, 29))
    x[bad, 17] = float("inf")
    qx, sx = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    hq.gated_norm_quant(hq.make_desc(K, 128, 32, "w4"), x, gate, None, signs_dev(signs), D, "none", 0.0, qx=qx, sx=sx)
    rows = [r for r in range(M) if r not in bad]
    check(value(x[rows], gate[rows], None, D, "none", 0.0), signs, None, qx[rows], sx[rows])
    assert not bool(torch.isfinite(sx[bad]).any()) and not bool(qx[bad].any())


@pytest.mark.parametrize("size", [0.0, 1e-44, 1e-40, 1e-37, 1e-33, 1e-20, 1.0, 1e30, 4e37])
def test_rows_of_any_size_without_a_norm(size):
    M, K = 3, 1024
    x, _, _, signs = make(M, K, 64, F32, None, seed=5)
    x = (x.double().clamp(-4, 4) * size).float()
    qx, sx = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    hq.gated_norm_quant(hq.make_desc(K, 128, 32, "w4"), x, None, None, signs_dev(signs), 64, "silu", 0.0, qx=qx, sx=sx)
    check(value(x, None, None, 64, "silu", 0.0), signs, None, qx, sx)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["x", "gate", "weight"])
def test_rows_that_are_not_finite(bad, where):
    M, K, D = 4, 1024, 128
    x, gate, w, signs = make(M, K, D, F32, F32, seed=6)
    clean = value(x, gate, w, D, "sigmoid", 1e-6)
    if where == "weight":
        w[5] = bad
    else:
        (x if where == "x" else gate)[1, 300] = bad
    h, qx, sx = torch.empty((M, K), device=DEV), torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    hq.gated_norm_quant(hq.make_desc(K, 128, 32, "w4"), x, gate, w, signs_dev(signs), D, "sigmoid", 1e-6, h=h, qx=qx, sx=sx)
    rows = [0, 2, 3] if where != "weight" else []
    if rows:
        check(clean[rows], signs, h[rows], qx[rows], sx[rows])
    if where == "gate" and bad == bad:  # a gate of 1 or 0
        y = clean.copy()
        y[1, 300] = value(x[1:2], None, w, D, "none", 1e-6)[0, 300] if bad > 0 else 0.0
        check(y, signs, h, qx, sx)
        return
    for r in sorted(set(range(4)) - set(rows)):
        assert not bool(torch.isfinite(sx[r])) and not bool(qx[r].any())
    if where == "x":  # other heads do not see it
        keep = [i for i in range(K) if i // D != 300 // D]
        check(clean[1:2][:, keep], signs, h[1:2][:, keep])
        assert bool(torch.isnan(h[1, 300]))


@pytest.mark.parametrize("codes", [False, True])
def test_rows_past_32_bits(codes):
    M, K, D, ld = 3, 1024, 128, 2 ** 30
    x, gate, w, signs = make(M, K, D, BF16, BF16, seed=11)
    far = [torch.empty(2 * ld + K, dtype=BF16, device=DEV).as_strided((M, K), (ld, 1)) for _ in range(2)]
    for t, v in zip(far, (x, gate)):
        t.copy_(v)
    qx, sx = (torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)) if codes else (None, None)
    hq.gated_norm_quant(hq.make_desc(K, 128, 64, "w4"), far[0], far[1], w, signs_dev(signs), D, "silu", 1e-6, h=far[0], qx=qx, sx=sx)
    check(value(x, gate, w, D, "silu", 1e-6), signs, far[0], qx, sx)


@pytest.mark.parametrize("M,K,D", [(3, 1024, 128), (700, 4096, 64), (5, 20480, 256)])
def test_group_sums_or_the_operand_alone(M, K, D):
    x, gate, w, signs = make(M, K, D, F32, F16, seed=10)
    d, sg = hq.make_desc(K, 128, 64, "w4"), signs_dev(signs)
    qx, gs, sx = torch.empty((M, K), dtype=torch.int8, device=DEV), Guarded((M, K // 64), torch.int32, DEV), torch.empty(M, device=DEV)
    hq.gated_norm_quant(d, x, gate, w, sg, D, "silu", gsum=gs.t, sx=sx)
    hq.gated_norm_quant(d, x, gate, w, sg, D, "silu", qx=qx, sx=sx)
    gs.check()
    assert torch.equal(gs.t, qx.view(M, -1, 64).to(torch.int32).sum(2, dtype=torch.int32))
    if M <= hq.HQ_MAX_M:
        n = hq.hq_act_operand_bytes(d, M)
        a, b = Guarded((n,), torch.uint8, DEV), Guarded((n,), torch.uint8, DEV)
        hq.gated_norm_quant(d, x, gate, w, sg, D, "silu", qop=a.t, sx=sx)
        hq.gated_norm_quant(d, x, gate, w, sg, D, "silu", qx=qx, qop=b.t, gsum=gs.t, sx=sx)
        a.check()
        assert torch.equal(a.t, b.t)


def test_a_captured_call_and_another_stream():
    M, K, D = 9, 4096, 128
    x, gate, w, signs = make(M, K, D, F32, BF16, seed=7)
    d, sg = hq.make_desc(K, 128, 64, "w4"), signs_dev(signs)
    h, qx, sx = torch.empty((M, K), dtype=F16, device=DEV), torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hq.gated_norm_quant(d, x, gate, w, sg, D, "silu", h=h, qx=qx, sx=sx, stream=s)
    s.synchronize()
    check(value(x, gate, w, D, "silu", 1e-6), signs, h, qx, sx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.gated_norm_quant(d, x, gate, w, sg, D, "silu", h=h, qx=qx, sx=sx, flags=hq.HQ_LAUNCH_PDL)
    x.mul_(-3.0)
    gate.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    check(value(x, gate, w, D, "silu", 1e-6), signs, h, qx, sx)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("K", [1024, 8192, 16384])
@pytest.mark.parametrize("gt", [F32, BF16, F16])
def test_finite_gates_of_any_size(gt, K, act):
    """A row for each gate, up to the type's largest; a quotient 1 / (1 + e^-gate) below 2^-126 is 0.  |x| <= 1/2, so silu's
    products stay finite."""
    sizes = [0.0, 1e-30, 50.0, 88.0, 100.0] + ([1e4] if gt == F16 else [1e30, 2.4e38]) + [torch.finfo(gt).max]
    gates = torch.tensor(sizes + [-s for s in sizes], device=DEV).to(gt)
    M, D = len(gates), 128
    x, _, _, signs = make(M, K, D, F32, None, seed=13)
    x, gate = (x / 8).clamp(-0.5, 0.5), gates.unsqueeze(1).expand(M, K).contiguous()
    z = gate.double().cpu().numpy()
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    s = np.where(s < 2.0 ** -126, 0.0, s)
    y = x.double().cpu().numpy() * (z * s if act == "silu" else s)
    d, sg = hq.make_desc(K, 128, 32, "w4"), signs_dev(signs)
    h, both = torch.empty((M, K), dtype=gt, device=DEV), torch.empty((M, K), dtype=gt, device=DEV)
    qx, sx = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    hq.gated_norm_quant(d, x, gate, None, None, D, act, h=h)
    hq.gated_norm_quant(d, x, gate, None, sg, D, act, h=both, qx=qx, sx=sx)
    check(y, signs, h, qx, sx)
    assert torch.equal(h, both)
    qx2, sx2 = torch.empty_like(qx), torch.empty_like(sx)  # beside the operand: another kernel
    qop = torch.empty(hq.hq_act_operand_bytes(d, M), dtype=torch.uint8, device=DEV)
    hq.gated_norm_quant(d, x, gate, None, sg, D, act, qx=qx2, qop=qop, sx=sx2)
    assert torch.equal(qx, qx2) and torch.equal(sx, sx2)


@pytest.mark.parametrize("M,K", [(16, 8192), (3, 16384)])
def test_the_sigmoid_keeps_its_accuracy_far_below_zero(M, K):
    """x is a power of two and h fp32, so h is the sigmoid as it was computed: power 2^-22, ln 2 as it is rounded 2^-22 at
    the far end, reciprocal 2^-23, three roundings: 13 * 2^-24."""
    gate = torch.linspace(-87.2, 20.0, M * K, dtype=torch.float64, device=DEV).float().view(M, K)
    x = 2.0 ** torch.randint(0, 10, (M, K), device=DEV).float()
    h, both = torch.empty((M, K), device=DEV), torch.empty((M, K), device=DEV)
    d, sg = hq.make_desc(K, 128, 32, "w4"), signs_dev(hq.hq_make_signs(1, K))
    hq.gated_norm_quant(d, x, gate, None, None, 128, "sigmoid", h=h)
    hq.gated_norm_quant(d, x, gate, None, sg, 128, "sigmoid", h=both, qx=torch.empty((M, K), dtype=torch.int8, device=DEV),
                        sx=torch.empty(M, device=DEV))
    want = x.double() / (1.0 + torch.exp(-gate.double()))
    for t in (h, both):
        assert float(((t.double() - want) / want).abs().max()) <= 13 * 2.0 ** -24


@pytest.mark.parametrize("K", [448, 1024, 1984, 2048, 4096, 8192])
@pytest.mark.parametrize("xt,gt", [(F32, BF16), (BF16, BF16), (F32, F16), (F16, F16)])
def test_codes_with_types_known_at_compile_time(xt, gt, K):
    """The same values in types that the kernel looks up at run time give the same bits."""
    M, D = 1500, 64
    x, gate, w, signs = make(M, K, D, xt, gt, seed=K, pad=8)
    d, sg = hq.make_desc(K, 128, 32, "w4"), signs_dev(signs)
    h, qx, sx = torch.empty((M, K), dtype=gt, device=DEV), torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    hq.gated_norm_quant(d, x, gate, w, sg, D, "silu", 1e-6, h=h, qx=qx, sx=sx)
    check(value(x, gate, w, D, "silu", 1e-6), signs, h, qx, sx)
    h2, qx2, sx2 = torch.empty_like(h), torch.empty_like(qx), torch.empty_like(sx)
    hq.gated_norm_quant(d, x, gate.float(), w, sg, D, "silu", 1e-6, h=h2, qx=qx2, sx=sx2)
    assert torch.equal(h, h2) and torch.equal(qx, qx2) and torch.equal(sx, sx2)
