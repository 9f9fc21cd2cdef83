"""Residual addition, RMS norm and int8 output in one pass, against a plain
computation in 64 bits.

Tolerances.  s = x + residual is one fp32 rounding, so residual_out is compared
bit for bit with the fp32 sum rounded to its type.  The sum of squares adds at
most 64 + 10 terms in a chain (the rest is a tree), so it is off by at most
2^-17 relative and rstd by half of that plus two roundings: h is within
2^-17 + eps / 2 of the value.  The rotation of a 32-block is 5 additions, 2
products and the product with the weight: |dz| <= 8 * 2^-24 * sum|w s| /
sqrt(32) over the block; a code is the rounding of c = 127 z / max|z|, so
|q - c| <= 1/2 + 127 * 2 |dz| / max|z| + 127 * 2^-22.
"""
import numpy as np
import pytest
import torch

from guard import Guarded
from quantized_speculative_verify_gb300 import hq

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def rotate64(y, signs):
    """The block rotation in 64 bits, as a matrix product."""
    i = np.arange(32)
    H = np.where(np.array([[bin(a & b).count("1") & 1 for b in i] for a in i]), -1.0, 1.0)
    bits = (signs[:, None] >> np.arange(32, dtype=np.uint32)) & 1
    z = (y * np.where(bits.reshape(-1), -1.0, 1.0)).reshape(y.shape[0], -1, 32)
    return (z @ H).reshape(y.shape) / np.sqrt(32.0)


def make(M, K, xt, rt, seed, pad=0, spread=30.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    big = torch.ones(K, device=DEV)
    big[torch.randint(0, K, (2,), generator=g, device=DEV)] = spread
    x = (torch.randn((M, K + pad), generator=g, device=DEV)[:, :K] * big).to(xt)
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))[:, :K]
    r = torch.randn((M, K + pad), generator=g, device=DEV).to(rt)[:, :K]
    w = 1.0 + 0.3 * torch.randn(K, generator=g, device=DEV)
    return x, r, w, hq.hq_make_signs(seed, K)


def signs_dev(signs):
    return torch.from_numpy(signs.view(np.int32)).to(DEV)


def check(x, r, w, signs, eps, res_out, h, qx, sx):
    K = x.shape[1]
    s32 = x.float() + r.float() if r is not None else x.float()
    if res_out is not None:
        assert torch.equal(res_out, s32.to(res_out.dtype))
    s = s32.double().cpu().numpy()
    w64 = w.double().cpu().numpy()
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    if h is not None:
        y = s * rstd * w64
        rel = 2.0 ** -17 + torch.finfo(h.dtype).eps / 2
        tiny = torch.finfo(h.dtype).smallest_normal
        assert np.all(np.abs(h.double().cpu().numpy() - y) <= rel * np.abs(y) + tiny)
    if qx is not None:
        z = rotate64(s * w64, signs)
        dz = 8 * 2.0 ** -24 * np.abs(s * w64).reshape(s.shape[0], -1, 32).sum(2).max(1, keepdims=True) / np.sqrt(32.0)
        amax = np.abs(z).max(1, keepdims=True)
        q = qx.cpu().numpy().astype(np.float64)
        c = 127.0 * z / amax
        off = np.abs(q - c) - 0.5
        lim = 254.0 * dz / amax + 127 * 2.0 ** -22
        assert np.all(off <= lim), f"worst {np.max(off - lim)}"
        assert np.abs(q).max(1).min() == 127  # the largest value of every row takes the largest code
        ref = (rstd * amax / 127.0)[:, 0]
        assert np.all(np.abs(sx.double().cpu().numpy() - ref) <= ref * (2.0 ** -17 + (dz / amax)[:, 0]))


CASES = [  # M, K, group, format, x, residual, h
    (1, 32, 32, "w4", F32, F32, F32), (1, 4096, 64, "w4", F32, BF16, BF16), (3, 256, 16, "w8", F16, F16, F16),
    (16, 4096, 64, "w4", F32, F32, F16), (17, 1056, 32, "w4", BF16, BF16, F32), (32, 2080, 16, "w4", F32, BF16, BF16),
    (33, 1024, 64, "w4", F16, F32, F16), (64, 512, 16, "w4", BF16, F32, BF16), (65, 2048, 128, "w8", BF16, BF16, BF16),
    (128, 8192, 256, "w4", F32, F32, F32), (5, 12288, 128, "w4", F32, BF16, BF16), (2, 16384, 64, "w8", F32, F16, F16),
    (2, 32768, 256, "w4", BF16, BF16, BF16), (1, 65536, 64, "w4", F32, F32, F16), (3, 9984, 32, "w4", F16, F16, F16),
]


@pytest.mark.parametrize("M,K,G,fmt,xt,rt,ht", CASES)
def test_norm_matches_64_bits(M, K, G, fmt, xt, rt, ht):
    x, r, w, signs = make(M, K, xt, rt, seed=M + K)
    d = hq.make_desc(K, 128, G, fmt)
    res_out, h = Guarded((M, K), rt, DEV), Guarded((M, K), ht, DEV)
    qx, sx, gs = Guarded((M, K), torch.int8, DEV), Guarded((M,), F32, DEV), Guarded((M, K // G), torch.int32, DEV)
    qop = Guarded((hq.hq_act_operand_bytes(d, M),), torch.uint8, DEV)
    hq.add_norm_quant(d, x, r, w, signs_dev(signs), 1e-5, residual_out=res_out.t, h=h.t, qx=qx.t, gsum=gs.t, qop=qop.t,
                      sx=sx.t)
    torch.cuda.synchronize()
    for t in (res_out, h, qx, sx, gs, qop):
        t.check()
    check(x, r, w, signs, 1e-5, res_out.t, h.t, qx.t, sx.t)
    assert torch.equal(gs.t, qx.t.view(M, K // G, G).to(torch.int32).sum(2, dtype=torch.int32))
    # the operand holds these codes: the GEMM on it equals the GEMM on the codes, bit for bit
    layer = hq.pack_layer(0.02 * torch.randn((128, K), device=DEV), G, fmt, signs)
    ws = torch.zeros(hq.hq_workspace_q8_bytes(layer.desc, M), dtype=torch.uint8, device=DEV)
    Y, Y8 = (torch.empty((M, 128), device=DEV) for _ in range(2))
    hq.hq_verify_gemm(layer.desc, layer.blob, qop.t, sx.t, M, Y, None, ws, hq.HQ_LAUNCH_EXACT_ORDER)
    hq.hq_verify_gemm_q8(layer.desc, layer.blob, qx.t, sx.t, None, M, Y8, None, ws, hq.HQ_LAUNCH_EXACT_ORDER)
    torch.cuda.synchronize()
    assert torch.equal(Y, Y8)


@pytest.mark.parametrize("M,K", [(300, 1024), (1000, 4096), (257, 8192)])
def test_norm_of_many_rows_without_an_operand(M, K):
    x, r, w, signs = make(M, K, BF16, BF16, seed=M)
    d = hq.make_desc(K, 128, 32, "w4")
    h, qx, sx = torch.empty_like(x), torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    out = torch.empty_like(r)
    hq.add_norm_quant(d, x, r, w, signs_dev(signs), 1e-6, residual_out=out, h=h, qx=qx, sx=sx)
    check(x, r, w, signs, 1e-6, out, h, qx, sx)


@pytest.mark.parametrize("M,K,G,xt,rt,ht,pad", [
    (3001, 1024, 32, F16, F16, F16, 0), (2500, 736, 16, F32, BF16, F16, 24), (1300, 4096, 64, BF16, F32, BF16, 0),
    (700, 8192, 128, F32, F32, F32, 8), (400, 16384, 64, BF16, BF16, BF16, 16), (1200, 2048, 32, BF16, None, F16, 0),
    (2100, 96, 32, BF16, BF16, F32, 0), (200, 16384, 32, F32, F32, BF16, 0)])
def test_norm_of_many_rows_of_every_type_in_place(M, K, G, xt, rt, ht, pad):
    x, r, w, signs = make(M, K, xt, rt or F32, seed=M + K, pad=pad)
    d = hq.make_desc(K, 128, G, "w4")
    r0 = r.clone() if rt else None
    h = torch.full((M, K + 8), 7.0, dtype=ht, device=DEV)
    qx, sx, gs = Guarded((M, K), torch.int8, DEV), Guarded((M,), F32, DEV), Guarded((M, K // G), torch.int32, DEV)
    hq.add_norm_quant(d, x, r if rt else None, w, signs_dev(signs), 1e-5, residual_out=r if rt else None, h=h[:, :K],
                      qx=qx.t, gsum=gs.t, sx=sx.t)
    torch.cuda.synchronize()
    for t in (qx, sx, gs):
        t.check()
    check(x, r0, w, signs, 1e-5, r if rt else None, h[:, :K], qx.t, sx.t)
    assert bool((h[:, K:] == 7.0).all())
    assert torch.equal(gs.t, qx.t.view(M, K // G, G).to(torch.int32).sum(2, dtype=torch.int32))


def test_norm_degenerate_rows_among_many():
    """Zero, NaN and infinite rows stay by themselves where a block takes several rows."""
    M, K = 1500, 2048
    x, r, w, signs = make(M, K, BF16, BF16, seed=9, spread=1.0)
    x[700], r[700] = 0, 0
    x[3, 17] = float("nan")
    r[1499, 2000] = float("inf")
    d = hq.make_desc(K, 128, 32, "w4")
    h, qx, sx = torch.empty_like(x), torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    hq.add_norm_quant(d, x, r, w, signs_dev(signs), 0.0, h=h, qx=qx, sx=sx)
    assert not h[700].any() and not qx[700].any() and float(sx[700]) == 0.0
    assert not torch.isfinite(sx[3]) and not torch.isfinite(sx[1499])
    keep = [i for i in range(M) if i not in (3, 700, 1499)]
    check(x[keep], r[keep], w, signs, 0.0, None, h[keep], qx[keep], sx[keep])


def test_norm_strided_rows_and_in_place_residual():
    M, K = 9, 736
    x, r, w, signs = make(M, K, F32, BF16, seed=5, pad=24)
    d = hq.make_desc(K, 128, 32, "w8")
    assert x.stride(0) == K + 24
    r0 = r.clone()
    hbuf = torch.full((M, K + 8), 7.0, dtype=F16, device=DEV)
    qx, sx = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    hq.add_norm_quant(d, x, r, w, signs_dev(signs), 1e-5, residual_out=r, h=hbuf[:, :K], qx=qx, sx=sx,
                      flags=hq.HQ_LAUNCH_PDL)
    check(x, r0, w, signs, 1e-5, r, hbuf[:, :K], qx, sx)
    assert bool((hbuf[:, K:] == 7.0).all())


def test_norm_alone_and_without_residual():
    M, K = 4, 512
    x, _, w, signs = make(M, K, BF16, BF16, seed=6)
    d = hq.make_desc(K, 128, 64, "w4")
    h = torch.empty((M, K), device=DEV)
    hq.add_norm_quant(d, x, None, w, None, 1e-5, h=h)
    check(x, None, w, signs, 1e-5, None, h, None, None)
    first = torch.empty_like(x)  # the first layer's residual is x itself
    hq.add_norm_quant(d, x, None, w, None, 1e-5, residual_out=first, h=x)  # h over x
    assert torch.equal(first.float().cpu(), make(M, K, BF16, BF16, seed=6)[0].float().cpu())
    assert np.allclose(x.float().cpu(), h.to(BF16).float().cpu(), rtol=2.0 ** -7, atol=0)


def test_norm_degenerate_rows():
    """Zero rows give zeros; NaN and infinities stay in their row and reach its scale."""
    M, K = 6, 256
    x, r, w, signs = make(M, K, F32, F32, seed=7, spread=1.0)
    x[1], r[1] = 0, 0
    x[2, 17] = float("nan")
    x[3, 200] = float("inf")
    x[4], r[4] = 1e-30, 0
    d = hq.make_desc(K, 128, 32, "w4")
    for eps in (0.0, 1e-6):
        h, qx, sx = torch.empty((M, K), device=DEV), torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
        hq.add_norm_quant(d, x, r, w, signs_dev(signs), eps, h=h, qx=qx, sx=sx)
        assert not h[1].any() and not qx[1].any() and float(sx[1]) == 0.0
        assert not torch.isfinite(sx[2]) and not torch.isfinite(sx[3])
        good = [0, 5]
        check(x[good], r[good], w, signs, eps, None, h[good], qx[good], sx[good])


def test_norm_on_a_side_stream_and_in_a_graph():
    M, K = 8, 1024
    x, r, w, signs = make(M, K, F32, BF16, seed=8)
    sg = signs_dev(signs)
    d = hq.make_desc(K, 128, 32, "w4")
    out, h = torch.empty_like(r), torch.empty_like(r)
    qx, sx = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        hq.add_norm_quant(d, x, r, w, sg, 1e-5, residual_out=out, h=h, qx=qx, sx=sx)
    st.synchronize()
    check(x, r, w, signs, 1e-5, out, h, qx, sx)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hq.add_norm_quant(d, x, r, w, sg, 1e-5, residual_out=out, h=h, qx=qx, sx=sx)
    x.copy_(make(M, K, F32, BF16, seed=9)[0])
    g.replay()
    torch.cuda.synchronize()
    check(x, r, w, signs, 1e-5, out, h, qx, sx)


@pytest.mark.parametrize("M,K,t,pad", [(1000, 8192, F16, 0), (2600, 640, BF16, 16), (1500, 4096, BF16, 0), (333, 12288, F16, 8)])
def test_norm_of_many_rows_behind_an_fp32_projection(M, K, t, pad):
    x, r, w, signs = make(M, K, F32, t, seed=M, pad=pad)
    d = hq.make_desc(K, 128, 32, "w8")
    out, h, qx, sx = (Guarded((M, K), t, DEV), Guarded((M, K), t, DEV), Guarded((M, K), torch.int8, DEV), Guarded((M,), F32, DEV))
    if pad:  # residual_out shares the residual's stride
        hq.add_norm_quant(d, x, r, w, signs_dev(signs), 1e-6, h=h.t, qx=qx.t, sx=sx.t)
    else:
        hq.add_norm_quant(d, x, r, w, signs_dev(signs), 1e-6, residual_out=out.t, h=h.t, qx=qx.t, sx=sx.t)
    torch.cuda.synchronize()
    for g in (out, h, qx, sx):
        g.check()
    check(x, r, w, signs, 1e-6, None if pad else out.t, h.t, qx.t, sx.t)


def outputs(d, x, r, w, signs, eps, qop):
    """Everything the call writes (qop: with the operand), and a GEMM's output of the operand."""
    M, K = x.shape
    h, qx, sx = torch.empty((M, K), device=DEV), torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    gs = torch.empty((M, K // d.group), dtype=torch.int32, device=DEV)
    op = torch.empty(hq.hq_act_operand_bytes(d, M), dtype=torch.uint8, device=DEV) if qop else None
    hq.add_norm_quant(d, x, r, w, signs_dev(signs), eps, h=h, qx=qx, gsum=gs, qop=op, sx=sx)
    Y = None
    if qop:
        layer = hq.pack_layer(0.02 * torch.randn((128, K), device=DEV), d.group, d.format, signs)
        Y = torch.empty((M, 128), device=DEV)
        hq.hq_verify_gemm(layer.desc, layer.blob, op, sx, M, Y, None, hq.workspace(layer.desc, M, DEV), hq.HQ_LAUNCH_EXACT_ORDER)
    assert torch.equal(gs, qx.view(M, K // d.group, d.group).to(torch.int32).sum(2, dtype=torch.int32))
    return h, qx, sx, Y


NONFINITE = [  # rows, features, group, format, x, residual, operand: direct with either encoding, through the ring
    (6, 256, 32, "w4", F32, F32, True), (40, 1024, 64, "w4", BF16, F32, True), (100, 512, 128, "w8", F16, BF16, True),
    (9, 16384, 64, "w8", BF16, BF16, True), (1500, 2048, 32, "w4", BF16, BF16, False), (700, 4096, 64, "w4", F32, F16, False),
    (900, 736, 32, "w4", F32, F32, False)]


@pytest.mark.parametrize("M,K,G,fmt,xt,rt,qop", NONFINITE)
def test_norm_infinities_of_any_pattern_reach_the_scale(M, K, G, fmt, xt, rt, qop):
    x, r, w, signs = make(M, K, xt, rt, seed=M, spread=1.0)
    inf = float("inf")
    x[0] = inf                              # every block of the row: infinities of both signs after the layer's
    x[1, 32:36] = inf                       # one block
    x[2, 64:96] = torch.tensor([inf, -inf], device=DEV).repeat(16).to(xt)
    x[3, K - 1], r[3, K - 2] = inf, -inf
    x[4, 40], r[4, 40] = inf, -inf          # their sum is NaN
    h, qx, sx, Y = outputs(hq.make_desc(K, 128, G, fmt), x, r, w, signs, 1e-6, qop)
    assert not torch.isfinite(sx[:5]).any() and not qx[:5].any()
    assert not torch.isfinite(h[torch.arange(5), [0, 33, 70, K - 1, 40]]).any()
    if qop:
        assert torch.isnan(Y[:5]).all() and torch.isfinite(Y[5:]).all()
    check(x[5:], r[5:], w, signs, 1e-6, None, h[5:], qx[5:], sx[5:])


@pytest.mark.parametrize("M,K,G,fmt,xt,rt,qop", NONFINITE)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_weights_that_are_not_finite_reach_every_scale(M, K, G, fmt, xt, rt, qop, bad):
    x, r, w, signs = make(M, K, xt, rt, seed=M, spread=1.0)
    w[K // 2] = bad
    h, qx, sx, Y = outputs(hq.make_desc(K, 128, G, fmt), x, r, w, signs, 1e-6, qop)
    assert not torch.isfinite(sx).any() and not qx.any()
    assert not torch.isfinite(h[:, K // 2]).any() and torch.isfinite(h[:, :K // 2]).all()
    if qop:
        assert not torch.isfinite(Y).any()


def check_far(x, r, w, signs, eps, res_out, h, qx, sx):
    """check() for rows of any size: what is below fp32's normal range is off by half of its smallest step more."""
    K = x.shape[1]
    s32 = x.float() + r.float() if r is not None else x.float()
    if res_out is not None:
        assert torch.equal(res_out, s32.to(res_out.dtype))
    zero = (s32 == 0).all(1)  # a size below the type's smallest step
    assert not h[zero].any() and not qx[zero].any() and not sx[zero].any()
    s32, h, qx, sx = s32[~zero], h[~zero], qx[~zero], sx[~zero]
    s, w64 = s32.double().cpu().numpy(), w.double().cpu().numpy()
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    y = s * rstd * w64
    rel, step = 2.0 ** -17 + torch.finfo(h.dtype).eps / 2, torch.finfo(h.dtype).smallest_normal
    assert np.all(np.abs(h.double().cpu().numpy() - y) <= rel * np.abs(y) + step)
    assert np.all(np.abs(h.double().cpu().numpy()).max(1) >= 0.5 * np.where(np.abs(y).max(1) > 4 * step, np.abs(y).max(1), 0))
    z = rotate64(s * w64, signs)
    dz = 8 * 2.0 ** -24 * np.abs(s * w64).reshape(s.shape[0], -1, 32).sum(2).max(1, keepdims=True) / np.sqrt(32.0)
    amax = np.abs(z).max(1, keepdims=True)
    q = qx.cpu().numpy().astype(np.float64)
    off = np.abs(q - 127.0 * z / amax) - 0.5
    assert np.all(off <= 254.0 * dz / amax + 127 * 2.0 ** -22)
    assert np.all(np.abs(q).max(1) == 127)
    ref = (rstd * amax / 127.0)[:, 0]
    assert np.all(np.abs(sx.double().cpu().numpy() - ref) <= ref * (2.0 ** -17 + (dz / amax)[:, 0]) + 4 * 2.0 ** -149)


SIZES = [1e-37, 1e-40, 3e-39, 1e-30, 2e-20, 1e-12, 1.0, 1e12, 3e19, 1e25, 3e37, 5e-45]


@pytest.mark.parametrize("M,K,G,fmt,xt,rt,qop", [
    (12, 256, 32, "w4", F32, F32, True), (40, 1024, 64, "w4", BF16, BF16, True), (100, 512, 128, "w8", F32, BF16, True),
    (16, 16384, 64, "w8", BF16, F32, True), (12, 65536, 64, "w4", BF16, BF16, False), (1500, 2048, 32, "w4", BF16, BF16, False),
    (700, 4096, 64, "w4", F32, BF16, False), (900, 736, 32, "w4", F32, F32, False), (400, 12288, 32, "w4", BF16, F32, False)])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("over", [None, "residual", "x"])
def test_norm_of_rows_of_any_size(M, K, G, fmt, xt, rt, qop, eps, over):
    """Rows down to a few of fp32's smallest steps and up to a tenth of its largest value."""
    x, r, w, signs = make(M, K, F32, F32, seed=M + K, spread=3.0)
    size = torch.ones(M, device=DEV)
    for i, f in enumerate(SIZES):
        size[(i * 37 + 3) % M] = f  # among rows of the common kind
    x, r = (x * size[:, None] / 3).to(xt), (r * size[:, None]).to(rt)
    if over == "x":
        r = None
    x0, r0 = x.clone(), None if r is None else r.clone()
    d = hq.make_desc(K, 128, G, fmt)
    out = r if over == "residual" else x if over == "x" else torch.empty_like(r)
    h, qx, sx = Guarded((M, K), F32, DEV), Guarded((M, K), torch.int8, DEV), Guarded((M,), F32, DEV)
    gs = Guarded((M, K // G), torch.int32, DEV)
    op = Guarded((hq.hq_act_operand_bytes(d, M),), torch.uint8, DEV) if qop else None
    hq.add_norm_quant(d, x, r, w, signs_dev(signs), eps, residual_out=out, h=h.t, qx=qx.t, gsum=gs.t, qop=op.t if qop else None,
                      sx=sx.t)
    torch.cuda.synchronize()
    for g in (h, qx, sx, gs):
        g.check()
    check_far(x0, r0, w, signs, eps, out, h.t, qx.t, sx.t)
    assert torch.equal(gs.t, qx.t.view(M, K // G, G).to(torch.int32).sum(2, dtype=torch.int32))
    if qop:
        op.check()
        layer = hq.pack_layer(0.02 * torch.randn((128, K), device=DEV), G, fmt, signs)
        ws = torch.zeros(hq.hq_workspace_q8_bytes(layer.desc, M), dtype=torch.uint8, device=DEV)
        Y, Y8 = (torch.empty((M, 128), device=DEV) for _ in range(2))
        hq.hq_verify_gemm(layer.desc, layer.blob, op.t, sx.t, M, Y, None, ws, hq.HQ_LAUNCH_EXACT_ORDER)
        hq.hq_verify_gemm_q8(layer.desc, layer.blob, qx.t, sx.t, None, M, Y8, None, ws, hq.HQ_LAUNCH_EXACT_ORDER)
        assert torch.equal(Y, Y8) and bool(torch.isfinite(Y).all())


def test_norm_of_one_tensor_as_x_residual_and_residual_out():
    for M, t in ((9, BF16), (1200, BF16), (9, F32)):
        x, _, w, signs = make(M, 512, F32, F32, seed=M)
        x = x.to(t)
        x[1] *= 1e-38
        x[2] = 0
        x[3] *= 1e30
        x0 = x.clone()
        h, qx, sx = torch.empty((M, 512), device=DEV), torch.empty((M, 512), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
        hq.add_norm_quant(hq.make_desc(512, 128, 32, "w4"), x, x, w, signs_dev(signs), 0.0, residual_out=x, h=h, qx=qx, sx=sx)
        assert not h[2].any() and not qx[2].any() and float(sx[2]) == 0.0
        keep = [i for i in range(M) if i != 2]
        check_far(x0[keep], x0[keep], w, signs, 0.0, x[keep], h[keep], qx[keep], sx[keep])
