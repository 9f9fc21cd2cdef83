"""The calls for a batch of requests on the host, without a GPU: arguments are
refused before anything is launched, sizes, and the binding's own checks."""
import ctypes

import pytest
import torch

from quantized_speculative_verify_gb300 import hq

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails its checks
E = hq.HQ_ERR_INVALID_ARG


def norm_call(**kw):
    a = dict(K=256, group=32, fmt="w4", x=FAKE, xt=hq.HQ_F32, ldx=256, res=FAKE, out=FAKE, rt=hq.HQ_BF16, ldr=256,
             w=FAKE, eps=1e-5, M=4, signs=FAKE, h=FAKE, ht=hq.HQ_F16, ldh=256, qx=FAKE, gsum=FAKE, qop=FAKE, sx=FAKE,
             flags=0)
    assert set(kw) <= set(a)
    a.update(kw)
    d = hq.make_desc(a["K"], 256, a["group"], a["fmt"])
    return hq.load().hq_add_norm_quant(ctypes.byref(d), a["x"], a["xt"], a["ldx"], a["res"], a["out"], a["rt"], a["ldr"],
                                       a["w"], a["eps"], a["M"], a["signs"], a["h"], a["ht"], a["ldh"], a["qx"],
                                       a["gsum"], a["qop"], a["sx"], a["flags"], None)


def test_norm_refuses_bad_arguments():
    assert norm_call(M=0) == hq.HQ_OK
    assert norm_call(M=0, x=None, w=None) == hq.HQ_OK
    bad = [dict(M=-1), dict(M=129), dict(M=(1 << 20) + 1, qop=None), dict(K=40), dict(K=0), dict(flags=2), dict(flags=4),
           dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(xt=3), dict(rt=-1), dict(ht=7),
           dict(x=None), dict(w=None), dict(signs=None), dict(sx=None), dict(x=FAKE + 4), dict(res=FAKE + 8),
           dict(out=FAKE + 2), dict(h=FAKE + 8), dict(w=FAKE + 4), dict(qx=FAKE + 4), dict(qop=FAKE + 8),
           dict(gsum=FAKE + 2), dict(ldx=255), dict(ldx=258), dict(ldr=260), dict(ldh=252), dict(ldh=257),
           dict(qx=None, gsum=None, qop=None, h=None, out=None), dict(signs=FAKE + 1), dict(sx=FAKE + 2)]
    for b in bad:
        assert norm_call(**b) == E, b


def test_norm_binding_checks_shapes_before_the_library():
    d = hq.make_desc(256, 256, 32, "w4")
    x, w = torch.zeros((3, 256)), torch.zeros(256)
    with pytest.raises(ValueError, match="256"):
        hq.add_norm_quant(d, torch.zeros((3, 128)), None, w, None, h=x)
    with pytest.raises(ValueError, match="residual"):
        hq.add_norm_quant(d, x, torch.zeros((2, 256)), w, None, h=x)
    with pytest.raises(ValueError, match="weight"):
        hq.add_norm_quant(d, x, None, torch.zeros(128), None, h=x)
    with pytest.raises(ValueError, match="qx"):
        hq.add_norm_quant(d, x, None, w, None, qx=torch.zeros((3, 256), dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        hq.add_norm_quant(d, torch.zeros((256, 3)).t(), None, w, None, h=x)
    with pytest.raises(TypeError, match="int32"):
        hq.add_norm_quant(d, torch.zeros((3, 256), dtype=torch.int32), None, w, None, h=x)
    with pytest.raises(ValueError, match="same type"):
        hq.add_norm_quant(d, x, x, w, None, residual_out=torch.zeros((3, 256), dtype=torch.float16))
    with pytest.raises(TypeError, match="CPU tensor"):
        hq.add_norm_quant(d, x, None, w, None, h=x)


def lora_call(**kw):
    a = dict(x=FAKE, xt=hq.HQ_F32, ldx=256, M=4, K=256, N=100, A=FAKE, B=FAKE, wt=hq.HQ_F16, n=3, r=16, ids=FAKE,
             ranks=FAKE, scale=FAKE, base=FAKE, ldb=100, Y=FAKE + 4096, ldy=100, ws=FAKE, flags=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return hq.load().hq_lora_apply(a["x"], a["xt"], a["ldx"], a["M"], a["K"], a["N"], a["A"], a["B"], a["wt"], a["n"],
                                   a["r"], a["ids"], a["ranks"], a["scale"], a["base"], a["ldb"], a["Y"], a["ldy"],
                                   a["ws"], a["flags"], None)


def test_lora_refuses_bad_arguments():
    assert lora_call(M=0) == hq.HQ_OK and lora_call(M=0, x=None, ids=None) == hq.HQ_OK
    bad = [dict(M=-1), dict(M=129), dict(K=0), dict(K=260), dict(K=65544), dict(N=0), dict(r=0), dict(r=12), dict(r=264),
           dict(n=0), dict(flags=2), dict(xt=5), dict(wt=hq.HQ_F32), dict(wt=9), dict(x=None), dict(A=None),
           dict(B=None), dict(ids=None), dict(Y=None), dict(ws=None), dict(x=FAKE + 8), dict(A=FAKE + 8),
           dict(B=FAKE + 2), dict(ws=FAKE + 4), dict(ids=FAKE + 1), dict(ranks=FAKE + 2), dict(scale=FAKE + 2),
           dict(base=FAKE + 2), dict(Y=FAKE + 3), dict(ldx=248), dict(ldx=258), dict(ldb=99), dict(ldy=99),
           dict(Y=FAKE, ldb=104)]
    for b in bad:
        assert lora_call(**b) == E, b
    size = hq.hq_lora_workspace_bytes
    assert size(4, 16) == 256 and size(128, 256) == 131072
    assert size(0, 16) == size(129, 16) == size(4, 0) == size(4, 12) == size(4, 264) == 0


def test_lora_binding_checks_shapes_before_the_library():
    x, A, B = torch.zeros((2, 64)), torch.zeros((3, 8, 64), dtype=torch.float16), torch.zeros((3, 40, 8), dtype=torch.float16)
    ids = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="B"):
        hq.lora_apply(x, A, B.to(torch.bfloat16), ids)
    with pytest.raises(ValueError, match="ids"):
        hq.lora_apply(x, A, B, ids.long())
    with pytest.raises(ValueError, match="A"):
        hq.lora_apply(torch.zeros((2, 72)), A, B, ids)
    with pytest.raises(ValueError, match="base"):
        hq.lora_apply(x, A, B, ids, base=torch.zeros((2, 39)))
    with pytest.raises(ValueError, match="workspace"):
        hq.lora_apply(x, A, B, ids, workspace=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(TypeError, match="CPU tensor"):
        hq.lora_apply(x, A, B, ids)
