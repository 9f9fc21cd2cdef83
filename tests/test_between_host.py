"""The calls between a batch's layers on the host, without a GPU: refusals
before anything is launched, rotary frequencies and their fixed-point form, and
the binding's own checks."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from quantized_speculative_verify_gb300 import hq, verify_batch
from test_batch_host import BAD_CACHES, FAKE, pages

E, U = hq.HQ_ERR_INVALID_ARG, hq.HQ_ERR_UNSUPPORTED
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


# ------------------------------------------------------------- frequencies ---
@pytest.mark.parametrize("rot", [2, 16, 64, 128, 250])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_plain_frequencies_are_the_powers_of_the_base(rot, base):
    f = hq.rope_freqs(rot, base)
    assert f.shape == (rot // 2,) and f[0] == 1.0
    assert np.allclose(f, base ** (-np.arange(rot // 2) * 2.0 / rot), rtol=1e-14, atol=0)
    assert np.array_equal(hq.rope_freqs(rot, base, "linear", factor=4.0), f / 4.0)


def test_scaled_frequencies_keep_the_fast_pairs_and_divide_the_slow_ones():
    rot, base, factor, original = 128, 10000.0, 8.0, 4096.0
    f = hq.rope_freqs(rot, base)
    turns = original * f / (2.0 * math.pi)
    b = hq.rope_freqs(rot, base, "bands", factor, original)
    assert np.array_equal(b[turns >= 4.0], f[turns >= 4.0])
    assert np.allclose(b[turns <= 1.0], f[turns <= 1.0] / factor, rtol=1e-15)
    mid = (turns > 1.0) & (turns < 4.0)
    t = (turns[mid] - 1.0) / 3.0
    assert mid.any() and np.allclose(b[mid], f[mid] * t + f[mid] / factor * (1.0 - t), rtol=1e-13)
    y = hq.rope_freqs(rot, base, "yarn", factor, original)
    where = [rot * math.log(original / (n * 2.0 * math.pi)) / (2.0 * math.log(base)) for n in (32.0, 1.0)]
    lo, hi = math.floor(where[0]), math.ceil(where[1])
    i = np.arange(rot // 2)
    t = np.clip((i - lo) / (hi - lo), 0.0, 1.0)
    assert 0 < lo < hi < rot // 2 and np.allclose(y, f / factor * t + f * (1.0 - t), rtol=1e-13)
    assert np.array_equal(y[:lo + 1], f[:lo + 1])
    n = hq.rope_freqs(rot, base, "ntk", factor)
    assert n[0] == 1.0 and np.isclose(n[-1], f[-1] / factor, rtol=1e-13)  # the slowest pair is divided by the factor
    for kind in ("linear", "ntk", "yarn", "bands"):
        assert np.array_equal(hq.rope_freqs(rot, base, kind, 1.0, original), f), kind


def test_frequencies_refuse_bad_arguments():
    out = np.zeros(64)

    def call(**kw):
        a = dict(rot=128, base=1e4, kind=3, factor=8.0, original=4096.0, low=1.0, high=32.0, out=out.ctypes.data)
        assert set(kw) <= set(a)
        a.update(kw)
        return hq.load().hq_rope_freqs(a["rot"], a["base"], a["kind"], a["factor"], a["original"], a["low"], a["high"], a["out"])
    assert call() == hq.HQ_OK
    bad = [dict(rot=0), dict(rot=3), dict(rot=65538), dict(base=1.0), dict(base=-3.0), dict(base=float("nan")),
           dict(base=float("inf")), dict(kind=-1), dict(kind=5), dict(factor=0.5), dict(factor=float("nan")), dict(factor=1e10),
           dict(original=0.0), dict(original=float("nan")), dict(original=1e19), dict(low=0.0), dict(low=32.0),
           dict(high=float("nan")), dict(high=1e19), dict(out=None), dict(kind=2, rot=2), dict(kind=1, factor=0.0)]
    for b in bad:
        assert call(**b) == E, b
    assert call(kind=0, factor=0.0, original=0.0, low=0.0, high=0.0) == hq.HQ_OK  # not used
    with pytest.raises(ValueError, match="kind"):
        hq.rope_freqs(64, kind="other")


def test_turns_are_the_frequencies_over_two_pi_rounded_to_2_to_the_minus_64():
    getcontext().prec = 90
    f = np.concatenate([hq.rope_freqs(128), hq.rope_freqs(64, 5e5, "yarn", 16.0, 8192.0),
                        [0.0, 5e-324, 1e-300, 2.0 ** -60, 2.0 ** -70, 1e-20, 0.1, 1.0, 3.0, math.pi]])
    t = hq.rope_turns(f, "cpu").numpy().view(np.uint64)
    for x, got in zip(f.tolist(), t.tolist()):
        exact = Decimal(x) / (2 * PI) * 2 ** 64
        assert abs(Decimal(got) - exact) <= Decimal("0.5000001"), x


def test_turns_refuse_bad_arguments():
    f, out = np.array([1.0, 0.5]), np.zeros(2, dtype=np.uint64)
    call = hq.load().hq_rope_turns
    assert call(f.ctypes.data, 2, out.ctypes.data) == hq.HQ_OK
    assert call(None, 2, out.ctypes.data) == E and call(f.ctypes.data, 2, None) == E
    assert call(f.ctypes.data, 0, out.ctypes.data) == E and call(f.ctypes.data, 32769, out.ctypes.data) == E
    for x in (-1e-9, 3.2, float("nan"), float("inf")):
        g = np.array([0.1, x])
        assert call(g.ctypes.data, 2, out.ctypes.data) == E, x
    with pytest.raises(ValueError, match="list"):
        hq.rope_turns(np.zeros((2, 3)), "cpu")


# ------------------------------------------------------------------ refusals ---
def test_rope_write_refuses_bad_arguments():
    lib = hq.load()

    def call(c=None, **kw):
        a = dict(kp=0, vp=1, t=hq.HQ_F16, q=FAKE, k=FAKE, v=FAKE, it=hq.HQ_F32, ldq=512, ldk=256, ldv=256, Hq=4, qw=FAKE, kw=FAKE,
                 eps=1e-6, turns=FAKE, rot=64, layout=0, gain=1.0, seqs=FAKE, starts=FAKE, B=2, rows=6, max_rows=4, parent=FAKE,
                 pos=FAKE, out=FAKE + 4096, ldo=512, flags=0)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.hq_rope_write(c or pages(), a["kp"], a["vp"], a["t"], a["q"], a["k"], a["v"], a["it"], a["ldq"], a["ldk"],
                                 a["ldv"], a["Hq"], a["qw"], a["kw"], a["eps"], a["turns"], a["rot"], a["layout"], a["gain"],
                                 a["seqs"], a["starts"], a["B"], a["rows"], a["max_rows"], a["parent"], a["pos"], a["out"],
                                 a["ldo"], a["flags"], None)
    assert call(B=0) == hq.HQ_OK and call(rows=0) == hq.HQ_OK
    nan, inf = float("nan"), float("inf")
    bad = [dict(kp=-1), dict(kp=2), dict(vp=2), dict(kp=1), dict(t=hq.HQ_F32), dict(it=hq.HQ_BF16), dict(it=9), dict(q=None), dict(k=None),
           dict(v=None), dict(out=None), dict(turns=None), dict(q=FAKE + 8), dict(k=FAKE + 4), dict(v=FAKE + 8),
           dict(out=FAKE + 8), dict(ldq=508), dict(ldq=514), dict(ldk=252), dict(ldv=255), dict(ldo=511), dict(ldo=516),
           dict(Hq=0), dict(Hq=65536), dict(qw=FAKE + 8), dict(kw=FAKE + 4), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
           dict(turns=FAKE + 4), dict(rot=0), dict(rot=8), dict(rot=72), dict(rot=144), dict(rot=-16), dict(layout=2),
           dict(layout=-1), dict(gain=nan), dict(gain=inf), dict(seqs=FAKE + 2), dict(starts=FAKE + 1), dict(B=-1),
           dict(B=65536), dict(rows=-1), dict(max_rows=0), dict(max_rows=129), dict(starts=None, rows=7), dict(parent=FAKE + 1),
           dict(pos=FAKE + 2), dict(flags=2), dict(out=FAKE), dict(it=hq.HQ_F16, out=FAKE, ldo=520)]
    for b in bad:
        assert call(**b) == E, b
    assert call(pages(n_pages=0)) == E and call(pages(row_bytes=192)) == U
    for kw in BAD_CACHES:
        assert call(pages(**kw), B=0) == E, kw
    assert call(parent=None, max_rows=5000, B=0) == hq.HQ_OK  # long prompts have no tree


def test_gated_norm_refuses_bad_arguments():
    def call(**kw):
        a = dict(K=256, group=32, fmt="w4", x=FAKE, xt=hq.HQ_F32, ldx=256, g=FAKE, gt=hq.HQ_BF16, ldg=256, act=2, w=FAKE, D=64,
                 eps=1e-5, M=4, signs=FAKE, h=FAKE + 65536, ht=hq.HQ_F16, ldh=256, qx=FAKE, gsum=FAKE, qop=FAKE, sx=FAKE, flags=0)
        assert set(kw) <= set(a)
        a.update(kw)
        d = hq.make_desc(a["K"], 256, a["group"], a["fmt"])
        return hq.load().hq_gated_norm_quant(ctypes.byref(d), a["x"], a["xt"], a["ldx"], a["g"], a["gt"], a["ldg"], a["act"],
                                             a["w"], a["D"], a["eps"], a["M"], a["signs"], a["h"], a["ht"], a["ldh"], a["qx"],
                                             a["gsum"], a["qop"], a["sx"], a["flags"], None)
    assert call(M=0) == hq.HQ_OK and call(M=0, x=None) == hq.HQ_OK
    bad = [dict(M=-1), dict(M=129), dict(M=(1 << 20) + 1, qop=None), dict(K=40), dict(flags=2), dict(eps=-1e-9),
           dict(eps=float("nan")), dict(eps=float("inf")), dict(xt=3), dict(gt=-1), dict(ht=7), dict(act=3), dict(act=-1),
           dict(D=32), dict(D=96), dict(D=512), dict(K=288, D=64, ldx=288, ldg=288, ldh=288), dict(x=None), dict(signs=None),
           dict(sx=None), dict(x=FAKE + 4), dict(g=FAKE + 8), dict(w=FAKE + 4), dict(h=FAKE + 8), dict(qx=FAKE + 4),
           dict(gsum=FAKE + 2), dict(qop=FAKE + 8), dict(signs=FAKE + 1), dict(sx=FAKE + 2), dict(ldx=255), dict(ldx=258),
           dict(ldg=252), dict(ldh=260), dict(qx=None, gsum=None, qop=None, h=None), dict(h=FAKE), dict(x=FAKE + 32, h=FAKE)]
    for b in bad:
        assert call(**b) == E, b


def history(**kw):
    a = dict(tokens=FAKE, len=FAKE, prompt=FAKE, status=FAKE, n_slots=4, cap=100)
    assert set(kw) <= set(a)
    a.update(kw)
    return hq.hq_history(*a.values())


def rules(**kw):
    a = dict(repetition=FAKE, presence=FAKE, frequency=FAKE, bias_starts=FAKE, bias_tokens=FAKE, bias_values=FAKE, masks=FAKE,
             ldmask=32, n_slots=4, n_bias=10, n_masks=3)
    assert set(kw) <= set(a)
    a.update(kw)
    return hq.hq_logit_rules(*a.values())


BAD_HISTORIES = [dict(tokens=0), dict(len=0), dict(status=0), dict(tokens=FAKE + 2), dict(len=FAKE + 1), dict(prompt=FAKE + 2),
                 dict(status=FAKE + 3), dict(n_slots=0), dict(n_slots=65537), dict(cap=0), dict(cap=(1 << 24) + 1)]


def test_greedy_tokens_refuses_bad_arguments():
    def call(**kw):
        a = dict(x=FAKE, t=hq.HQ_F32, ld=1000, V=1000, h=history(), r=rules(), ids=FAKE, seqs=FAKE, starts=FAKE, B=2, rows=6,
                 max_rows=4, parent=FAKE, tokens=FAKE, out=FAKE + 65536, ot=hq.HQ_F32, ldo=1000, greedy=FAKE, ws=FAKE, flags=0)
        assert set(kw) <= set(a)
        a.update(kw)
        return hq.load().hq_greedy_tokens(a["x"], a["t"], a["ld"], a["V"], a["h"], a["r"], a["ids"], a["seqs"], a["starts"], a["B"],
                                          a["rows"], a["max_rows"], a["parent"], a["tokens"], a["out"], a["ot"], a["ldo"],
                                          a["greedy"], a["ws"], a["flags"], None)
    assert call(B=0) == hq.HQ_OK and call(rows=0) == hq.HQ_OK
    bad = [dict(t=3), dict(ot=hq.HQ_BF16), dict(t=hq.HQ_F16, ot=hq.HQ_BF16), dict(V=0), dict(V=(1 << 24) + 1), dict(ld=999),
           dict(ldo=999), dict(x=None), dict(greedy=None), dict(ws=None), dict(x=FAKE + 2), dict(t=hq.HQ_F16, ot=hq.HQ_F16, x=FAKE + 1),
           dict(out=FAKE + 65538), dict(greedy=FAKE + 2), dict(ws=FAKE + 8), dict(ids=FAKE + 1), dict(seqs=FAKE + 2),
           dict(starts=FAKE + 3), dict(parent=FAKE + 2), dict(tokens=FAKE + 1), dict(B=-1), dict(B=65536), dict(rows=-1),
           dict(rows=(1 << 26) + 1), dict(max_rows=0), dict(max_rows=129), dict(starts=None, rows=7), dict(flags=2),
           dict(out=FAKE, ldo=1001), dict(t=hq.HQ_F16, out=FAKE, ot=hq.HQ_F32)]
    for b in bad:
        assert call(**b) == E, b
    for h in BAD_HISTORIES:
        assert call(h=history(**h), B=0) == E, h
    for r in [dict(n_slots=-1), dict(n_slots=65537), dict(n_bias=-1), dict(n_masks=-1), dict(repetition=FAKE + 1),
              dict(presence=FAKE + 2), dict(frequency=FAKE + 3), dict(bias_starts=FAKE + 2), dict(bias_tokens=FAKE + 1),
              dict(bias_values=FAKE + 2), dict(masks=FAKE + 2), dict(bias_tokens=0), dict(bias_values=0), dict(ldmask=31)]:
        assert call(r=rules(**r), B=0) == E, r
    assert call(h=None, r=None, B=0) == hq.HQ_OK
    size = hq.hq_greedy_tokens_workspace_bytes
    assert size(0) == size(-1) == size((1 << 26) + 1) == 0 and size(1) >= 16 + 4 * 16384 and size(4) == 4 * size(1)
    assert size(1 << 26) <= 16 * (1 << 26) + (17 << 20)
    assert all(size(n) <= size(n + 1) for n in range(1, 200))


def test_tree_accept_batch_refuses_bad_arguments():
    def call(**kw):
        a = dict(g=FAKE, parent=FAKE, tokens=FAKE, seqs=FAKE, starts=FAKE, B=2, rows=6, max_rows=4, h=history(), path=FAKE, ld=4,
                 n=FAKE, bonus=FAKE, flags=0)
        assert set(kw) <= set(a)
        a.update(kw)
        return hq.load().hq_tree_accept_batch(a["g"], a["parent"], a["tokens"], a["seqs"], a["starts"], a["B"], a["rows"],
                                              a["max_rows"], a["h"], a["path"], a["ld"], a["n"], a["bonus"], a["flags"], None)
    assert call(B=0) == hq.HQ_OK and call(B=0, g=None, path=None) == hq.HQ_OK
    bad = [dict(g=None), dict(tokens=None), dict(path=None), dict(n=None), dict(bonus=None), dict(g=FAKE + 2),
           dict(parent=FAKE + 1), dict(tokens=FAKE + 2), dict(seqs=FAKE + 3), dict(starts=FAKE + 1), dict(path=FAKE + 2),
           dict(n=FAKE + 2), dict(bonus=FAKE + 1), dict(B=-1), dict(B=65536), dict(rows=-1), dict(max_rows=0), dict(max_rows=129),
           dict(starts=None, rows=7), dict(ld=3), dict(flags=2)]
    for b in bad:
        assert call(**b) == E, b
    for h in BAD_HISTORIES:
        assert call(h=history(**h), B=0) == E, h
        assert hq.load().hq_history_status(history(**h), None) == E, h
    assert hq.load().hq_history_status(None, None) == E


# ------------------------------------------------------------------- binding ---
I32 = dict(dtype=torch.int32)


@pytest.fixture
def host_pointers(monkeypatch):
    monkeypatch.setattr(hq, "_ptr", lambda t: None if t is None else t.data_ptr())


def small_cache():
    return hq.PagedCache(torch.zeros((2, 4, 1, 16, 64), dtype=torch.float16), torch.zeros(4, **I32), torch.zeros((2, 2), **I32),
                         torch.zeros(2, **I32))


def test_rope_binding_checks(host_pointers):
    cache, turns = small_cache(), hq.rope_turns(hq.rope_freqs(32), "cpu")
    q, k = torch.zeros((4, 2, 64)), torch.zeros((4, 1, 64))

    def bad(match, **kw):
        a = dict(cache=cache, k_plane=0, v_plane=1, q=q, k=k, v=k, turns=turns, starts=None, max_rows=2)
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            hq.rope_write(**a)
    bad("expected", q=torch.zeros((4, 2, 128)))
    bad("expected", k=torch.zeros((4, 2, 64)))
    bad("expected", v=torch.zeros((3, 1, 64)))
    bad("same type", k=k.half())
    bad("turns", turns=torch.zeros(16))
    bad("turns", turns=torch.zeros(32, dtype=torch.int64)[::2])
    bad("layout", layout="other")
    bad("max_rows", max_rows=0)
    bad("the cache has 2", max_rows=1)
    bad("parent", parent=torch.zeros(3, **I32))
    bad("positions", positions=torch.zeros(4))
    bad("q_weight", q_weight=torch.zeros(32))
    bad("k_weight", k_weight=torch.zeros(64, dtype=torch.float16))
    bad("out", out=torch.zeros((4, 2, 64)))
    with pytest.raises(hq.HQError):
        hq.rope_write(cache, 0, 1, q, k, k, turns[:4], torch.zeros(1, **I32), 2)  # 8 elements: not a multiple of 16


def test_gated_norm_binding_checks():
    d = hq.make_desc(256, 256, 32, "w4")
    x = torch.zeros((3, 256))
    with pytest.raises(ValueError, match="features"):
        hq.gated_norm_quant(d, torch.zeros((3, 128)), None, None, None, 64, h=x)
    with pytest.raises(ValueError, match="act"):
        hq.gated_norm_quant(d, x, x, None, None, 64, act="tanh", h=x)
    with pytest.raises(ValueError, match="gate"):
        hq.gated_norm_quant(d, x, torch.zeros((2, 256)), None, None, 64, h=x)
    with pytest.raises(ValueError, match="weight"):
        hq.gated_norm_quant(d, x, x, torch.zeros(256), None, 64, h=x)
    with pytest.raises(ValueError, match="signs"):
        hq.gated_norm_quant(d, x, x, torch.zeros(64), torch.zeros(4, **I32), 64, qx=torch.zeros((3, 256), dtype=torch.int8))
    with pytest.raises(ValueError, match="qx"):
        hq.gated_norm_quant(d, x, x, torch.zeros(64), None, 64, qx=torch.zeros((3, 256)))
    with pytest.raises(ValueError, match="contiguous"):
        hq.gated_norm_quant(d, torch.zeros((256, 3)).t(), None, None, None, 64, h=x)
    with pytest.raises(TypeError, match="int32"):
        hq.gated_norm_quant(d, torch.zeros((3, 256), **I32), None, None, None, 64, h=x)
    with pytest.raises(TypeError, match="CPU tensor"):
        hq.gated_norm_quant(d, x, None, None, None, 64, h=x)


def test_history_and_rules_check_and_keep_their_tensors(host_pointers):
    z = torch.zeros
    with pytest.raises(ValueError, match="tokens"):
        hq.History(z(4, **I32), z(4, **I32))
    with pytest.raises(ValueError, match="lens"):
        hq.History(z((4, 9), **I32), z(3, **I32))
    with pytest.raises(ValueError, match="prompt"):
        hq.History(z((4, 9), **I32), z(4, **I32), z(4))
    with pytest.raises(ValueError, match="slots"):
        hq.History(z((0, 9), **I32), z(0, **I32))
    h = hq.History(z((4, 9), **I32), z(4, **I32))
    for name in ("tokens", "lens", "prompt", "status"):
        with pytest.raises(AttributeError, match=name):
            setattr(h, name, z((4, 9), **I32))
    h.lens += 2
    with pytest.raises(ValueError, match="presence"):
        hq.LogitRules(4, presence=z(3))
    with pytest.raises(ValueError, match="bias starts"):
        hq.LogitRules(4, bias=(z(4, **I32), z(2, **I32), z(2)))
    with pytest.raises(ValueError, match="bias values"):
        hq.LogitRules(4, bias=(z(5, **I32), z(2, **I32), z(3)))
    with pytest.raises(ValueError, match="masks"):
        hq.LogitRules(4, masks=z((4, 9)))
    r = hq.LogitRules(4, repetition=z(4), masks=z((3, 9), **I32))
    with pytest.raises(AttributeError, match="masks"):
        r.masks = z((3, 9), **I32)


def test_greedy_and_accept_binding_checks(host_pointers):
    x, z = torch.zeros((4, 100)), torch.zeros
    with pytest.raises(TypeError, match="fp32"):
        hq.greedy_tokens(x.double(), None, 1)
    with pytest.raises(ValueError, match="max_rows"):
        hq.greedy_tokens(x, None, 0)
    with pytest.raises(ValueError, match="words"):
        hq.greedy_tokens(x, None, 1, rules=hq.LogitRules(4, masks=z((4, 3), **I32)))
    with pytest.raises(ValueError, match="out"):
        hq.greedy_tokens(x, None, 1, out=x.half())
    with pytest.raises(ValueError, match="mask_ids"):
        hq.greedy_tokens(x, None, 1, mask_ids=z(3, **I32))
    with pytest.raises(ValueError, match="workspace"):
        hq.greedy_tokens(x, None, 1, workspace=z(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        hq.greedy_tokens(z((100, 4)).t(), None, 1)
    g = z(4, **I32)
    with pytest.raises(ValueError, match="tokens"):
        hq.tree_accept_batch(g, None, z(3, **I32), None, 2)
    with pytest.raises(ValueError, match="greedy"):
        hq.tree_accept_batch(g.long(), None, g, None, 2)
    with pytest.raises(ValueError, match="path"):
        hq.tree_accept_batch(g, None, g, None, 2, path=z((2, 1), **I32))
    with pytest.raises(ValueError, match="bonus"):
        hq.tree_accept_batch(g, None, g, None, 2, bonus=z(3, **I32))


class Stop(Exception):
    pass


def test_the_step_of_the_command_has_its_frequencies_gain(monkeypatch):
    """Frequencies for contexts four times as long, of the kind whose rotated elements have a gain."""
    seen = {}

    def layer(*a, **kw):
        seen.update(kw)
        raise Stop
    monkeypatch.setattr("sys.argv", ["verify_batch"])
    monkeypatch.setattr(verify_batch, "BatchLayer", layer)
    with pytest.raises(Stop):
        verify_batch.main()
    assert np.array_equal(seen["freqs"], hq.rope_freqs(128, kind="yarn", factor=4.0, original=8192))
    assert seen["gain"] == pytest.approx(0.1 * math.log(4.0) + 1.0)


def test_a_layer_without_rotary_positions_refuses_what_goes_with_them():
    for bad in (dict(gain=1.1), dict(q_norm=torch.ones(64)), dict(k_norm=torch.ones(64))):
        with pytest.raises(ValueError, match="rotary"):
            verify_batch.BatchLayer(512, 8, 2, 64, 4, 1, 8, **bad)
