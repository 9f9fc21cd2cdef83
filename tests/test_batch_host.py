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


@pytest.mark.parametrize("signs", [torch.zeros(7, dtype=torch.int32), torch.zeros(9, dtype=torch.int32),
                                   torch.zeros(8), torch.zeros((2, 4), dtype=torch.int32),
                                   torch.zeros(16, dtype=torch.int32)[::2]])
def test_norm_binding_checks_the_signs(signs):
    """A word per 32 features: a shorter vector would be read past its end."""
    d = hq.make_desc(256, 256, 32, "w4")
    x = torch.zeros((3, 256))
    with pytest.raises(ValueError, match="signs"):
        hq.add_norm_quant(d, x, None, torch.zeros(256), signs, qx=torch.zeros((3, 256), dtype=torch.int8), sx=torch.zeros(3))


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


def pages(**kw):
    a = dict(pool=FAKE, ref=FAKE, table=FAKE, len=FAKE, status=FAKE, scratch=FAKE, plane_bytes=100 * 2 * 16 * 256,
             n_planes=2, n_pages=100, n_seqs=8, max_pages=10, page_size=16, heads=2, row_bytes=256)
    assert set(kw) <= set(a)
    a.update(kw)
    return hq.hq_pages(**a)


BAD_CACHES = [dict(pool=0), dict(ref=0), dict(table=0), dict(len=0), dict(status=0), dict(scratch=0), dict(pool=FAKE + 8),
              dict(scratch=FAKE + 4), dict(ref=FAKE + 2), dict(table=FAKE + 1), dict(len=FAKE + 2), dict(status=FAKE + 3),
              dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(page_size=0), dict(row_bytes=0),
              dict(row_bytes=24), dict(row_bytes=8192), dict(n_planes=0), dict(heads=0), dict(n_pages=0),
              dict(n_pages=101), dict(n_pages=(1 << 24) + 1), dict(n_seqs=0), dict(n_seqs=8193), dict(max_pages=0),
              dict(max_pages=(1 << 20) + 1), dict(plane_bytes=100 * 2 * 16 * 256 - 16), dict(plane_bytes=100 * 2 * 16 * 256 + 8),
              dict(plane_bytes=-16), dict(n_pages=1 << 24, page_size=256, plane_bytes=1 << 60)]


def test_page_operations_refuse_bad_arguments():
    lib = hq.load()
    ok = pages()
    calls = {
        "fork": lambda c, n=2, a=FAKE, b=FAKE, f=0: lib.hq_pages_fork(c, a, b, n, f, None),
        "extend": lambda c, n=2, a=FAKE, b=FAKE, f=0: lib.hq_pages_extend(c, a, b, n, f, None),
        "free": lambda c, n=2, a=FAKE, b=FAKE, f=0: lib.hq_pages_free(c, a if b else None, n, f, None),
        "compact": lambda c, n=2, a=FAKE, b=FAKE, f=0: lib.hq_pages_compact(c, a, b, FAKE, 4, 4, FAKE, n, f, None),
        "copy": lambda c, n=2, a=FAKE, b=FAKE, f=0: lib.hq_pages_copy(c, a, b, n, f, None),
    }
    for name, call in calls.items():
        assert call(ok, n=0) == hq.HQ_OK, name
        for kw in BAD_CACHES:
            assert call(pages(**kw), n=0) == E, (name, kw)
        assert call(None) == E and call(ok, n=-1) == E and call(ok, a=None) == E and call(ok, b=None) == E, name
        assert call(ok, f=2) == E and call(ok, a=FAKE + 2) == E, name
        assert call(ok, n=65536) == E and (name == "copy" or call(ok, n=9) == E), name
    assert lib.hq_pages_compact(ok, FAKE, FAKE, FAKE, 3, 4, FAKE, 2, 0, None) == E
    assert lib.hq_pages_compact(ok, FAKE, FAKE, FAKE, 4, -1, FAKE, 2, 0, None) == E
    assert lib.hq_pages_compact(ok, FAKE, FAKE, None, 4, 4, FAKE, 2, 0, None) == E
    assert lib.hq_pages_compact(ok, FAKE, FAKE, FAKE, 4, 4, None, 2, 0, None) == E
    assert lib.hq_pages_status(None, None) == E
    for kw in BAD_CACHES:
        assert lib.hq_pages_status(pages(**kw), None) == E, kw
        if not set(kw) & {"pool", "ref", "table", "len", "status", "scratch"}:
            assert lib.hq_pages_scratch_bytes(pages(**kw)) == 0, kw
    assert lib.hq_pages_scratch_bytes(pages(pool=0, ref=0, table=0, len=0, status=0, scratch=0)) \
        == lib.hq_pages_scratch_bytes(ok) > 0
    assert hq.status_string(hq.HQ_ERR_NO_PAGES) == "HQ_ERR_NO_PAGES"


def test_page_writes_refuse_bad_arguments():
    lib = hq.load()

    def call(c=None, **kw):
        a = dict(kp=0, vp=1, k=FAKE, v=FAKE, it=hq.HQ_F32, ldk=256, ldv=256, t=hq.HQ_F16, seqs=FAKE, starts=FAKE, B=2,
                 rows=6, max_rows=3, flags=0)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.hq_pages_write(c or pages(), a["kp"], a["vp"], a["k"], a["v"], a["it"], a["ldk"], a["ldv"], a["t"],
                                  a["seqs"], a["starts"], a["B"], a["rows"], a["max_rows"], a["flags"], None)
    assert call(B=0) == hq.HQ_OK and call(rows=0) == hq.HQ_OK
    bad = [dict(kp=-1), dict(kp=2), dict(vp=2), dict(k=None), dict(v=None), dict(k=FAKE + 4), dict(v=FAKE + 8), dict(it=3),
           dict(it=hq.HQ_BF16), dict(t=hq.HQ_F32), dict(ldk=255), dict(ldv=252), dict(ldk=257), dict(B=-1), dict(B=65536),
           dict(rows=-1), dict(max_rows=0), dict(starts=None, rows=5), dict(starts=FAKE + 2), dict(seqs=FAKE + 1),
           dict(flags=2)]
    for b in bad:
        assert call(**b) == E, b
    assert call(pages(n_pages=0)) == E


def test_paged_cache_binding_checks():
    z = torch.zeros
    i = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="fp16 or bf16"):
        hq.PagedCache(z((2, 4, 1, 16, 64)), z(4, **i), z((2, 2), **i), z(2, **i))
    with pytest.raises(ValueError, match="ref"):
        hq.PagedCache(z((2, 4, 1, 16, 64), dtype=torch.float16), z(5, **i), z((2, 2), **i), z(2, **i))
    with pytest.raises(ValueError, match="lens"):
        hq.PagedCache(z((2, 4, 1, 16, 64), dtype=torch.float16), z(4, **i), z((2, 2), **i), z(3, **i))
    with pytest.raises(hq.HQError):
        hq.PagedCache(z((2, 4, 1, 24, 64), dtype=torch.float16), z(4, **i), z((2, 2), **i), z(2, **i))
    with pytest.raises(TypeError, match="CPU tensor"):
        hq.PagedCache(z((2, 4, 1, 16, 64), dtype=torch.float16), z(4, **i), z((2, 2), **i), z(2, **i))


def test_a_paged_cache_keeps_the_tensors_whose_addresses_it_holds(monkeypatch):
    monkeypatch.setattr(hq, "_ptr", lambda t: t.data_ptr())
    i = dict(dtype=torch.int32)
    cache = hq.PagedCache(torch.zeros((2, 4, 1, 16, 64), dtype=torch.float16), torch.zeros(4, **i), torch.zeros((2, 2), **i),
                          torch.zeros(2, **i))
    was = {k: getattr(cache, k) for k in ("pool", "ref", "table", "lens", "status", "scratch")}
    for k, t in was.items():
        with pytest.raises(AttributeError, match=k):
            setattr(cache, k, t.clone())
        assert getattr(cache, k) is t
    cache.lens += 3  # in place
    cache.lens[1] = 5
    assert cache.lens.tolist() == [3, 5] and cache.lens is was["lens"] and cache.c.len == cache.lens.data_ptr()


@pytest.mark.parametrize("max_rows", [0, -1])
def test_binding_refuses_batches_without_rows_a_sequence(monkeypatch, max_rows):
    monkeypatch.setattr(hq, "_ptr", lambda t: t.data_ptr())
    i = dict(dtype=torch.int32)
    cache = hq.PagedCache(torch.zeros((2, 4, 1, 16, 64), dtype=torch.float16), torch.zeros(4, **i), torch.zeros((2, 2), **i),
                          torch.zeros(2, **i))
    x = torch.zeros((4, 1, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="max_rows"):
        hq.pages_write(cache, 0, 1, x, x, None, max_rows)
    with pytest.raises(ValueError, match="max_rows"):
        hq.prefix_attention(cache, 0, 1, x, None, max_rows, 0, 16, 0.1)


def test_prefix_attention_refuses_bad_arguments():
    lib = hq.load()

    def call(c=None, **kw):
        a = dict(kp=0, vp=1, t=hq.HQ_F16, q=FAKE, ldq=512, seqs=FAKE, starts=FAKE, B=2, rows=6, max_rows=4, parent=FAKE,
                 Hq=4, shared=20, max_len=150, scale=0.1, out=FAKE, ot=hq.HQ_F16, ldo=512, ws=FAKE, flags=0)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.hq_prefix_attention(c or pages(), a["kp"], a["vp"], a["t"], a["q"], a["ldq"], a["seqs"], a["starts"],
                                       a["B"], a["rows"], a["max_rows"], a["parent"], a["Hq"], a["shared"], a["max_len"],
                                       a["scale"], a["out"], a["ot"], a["ldo"], a["ws"], a["flags"], None)
    assert call(B=0) == hq.HQ_OK and call(rows=0) == hq.HQ_OK
    bad = [dict(kp=-1), dict(vp=2), dict(t=hq.HQ_F32), dict(ot=hq.HQ_BF16), dict(ot=5), dict(q=None), dict(out=None),
           dict(ws=None), dict(q=FAKE + 8), dict(out=FAKE + 4), dict(ws=FAKE + 8), dict(ldq=511), dict(ldq=516),
           dict(ldo=504), dict(seqs=FAKE + 2), dict(starts=FAKE + 1), dict(parent=FAKE + 2), dict(B=-1), dict(B=65536),
           dict(rows=-1), dict(max_rows=0), dict(max_rows=129), dict(starts=None, rows=7), dict(Hq=3), dict(Hq=0),
           dict(shared=-1), dict(shared=150), dict(max_len=0), dict(max_len=161), dict(scale=float("nan")),
           dict(scale=float("inf")), dict(flags=2), dict(rows=1 << 27, ldq=512)]
    for b in bad:
        assert call(**b) == E, b
    U = hq.HQ_ERR_UNSUPPORTED
    assert call(pages(row_bytes=192)) == U
    assert call(pages(n_pages=0)) == E
    assert call(pages(plane_bytes=1 << 40)) == U
    size = hq.hq_prefix_attention_workspace_bytes
    assert size(2, 6, 4, 4, 2, 128) > 16
    for z in ((0, 6, 4, 4, 2, 128), (2, 0, 4, 4, 2, 128), (2, 6, 129, 4, 2, 128), (2, 6, 4, 5, 2, 128), (2, 6, 4, 4, 2, 96)):
        assert size(*z) == 0, z


def test_prefix_attention_workspace_serves_smaller_calls():
    size = hq.hq_prefix_attention_workspace_bytes
    for Hq, Hkv, D in ((32, 8, 128), (8, 8, 64), (64, 1, 128), (40, 5, 64)):
        for m in (1, 5, 16, 128):
            sizes = [size(1, rows, m, Hq, Hkv, D) for rows in range(1, 700, 3)]
            assert sizes == sorted(sizes)
            assert size(7, 50, m, Hq, Hkv, D) == size(50, 50, m, Hq, Hkv, D) <= size(1, 50, min(128, m + 1), Hq, Hkv, D)


@pytest.mark.parametrize("scale,ok", [(3.0e38, False), (-3.0e38, False), (2.4e38, False), (2.3e38, True), (-2.3e38, True)])
def test_prefix_attention_refuses_scales_without_a_base_2_form(scale, ok):
    """scale * log2(e) enters every score: an infinity there would make NaN of a score of 0."""
    rc = hq.load().hq_prefix_attention(pages(), 0, 1, hq.HQ_F16, FAKE, 512, None, None, 0, 6, 4, None, 4, 20, 150, scale, FAKE,
                                       hq.HQ_F16, 512, FAKE, 0, None)  # no sequences: nothing is launched
    assert rc == (hq.HQ_OK if ok else E)
