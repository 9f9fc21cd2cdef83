"""Calls with an explicit `stream` that make their outputs and workspaces themselves.

The other stream is kept busy for a while, so the call's kernels wait behind
it.  Meanwhile the current stream allocates and fills buffers of the sizes that
the call used: none of them may be memory that the waiting kernels still use,
and no fill of the call's own may run ahead of or between them.
"""
import pytest
import torch

from quantized_speculative_verify_gb300 import hq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def behind_a_busy_stream(call, sizes):
    """call(stream) on a stream with work ahead of it, the current stream going on meanwhile."""
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    call(None)  # launch set-up happens here
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
        out = call(stream)
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
        current.synchronize()
        side.synchronize()
        del junk
        yield out
    # let go on the current stream while it still reads it
    out = call(side)
    current.wait_stream(side)
    torch.cuda._sleep(100_000_000)
    copies = [t.clone() for t in (out if isinstance(out, tuple) else (out,))]
    del out
    with torch.cuda.stream(side):
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del junk
    yield tuple(copies) if len(copies) > 1 else copies[0]


def test_adapters():
    M, K, N, r = 24, 512, 1000, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((M, K), generator=g, device=DEV).half()
    A, B = (torch.randn(s, generator=g, device=DEV).half() for s in ((4, r, K), (4, N, r)))
    ids = (torch.arange(M, device=DEV) % 4).to(torch.int32)
    ref = hq.lora_apply(x, A, B, ids)
    for got in behind_a_busy_stream(lambda s: hq.lora_apply(x, A, B, ids, stream=s),
                                    [hq.hq_lora_workspace_bytes(M, r), M * N * 4]):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("B", [3, 40])
def test_prefix_attention(B):
    cache = hq.PagedCache.empty(2, 40 * 8, 2, 16, 128, B, 8)
    g = torch.Generator(device=DEV).manual_seed(2)
    cache.pool.normal_(generator=g)
    cache.table.copy_(torch.randint(0, 40 * 8, (B, 8), generator=g, device=DEV).to(torch.int32))
    cache.table[:, :6] = cache.table[:1, :6].clone()
    cache.lens.fill_(120)
    q = torch.randn((B, 32, 128), generator=g, device=DEV).half()
    ref = hq.prefix_attention(cache, 0, 1, q, None, 1, 96, 128, 0.1)
    need = hq.hq_prefix_attention_workspace_bytes(B, B, 1, 32, 2, 128)
    for got in behind_a_busy_stream(lambda s: hq.prefix_attention(cache, 0, 1, q, None, 1, 96, 128, 0.1, stream=s),
                                    [need, q.nbytes]):
        assert torch.equal(got, ref)


def test_tree_attention():
    M, Hq, Hkv, L, D = 16, 8, 2, 300, hq.HQ_ATTN_HEAD_DIM
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn((M, Hq, D), generator=g, device=DEV).half()
    k, v = (torch.randn((Hkv, 512, D), generator=g, device=DEV).half() for _ in range(2))
    parent = torch.tensor([max(0, i - 1) for i in range(M)], dtype=torch.int32, device=DEV)
    ref = hq.tree_attention(q, k, v, L, parent, 0.1)
    for got in behind_a_busy_stream(lambda s: hq.tree_attention(q, k, v, L, parent, 0.1, stream=s),
                                    [hq.hq_tree_attention_workspace_bytes(Hkv), M * Hq * D * 4]):
        assert torch.equal(got, ref)


def test_tree_accept():
    M, V = 16, 5000
    g = torch.Generator(device=DEV).manual_seed(4)
    logits = torch.randn((M, V), generator=g, device=DEV)
    parent = torch.tensor([max(0, i - 1) for i in range(M)], dtype=torch.int32, device=DEV)
    tokens = torch.cat([torch.zeros(1, device=DEV), logits.argmax(1)[:-1]]).to(torch.int32)
    ref = hq.tree_accept(logits, parent, tokens)
    for got in behind_a_busy_stream(lambda s: hq.tree_accept(logits, parent, tokens, stream=s),
                                    [hq.hq_tree_accept_workspace_bytes(M, V), 4 * M]):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_delta_tree():
    M, H, D = 8, 4, hq.HQ_DELTA_HEAD_DIM
    g = torch.Generator(device=DEV).manual_seed(5)
    state = torch.randn((H, D, D), generator=g, device=DEV)
    q, k, v = (torch.randn((M, H, D), generator=g, device=DEV) / D ** 0.5 for _ in range(3))
    a, b = (torch.rand((M, H), generator=g, device=DEV) for _ in range(2))
    parent = torch.tensor([max(0, i - 1) for i in range(M)], dtype=torch.int32, device=DEV)
    ref = hq.delta_tree(state, q, k, v, a, b, parent)
    for got in behind_a_busy_stream(lambda s: hq.delta_tree(state, q, k, v, a, b, parent, stream=s), [M * H * D * 4]):
        assert torch.equal(got, ref)


def test_pack_unpack_and_linear():
    K, N, M = 512, 640, 16
    signs = hq.hq_make_signs(6, K)
    g = torch.Generator(device=DEV).manual_seed(6)
    W = torch.randn((K, N), generator=g, device=DEV).t()  # packed from a copy of its own
    X = torch.randn((M, K), generator=g, device=DEV)
    layer = hq.pack_layer(W, 64, "w4", signs)
    ws = hq.workspace(layer.desc, M, DEV)
    flags = hq.HQ_LAUNCH_EXACT_ORDER
    sizes = [hq.hq_act_operand_bytes(layer.desc, M), 4 * M, M * N * 4]
    ref = hq.verify_linear(layer, X, ws, flags=flags)
    for got in behind_a_busy_stream(lambda s: hq.verify_linear(layer, X, ws, flags=flags, stream=s), sizes):
        assert torch.equal(got, ref)
    ref = hq.unpack(layer)
    for got in behind_a_busy_stream(lambda s: hq.unpack(layer, s), [t.nbytes for t in ref]):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    for got in behind_a_busy_stream(lambda s: hq.pack_layer(W, 64, "w4", signs, s).blob, [K * N * 4, layer.blob.numel()]):
        assert torch.equal(got, layer.blob)
    parts = [W[:128], W[128:]]
    fused = hq.pack_fused(parts, 64, "w4", signs).layer.blob
    for got in behind_a_busy_stream(lambda s: hq.pack_fused(parts, 64, "w4", signs, s).layer.blob,
                                    [K * 128 * 4, K * 512 * 4, fused.numel()]):
        assert torch.equal(got, fused)
