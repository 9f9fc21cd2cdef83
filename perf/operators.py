"""Performance cases of the operators a batch of requests adds to the verify pass.

Four operators: the residual addition with RMS norm and int8 output that feeds a quantized layer; low-rank adapters
of many requests beside a shared projection; the page table of a paged key/value cache (fork, extend with copy on
write, write, compact, free); and attention of a batch whose sequences share a long prefix, over that cache.

``own`` selects what run() computes: False, the operators in elementary torch operations; True, the calls of this
repository's library.  Both take the same state from prepare().
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
DEV = "cuda"


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # one sequence decoding one token: the norm before a projection of the 9B-class decoder (hidden 4096);
        # x is the previous projection's fp32 output, the residual stream is bf16
        dict(name="norm_token", op="norm", rows=1, width=4096, x="f32", res="bf16", h="bf16"),
        # eight trees of 16 nodes through a layer of the 8192-wide sweep
        dict(name="norm_trees", op="norm", rows=128, width=8192, x="f32", res="f32", h="f16"),
        # a long prompt's rows, everything in 16 bits
        dict(name="norm_prompt", op="norm", rows=8190, width=8192, x="bf16", res="bf16", h="bf16"),
        # eight requests, one token each, an adapter of their own each, beside the o projection
        dict(name="lora_tokens", op="lora", rows=8, n_in=4096, n_out=4096, adapters=16, distinct=8, rank=16, none=0,
             x="f16", w="f16"),
        # eight trees of 16 nodes, five adapters, one tree without, beside the fused gate+up projection
        dict(name="lora_trees", op="lora", rows=128, n_in=4096, n_out=24576, adapters=24, distinct=5, rank=64, none=16,
             x="bf16", w="bf16"),
        # every row another request, beside the down projection; ragged rank; activations in fp32
        dict(name="lora_rows", op="lora", rows=97, n_in=12288, n_out=4096, adapters=97, distinct=96, rank=64, none=1,
             x="f32", w="bf16"),
        # four requests, one token each, behind a short system prompt
        dict(name="attn_few", op="attn", batch=4, nodes=1, shared=1000, suffix=200, heads=32, kv=8, dim=128, page=16,
             type="f16"),
        # a full server decoding one token per request behind a long shared document
        dict(name="attn_wide", op="attn", batch=128, nodes=1, shared=32768, suffix=1024, heads=32, kv=8, dim=128,
             page=64, type="bf16"),
        # draft trees of up to 16 nodes for 48 requests behind a shared prompt
        dict(name="attn_trees", op="attn", batch=48, nodes=16, shared=12345, suffix=700, heads=32, kv=8, dim=128,
             page=32, type="f16"),
        # one verify step's page work for four requests: fork, grow by the tree, write one layer's rows, keep the path
        dict(name="pages_step", op="pages", parents=4, kids=1, length=900, add=16, evict=False, page=16, planes=8,
             heads=8, dim=128, type="f16"),
        # 96 branches forked from two long prompts
        dict(name="pages_fan", op="pages", parents=2, kids=48, length=8000, add=16, evict=False, page=64, planes=16,
             heads=8, dim=128, type="bf16"),
        # half the positions of long sequences dropped in a fork, all planes rewritten
        dict(name="pages_evict", op="pages", parents=6, kids=1, length=16000, add=0, evict=True, page=32, planes=16,
             heads=8, dim=128, type="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "lora", "attn", "pages"])
    t16 = rng.choice(["f16", "bf16"])
    if op == "norm":
        width = 32 * _log(rng, 8, 512)
        return dict(op=op, rows=_log(rng, 1, min(8190, 8190 * 4096 // width)), width=width,
                    x=rng.choice(["f32", t16]), res=rng.choice(["f32", t16]), h=t16)
    if op == "lora":
        rows = _log(rng, 1, 128)
        distinct = _log(rng, 1, max(1, rows // 2)) if rng.random() < 0.6 else rows
        rank = 8 * _log(rng, 1, 8)
        n_in = 8 * _log(rng, 32, 1536)
        most = 96 * 64 * 16384 // (max(distinct, 8) * rank) - n_in
        return dict(op=op, rows=rows, n_in=n_in, n_out=_log(rng, 128, max(129, min(24576, most))), distinct=distinct,
                    adapters=distinct + rng.randrange(8), rank=rank, none=rng.randrange(rows - distinct + 1),
                    x=rng.choice(["f32", t16]), w=t16)
    if op == "attn":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 8])
        batch = _log(rng, 1, 128)
        nodes = rng.choice([1, 1, _log(rng, 1, 32)])
        most = 128 * 32 * 32768 // (batch * nodes * heads)
        return dict(op=op, batch=batch, nodes=nodes, shared=_log(rng, 1, max(1, min(32768, most // 2))),
                    suffix=_log(rng, 1, min(1024, most // 2)), heads=heads, kv=kv, dim=rng.choice([64, 128, 128]),
                    page=rng.choice([16, 32, 64, 128]), type=t16)
    evict = rng.random() < 0.4
    parents = _log(rng, 1, 6)
    return dict(op=op, parents=parents, kids=1 if evict else _log(rng, 1, 48 // parents + 1),
                length=_log(rng, 20, 16000 if evict else 8000), add=0 if evict else _log(rng, 1, 64), evict=evict,
                page=rng.choice([16, 32, 64, 128]), planes=rng.choice([2, 4, 8, 16]), heads=rng.choice([1, 2, 4, 8]),
                dim=rng.choice([64, 128]), type=t16)


def _spread(n, most, least=1, step=0.6180339887498949):
    """n whole numbers over [least, most], the first one `most`."""
    return [most if i == 0 else least + int((most - least) * ((i * step) % 1.0)) for i in range(n)]


def _ranks(c):
    return [max(1, c["rank"] >> (i % 3)) for i in range(c["adapters"])]


def _attn_sizes(c):
    """Rows of each sequence, and its length with them."""
    rows = _spread(c["batch"], c["nodes"], max(1, c["nodes"] // 2))
    own_len = _spread(c["batch"], c["suffix"], 0, 0.7548776662466927)
    return rows, [c["shared"] + s + m for s, m in zip(own_len, rows)]


def _page_sizes(c):
    """Each parent's length; each child's parent, and the positions it keeps."""
    lengths = _spread(c["parents"], c["length"], max(1, c["length"] // 2))
    src = [i // c["kids"] for i in range(c["parents"] * c["kids"])]
    if c["evict"]:
        keep = [(lengths[p] + 1) // 2 for p in src]
    else:
        keep = _spread(len(src), max(0, (c["add"] - 1) // 2), 0)
    return lengths, src, keep


def work(c):
    if c["op"] == "norm":
        n = c["rows"] * c["width"]
        return {"bytes": n * (BYTES[c["x"]] + 2 * BYTES[c["res"]] + BYTES[c["h"]] + 1) + 4 * c["width"] + 4 * c["rows"],
                "flops": 16 * n}
    if c["op"] == "lora":
        r = _ranks(c)[:c["distinct"]]
        used = c["rows"] - c["none"]
        mean = sum(r) / len(r)
        return {"bytes": sum(r) * (c["n_in"] + c["n_out"]) * BYTES[c["w"]] + used * c["n_in"] * BYTES[c["x"]]
                + 8 * c["rows"] * c["n_out"], "flops": 2 * used * mean * (c["n_in"] + c["n_out"])}
    if c["op"] == "attn":
        rows, lens = _attn_sizes(c)
        kv = 2 * c["kv"] * c["dim"] * 2
        return {"bytes": kv * (c["shared"] + sum(n - c["shared"] for n in lens)) + 4 * sum(rows) * c["heads"] * c["dim"],
                "flops": 4 * c["dim"] * c["heads"] * sum(m * (n - m / 2) for m, n in zip(rows, lens))}
    lengths, src, keep = _page_sizes(c)
    row = c["heads"] * c["dim"] * 2
    if c["evict"]:
        moved = sum(keep) * row * c["planes"]
        return {"bytes": 2 * moved, "flops": 0}
    part = sum(lengths[p] % c["page"] for p in src)
    return {"bytes": 2 * (part + sum(keep)) * row * c["planes"] + len(src) * c["add"] * 2 * row * 3
            + 8 * sum(-(-lengths[p] // c["page"]) for p in src), "flops": 0}


# ------------------------------------------------------------------ inputs ---
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 17)
    return {"norm": _prepare_norm, "lora": _prepare_lora, "attn": _prepare_attn, "pages": _prepare_pages}[c["op"]](c, g)


def _prepare_norm(c, g):
    M, K = c["rows"], c["width"]
    s = dict(c)
    # a few channels are far larger than the others, as in the activations of a trained decoder
    big = torch.ones(K, device=DEV)
    big[torch.randperm(K, generator=g, device=DEV)[:2]] = 30.0
    s["xs"] = (torch.randn((M, K), generator=g, device=DEV) * big).to(TYPES[c["x"]])
    s["rs"] = (torch.randn((M, K), generator=g, device=DEV) * 2.0 * big).to(TYPES[c["res"]])
    s["weight"] = 1.0 + 0.2 * torch.randn(K, generator=g, device=DEV)
    # the layer's random signs: bit k % 32 of word k / 32 set means feature k is negated
    s["signs"] = torch.randint(-2 ** 31, 2 ** 31, (K // 32,), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    bits = (s["signs"].unsqueeze(1) >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
    s["pm"] = (1.0 - 2.0 * bits).reshape(K).float()
    i = torch.arange(32, device=DEV)
    odd = sum(((i.unsqueeze(1) & i.unsqueeze(0)) >> b) & 1 for b in range(5)) & 1
    s["hadamard"] = (1.0 - 2.0 * odd).float()
    if own:
        from quantized_speculative_verify_gb300 import hq
        s["hq"], s["desc"] = hq, hq.make_desc(K, 128, 32, "w4")
        s["res_out"] = torch.empty_like(s["rs"])
        s["h_out"] = torch.empty((M, K), dtype=TYPES[c["h"]], device=DEV)
        s["qx"] = torch.empty((M, K), dtype=torch.int8, device=DEV)
        s["sx"] = torch.empty(M, dtype=torch.float32, device=DEV)
        s["values"] = torch.empty((M, K), dtype=TYPES[c["h"]], device=DEV)
    return s


def _prepare_lora(c, g):
    M, K, N, n, r = c["rows"], c["n_in"], c["n_out"], c["adapters"], c["rank"]
    s = dict(c)
    wt = TYPES[c["w"]]
    s["xs"] = torch.randn((M, K), generator=g, device=DEV).to(TYPES[c["x"]])
    s["A"] = (torch.randn((n, r, K), generator=g, device=DEV) / math.sqrt(K)).to(wt)
    s["B"] = (torch.randn((n, N, r), generator=g, device=DEV) / math.sqrt(r)).to(wt)
    s["ranks"] = _ints(_ranks(c))
    s["scale"] = 0.5 + torch.rand(n, generator=g, device=DEV)
    s["base"] = torch.randn((M, N), generator=g, device=DEV)
    # every one of the first `distinct` adapters is used; requests' rows lie next to one another
    ids = [-1] * c["none"] + [i * c["distinct"] // (M - c["none"]) for i in range(M - c["none"])]
    s["ids"] = _ints(ids)
    if own:
        from quantized_speculative_verify_gb300 import hq
        s["hq"] = hq
        s["Y"] = torch.empty((M, N), dtype=torch.float32, device=DEV)
        s["ws"] = torch.zeros(hq.hq_lora_workspace_bytes(M, r), dtype=torch.uint8, device=DEV)
    return s


def _make_cache(c, g, lengths, n_seqs, n_pages, planes, max_pages, kv):
    """Pool, counts, tables and lengths of a cache whose first len(lengths) sequences are filled; pages in any order."""
    ps = c["page"]
    pool = torch.randn((planes, n_pages, kv, ps, c["dim"]), generator=g, device=DEV, dtype=torch.float32).to(TYPES[c["type"]]) \
        if planes * n_pages * kv * ps * c["dim"] < 2 ** 28 else torch.empty((planes, n_pages, kv, ps, c["dim"]),
                                                                            dtype=TYPES[c["type"]], device=DEV).normal_(generator=g)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=DEV)
    ref = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(lengths):
        p = -(-n // ps)
        table[i, :p] = order[at:at + p]
        at += p
    ref[order[:at].long()] = 1
    lens = torch.zeros(n_seqs, dtype=torch.int32, device=DEV)
    lens[:len(lengths)] = _ints(lengths)
    return pool, ref, table, lens, order, at


def _prepare_attn(c, g):
    s = dict(c)
    ps, B = c["page"], c["batch"]
    rows, lens = _attn_sizes(c)
    first = c["shared"] // ps  # whole pages of the prefix are shared; its last rows lie in each sequence's own page
    max_pages = -(-max(lens) // ps)
    n_pages = first + sum(-(-n // ps) - first for n in lens) + 3
    pool, ref, table, ln, order, at = _make_cache(c, g, [first * ps], B, n_pages, 2, max_pages, c["kv"])
    for b, n in enumerate(lens):
        p = -(-n // ps) - first
        table[b, :first] = table[0, :first]
        table[b, first:first + p] = order[at:at + p]
        at += p
    ref[order[:first].long()] = B
    ref[order[first:at].long()] = 1
    rest = c["shared"] % ps
    if rest:  # the same rows in every sequence's own copy of the page
        pages = table[:, first].long()
        pool[:, pages, :, :rest] = pool[:, pages[:1], :, :rest]
    ln.copy_(_ints(lens))
    starts = [0]
    for m in rows:
        starts.append(starts[-1] + m)
    s["n_rows"] = starts[-1]
    s["q"] = (1.5 * torch.randn((starts[-1], c["heads"], c["dim"]), generator=g, device=DEV)).to(TYPES[c["type"]])
    u = torch.rand(starts[-1], generator=g, device=DEV).tolist()
    parent = []
    for b, m in enumerate(rows):
        parent += [0] + [max(0, i - 1 - int(u[starts[b] + i] * 3)) for i in range(1, m)]
    s["parent"], s["starts"] = _ints(parent), _ints(starts)
    s["pool"], s["ref"], s["table"], s["lens"] = pool, ref, table, ln
    s["max_len"] = max(lens)
    # for the plain form: each row's sequence and place in it
    s["row_seq"] = torch.tensor([b for b, m in enumerate(rows) for _ in range(m)], device=DEV)
    s["row_node"] = torch.tensor([i for m in rows for i in range(m)], device=DEV)
    s["scale"] = 1.0 / math.sqrt(c["dim"])
    if own:
        from quantized_speculative_verify_gb300 import hq
        s["hq"] = hq
        s["cache"] = hq.PagedCache(pool, ref, table, ln)
        s["out"] = torch.empty_like(s["q"])
        s["ws"] = torch.zeros(hq.hq_prefix_attention_workspace_bytes(B, starts[-1], c["nodes"], c["heads"], c["kv"], c["dim"]),
                              dtype=torch.uint8, device=DEV)
    return s


def _prepare_pages(c, g):
    s = dict(c)
    ps = c["page"]
    lengths, src, keep = _page_sizes(c)
    n, P = len(src), c["parents"]
    max_pages = -(-(c["length"] + c["add"]) // ps)
    held = sum(-(-x // ps) for x in lengths)
    more = sum(-(-k // ps) + 1 for k in keep) if c["evict"] else n * (c["add"] // ps + 3)
    pool, ref, table, lens, _, _ = _make_cache(c, g, lengths, P + n, held + more + 5, c["planes"], max_pages, c["heads"])
    s["pool"], s["ref"], s["table"], s["lens"] = pool, ref, table, lens
    s["src"], s["dst"] = _ints(src), torch.arange(P, P + n, device=DEV, dtype=torch.int32)
    s["grow"] = _ints([c["add"]] * n)
    s["starts"] = torch.arange(n + 1, device=DEV, dtype=torch.int32) * c["add"]
    # a kept position is named by its distance from `base`, the last position that stays where it is
    s["base"] = _ints([-1 if c["evict"] else lengths[p] for p in src])
    room = [lengths[p] if c["evict"] else c["add"] - 1 for p in src]
    wide = max(1, max(keep))
    rows = []
    for i in range(n):
        pick = torch.randperm(max(1, room[i]), generator=g, device=DEV)[:keep[i]].sort().values.to(torch.int32) + 1
        rows.append(torch.cat([pick, torch.full((wide - keep[i],), -1, dtype=torch.int32, device=DEV)]))
    s["keep"], s["n_keep"] = torch.stack(rows), _ints(keep)
    s["k"] = torch.randn((n * c["add"], c["heads"], c["dim"]), generator=g, device=DEV)
    s["v"] = torch.randn((n * c["add"], c["heads"], c["dim"]), generator=g, device=DEV)
    if own:
        from quantized_speculative_verify_gb300 import hq
        s["hq"], s["cache"] = hq, hq.PagedCache(pool, ref, table, lens)
    return s


# --------------------------------------------------------------- the passes ---
def run(s):
    return {"norm": _run_norm, "lora": _run_lora, "attn": _run_attn, "pages": _run_pages}[s["op"]](s)


def _run_norm(s):
    if own:
        s["hq"].add_norm_quant(s["desc"], s["xs"], s["rs"], s["weight"], s["signs"], EPS, residual_out=s["res_out"],
                               h=s["h_out"], qx=s["qx"], sx=s["sx"])
        torch.mul(s["qx"], s["sx"].unsqueeze(1), out=s["values"])  # the codes as the values they stand for
        return {"residual": s["res_out"], "h": s["h_out"], "scale": s["sx"], "values": s["values"]}
    M, K = s["xs"].shape
    t = s["xs"].float() + s["rs"].float()
    y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["weight"]
    z = ((y * s["pm"]).view(-1, 32) @ s["hadamard"]).view(M, K) * (1.0 / math.sqrt(32.0))
    sx = z.abs().amax(1) / 127.0
    q = torch.clamp(torch.round(z / sx.unsqueeze(1)), -127, 127)
    return {"residual": t.to(s["rs"].dtype), "h": y.to(TYPES[s["h"]]), "scale": sx,
            "values": (q * sx.unsqueeze(1)).to(TYPES[s["h"]])}


def _run_lora(s):
    if own:
        s["hq"].lora_apply(s["xs"], s["A"], s["B"], s["ids"], s["ranks"], s["scale"], base=s["base"], Y=s["Y"], workspace=s["ws"])
        return s["Y"]
    ids = s["ids"].clamp(min=0).long()
    on = torch.where(s["ids"] >= 0, s["scale"][ids], torch.zeros_like(s["scale"][ids]))
    t = torch.bmm(s["A"][ids].float(), s["xs"].float().unsqueeze(2)).squeeze(2)
    live = torch.arange(s["rank"], device=DEV) < s["ranks"][ids].unsqueeze(1)
    t = torch.where(live, t, torch.zeros_like(t))
    d = torch.bmm(s["B"][ids].float(), t.unsqueeze(2)).squeeze(2)
    return s["base"] + on.unsqueeze(1) * d


def _ancestors(parent, seq, node, B, m):
    """visible [B][m][m]: node j is node i itself or one of its ancestors."""
    a = torch.eye(m, device=DEV).expand(B, m, m).clone()
    a[seq, node, parent.long()] = 1.0
    for _ in range(max(1, (m - 1).bit_length())):
        a = (torch.bmm(a, a) > 0).float()
    return a > 0


def _run_attn(s):
    if own:
        s["hq"].prefix_attention(s["cache"], 0, 1, s["q"], s["starts"], s["nodes"], s["shared"], s["max_len"], s["scale"],
                                 parent=s["parent"], out=s["out"], workspace=s["ws"])
        return s["out"]
    B, m, H, kv, D, ps, P = s["batch"], s["nodes"], s["heads"], s["kv"], s["dim"], s["page"], s["shared"]
    G, R, pool, table = H // kv, s["n_rows"], s["pool"], s["table"].long()
    q = s["q"].float().view(R, kv, G, D) * s["scale"]
    # the shared positions, once for all rows
    pre = pool[:, table[0, :-(-P // ps)]].float().transpose(1, 2).reshape(2, kv, -1, D)[:, :, :P]
    s1 = torch.matmul(q.permute(1, 0, 2, 3).reshape(kv, R * G, D), pre[0].transpose(1, 2)).view(kv, R, G, P)
    # each sequence's own positions, padded to the longest
    c0 = P // ps
    mine = pool[:, table[:, c0:].clamp(min=0)].float().transpose(2, 3).reshape(2, B, kv, -1, D)
    pos = torch.arange(c0 * ps, c0 * ps + mine.shape[3], device=DEV)
    old = (s["lens"] - (s["starts"][1:] - s["starts"][:-1])).long()
    tree = _ancestors(s["parent"], s["row_seq"], s["row_node"], B, m)
    at = pos.unsqueeze(0) - old.unsqueeze(1)
    in_tree = torch.gather(tree, 2, at.clamp(0, m - 1).unsqueeze(1).expand(B, m, -1)) & (at >= 0).unsqueeze(1) \
        & (pos < s["lens"].unsqueeze(1)).unsqueeze(1)
    vis = ((pos >= P) & (at < 0)).unsqueeze(1) | in_tree
    qp = torch.zeros((B, m, kv, G, D), device=DEV)
    qp[s["row_seq"], s["row_node"]] = q
    s2 = torch.matmul(qp.permute(0, 2, 1, 3, 4).reshape(B, kv, m * G, D), mine[0].transpose(2, 3)).view(B, kv, m, G, -1)
    s2 = s2.masked_fill(~vis.unsqueeze(1).unsqueeze(3), -math.inf).permute(0, 2, 1, 3, 4)
    x2 = s2[s["row_seq"], s["row_node"]].permute(1, 0, 2, 3)  # [kv][R][G][own positions]
    top = torch.maximum(s1.amax(3, keepdim=True), x2.amax(3, keepdim=True))
    e1, e2 = torch.exp(s1 - top), torch.exp(x2 - top)
    total = e1.sum(3) + e2.sum(3)
    o = torch.matmul(e1.view(kv, R * G, P), pre[1]).view(kv, R, G, D)
    ep = torch.zeros((B, m, kv, G, mine.shape[3]), device=DEV)
    ep[s["row_seq"], s["row_node"]] = e2.permute(1, 0, 2, 3)
    clean = torch.where((pos < s["lens"].unsqueeze(1)).view(B, 1, -1, 1), mine[1], torch.zeros_like(mine[1]))
    o2 = torch.matmul(ep.permute(0, 2, 1, 3, 4).reshape(B, kv, m * G, -1), clean).view(B, kv, m, G, D)
    o = o + o2.permute(0, 2, 1, 3, 4)[s["row_seq"], s["row_node"]].permute(1, 0, 2, 3)
    return (o / total.unsqueeze(3)).permute(1, 0, 2, 3).reshape(R, H, D).to(s["q"].dtype)


def _run_pages(s):
    out = {"pool": s["pool"], "table": s["table"], "ref": s["ref"], "lens": s["lens"]}
    if own:
        hq, c = s["hq"], s["cache"]
        hq.pages_free(c, s["dst"])
        hq.pages_fork(c, s["src"], s["dst"])
        if s["add"]:
            hq.pages_extend(c, s["dst"], s["grow"])
            hq.pages_write(c, 0, 1, s["k"], s["v"], s["starts"], s["add"], seqs=s["dst"])
        hq.pages_compact(c, s["dst"], s["base"], s["keep"], s["n_keep"])
        return out
    ps, table, ref, lens, pool, dst = s["page"], s["table"], s["ref"], s["lens"], s["pool"], s["dst"].long()
    cols = torch.arange(table.shape[1], device=DEV)

    def count(pages, by):  # adds `by` to the counts of the pages that are there
        ref.index_add_(0, pages.clamp(min=0).reshape(-1).long(), torch.where(pages >= 0, by, 0).reshape(-1).to(torch.int32))

    def lowest():  # free pages first, each in ascending order
        return torch.argsort((ref != 0).to(torch.int8), stable=True).to(torch.int32)

    def place(new):  # free pages for the True places of [sequences][columns], in that order
        k = torch.cumsum(new.reshape(-1).to(torch.int32), 0) - 1
        return lowest()[k.clamp(min=0).long()].view(new.shape)

    # free what the children hold
    count(table[dst], -1)
    table[dst] = -1
    lens[dst] = 0
    # fork: the same pages, held once more
    table[dst] = table[s["src"].long()]
    lens[dst] = lens[s["src"].long()]
    count(table[dst], 1)
    if s["add"]:
        # extend: a shared last page that is to be written is replaced by a copy, new pages follow
        n0 = lens[dst].long()
        n1 = n0 + s["grow"]
        old = table[dst]
        last = (n0 // ps).clamp(max=table.shape[1] - 1)
        part = torch.gather(old, 1, last.unsqueeze(1)).squeeze(1)
        cow = (n0 % ps > 0) & (ref[part.clamp(min=0).long()] > 1) & (s["grow"] > 0)
        new = ((cols >= -(-n0 // ps).unsqueeze(1)) & (cols < -(-n1 // ps).unsqueeze(1))) \
            | (cow.unsqueeze(1) & (cols == last.unsqueeze(1)))
        page = place(new)
        now = torch.where(new, page, old)
        count(torch.where(cow, part, torch.full_like(part, -1)), -1)
        count(torch.where(new, page, torch.full_like(page, -1)), 1)
        table[dst] = now
        lens[dst] = n1.to(torch.int32)
        to = torch.gather(now, 1, last.unsqueeze(1)).squeeze(1)
        used = (torch.arange(ps, device=DEV) < (n0 % ps).unsqueeze(1)) & cow.unsqueeze(1)
        a, b = part.clamp(min=0).long(), to.clamp(min=0).long()
        pool[:, b] = torch.where(used.view(1, -1, 1, ps, 1), pool[:, a], pool[:, b])
        # write one layer's new rows
        p = (n0.unsqueeze(1) + torch.arange(s["add"], device=DEV)).reshape(-1)
        pg = torch.gather(now, 1, (p.view(len(dst), -1) // ps)).reshape(-1).long()
        pool[0, pg, :, p % ps] = s["k"].to(pool.dtype)
        pool[1, pg, :, p % ps] = s["v"].to(pool.dtype)
    # compact: kept position d goes to base + 1 + d; pages that change and are shared are replaced, the rest is freed
    base, nk, keep = s["base"].long(), s["n_keep"].long(), s["keep"].long()
    wide = keep.shape[1]
    d = torch.arange(wide, device=DEV)
    moved = (keep != d + 1) & (d < nk.unsqueeze(1))
    d0 = torch.where(moved.any(1), moved.int().argmax(1), nk)
    p0, n1 = base + 1 + d0, base + 1 + nk
    old = table[dst]
    changed = (cols >= (p0 // ps).unsqueeze(1)) & (cols * ps < n1.unsqueeze(1)) & (d0 < nk).unsqueeze(1)
    new = changed & (ref[old.clamp(min=0).long()] > 1)
    page = place(new)
    now = torch.where(new, page, torch.where(cols * ps < n1.unsqueeze(1), old, torch.full_like(old, -1)))
    count(torch.where(now != old, old, torch.full_like(old, -1)), -1)
    count(torch.where(new, page, torch.full_like(page, -1)), 1)
    table[dst] = now
    lens[dst] = n1.to(torch.int32)
    # every row of the changed pages; rows past the end repeat the last one, a sequence without any repeats its first
    j = torch.arange(wide + ps, device=DEV).unsqueeze(0)
    p = torch.minimum((p0 // ps * ps).unsqueeze(1) + j, (n1 - 1).unsqueeze(1))
    p = torch.where((d0 < nk).unsqueeze(1), p, torch.zeros_like(p))
    k = torch.gather(keep, 1, (p - base.unsqueeze(1) - 1).clamp(0, wide - 1)) + base.unsqueeze(1)
    frm = torch.where((p >= p0.unsqueeze(1)) & (d0 < nk).unsqueeze(1), k, p)
    a = torch.gather(old, 1, frm // ps).reshape(-1).long()
    b = torch.gather(now, 1, p // ps).reshape(-1).long()
    pool[:, b, :, (p % ps).reshape(-1)] = pool[:, a, :, (frm % ps).reshape(-1)]
    return out


# ------------------------------------------------------- the same in 64 bits ---
def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "lora": _exact_lora, "attn": _exact_attn, "pages": _exact_pages}[c["op"]](s)


def _exact_norm(s):
    t = s["xs"].double() + s["rs"].double()
    y = t / torch.sqrt((t ** 2).sum(1, keepdim=True) / t.shape[1] + EPS) * s["weight"].double()
    z = y * s["pm"].double()
    for half in (1, 2, 4, 8, 16):  # the butterfly of the Hadamard product, one stride after the other
        u = z.view(z.shape[0], -1, 2, half)
        z = torch.stack([u[:, :, 0] + u[:, :, 1], u[:, :, 0] - u[:, :, 1]], 2).reshape(z.shape)
    z = z / math.sqrt(32.0)
    sx = z.abs().max(1).values / 127.0
    return {"residual": t, "h": y, "scale": sx, "values": torch.round(z / sx[:, None]).clamp(-127, 127) * sx[:, None]}


def _exact_lora(s):
    y = s["base"].double()
    for m, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            r = int(s["ranks"][a])
            y[m] += s["scale"][a].double() * (s["B"][a, :, :r].double() @ (s["A"][a, :r].double() @ s["xs"][m].double()))
    return y


def _exact_attn(s):
    ps, kv, H, D = s["page"], s["kv"], s["heads"], s["dim"]
    starts, lens, parent = s["starts"].tolist(), s["lens"].tolist(), s["parent"].tolist()
    if sum((starts[b + 1] - starts[b]) * n for b, n in enumerate(lens)) * H * D > 8e11:
        return None
    out = torch.zeros((s["n_rows"], H, D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        both = s["pool"][:, s["table"][b, :-(-n // ps)].long()].double().permute(0, 2, 1, 3, 4).reshape(2, kv, -1, D)[:, :, :n]
        r0, m = starts[b], starts[b + 1] - starts[b]
        hide = torch.zeros((m, n), dtype=torch.bool, device=DEV)
        hide[:, n - m:] = True
        rows, cols = [], []
        for i in range(m):
            j = i
            while True:
                rows.append(i)
                cols.append(n - m + j)
                if j == 0:
                    break
                j = parent[r0 + j]
        hide[rows, cols] = False
        q = s["q"][r0:r0 + m].double().view(m, kv, H // kv, D).permute(1, 2, 0, 3)
        x = (q @ both[0].unsqueeze(1).transpose(2, 3)) * s["scale"]
        x = x.masked_fill(hide, -math.inf)
        w = torch.exp(x - x.max(3, keepdim=True).values)
        out[r0:r0 + m] = ((w @ both[1].unsqueeze(1)) / w.sum(3, keepdim=True)).permute(2, 0, 1, 3).reshape(m, H, D)
    return out


def _exact_pages(s):
    if s["pool"].numel() > 3e8:
        return None
    ps, table, ref, lens = s["page"], s["table"].tolist(), s["ref"].tolist(), s["lens"].tolist()
    pool = s["pool"].double()
    dst, src, starts = s["dst"].tolist(), s["src"].tolist(), s["starts"].tolist()

    def free_pages():
        return iter([p for p, n in enumerate(ref) if n == 0])

    for a, b in zip(src, dst):
        table[b] = list(table[a])
        lens[b] = lens[a]
        for p in table[b]:
            if p >= 0:
                ref[p] += 1
    if s["add"]:
        get, shared = free_pages(), list(ref)
        for i, b in enumerate(dst):
            n = lens[b]
            at = n // ps
            if n % ps and shared[table[b][at]] > 1:
                page = next(get)
                pool[:, page, :, :n % ps] = pool[:, table[b][at], :, :n % ps]
                ref[table[b][at]] -= 1
                ref[page] += 1
                table[b][at] = page
            for at in range(-(-n // ps), -(-(n + s["add"]) // ps)):
                table[b][at] = next(get)
                ref[table[b][at]] += 1
            lens[b] = n + s["add"]
            for r in range(s["add"]):
                pool[0, table[b][(n + r) // ps], :, (n + r) % ps] = s["k"][starts[i] + r].double()
                pool[1, table[b][(n + r) // ps], :, (n + r) % ps] = s["v"][starts[i] + r].double()
    get, shared = free_pages(), list(ref)
    for i, b in enumerate(dst):
        base = int(s["base"][i])
        kept = s["keep"][i, :int(s["n_keep"][i])].tolist()
        was, end = list(table[b]), base + 1 + len(kept)
        d0 = next((d for d, k in enumerate(kept) if k != d + 1), None)
        if d0 is not None:
            lo = (base + 1 + d0) // ps
            whole = pool[:, [p for p in was if p >= 0]].transpose(2, 3).flatten(1, 2)  # every position's row, as it was
            for at in range(lo, -(-end // ps)):
                if shared[was[at]] > 1:
                    table[b][at] = next(get)
                    ref[was[at]] -= 1
                    ref[table[b][at]] += 1
                a, z = at * ps, min(end, at * ps + ps)
                frm = [p if p < base + 1 + d0 else base + kept[p - base - 1] for p in range(a, z)]
                pool[:, table[b][at], :, :z - a] = whole[:, frm].transpose(1, 2)
        for at in range(-(-end // ps), len(was)):
            if was[at] >= 0:
                ref[was[at]] -= 1
                table[b][at] = -1
        lens[b] = end
    return {"pool": pool, "table": _ints(table), "ref": _ints(ref), "lens": _ints(lens)}
