"""Performance cases of what stands between the calls of a batch's verify step.

Four operators: rotary positions of q and k with the write of k and v into the paged cache; penalties, biases and
grammar masks on the logits with the greedy token of every row; the acceptance of a batch of draft trees, which grows
the requests' histories; and the norm per head with its gate that feeds the quantized output projection.

``own`` selects what run() computes: False, the operators in elementary torch operations; True, the calls of this
repository's library.  Both take the same state from prepare().
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # four requests decoding one token each: q, k and v are the fused projection's fp32 columns (hidden 4096,
        # heads of 128, kv 1024)
        dict(name="rope_tokens", op="rope", batch=4, nodes=1, tree=False, context=1000, heads=32, kv=8, dim=128, rot=128,
             layout="half", kind="plain", norm=False, page=16, x="f32", type="f16"),
        # eight draft trees of up to 16 nodes far into long contexts, frequencies scaled for them, q and k normed per head
        dict(name="rope_trees", op="rope", batch=8, nodes=16, tree=True, context=30000, heads=32, kv=8, dim=128, rot=64,
             layout="half", kind="yarn", norm=True, page=64, x="f32", type="bf16"),
        # prompts of ragged lengths in one pass, everything in 16 bits, interleaved pairs
        dict(name="rope_prompts", op="rope", batch=3, nodes=4095, tree=False, context=0, heads=32, kv=8, dim=128, rot=128,
             layout="interleaved", kind="bands", norm=False, page=64, x="bf16", type="bf16"),
        # one request's next token: the LM head's fp32 row of 151552 logits, penalties from its history
        dict(name="pick_token", op="pick", batch=1, nodes=1, vocab=151552, history=500, bias=0, masked=0, out=False,
             x="f32"),
        # eight trees of up to 16 nodes, a grammar on every second request, a hundred biased tokens each
        dict(name="pick_trees", op="pick", batch=8, nodes=16, vocab=151552, history=2000, bias=100, masked=2, out=False,
             x="f32"),
        # a small vocabulary of odd size in 16 bits; the adjusted logits are kept (for a sampler)
        dict(name="pick_odd", op="pick", batch=5, nodes=7, vocab=32003, history=777, bias=13, masked=1, out=True, x="bf16"),
        # a full server, one token per request, long histories, the adjusted logits kept
        dict(name="pick_wide", op="pick", batch=128, nodes=1, vocab=151552, history=16000, bias=0, masked=3, out=True,
             x="f32"),
        # the 16-node tree of one request
        dict(name="accept_one", op="accept", batch=1, nodes=16),
        # a full server's trees, as wide as they may be
        dict(name="accept_many", op="accept", batch=512, nodes=128),
        # one token's heads behind the delta-rule layer: fp32 values, a gate in bf16, codes for the output projection
        dict(name="gate_token", op="gate", rows=1, heads=32, dim=128, act="silu", norm=True, codes=True, x="f32", h="bf16"),
        # eight trees of 16 nodes, an attention's output gate without a norm, 8192 wide
        dict(name="gate_trees", op="gate", rows=128, heads=64, dim=128, act="sigmoid", norm=False, codes=True, x="f32",
             h="f16"),
        # a long prompt's rows, all in 16 bits (its output product is one in 16 bits)
        dict(name="gate_prompt", op="gate", rows=8190, heads=64, dim=128, act="silu", norm=True, codes=False, x="bf16",
             h="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "pick", "accept", "gate"])
    t16 = rng.choice(["f16", "bf16"])
    if op == "rope":
        tree = rng.random() < 0.4
        batch = _log(rng, 1, 64)
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 128, 128, 256])
        heads, x = kv * rng.choice([1, 2, 4, 5]), rng.choice(["f32", t16])
        most = max(2, 9000 * 48 * 128 * 4 // (batch * (heads + 2 * kv) * dim * (BYTES[x] + 2)))
        nodes = _log(rng, 2, min(64, most)) if tree else rng.choice([1, _log(rng, 2, min(4095, most))])
        return dict(op=op, batch=batch, nodes=nodes, tree=tree,
                    context=_log(rng, 1, 30000 * 1024 // (max(1024, kv * dim) * -(-batch // 8))), heads=heads, kv=kv, dim=dim,
                    rot=16 * rng.randint(1, dim // 16), layout=rng.choice(["half", "interleaved"]),
                    kind=rng.choice(["plain", "linear", "ntk", "yarn", "bands"]), norm=rng.random() < 0.4,
                    page=rng.choice([16, 32, 64, 128]), x=x, type=t16)
    if op == "pick":
        batch = _log(rng, 1, 128)
        return dict(op=op, batch=batch, nodes=rng.choice([1, _log(rng, 1, max(1, min(64, 128 // batch)))]),
                    vocab=_log(rng, 1000, 140000), history=_log(rng, 1, 16000), bias=rng.choice([0, _log(rng, 1, 300)]),
                    masked=rng.randrange(4), out=rng.random() < 0.5, x=rng.choice(["f32", "f32", t16]))
    if op == "accept":
        return dict(op=op, batch=_log(rng, 1, 512), nodes=_log(rng, 1, 128))
    heads, dim, codes = _log(rng, 1, 64), rng.choice([64, 128, 128, 256]), rng.random() < 0.6
    x = rng.choice(["f32", t16])
    most = 8190 * 64 * 128 * 6 // (heads * dim * (BYTES[x] + 4)) // (4 if codes else 1)
    return dict(op=op, rows=_log(rng, 1, min(8190, most)), heads=heads, dim=dim, act=rng.choice(["silu", "sigmoid", "none"]),
                norm=rng.random() < 0.6, codes=codes, x=x, h=t16)


def _spread(n, most, least=1, step=0.6180339887498949):
    """n whole numbers over [least, most], the first one `most`."""
    return [most if i == 0 else least + int((most - least) * ((i * step) % 1.0)) for i in range(n)]


def _rows(c):
    """Rows of each sequence."""
    return _spread(c["batch"], c["nodes"], max(1, c["nodes"] // 2))


def _lengths(c):
    """Positions that each sequence holds before these rows."""
    return _spread(c["batch"], c["context"], c["context"] // 2, 0.7548776662466927)


def _histories(c):
    return _spread(c["batch"], c["history"], c["history"] // 2, 0.7548776662466927)


def _masked(c, b):
    return c["masked"] > 0 and b % c["masked"] == 0


def work(c):
    if c["op"] == "rope":
        n = sum(_rows(c)) * (c["heads"] + 2 * c["kv"]) * c["dim"]
        return {"bytes": n * (BYTES[c["x"]] + 2), "flops": 6 * sum(_rows(c)) * (c["heads"] + c["kv"]) * c["rot"] // 2}
    if c["op"] == "pick":
        m = _rows(c)
        n = sum(m) * c["vocab"]
        return {"bytes": n * BYTES[c["x"]] * (2 if c["out"] else 1)
                + sum(r for b, r in enumerate(m) if _masked(c, b)) * 4 * (-(-c["vocab"] // 32))
                + 4 * sum(_histories(c)) + 8 * c["batch"] * c["bias"] + 12 * sum(m), "flops": n}
    if c["op"] == "accept":
        return {"bytes": 16 * sum(_rows(c)) + 12 * c["batch"], "flops": 4 * sum(_rows(c))}
    n = c["rows"] * c["heads"] * c["dim"]
    return {"bytes": n * (BYTES[c["x"]] + 2 * BYTES[c["h"]] + (1 if c["codes"] else 0)) + 4 * c["dim"] + 4 * c["rows"],
            "flops": (14 if c["codes"] else 8) * n}


# ------------------------------------------------------------------ inputs ---
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 29)
    return {"rope": _prepare_rope, "pick": _prepare_pick, "accept": _prepare_accept, "gate": _prepare_gate}[c["op"]](c, g)


def _starts(rows):
    starts = [0]
    for m in rows:
        starts.append(starts[-1] + m)
    return starts


def _trees(rows, g):
    """Parents of a draft tree per sequence: each node hangs below one of the three before it."""
    u = torch.rand(sum(rows), generator=g, device=DEV).tolist()
    at, parent = 0, []
    for m in rows:
        parent += [0] + [max(0, i - 1 - int(u[at + i] * 3)) for i in range(1, m)]
        at += m
    return parent


def _places(s, rows):
    """For the plain forms: each row's sequence and place in it."""
    n = torch.tensor(rows, device=DEV)
    s["row_seq"] = torch.repeat_interleave(torch.arange(len(rows), device=DEV), n)
    s["row_node"] = torch.arange(int(sum(rows)), device=DEV) - (torch.cumsum(n, 0) - n)[s["row_seq"]]


def _freqs(c):
    """Radians a position of each pair: powers of the base, slowed down for contexts longer than the trained one."""
    half, base, factor, original = c["rot"] // 2, 10000.0, 8.0, 4096.0
    if c["kind"] == "ntk":
        base *= factor ** (c["rot"] / max(1, c["rot"] - 2))
    f = [base ** (-2.0 * i / c["rot"]) for i in range(half)]
    if c["kind"] == "linear":
        return [x / factor for x in f]
    if c["kind"] == "bands":  # wavelengths: short ones as they are, long ones divided, a ramp between
        r = [min(1.0, max(0.0, (original * x / (2.0 * math.pi) - 1.0) / (4.0 - 1.0))) for x in f]
        return [x * t + x / factor * (1.0 - t) for x, t in zip(f, r)]
    if c["kind"] == "yarn":  # the same ramp over the pairs' numbers, between those that turn 32 times and once
        where = [c["rot"] * math.log(original / (t * 2.0 * math.pi)) / (2.0 * math.log(base)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(where[0]), 0), min(math.ceil(where[1]), c["rot"] - 1)
        r = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(half)]
        return [x / factor * t + x * (1.0 - t) for x, t in zip(f, r)]
    return f


def _prepare_rope(c, g):
    s = dict(c)
    rows, before = _rows(c), _lengths(c)
    lens = [n + m for n, m in zip(before, rows)]
    starts, ps, R = _starts(rows), c["page"], sum(rows)
    held = [-(-n // ps) for n in lens]
    s["pool"] = torch.zeros((2, sum(held) + 1, c["kv"], ps, c["dim"]), dtype=TYPES[c["type"]], device=DEV)
    order = torch.randperm(sum(held) + 1, generator=g, device=DEV).to(torch.int32)
    s["table"] = torch.full((c["batch"], max(held)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, p in enumerate(held):
        s["table"][b, :p] = order[at:at + p]
        at += p
    s["ref"] = torch.ones(sum(held) + 1, dtype=torch.int32, device=DEV)
    s["lens"], s["starts"] = _ints(lens), _ints(starts)
    s["parent"] = _ints(_trees(rows, g)) if c["tree"] else None
    # one projection's columns, q first, then k and v
    q, kv = c["heads"] * c["dim"], c["kv"] * c["dim"]
    y = torch.randn((R, q + 2 * kv), generator=g, device=DEV).to(TYPES[c["x"]])
    s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, c["dim"])) for t in y.split([q, kv, kv], 1))
    s["qw"], s["kw"] = ((1.0 + 0.2 * torch.randn(c["dim"], generator=g, device=DEV)) if c["norm"] else None for _ in range(2))
    s["freqs"] = torch.tensor(_freqs(c), dtype=torch.float64, device=DEV)
    s["gain"] = 0.1 * math.log(8.0) + 1.0 if c["kind"] == "yarn" else 1.0
    _places(s, rows)
    if own:
        from quantized_speculative_verify_gb300 import hq
        s["hq"], s["cache"] = hq, hq.PagedCache(s["pool"], s["ref"], s["table"], s["lens"])
        s["turns"] = hq.rope_turns(_freqs(c), DEV)
        s["out"] = torch.empty((R, c["heads"], c["dim"]), dtype=TYPES[c["type"]], device=DEV)
    return s


def _prepare_pick(c, g):
    s = dict(c)
    rows, hist = _rows(c), _histories(c)
    B, V, R = c["batch"], c["vocab"], sum(rows)
    # a few tokens well above the rest; text repeats itself: the history's tokens lie near the front of the vocabulary
    x = 2.0 * torch.randn((R, V), generator=g, device=DEV)
    high = (torch.randint(0, V, (R, 1), generator=g, device=DEV) + torch.arange(20, device=DEV) * (V // 20)) % V
    x.scatter_add_(1, high, 8.0 + 2.0 * torch.rand((R, 20), generator=g, device=DEV))
    s["logits"] = x.to(TYPES[c["x"]])
    u = torch.rand((B, max(hist)), generator=g, device=DEV)
    s["tokens"] = (V * u ** 4).to(torch.int32).clamp(max=V - 1)
    s["lens"], s["prompt"] = _ints(hist), _ints([n // 2 for n in hist])
    s["draft"] = (V * torch.rand(R, generator=g, device=DEV) ** 4).to(torch.int32).clamp(max=V - 1)
    s["starts"], s["parent"] = _ints(_starts(rows)), _ints(_trees(rows, g))
    s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device=DEV)
    s["presence"] = 0.5 * torch.rand(B, generator=g, device=DEV)
    s["frequency"] = 0.2 * torch.rand(B, generator=g, device=DEV)
    if c["bias"]:
        n = min(c["bias"], V)
        s["bias_tokens"] = torch.cat([torch.randperm(V, generator=g, device=DEV)[:n] for _ in range(B)]).to(torch.int32)
        s["bias_values"] = 4.0 * torch.randn(B * n, generator=g, device=DEV)
        s["bias_starts"] = _ints([b * n for b in range(B + 1)])
    _places(s, rows)
    if c["masked"]:  # a bit for each token; a grammar allows few, some states of it most
        on = [_masked(c, b) for b in range(B)]
        ids, n = [], 0
        for b, m in enumerate(rows):
            ids += list(range(n, n + m)) if on[b] else [-1] * m
            n += m if on[b] else 0
        words = -(-V // 32)
        bits = [torch.randint(-2 ** 31, 2 ** 31, (n, words), generator=g, device=DEV, dtype=torch.int64) for _ in range(3)]
        s["masks"] = (bits[0] & bits[1] & bits[2]).to(torch.int32)
        s["mask_ids"] = _ints(ids)
    if own:
        from quantized_speculative_verify_gb300 import hq
        s["hq"], s["state"] = hq, hq.History(s["tokens"], s["lens"], s["prompt"])
        s["rules"] = hq.LogitRules(B, repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                   bias=(s["bias_starts"], s["bias_tokens"], s["bias_values"]) if c["bias"] else None,
                                   masks=s.get("masks"))
        s["greedy"] = torch.empty(R, dtype=torch.int32, device=DEV)
        s["adjusted"] = torch.empty_like(s["logits"]) if c["out"] else None
        s["ws"] = torch.zeros(hq.hq_greedy_tokens_workspace_bytes(R), dtype=torch.uint8, device=DEV)
    return s


def _prepare_accept(c, g):
    s = dict(c)
    rows = _rows(c)
    B, R, V = c["batch"], sum(rows), 151552
    s["starts"], s["parent"] = _ints(_starts(rows)), _ints(_trees(rows, g))
    s["draft"] = torch.randint(0, V, (R,), generator=g, device=DEV).to(torch.int32)
    _places(s, rows)
    # the model's token after a node is the draft of the child that names it last, where it agrees with the draft at all
    s["greedy"] = torch.randint(0, V, (R,), generator=g, device=DEV).to(torch.int32)
    first = s["starts"][:-1].long()[s["row_seq"]]
    child = torch.arange(R, device=DEV)
    last = torch.full((R,), -1, dtype=torch.int64, device=DEV)
    last.scatter_reduce_(0, first + s["parent"].long(), torch.where(s["row_node"] > 0, child, torch.full_like(child, -1)), "amax")
    agree = (last >= 0) & (torch.rand(R, generator=g, device=DEV) < 0.85)
    s["greedy"] = torch.where(agree, s["draft"][last.clamp(min=0)], s["greedy"])
    s["before"] = torch.randint(0, 500, (B,), generator=g, device=DEV).to(torch.int32)
    s["tokens"] = torch.zeros((B, 500 + c["nodes"]), dtype=torch.int32, device=DEV)
    s["lens"] = s["before"].clone()
    if own:
        from quantized_speculative_verify_gb300 import hq
        s["hq"], s["state"] = hq, hq.History(s["tokens"], s["lens"])
        s["path"] = torch.empty((B, c["nodes"]), dtype=torch.int32, device=DEV)
        s["n"], s["bonus"] = torch.empty(B, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
    return s


def _prepare_gate(c, g):
    s = dict(c)
    M, K = c["rows"], c["heads"] * c["dim"]
    s["xs"] = (0.5 * torch.randn((M, K), generator=g, device=DEV)).to(TYPES[c["x"]])
    s["gates"] = (1.5 * torch.randn((M, K), generator=g, device=DEV)).to(TYPES[c["h"]])
    s["weight"] = 1.0 + 0.2 * torch.randn(c["dim"], generator=g, device=DEV) if c["norm"] else None
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
        s["h_out"] = torch.empty((M, K), dtype=TYPES[c["h"]], device=DEV)
        if c["codes"]:
            s["qx"] = torch.empty((M, K), dtype=torch.int8, device=DEV)
            s["sx"] = torch.empty(M, dtype=torch.float32, device=DEV)
            s["values"] = torch.empty((M, K), dtype=TYPES[c["h"]], device=DEV)
    return s


# --------------------------------------------------------------- the passes ---
def run(s):
    return {"rope": _run_rope, "pick": _run_pick, "accept": _run_accept, "gate": _run_gate}[s["op"]](s)


def _ancestors(s):
    """[B][m][m]: node j is node i itself or one of its ancestors (rows past a sequence's own: themselves)."""
    B, m = s["batch"], s["nodes"]
    a = torch.eye(m, device=DEV).expand(B, m, m).clone()
    a[s["row_seq"], s["row_node"], s["parent"].long()] = 1.0
    for _ in range(max(1, (m - 1).bit_length())):
        a = (torch.bmm(a, a) > 0).float()
    return a


def _head_norm(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _run_rope(s):
    if own:
        s["hq"].rope_write(s["cache"], 0, 1, s["q"], s["k"], s["v"], s["turns"], s["starts"], s["nodes"], s["layout"],
                           gain=s["gain"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, parent=s["parent"], out=s["out"])
        return {"q": s["out"], "pool": s["pool"]}
    b, i, r, ps = s["row_seq"], s["row_node"], s["rot"], s["page"]
    place = (s["lens"] - (s["starts"][1:] - s["starts"][:-1])).long()[b] + i  # in the cache
    at = place if s["parent"] is None else place - i + (_ancestors(s).sum(2).long() - 1)[b, i]
    a = at.double().unsqueeze(1) * s["freqs"]
    c, n = (torch.cos(a) * s["gain"]).float().unsqueeze(1), (torch.sin(a) * s["gain"]).float().unsqueeze(1)

    def rotated(x, weight):
        x = x.float()
        if weight is not None:
            x = _head_norm(x, weight)
        if s["layout"] == "half":
            u, v = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat([u * c - v * n, v * c + u * n], 2)
        else:
            u, v = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack([u * c - v * n, v * c + u * n], 3).flatten(2)
        return torch.cat([y, x[..., r:]], 2).to(TYPES[s["type"]])

    page = s["table"][b, place // ps].long()
    s["pool"][0, page, :, place % ps] = rotated(s["k"], s["kw"])
    s["pool"][1, page, :, place % ps] = s["v"].to(TYPES[s["type"]])
    return {"q": rotated(s["q"], s["qw"]), "pool": s["pool"]}


def _run_pick(s):
    if own:
        s["hq"].greedy_tokens(s["logits"], s["starts"], s["nodes"], parent=s["parent"], tokens=s["draft"], history=s["state"],
                              rules=s["rules"], mask_ids=s.get("mask_ids"), out=s["adjusted"], greedy=s["greedy"],
                              workspace=s["ws"])
        return {"greedy": s["greedy"], "adjusted": s["adjusted"]}
    B, m, V, b, i = s["batch"], s["nodes"], s["vocab"], s["row_seq"], s["row_node"]
    col = torch.arange(s["tokens"].shape[1], device=DEV)
    held = (col < s["lens"].unsqueeze(1)).to(torch.int32)
    made = held * (col >= s["prompt"].unsqueeze(1))
    # the drafted tokens on each row's path, its own among them, the root's not (it is in the history)
    drafts = torch.zeros((B, m), dtype=torch.int64, device=DEV)
    drafts[b, i] = s["draft"].long()
    on = _ancestors(s).to(torch.int32)
    on[:, :, 0] = 0
    none = torch.zeros((B, V), dtype=torch.int32, device=DEV)
    seen, count = (none.scatter_add(1, s["tokens"].long(), w)[b].scatter_add_(1, drafts[b], on[b, i]) for w in (held, made))
    x = s["logits"].float()
    rep, pres, freq = (s[k][b].unsqueeze(1) for k in ("repetition", "presence", "frequency"))
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = torch.where(count > 0, x - freq * count - pres, x)
    if s["bias"]:
        bias = torch.zeros((B, V), device=DEV).scatter_(1, s["bias_tokens"].view(B, -1).long(), s["bias_values"].view(B, -1))
        x = x + bias[b]
    top = torch.arange(V, device=DEV)
    if s["masked"]:
        ids = s["mask_ids"].long()
        word = s["masks"][ids.clamp(min=0)][:, top // 32]
        x = torch.where((ids >= 0).unsqueeze(1) & ((word >> (top % 32)) & 1 == 0), torch.full_like(x, -math.inf), x)
    most = x.amax(1, keepdim=True)
    greedy = torch.where(x == most, top, V).amin(1)
    greedy = torch.where(most.squeeze(1) > -math.inf, greedy, torch.full_like(greedy, -1)).to(torch.int32)
    return {"greedy": greedy, "adjusted": x.to(s["logits"].dtype) if s["out"] else None}


def _run_accept(s):
    s["lens"].copy_(s["before"])  # every pass starts from the same histories
    if own:
        s["hq"].tree_accept_batch(s["greedy"], s["parent"], s["draft"], s["starts"], s["nodes"], history=s["state"],
                                  path=s["path"], n_accept=s["n"], bonus=s["bonus"])
        return {"path": s["path"], "n": s["n"], "bonus": s["bonus"], "tokens": s["tokens"], "lens": s["lens"]}
    B, m, b, i = s["batch"], s["nodes"], s["row_seq"], s["row_node"]
    greedy, draft = (torch.full((B, m), -1, dtype=torch.int64, device=DEV) for _ in range(2))
    parent, real = torch.zeros((B, m), dtype=torch.int64, device=DEV), torch.zeros((B, m), dtype=torch.bool, device=DEV)
    greedy[b, i], draft[b, i], parent[b, i], real[b, i] = s["greedy"].long(), s["draft"].long(), s["parent"].long(), True
    node = torch.arange(m, device=DEV)
    over = _ancestors(s)
    agrees = (node == 0) | (real & (draft == torch.gather(greedy, 1, parent)))
    depth = over.sum(2).long() - 1
    valid = real & (torch.bmm(over, (~agrees).float().unsqueeze(2)).squeeze(2) == 0)
    best = (torch.where(valid, depth, -1) * m + (m - 1 - node)).argmax(1, keepdim=True)
    n = torch.gather(depth, 1, best)
    on = (over[torch.arange(B, device=DEV), best.squeeze(1)] > 0) & (node > 0)
    at = torch.where(on, depth - 1, m)
    path = torch.full((B, m + 1), -1, dtype=torch.int64, device=DEV).scatter_(1, at, node.expand(B, m))[:, :m]
    bonus = torch.gather(greedy, 1, best)
    # the histories grow by the accepted drafts and the model's own token
    grown = torch.where(node < n, torch.gather(draft, 1, path.clamp(min=0)), bonus)
    to = torch.where(node <= n, s["before"].long().unsqueeze(1) + node, s["tokens"].shape[1])
    wide = torch.cat([s["tokens"], s["tokens"][:, :1]], 1).scatter_(1, to, grown.to(torch.int32))
    s["tokens"].copy_(wide[:, :-1])
    s["lens"].add_(n.squeeze(1).to(torch.int32) + 1)
    return {"path": path.to(torch.int32), "n": n.squeeze(1).to(torch.int32), "bonus": bonus.squeeze(1).to(torch.int32),
            "tokens": s["tokens"], "lens": s["lens"]}


def _run_gate(s):
    if own:
        if not s["codes"]:
            s["hq"].gated_norm_quant(s["desc"], s["xs"], s["gates"], s["weight"], None, s["dim"], s["act"], EPS, h=s["h_out"])
            return {"h": s["h_out"]}
        s["hq"].gated_norm_quant(s["desc"], s["xs"], s["gates"], s["weight"], s["signs"], s["dim"], s["act"], EPS,
                                 h=s["h_out"], qx=s["qx"], sx=s["sx"])
        torch.mul(s["qx"], s["sx"].unsqueeze(1), out=s["values"])  # the codes as the values they stand for
        return {"h": s["h_out"], "scale": s["sx"], "values": s["values"]}
    M, K = s["xs"].shape
    x, z = s["xs"].float().view(M, -1, s["dim"]), s["gates"].float()
    if s["weight"] is not None:
        x = _head_norm(x, s["weight"])
    if s["act"] != "none":
        z = torch.sigmoid(z) * (z if s["act"] == "silu" else 1.0)
    y = x.reshape(M, K) * z
    if not s["codes"]:
        return {"h": y.to(TYPES[s["h"]])}
    z = ((y * s["pm"]).view(-1, 32) @ s["hadamard"]).view(M, K) * (1.0 / math.sqrt(32.0))
    sx = z.abs().amax(1) / 127.0
    q = torch.clamp(torch.round(z / sx.unsqueeze(1)), -127, 127)
    return {"h": y.to(TYPES[s["h"]]), "scale": sx, "values": (q * sx.unsqueeze(1)).to(TYPES[s["h"]])}


# ------------------------------------------------------- the same in 64 bits ---
def exact(c, seed):
    s = prepare(c, seed)
    return {"rope": _exact_rope, "pick": _exact_pick, "accept": _exact_accept, "gate": _exact_gate}[c["op"]](s)


def _paths(s, b):
    """The nodes from the root to each node of sequence b's tree."""
    first, last = int(s["starts"][b]), int(s["starts"][b + 1])
    parent, found = s["parent"][first:last].tolist(), [[0]]
    for i in range(1, last - first):
        found.append(found[parent[i]] + [i])
    return first, found


def _exact_rope(s):
    starts, lens, table, ps, r, D = s["starts"].tolist(), s["lens"].tolist(), s["table"].tolist(), s["page"], s["rot"], s["dim"]
    at, page, slot = [], [], []
    for b, n in enumerate(lens):
        m = starts[b + 1] - starts[b]
        deep = list(range(m)) if s["parent"] is None else [len(p) - 1 for p in _paths(s, b)[1]]
        at += [n - m + d for d in deep]
        page += [table[b][(n - m + i) // ps] for i in range(m)]
        slot += [(n - m + i) % ps for i in range(m)]
    turn = torch.polar(torch.full((len(at), r // 2), float(s["gain"]), dtype=torch.float64, device=DEV),
                       torch.outer(torch.tensor(at, dtype=torch.float64, device=DEV), s["freqs"])).unsqueeze(1)

    def rotated(x, weight):  # pairs as complex numbers
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + EPS) * weight.double()
        part = x[..., :r]
        if s["layout"] == "half":
            y = torch.view_as_real(torch.complex(*part.chunk(2, -1)) * turn).transpose(-1, -2)
        else:
            y = torch.view_as_real(torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn)
        return torch.cat([y.flatten(-2), x[..., r:]], -1)

    pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device=DEV)
    pool[0, page, :, slot] = rotated(s["k"], s["kw"])
    pool[1, page, :, slot] = s["v"].double()
    return {"q": rotated(s["q"], s["qw"]), "pool": pool}


def _exact_pick(s):
    V, words = s["vocab"], -(-s["vocab"] // 32)
    rows, greedy = [], []
    for b in range(s["batch"]):
        first, paths = _paths(s, b)
        text, made = s["tokens"][b, :int(s["lens"][b])].long(), int(s["prompt"][b])
        for i, path in enumerate(paths):
            drafted = s["draft"][[first + j for j in path[1:]]].long() if len(path) > 1 else text[:0]
            after = torch.bincount(torch.cat([text[made:], drafted]), minlength=V).double()
            there = torch.bincount(torch.cat([text, drafted]), minlength=V) > 0
            x = s["logits"][first + i].double()
            rep = float(s["repetition"][b])
            x[there] = torch.where(x[there] > 0, x[there] / rep, x[there] * rep)
            x = x - after * float(s["frequency"][b]) - (after > 0).double() * float(s["presence"][b])
            if s["bias"]:
                lo, hi = int(s["bias_starts"][b]), int(s["bias_starts"][b + 1])
                x[s["bias_tokens"][lo:hi].long()] += s["bias_values"][lo:hi].double()
            if s["masked"] and int(s["mask_ids"][first + i]) >= 0:
                word = s["masks"][int(s["mask_ids"][first + i])].view(words, 1).long()
                allowed = ((word >> torch.arange(32, device=DEV)) & 1).flatten()[:V] > 0
                x = x.masked_fill(~allowed, -math.inf)
            if s["out"]:
                rows.append(x)
            most = x.max()
            greedy.append(int((x == most).nonzero()[0]) if float(most) > -math.inf else -1)
    return {"greedy": _ints(greedy), "adjusted": torch.stack(rows) if s["out"] else None}


def _exact_accept(s):
    tokens, before = s["tokens"].clone(), s["before"].tolist()
    lens, path, counts, bonus = [], [], [], []
    for b in range(s["batch"]):
        first, paths = _paths(s, b)
        greedy = s["greedy"][first:first + len(paths)].tolist()
        draft = s["draft"][first:first + len(paths)].tolist()
        best = [0]
        for p in paths:
            if len(p) > len(best) and all(draft[j] == greedy[i] for i, j in zip(p, p[1:])):
                best = p
        more = [draft[j] for j in best[1:]] + [greedy[best[-1]]]
        tokens[b, before[b]:before[b] + len(more)] = _ints(more)
        lens.append(before[b] + len(more))
        path.append(best[1:] + [-1] * (s["nodes"] - len(best) + 1))
        counts.append(len(best) - 1)
        bonus.append(more[-1])
    return {"path": _ints(path), "n": _ints(counts), "bonus": _ints(bonus), "tokens": tokens, "lens": _ints(lens)}


def _exact_gate(s):
    M, K = s["xs"].shape
    x, z = s["xs"].double().view(M, -1, s["dim"]), s["gates"].double()
    if s["weight"] is not None:
        x = x / torch.sqrt((x ** 2).sum(2, keepdim=True) / s["dim"] + EPS) * s["weight"].double()
    y = x.reshape(M, K) * {"none": z, "sigmoid": 1.0 / (1.0 + torch.exp(-z)), "silu": z / (1.0 + torch.exp(-z))}[s["act"]]
    if not s["codes"]:
        return {"h": y}
    z = y * s["pm"].double()
    for half in (1, 2, 4, 8, 16):  # the butterfly of the Hadamard product, one stride after the other
        u = z.view(M, -1, 2, half)
        z = torch.stack([u[:, :, 0] + u[:, :, 1], u[:, :, 0] - u[:, :, 1]], 2).reshape(z.shape)
    z = z / math.sqrt(32.0)
    sx = z.abs().max(1).values / 127.0
    return {"h": y, "scale": sx, "values": torch.round(z / sx[:, None]).clamp(-127, 127) * sx[:, None]}
