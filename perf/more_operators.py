"""Measured cases of what a decode loop has around its ternary projections and its 4-bit key/value cache: rotary
positions, the attention weight that cached tokens gather, eviction by that weight, and products with 4-bit weights.

Rotary positions. Pair i of a head's first `dims` numbers (half layout: numbers i and i + dims / 2; interleaved: 2 i and
2 i + 1) is turned by the angle p f_i of the row's position p, and multiplied by a magnitude; the rest of the head stays:

    f_i = base^(-2 i / dims)
    linear         f_i / factor
    ntk            base^(-2 i / dims) with base * factor^(dims / (dims - 2)) in place of base
    by_parts       f_i (1 - r) + f_i / factor r,  r = clamp((i - a) / max(b - a, 0.001), 0, 1), a = max(floor(d(high)), 0),
                   b = min(ceil(d(low)), dims - 1), d(n) = dims / 2 ln(original / (2 pi n)) / ln(base);
                   the magnitude is 0.1 ln(factor) + 1
    by_wavelength  f_i (t + (1 - t) / factor),  t = clamp((original f_i / (2 pi) - low) / (high - low), 0, 1)

Gathered weight. The cache holds keys and values as 4-bit codes in pages of 64 tokens (see operators.py for the format);
beside it lies one fp32 number for each page, key/value head and place. A call's queries vote: of each sequence's n new
tokens the last `voters` (0: all), each with the softmax weights of the positions that it sees (j <= p, and within the
window or among the first tokens). For a token that is older than the call: decay * mass + votes; for the call's own
tokens: votes. Votes of the query heads that share a key/value head are added up.

Eviction. A sequence of more than `limit` cached tokens keeps `budget` of them in each key/value head: the first
`sinks`, the last `recent`, and the ones of the greatest mass among the others (ties: the earlier one); in order, at
places 0, 1, ... of the pages that a second table names, with their mass. Shorter sequences keep all tokens.

Products with 4-bit weights. A row of N x K weights is held as codes 0..15, code k in byte k / 2 (even k: low nibble), with an
fp16 scale and a zero point (8 where none are given) for each group of K: w = scale (code - zero); out = x w^T in fp32.
"""
import math

import torch

own = False

PAGE = 64

# heads of the queries, heads of the cache, dimension: 4:1 sharing as in the 2560-wide decode workload, and generic ones
HEADS = ((20, 5, 128), (32, 8, 64), (12, 12, 64), (16, 2, 128), (28, 4, 128), (8, 1, 128), (24, 8, 64))
SCALINGS = ("none", "linear", "ntk", "by_parts", "by_wavelength")


def _rope(name, rows, heads, dims, layout, scaling, first, dtype):
    c = {"op": "rope", "rows": rows, "q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "dims": dims, "layout": layout,
         "scaling": scaling, "base": 500000.0, "factor": 1.0 if scaling == "none" else 8.0, "original": 8192, "first": first, "dtype": dtype}
    return dict(c, name=name) if name else c


def _mass(name, batch, heads, q, ctx, dtype="bf16", window=0, sinks=0, voters=0, decay=1.0):
    """q and ctx: the least and the greatest number of new tokens and of tokens cached before them."""
    c = {"op": "mass", "batch": batch, "q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "q_min": q[0], "q_max": q[1],
         "ctx_min": ctx[0], "ctx_max": ctx[1], "dtype": dtype, "window": window, "sinks": sinks, "voters": voters, "decay": decay}
    return dict(c, name=name) if name else c


def _evict(name, batch, heads, lengths, budget, limit, sinks, recent):
    c = {"op": "evict", "batch": batch, "kv_heads": heads[1], "dim": heads[2], "q_min": 0, "q_max": 0, "ctx_min": lengths[0],
         "ctx_max": lengths[1], "budget": budget, "limit": limit, "sinks": sinks, "recent": recent}
    return dict(c, name=name) if name else c


def _w4(name, rows, n, k, group, zeros, dtype):
    c = {"op": "w4", "rows": rows, "N": n, "K": k, "group": group, "zeros": zeros, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    h2b = HEADS[0]
    return [
        # one user's decode step far into a scaled context: one token's queries and keys
        _rope("rope_token", 1, h2b, 128, "half", "by_parts", 131006, "f32"),
        # prompts of 16,000 tokens in all as the projections give them, fp32
        _rope("rope_prompts", 16001, h2b, 128, "half", "none", 0, "f32"),
        # the first steps after a short question: latency alone
        _mass("mass_short", 1, h2b, (1, 1), (76, 76)),
        # one user with a very long context: the whole GPU on one sequence
        _mass("mass_long", 1, h2b, (1, 1), (131006, 131006)),
        # a server's decode step over contexts of unlike lengths, fp32 queries, old votes fading
        _mass("mass_batch", 64, h2b, (1, 1), (17, 8175), "f32", decay=0.98),
        # prompts whose last 64 tokens vote on all before them
        _mass("mass_last", 5, h2b, (999, 9001), (0, 70), voters=64),
        # a prompt all of whose tokens vote
        _mass("mass_prompt", 1, h2b, (2048, 2048), (0, 0)),
        # one very long cache is cut to 4096 tokens
        _evict("evict_long", 1, h2b, (131007, 131007), 4096, 8192, 4, 1024),
        # a server's caches of unlike lengths are cut to 2048 tokens where they are longer
        _evict("evict_batch", 48, h2b, (501, 16001), 2048, 2048, 4, 256),
        # one token through one layer's matrix
        _w4("layer_token", 1, 2560, 6912, 128, False, "bf16"),
        # one token's logits
        _w4("head_token", 1, 131072, 2560, 128, False, "f32"),
        # the logits of a server's decode step, zero points, small groups
        _w4("head_batch", 16, 131071, 2560, 64, True, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "rope", "mass", "mass", "mass", "mass", "evict", "evict", "w4", "w4", "w4"))
    heads, dtype = rng.choice(HEADS), rng.choice(("bf16", "f32"))
    width = heads[1] * heads[2] / 640
    if op == "rope":
        heads = heads[:2] + (rng.choice((heads[2], heads[2], 80, 96, 256)),)
        rows = _log(rng, 1, 16000 * 3200 / ((heads[0] + heads[1]) * heads[2]))
        dims = heads[2] // rng.choice((1, 1, 2)) // 8 * 8
        return _rope(None, rows, heads, dims, rng.choice(("half", "interleaved")), rng.choice(SCALINGS), _log(rng, 1, 1000000), dtype)
    if op == "evict":
        total = _log(rng, 64, 400000 / width)
        batch = min(_log(rng, 1, 64), total)
        top = max(1, min(total // batch, 131000))
        budget = max(1, _log(rng, 1, top))
        sinks = min(rng.choice((0, 1, 4, 70)), budget)
        return _evict(None, batch, heads, (top // rng.choice((1, 3, 20)), top), budget, budget + rng.choice((0, 0, top // 8)), sinks,
                      rng.randint(0, budget - sinks))
    if op == "w4":
        k = 128 * _log(rng, 1, 64)
        return _w4(None, _log(rng, 1, 32), _log(rng, 16, min(131072, 131072 * 2560 // k)), k, rng.choice((32, 64, 128)), rng.random() < 0.5, dtype)
    window, sinks = (0, 0) if rng.random() < 0.6 else (_log(rng, 1, 5000), rng.choice((0, 1, 4, 70)))
    decay = rng.choice((1.0, 0.95))
    if rng.random() < 0.6:  # a few voting queries a sequence
        total = _log(rng, 64, 250000 / width)
        batch = min(_log(rng, 1, 64), total)
        top = max(1, min(total // batch, 131000))
        q = rng.choice((1, 1, 1, 2, 5, 8))
        return _mass(None, batch, heads, (1 if q > 4 else q, q), (top // rng.choice((1, 3, 20)), top), dtype, window, sinks, 0, decay)
    pairs = _log(rng, 20000, 2.0e6 * 2560 / (heads[0] * heads[2]))  # voting queries times what they see, in all
    batch = rng.choice((1, 1, 2, 5))
    n = min(2000, max(9, _log(rng, 9, math.sqrt(2 * pairs / batch))))
    voters = rng.choice((0, 16, 33, 64, 200))
    ctx = 0 if rng.random() < 0.4 else min(9000, max(0, int(pairs / batch / n) - n // 2))
    return _mass(None, batch, heads, (max(1, n // rng.choice((1, 1, 4))), n), (ctx // 2, ctx), dtype, window, sinks, voters, decay)


def _lengths(case):
    """Each sequence's new tokens and cached tokens (the new ones among them): spread over the case's ranges, the same for every seed."""
    new, kv = [], []
    for b in range(case["batch"]):
        u, v = ((b + 1) * 0.6180339887498949) % 1.0, ((b + 1) * 0.7548776662466927) % 1.0
        if case["batch"] == 1:
            u = v = 1.0
        new.append(case["q_min"] + int(round(u * (case["q_max"] - case["q_min"]))))
        kv.append(new[-1] + case["ctx_min"] + int(round(v * (case["ctx_max"] - case["ctx_min"]))))
    return new, kv


def _frequencies(case):
    """The angle that one position adds to each pair, in 64 bits, and the magnitude."""
    dims, base, s = case["dims"], case["base"], case["factor"]
    i = torch.arange(dims // 2, dtype=torch.float64)
    if case["scaling"] == "ntk" and dims > 2:
        base = base * s ** (dims / (dims - 2))
    f = base ** (-2.0 * i / dims)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "by_parts":
        at = lambda n: dims / 2 * math.log(case["original"] / (2 * math.pi * n)) / math.log(base)  # noqa: E731
        a, b = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), dims - 1)
        r = ((i - a) / max(b - a, 0.001)).clamp(0, 1)
        return f * (1 - r) + f / s * r, 0.1 * math.log(s) + 1
    if case["scaling"] == "by_wavelength":
        t = ((case["original"] * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f * (t + (1 - t) / s)
    return f, 1.0


def _rho(t):
    return (t & ~7) | ((t & 3) << 1) | ((t >> 2) & 1)


def _fields(pages, dim):
    """Views of a cache's pages (pages x heads x block bytes): key rows, value rows, parameters."""
    at = PAGE * dim // 2
    return (pages[:, :, :at].unflatten(2, (PAGE, dim // 2)), pages[:, :, at:2 * at].unflatten(2, (PAGE, dim // 2)),
            pages[:, :, 2 * at:].view(torch.float16).unflatten(2, (PAGE, 4)))


def _keys(pages, dim, page, off):
    """The fp32 keys at places `page`, `off` (any shape): that shape x heads x dim. Nibble n of word w is dimension w + dim / 8 n."""
    fk, _, fp = _fields(pages, dim)
    words = fk[page, :, _rho(off)]
    par = fp[page, :, _rho(off)].float()
    code = torch.stack((words & 15, words >> 4), -1).flatten(-2).unflatten(-1, (dim // 8, 8)).transpose(-1, -2).flatten(-2)
    return code.float() * par[..., 0:1] + par[..., 1:2]


def _table(lengths, ids):
    """A page table that deals the pages `ids` out to sequences of these lengths, in order."""
    need = [-(-n // PAGE) for n in lengths]
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table.cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    t = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    state = {"case": case}
    if case["op"] == "rope":
        # a batch's rows: positions run on within a sequence, and begin anew at every thousandth row or so
        row = torch.arange(case["rows"], device="cuda")
        state["positions"] = (case["first"] + row % 997 + 13 * (row // 997)).to(torch.int32)
        state["q"] = rand(case["rows"], case["q_heads"], case["dim"]).to(t)
        state["k"] = rand(case["rows"], case["kv_heads"], case["dim"]).to(t)
        f, state["magnitude"] = _frequencies(case)
        state["frequencies"] = f.cuda()
        if own:  # the table that a program keeps for its model
            from ternary_weight_gb300 import binding
            state["table"] = binding.Rope(case["dims"], base=case["base"], layout=case["layout"], scaling=case["scaling"],
                                          factor=case["factor"], original=case["original"])
        return state
    if case["op"] == "w4":
        groups = case["K"] // case["group"]
        state["codes"] = byte(case["N"], case["K"] // 2)
        state["scales"] = (0.01 * (0.3 + torch.rand(case["N"], groups, generator=g, device="cuda"))).half()
        state["zeros"] = torch.randint(5, 11, (case["N"], groups), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        # activations have channels much larger than the others
        state["x"] = (rand(case["rows"], case["K"]) * (0.5 + rand(1, case["K"]).abs() ** 3)).to(t)
        return state
    new, kv = _lengths(case)
    h, d = case["kv_heads"], case["dim"]
    keeps = [] if case["op"] == "mass" else [n if n <= case["limit"] else case["budget"] for n in kv]
    need, more = sum(-(-n // PAGE) for n in kv), sum(-(-n // PAGE) for n in keeps)
    n_pages = need + more + 3
    ids = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed + 1)).to(torch.int32)  # a used pool: pages lie in any order
    pages = byte(n_pages, h, PAGE * d + 512)
    step = 0.05 + 0.1 * torch.rand(n_pages, h, PAGE, 2, generator=g, device="cuda")
    base = (0.3 * rand(n_pages, h, PAGE, 2) - 7.5) * step
    _fields(pages, d)[2].copy_(torch.stack((step, base), -1).flatten(-2))
    # few tokens hold most of the weight; of a step's votes a token gets thousandths
    state["mass"] = torch.exp(2.0 * rand(n_pages, h, PAGE)) * (1.0 if case["op"] == "evict" else 0.001)
    if case["op"] == "evict":  # weights that are equal, and tokens that never got any
        state["mass"] = torch.where(state["mass"] < 0.5, 0.0, (state["mass"] * 64).round() / 64)
    state["pages"], state["table"] = pages, _table(kv, ids)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    state["kv_len"], state["max_kv"] = i32(kv), max(kv)
    state["cu_q"], state["rows"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda(), sum(new)
    if case["op"] == "evict":
        state["into"] = _table(keeps, ids[need:])
        state["most"] = max(keeps)
    else:
        state["q"], state["max_q"] = (3.0 * rand(sum(new), case["q_heads"], d)).to(t), max(new)
        state["out"] = state["mass"].clone()
    if own:  # the handles that a program keeps beside its pool of pages and its batch
        from ternary_weight_gb300 import binding
        state["cache"] = binding.KV4Cache(n_pages, h, d, pages=pages.view(-1))
        state["batch"] = binding.KV4Batch(state["cu_q"], state["kv_len"], state["table"], state["rows"], max(1, max(new)), max(kv))
    return state


def run(state):
    case = state["case"]
    if own:
        from ternary_weight_gb300 import binding
        if case["op"] == "rope":
            return binding.rope(state["table"], state["positions"], state["q"], state["k"])
        if case["op"] == "w4":
            return binding.w4_matmul(state["x"], state["codes"], state["scales"], zeros=state["zeros"])
        if case["op"] == "mass":
            return binding.kv4_attention_mass(state["cache"], state["batch"], state["q"], 1.0 / math.sqrt(case["dim"]), state["mass"],
                                              decay=case["decay"], window=case["window"], sinks=case["sinks"], voters=case["voters"],
                                              out=state["out"])
        length = binding.kv4_evict(state["cache"], state["batch"], state["mass"], case["budget"], limit=case["limit"], sinks=case["sinks"],
                                   recent=case["recent"], into=state["into"])
        return state["pages"], state["mass"], length
    if case["op"] == "rope":
        angle = state["positions"].double()[:, None] * state["frequencies"]
        cos, sin = ((f(angle) * state["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
        return tuple(_turned(state[x], cos, sin, case) for x in ("q", "k"))
    if case["op"] == "w4":
        codes = torch.stack((state["codes"] & 15, state["codes"] >> 4), -1).flatten(1).float().unflatten(1, (-1, case["group"]))
        zeros = 8.0 if state["zeros"] is None else state["zeros"].float()[..., None]
        return state["x"].float() @ ((codes - zeros) * state["scales"].float()[..., None]).flatten(1).T
    return _gathered(state) if case["op"] == "mass" else _evicted(state)


def _turned(x, cos, sin, case):
    dims, t = case["dims"], x.float()
    if case["layout"] == "half":
        a, b = t[..., :dims // 2], t[..., dims // 2:dims]
        both = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = t[..., 0:dims:2], t[..., 1:dims:2]
        both = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((both, t[..., dims:]), -1).to(x.dtype)


def _gathered(state):
    """All sequences at once, padded to the longest: softmax weights of the voting queries, added up for each cached token."""
    case = state["case"]
    b, h, d = case["batch"], case["kv_heads"], case["dim"]
    r = case["q_heads"] // h
    n = min(state["max_q"], case["voters"]) if case["voters"] else state["max_q"]
    kv, cu = state["kv_len"].long()[:, None], state["cu_q"].long()
    count = (cu[1:] - cu[:-1])[:, None]
    back = torch.arange(n, device="cuda")  # 0: a sequence's last query
    votes = back < count
    q = state["q"].float()[(cu[1:, None] - 1 - back).clamp(min=0)].unflatten(2, (h, r))
    at = kv - 1 - back  # positions of the queries
    j = torch.arange(state["max_kv"], device="cuda").expand(b, -1)
    page = state["table"].gather(1, j // PAGE).long().clamp(min=0)
    here = j < kv
    s = torch.einsum("bnhrd,blhd->bhrnl", q, _keys(state["pages"], d, page, j % PAGE)) * (1.0 / math.sqrt(d))
    sees = (j[:, None, :] <= at[..., None]) & votes[..., None]
    if case["window"]:
        sees = sees & ((j[:, None, :] > at[..., None] - case["window"]) | (j[:, None, :] < case["sinks"]))
    s = s.masked_fill(~sees[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    votes = (s / s.sum(-1, keepdim=True).clamp(min=1e-30)).sum((2, 3)).transpose(1, 2)  # batch x tokens x heads
    old = state["mass"][page, :, j % PAGE]
    new = torch.where((j < kv - count)[..., None], case["decay"] * old + votes, votes)
    state["out"][page[here], :, (j % PAGE)[here]] = new[here]
    return state["out"]


def _evicted(state):
    """All sequences at once, padded to the longest: the kept tokens of each head by a stable sort of the masses, then one gather."""
    case, pages, mass = state["case"], state["pages"], state["mass"]
    b, h = case["batch"], case["kv_heads"]
    kv = state["kv_len"].long()[:, None]
    cut = kv > case["limit"]
    keeps = torch.where(cut, case["budget"], kv)
    j = torch.arange(state["max_kv"], device="cuda").expand(b, -1)
    page = state["table"].gather(1, j // PAGE).long().clamp(min=0)
    weight = mass[page, :, j % PAGE].transpose(1, 2)  # batch x heads x tokens
    sure = ~cut | (j < case["sinks"]) | (j >= kv - case["recent"])
    weight = weight.masked_fill(sure[:, None], math.inf).masked_fill((j >= kv)[:, None], -math.inf)
    order = weight.sort(dim=-1, descending=True, stable=True).indices[..., :state["most"]]
    to = torch.arange(order.shape[2], device="cuda").expand(b, h, -1)
    there = to < keeps[..., None]
    at = torch.where(there, order, state["max_kv"]).sort(dim=-1).values
    head = torch.arange(h, device="cuda")[:, None].expand(b, h, to.shape[2])[there]
    seq = torch.arange(b, device="cuda")[:, None, None].expand_as(to)[there]
    at, to = at[there], to[there]
    p0, p1 = state["table"][seq, at // PAGE].long(), state["into"][seq, to // PAGE].long()
    o0, o1 = at % PAGE, to % PAGE
    fk, fv, fp = _fields(pages, case["dim"])
    fk[p1, head, _rho(o1)] = fk[p0, head, _rho(o0)]
    fp[p1, head, _rho(o1)] = fp[p0, head, _rho(o0)]
    v = fv[p0, head, o0]
    if case["dim"] == 128:  # the halves of a value row are exchanged where bit 1 of its place is set
        v = torch.where((((o0 ^ o1) & 2) != 0)[:, None], v.roll(v.shape[1] // 2, -1), v)
    fv[p1, head, o1] = v
    mass[p1, head, o1] = mass[p0, head, o0]
    return pages, mass, keeps[:, 0].to(torch.int32)


def _seen(case):
    """For each sequence: the pairs of a voting query and a position it sees, and the positions that any of them sees."""
    got = []
    for n, kv in zip(*_lengths(case)):
        votes = min(n, case["voters"]) if case["voters"] else n
        w, s = case["window"] or kv, case["sinks"]
        pairs = 0
        for p in (range(kv - votes, kv) if case["window"] else ()):
            low = max(0, p - w + 1)
            pairs += p + 1 - low + min(s, low)
        if not case["window"]:
            pairs = votes * (2 * kv - votes + 1) // 2
        low = max(0, kv - votes - w + 1)
        got.append((pairs, kv - low + min(s, low), votes))
    return got


def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "rope":
        numbers = case["rows"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * numbers * size + 4 * case["rows"], "flops": 3 * numbers * case["dims"] / case["dim"]}
    if case["op"] == "w4":
        groups = case["N"] * case["K"] // case["group"]
        return {"bytes": case["N"] * case["K"] // 2 + groups * (3 if case["zeros"] else 2) + case["rows"] * (case["K"] * size + 4 * case["N"]),
                "flops": 2 * case["rows"] * case["N"] * case["K"]}
    new, kv = _lengths(case)
    vector = case["dim"] // 2 + 4  # bytes of a stored vector
    if case["op"] == "evict":
        moved = sum(n if n <= case["limit"] else case["budget"] for n in kv)
        read = sum(n for n in kv if n > case["limit"])
        return {"bytes": case["kv_heads"] * (4 * read + 2 * moved * (2 * vector + 4)), "flops": 0}
    seen = _seen(case)
    touched = [n if case["decay"] != 1.0 else min(n, max(s, m)) for (_, s, _), m, n in zip(seen, new, kv)]
    old = sum(t - min(m, t) for t, m in zip(touched, new))
    return {"bytes": case["kv_heads"] * (sum(s for _, s, _ in seen) * vector + 4 * (old + sum(touched)))
            + sum(v for _, _, v in seen) * case["q_heads"] * case["dim"] * size,
            "flops": 2 * case["dim"] * case["q_heads"] * sum(p for p, _, _ in seen)}


def exact(case, seed):
    """From the definitions, in 64 bits: pair by pair, sequence by sequence, head by head."""
    state = prepare(case, seed)
    if case["op"] == "rope":
        outs = []
        where = state["positions"].to(torch.float64)
        for x in (state["q"].double(), state["k"].double()):
            y = x.clone()
            for i in range(case["dims"] // 2):
                a, b = (i, i + case["dims"] // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
                turn = torch.polar(torch.full_like(where, state["magnitude"]), where * state["frequencies"][i])
                z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
                y[..., a], y[..., b] = z.real, z.imag
            outs.append(y)
        return tuple(outs)
    if case["op"] == "w4":
        parts = []
        for rows in torch.arange(case["N"], device="cuda").split(16384):
            w = torch.empty(len(rows), case["K"], dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = state["codes"][rows] % 16, state["codes"][rows] // 16
            zero = 8 if state["zeros"] is None else state["zeros"][rows].double().repeat_interleave(case["group"], 1)
            parts.append(state["x"].double() @ ((w - zero) * state["scales"][rows].double().repeat_interleave(case["group"], 1)).T)
        return torch.cat(parts, 1)
    new, kv = _lengths(case)
    table, mass, d = state["table"].tolist(), state["mass"].double(), case["dim"]
    if case["op"] == "evict":
        into, moved = state["into"].tolist(), mass.clone()
        for b, n in enumerate(kv):
            line = mass[table[b][:-(-n // PAGE)]].transpose(0, 1).flatten(1)[:, :n]  # heads x tokens
            if n > case["limit"]:
                middle = torch.arange(case["sinks"], n - case["recent"], device="cuda")
                count = case["budget"] - case["sinks"] - case["recent"]
                kept = []
                for row in line:
                    # the greatest value that `count` tokens reach; above it all are kept, at it the earliest
                    least = torch.topk(row[middle], count).values[-1] if count else math.inf
                    above, level = middle[row[middle] > least], middle[row[middle] == least]
                    chosen = torch.cat((above, level[:count - len(above)])) if count else middle[:0]
                    ends = torch.cat((torch.arange(case["sinks"], device="cuda"), torch.arange(n - case["recent"], n, device="cuda")))
                    kept.append(row[torch.cat((chosen, ends)).sort().values])
                line = torch.stack(kept)
            for p in range(0, line.shape[1], PAGE):
                part = line[:, p:p + PAGE]
                moved[into[b][p // PAGE], :, :part.shape[1]] = part
        return None, moved, None
    out, last = state["out"].double(), 0
    word, place = torch.arange(d, device="cuda") % (d // 8), torch.arange(d, device="cuda") // (d // 8)
    order = torch.tensor([(t & ~7) | ((t & 3) << 1) | ((t >> 2) & 1) for t in range(PAGE)], device="cuda")
    share = case["q_heads"] // case["kv_heads"]
    for b, (n, length) in enumerate(zip(new, kv)):
        last += n
        votes = min(n, case["voters"]) if case["voters"] else n
        mine = table[b][:-(-length // PAGE)]
        query = torch.arange(length - votes, length, device="cuda")[:, None]
        other = torch.arange(length, device="cuda")[None, :]
        hidden = other > query
        if case["window"]:
            hidden = hidden | ((other <= query - case["window"]) & (other >= case["sinks"]))
        for head in range(case["kv_heads"]):
            block = state["pages"][mine, head]
            codes = block[:, :PAGE * d // 2].reshape(-1, PAGE, d // 2)[:, order].reshape(-1, d // 2)[:length]
            pair = codes[:, word * 4 + place // 2].to(torch.int64)
            params = block[:, PAGE * d:].reshape(-1, PAGE, 8)[:, order].contiguous().view(torch.float16).reshape(-1, 4)[:length].double()
            keys = params[:, :1] * torch.where(place % 2 == 1, pair >> 4, pair & 15).double() + params[:, 1:2]
            total = torch.zeros(length, dtype=torch.float64, device="cuda")
            for one in range(head * share, (head + 1) * share):
                score = (state["q"][last - votes:last, one].double() @ keys.T) / math.sqrt(d)
                total += torch.softmax(score.masked_fill(hidden, -math.inf), -1).sum(0)
            before = mass[mine, head].flatten()[:length] * case["decay"]
            before[length - n:] = 0.0
            full = out[mine, head].flatten()
            full[:length] = before + total
            out[mine, head] = full.view(-1, PAGE)
    return out
