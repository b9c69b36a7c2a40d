"""Measured cases of the 4-bit key/value cache operators: writing a cache, reading it back, and attention over it.

The cache holds 4-bit codes in pages of 64 tokens. One vector (a key or a value of one token and one key/value head, D
numbers) is stored as D codes 0..15, a step and a base, both fp16; it stands for step * code + base:

    lo, hi = the least and the greatest x, each clamped to [-61440, 61440]
    base = fp16(lo), step = fp16((hi - lo) / 15)          (fp32 subtraction and division, then one rounding)
    code = clamp(rne((x - base) / step), 0, 15), 0 where step is 0   (the quotient rounded once, ties to even)

A page holds, for each head, one block of 64 * D + 512 bytes, with W = D / 8 words of 32 bits a vector:

    key codes    row rho(t) of W words, rho(t) = (t & ~7) | (t & 3) << 1 | (t >> 2) & 1 for token t of the page;
                 nibble n of word w is the code of dimension w + W * n
    value codes  row t of W words, the same nibbles; with D = 128 the row's two halves are exchanged where t & 2
    parameters   row rho(t): key step, key base, value step, value base

A batch is `cu_q` (where each sequence's tokens begin in the packed rows), `kv_len` (each sequence's cached tokens, the
call's own among them: a call's tokens are a sequence's last ones) and `page_table`. Query i of a sequence with n queries
and L cached tokens has position p = L - n + i and sees position j where j <= p and (j > p - window or j < sinks); window 0
stands for all.
"""
import math

import torch

own = False

PAGE = 64

# heads of the queries, heads of the cache, dimension: 4:1 sharing as in the 2560-wide decode workload, and generic ones
HEADS = ((20, 5, 128), (32, 8, 64), (12, 12, 64), (16, 2, 128), (28, 4, 128), (8, 1, 128), (24, 8, 64))


def _case(name, op, batch, heads, q, ctx, dtype="bf16", window=0, sinks=0):
    """q and ctx: the least and the greatest number of new tokens and of tokens cached before them."""
    c = {"op": op, "batch": batch, "q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "q_min": q[0], "q_max": q[1],
         "ctx_min": ctx[0], "ctx_max": ctx[1], "dtype": dtype, "window": window, "sinks": sinks}
    return dict(c, name=name) if name else c


def listed():
    h2b = HEADS[0]
    return [
        # one user's decode step: one token's keys and values, fp32 as the projections give them
        _case("write_token", "write", 1, h2b, (1, 1), (511, 511), "f32"),
        # a server's decode step: one token of each of 96 sequences
        _case("write_batch", "write", 96, h2b, (1, 1), (0, 4000)),
        # five prompts of unlike lengths arrive at once
        _case("write_prompts", "write", 5, h2b, (999, 9001), (0, 70)),
        # six whole caches are read back, to hand them to a consumer of bf16 keys and values
        _case("read_caches", "read", 6, h2b, (501, 23999), (0, 0)),
        # the first steps after a short question: latency alone
        _case("decode_short", "attend", 1, h2b, (1, 1), (76, 76)),
        # one user with a very long context: the whole GPU on one sequence
        _case("decode_long", "attend", 1, h2b, (1, 1), (131006, 131006)),
        # a server's decode step over contexts of unlike lengths, fp32 queries
        _case("decode_batch", "attend", 64, h2b, (1, 1), (17, 8175), "f32"),
        # streaming sequences: a window and the first tokens, whatever the length
        _case("decode_window", "attend", 24, HEADS[1], (1, 1), (3001, 65007), "bf16", 2048, 4),
        # drafted tokens are checked: a few queries a sequence
        _case("decode_draft", "attend", 16, h2b, (3, 7), (1001, 12005)),
        # a short prompt, fp32 queries
        _case("prompt_128", "attend", 1, h2b, (128, 128), (0, 0), "f32"),
        # a long prompt from nothing: bound by the products
        _case("prompt_4096", "attend", 1, h2b, (4096, 4096), (0, 0)),
        # prompts in chunks behind cached contexts, with a window
        _case("prompt_chunks", "attend", 4, HEADS[1], (201, 1501), (0, 20011), "bf16", 1024, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend", "attend"))
    heads, dtype = rng.choice(HEADS), rng.choice(("bf16", "bf16", "f32"))
    width = heads[1] * heads[2] / 640
    if op != "attend":  # tokens in all: at most those of the largest such listed case
        total = _log(rng, 2, 60000 / width / (2 if dtype == "f32" else 1) / (1.7 if op == "write" else 1))
        batch = min(_log(rng, 1, 128), total)
        top = max(1, total // batch)
        return _case(None, op, batch, heads, (rng.randint(max(1, top // 8), top), top), (0, rng.randint(0, 500) if op == "write" else 0), dtype)
    window, sinks = (0, 0) if rng.random() < 0.5 else (_log(rng, 1, 5000), rng.choice((0, 1, 4, 70)))
    if rng.random() < 0.6:  # a few queries a sequence
        total = _log(rng, 64, 250000 / width)
        batch = min(_log(rng, 1, 128), total)
        top = max(1, min(total // batch, 131000))
        q = rng.choice((1, 1, 1, 2, 5, 8))
        return _case(None, op, batch, heads, (1 if q > 4 else q, q), (top // rng.choice((1, 3, 20)), top), dtype, window, sinks)
    pairs = _log(rng, 20000, 8.0e6 * 2560 / (heads[0] * heads[2]))  # queries times what they see, in all
    batch = rng.choice((1, 1, 2, 5))
    n = min(4000, max(9, _log(rng, 9, math.sqrt(2 * pairs / batch))))
    sees = int(pairs / batch / n)
    ctx = 0 if rng.random() < 0.4 else min(30000, max(0, (sees if not window else 10 * window) - n // 2))
    return _case(None, op, batch, heads, (max(1, n // rng.choice((1, 1, 4))), n), (ctx // 2, ctx), dtype, window, sinks)


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


def _raw(case, seed):
    """The floating inputs, packed sequence by sequence: keys and values of every cached token, and the queries."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, kv = _lengths(case)
    t = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    h, d = case["kv_heads"], case["dim"]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    # keys have channels of their own mean and size, values a size of their own for each token
    k = (rand(sum(kv), h, d) * (0.5 + rand(1, h, d).abs()) + rand(1, h, d)).to(t)
    v = (rand(sum(kv), h, d) * (0.2 + rand(sum(kv), h, 1).abs())).to(t)
    q = (rand(sum(new), case["q_heads"], d) * 1.2).to(t) if case["op"] == "attend" else None
    return new, kv, k, v, q


def _quantise(x):
    """Codes (uint8), step and base (fp16) of the vectors along the last axis. The quotient is in 64 bits: next to a border 32 lose the code."""
    x = x.float().clamp(-61440.0, 61440.0)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    base, step = lo.half(), ((hi - lo) / 15.0).half()
    code = torch.round((x.double() - base.double()) / step.double()).clamp(0, 15)
    return torch.where(step == 0, torch.zeros_like(code), code).to(torch.uint8), step, base


def _rho(t):
    return (t & ~7) | ((t & 3) << 1) | ((t >> 2) & 1)


def _words(code):
    """Codes along the last axis as the bytes of the W words that hold them."""
    d = code.shape[-1]
    c = code.unflatten(-1, (8, d // 8)).transpose(-1, -2).reshape(*code.shape[:-1], d // 2, 2)
    return c[..., 0] | (c[..., 1] << 4)


def _codes(words):
    """The inverse of _words."""
    w = words.shape[-1] // 4
    c = torch.stack((words & 15, words >> 4), -1).reshape(*words.shape[:-1], w, 8)
    return c.transpose(-1, -2).flatten(-2)


def _swap(words, off):
    """Exchanges the halves of a 128-wide value row where bit 1 of the token's place in its page is set; its own inverse."""
    n = words.shape[-1]
    return torch.where(((off & 2) != 0)[..., None, None], words.roll(n // 2, -1), words) if n == 64 else words


def _fields(pages, dim):
    """Views of a cache's pages (pages x heads x block bytes): key rows, value rows, parameters."""
    n, h = pages.shape[0], pages.shape[1]
    at = PAGE * dim // 2
    return (pages[:, :, :at].unflatten(2, (PAGE, dim // 2)), pages[:, :, at:2 * at].unflatten(2, (PAGE, dim // 2)),
            pages[:, :, 2 * at:].view(torch.float16).unflatten(2, (PAGE, 4)))


def _store(pages, page, off, k, v):
    """Quantises k and v (tokens x heads x dim) into the tokens' places."""
    fk, fv, fp = _fields(pages, k.shape[-1])
    ck, sk, bk = _quantise(k)
    cv, sv, bv = _quantise(v)
    fk[page, :, _rho(off)] = _words(ck)
    fv[page, :, off] = _swap(_words(cv), off)
    fp[page, :, _rho(off)] = torch.cat((sk, bk, sv, bv), -1)


def _load(pages, dim, page, off):
    """The fp32 keys and values at places `page`, `off` (any shape): that shape x heads x dim."""
    fk, fv, fp = _fields(pages, dim)
    par = fp[page, :, _rho(off)].float()
    k = _codes(fk[page, :, _rho(off)]).float() * par[..., 0:1] + par[..., 1:2]
    v = _codes(_swap(fv[page, :, off], off)).float() * par[..., 2:3] + par[..., 3:4]
    return k, v


def prepare(case, seed):
    new, kv, k, v, q = _raw(case, seed)
    need = [-(-n // PAGE) for n in kv]
    n_pages, wide = sum(need) + 3, max(need)
    g = torch.Generator().manual_seed(seed + 1)
    ids = torch.randperm(n_pages, generator=g)[:sum(need)].to(torch.int32)  # a used pool: pages lie in any order
    table = torch.full((len(kv), wide), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    table = table.cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cum = lambda x: torch.tensor([0] + x).cumsum(0)  # noqa: E731
    seq = torch.repeat_interleave(torch.arange(len(kv)), torch.tensor(kv)).cuda()
    pos = torch.arange(sum(kv), device="cuda") - cum(kv).cuda()[seq]
    page, off = table[seq, pos // PAGE].long(), pos % PAGE
    fresh = pos >= i32([n - m for n, m in zip(kv, new)])[seq]
    # pages come with what their last user left in them
    pages = torch.full((n_pages, case["kv_heads"], PAGE * case["dim"] + 512), 255, dtype=torch.uint8, device="cuda")
    if case["op"] == "write":
        old = ~fresh
        if bool(old.any()):
            _store(pages, page[old], off[old], k[old], v[old])
    else:
        for i in range(0, len(pos), 1 << 17):
            j = slice(i, i + (1 << 17))
            _store(pages, page[j], off[j], k[j], v[j])
    state = {"case": case, "pages": pages, "table": table, "cu_q": cum(new).to(torch.int32).cuda(), "kv_len": i32(kv),
             "page": page[fresh], "off": off[fresh], "rows": sum(new), "max_q": max(new), "max_kv": max(kv)}
    if case["op"] == "write":
        state["k"], state["v"] = k[fresh], v[fresh]
    state["q"] = q
    state["dtype"] = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    if own:  # the handles that a program keeps beside its pool of pages and its batch
        from ternary_weight_gb300 import binding
        state["cache"] = binding.KV4Cache(n_pages, case["kv_heads"], case["dim"], pages=pages.view(-1))
        state["batch"] = binding.KV4Batch(state["cu_q"], state["kv_len"], table, state["rows"], state["max_q"], state["max_kv"])
    return state


def run(state):
    case = state["case"]
    scale = 1.0 / math.sqrt(case["dim"])
    if own:
        from ternary_weight_gb300 import binding
        if case["op"] == "attend":
            return binding.kv4_attention(state["cache"], state["batch"], state["q"], scale, window=case["window"], sinks=case["sinks"])
        if case["op"] == "write":
            binding.kv4_append(state["cache"], state["batch"], state["k"], state["v"])
        return binding.kv4_read(state["cache"], state["batch"], state["dtype"])
    if case["op"] == "attend":
        return _attend(state, scale)
    if case["op"] == "write":
        _store(state["pages"], state["page"], state["off"], state["k"], state["v"])
    k, v = _load(state["pages"], case["dim"], state["page"], state["off"])
    return k.to(state["dtype"]), v.to(state["dtype"])


def _attend(state, scale):
    """All sequences at once, padded to the longest: scores of what the window and the first tokens leave, softmax, values."""
    case, q = state["case"], state["q"]
    b, n = case["batch"], state["max_q"]
    h, d = case["kv_heads"], case["dim"]
    r = case["q_heads"] // h
    kv, cu = state["kv_len"].long()[:, None], state["cu_q"].long()
    count = (cu[1:] - cu[:-1])[:, None]
    row = torch.arange(n, device="cuda")
    pad = torch.zeros(b, n, h, r, d, device="cuda")
    there = row < count
    pad[there] = q.float().unflatten(1, (h, r))
    at = kv - count + row  # positions of the queries
    j, double = torch.arange(state["max_kv"], device="cuda").expand(b, -1), None
    if case["window"] and case["sinks"] + case["window"] + n - 1 < state["max_kv"]:  # only what can be seen
        first = (at[:, :1] - case["window"] + 1).clamp(min=0)
        late = first + torch.arange(case["window"] + n - 1, device="cuda")
        j = torch.cat((torch.arange(case["sinks"], device="cuda").expand(b, -1), late), 1)
        double = torch.cat((torch.zeros_like(j[:, :case["sinks"]], dtype=torch.bool), late < case["sinks"]), 1)
    page = state["table"].gather(1, (j // PAGE).clamp(max=state["table"].shape[1] - 1)).long().clamp(min=0)
    k, v = _load(state["pages"], d, page, j % PAGE)
    here = (j < kv)[..., None, None]
    k, v = torch.where(here, k, 0.0), torch.where(here, v, 0.0)
    s = torch.einsum("bnhrd,blhd->bhrnl", pad, k) * scale
    sees = j[:, None, :] <= at[..., None]
    if case["window"]:
        sees = sees & ((j[:, None, :] > at[..., None] - case["window"]) | (j[:, None, :] < case["sinks"]))
    if double is not None:
        sees = sees & ~double[:, None, :]
    s = s.masked_fill(~sees[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    o = torch.einsum("bhrnl,blhd->bnhrd", s, v) / s.sum(-1).permute(0, 3, 1, 2)[..., None].clamp(min=1e-30)
    return o[there].flatten(1, 2).bfloat16()


def _seen(case):
    """For each sequence: the pairs of a query and a position it sees, and the positions that any query sees."""
    got = []
    for n, kv in zip(*_lengths(case)):
        w, s = case["window"] or kv, case["sinks"]
        pairs = 0
        for p in (range(kv - n, kv) if case["window"] else ()):
            low = max(0, p - w + 1)
            pairs += p + 1 - low + min(s, low)
        if not case["window"]:
            pairs = n * (2 * kv - n + 1) // 2
        low = max(0, kv - n - w + 1)
        got.append((pairs, kv - low + min(s, low)))
    return got


def work(case):
    new, _ = _lengths(case)
    size = 4 if case["dtype"] == "f32" else 2
    vector = case["dim"] // 2 + 4  # bytes of a stored vector
    if case["op"] == "attend":
        seen = _seen(case)
        values = sum(new) * case["q_heads"] * case["dim"]
        return {"bytes": sum(s for _, s in seen) * case["kv_heads"] * 2 * vector + values * (size + 2),
                "flops": 4 * case["dim"] * case["q_heads"] * sum(p for p, _ in seen)}
    vectors = 2 * sum(new) * case["kv_heads"]
    sides = 2 if case["op"] == "write" else 1  # the vectors go in and come back, or only come back
    return {"bytes": vectors * (vector + sides * case["dim"] * size), "flops": vectors * case["dim"] * 4 * sides}


def exact(case, seed):
    """From the definition, sequence by sequence in 64 bits: the stored parameters are what fp32 and fp16 make of a vector's ends, all else is 64-bit."""
    new, kv, k, v, q = _raw(case, seed)

    def stands_for(x):
        x = torch.clamp(x.double(), -61440.0, 61440.0)
        low, high = x.min(-1).values.float(), x.max(-1).values.float()
        base, step = low.to(torch.float16).double()[..., None], ((high - low) / 15.0).to(torch.float16).double()[..., None]
        quotient = torch.where(step > 0, (x - base) / torch.where(step > 0, step, 1.0), 0.0)
        return base + step * torch.clamp(torch.round(quotient), 0.0, 15.0)

    outs, last, first = [], 0, 0
    for n, length in zip(new, kv):
        mine = slice(last, last + length)
        last += length
        if case["op"] != "attend":
            mine = slice(last - n, last)
            outs.append((stands_for(k[mine]), stands_for(v[mine])))
            continue
        place = torch.arange(length - n, length, device="cuda")[:, None]
        other = torch.arange(length, device="cuda")[None, :]
        hidden = other > place
        if case["window"]:
            hidden = hidden | ((other <= place - case["window"]) & (other >= case["sinks"]))
        part = torch.empty(n, case["q_heads"], case["dim"], dtype=torch.float64, device="cuda")
        share = case["q_heads"] // case["kv_heads"]
        for head in range(case["kv_heads"]):
            keys, values = stands_for(k[mine, head]), stands_for(v[mine, head])
            for one in range(head * share, (head + 1) * share):
                score = (q[first:first + n, one].double() @ keys.T) / math.sqrt(case["dim"])
                part[:, one] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ values
        outs.append(part)
        first += n
    if case["op"] == "attend":
        return torch.cat(outs)
    return torch.cat([o[0] for o in outs]), torch.cat([o[1] for o in outs])
