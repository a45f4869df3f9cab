"""Performance cases of the operators between a block's projections and its
attention's output: the step of a paged cache (block tables and slot maps),
the norms and the rotation of queries and keys with the store into a cache of
4 bits, and attention over that cache.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, in 64 where values are compared with a rounding's borders, rounded
once at the end) or, where ``own`` is true, by the calls a user makes of the
package.

The cache is uint8 ``[pages, kv_heads, page_size / 16, 2, 9 * D]``: of each 16
tokens of a head first the keys, then the values, each 16 rows of D / 2 bytes
(E2M1, the even column in the low nibble) and 16 rows of D / 16 scales (E4M3,
one per 16 columns).
"""
import math
import random

import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # 64 decoding requests, a token each: where the tokens go, and now and then a new page
        dict(name="step_decode", op="step", R=64, new=1, ctx=4096, page=16, finished=0.0),
        # a full batch of prompt chunks while some requests end
        dict(name="step_prompts", op="step", R=512, new=128, ctx=2048, page=64, finished=0.1),
        # one token's queries, keys and values between the projections and the attention: latency
        dict(name="rope_decode", op="rope", T=1, Hq=32, Hkv=8, D=128, rot=128, cached=True, page=16, gated=False,
             interleaved=False),
        # a long prompt into the cache
        dict(name="rope_prompt", op="rope", T=8192, Hq=32, Hkv=8, D=128, rot=128, cached=True, page=64, gated=False,
             interleaved=False),
        # wide heads, a quarter of them rotated, queries beside their gates; keys kept in 16 bits
        dict(name="rope_wide", op="rope", T=1001, Hq=16, Hkv=2, D=256, rot=64, cached=False, page=16, gated=True,
             interleaved=False),
        # one token of one request: latency
        dict(name="attn_one", op="attn", R=1, new=1, ctx=4096, Hq=32, Hkv=8, D=128, page=64, window=0, sinks=False,
             lse=False),
        # a serving batch of ragged contexts, small pages
        dict(name="attn_batch", op="attn", R=64, new=1, ctx=8192, Hq=64, Hkv=8, D=128, page=16, window=0, sinks=False,
             lse=False),
        # a serving batch of a layer with a sliding window and sinks
        dict(name="attn_window", op="attn", R=128, new=1, ctx=4096, Hq=64, Hkv=8, D=64, page=32, window=128, sinks=True,
             lse=False),
        # two requests with very long contexts, five queries to a key head
        dict(name="attn_long", op="attn", R=2, new=1, ctx=262144, Hq=40, Hkv=8, D=128, page=128, window=0, sinks=False,
             lse=True),
        # drafted tokens verified together
        dict(name="attn_draft", op="attn", R=16, new=5, ctx=16384, Hq=32, Hkv=8, D=128, page=32, window=0, sinks=False,
             lse=False),
        # chunks of prompts behind what is cached already: bound by the matrix products
        dict(name="attn_prompts", op="attn", R=4, new=2048, ctx=8192, Hq=32, Hkv=8, D=128, page=64, window=0,
             sinks=False, lse=False),
        # odd chunks, wide heads
        dict(name="attn_wide", op="attn", R=3, new=777, ctx=3001, Hq=16, Hkv=2, D=256, page=16, window=0, sinks=False,
             lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "rope", "rope", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "step":
        R = _log(rng, 1, 512)
        return dict(op=op, R=R, new=_log(rng, 1, max(1, min(2048, 65536 // R))), ctx=_log(rng, 16, 4096), page=page,
                    finished=rng.choice([0.0, 0.1, 0.4]))
    D = rng.choice([64, 128, 128, 256])
    if op == "rope":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.randint(1, 8)
        T = _log(rng, 1, 16384)
        while T * (Hq + 2 * Hkv) * D > 8192 * 48 * 128:
            T //= 2
        return dict(op=op, T=max(1, T), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, D // 4]),
                    cached=rng.random() < 0.6, page=page, gated=rng.random() < 0.3, interleaved=rng.random() < 0.3)
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
    R, new = rng.choice([(_log(rng, 1, 128), 1), (_log(rng, 1, 32), rng.randint(2, 8)),
                         (_log(rng, 1, 8), _log(rng, 16, 2048))])
    ctx = _log(rng, 1, 262144) + new - 1
    while R > 1 and R * new * Hq * ctx > 4 * 2048 * 32 * 8192:
        R //= 2
    while ctx > 16 and (R * ctx * Hkv * D > 64 * 8192 * 8 * 128 or R * new * Hq * ctx * D > 4 * 2048 * 32 * 6144 * 128):
        ctx //= 2
    return dict(op=op, R=R, new=min(new, ctx), ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, page=page,
                window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), sinks=rng.random() < 0.25, lse=rng.random() < 0.3)


def _spread(n, low, high):
    """n whole numbers over [low, high], the first of them high; the same for every seed."""
    return [high - int((high - low + 1) * (i * 0.6180339887498949 % 1.0)) for i in range(n)]


def _requests(case):
    """(lengths with the new tokens, new tokens) of an attention's requests; of several, one is of one token and
    one has nothing to do."""
    R = case["R"]
    new = _spread(R, max(1, case["new"] // 2), case["new"])
    length = [max(a, b) for a, b in zip(_spread(R, max(1, case["ctx"] // 2), case["ctx"]), new)]
    if R >= 8:
        length[2], new[2] = 1, 1
        new[5] = 0
    return length, new


def _visible(case):
    """(pairs of a query and a key that it sees, keys that some query of their request sees)."""
    pairs = keys = 0
    for n, q in zip(*_requests(case)):
        w = case["window"] or n
        first = n - q  # position of the first query
        full = max(0, min(n, w) - first)  # queries that see every key before them
        full = min(full, q)
        pairs += full * first + full * (full + 1) // 2 + (q - full) * w
        keys += n - max(0, first - w + 1) if q else 0
    return pairs, keys


# --------------------------------------------------------------------- inputs
def _nibbles(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _quantised(u):
    """[..., D] in 32 bits -> (codes of E2M1 [..., D], scales in E4M3 [..., D / 16]), each step in 32 bits."""
    b = u.unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    a = torch.where(s > 0, b.abs() / s, torch.zeros_like(b))
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return (code + 8 * (b < 0)).to(torch.uint8).flatten(-2), scale


def _values(code, scale):
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=code.device)
    return (table[code.int()].unflatten(-1, (-1, 16)) * scale.float().unsqueeze(-1)).flatten(-2)


def _cache(pages, case, g):
    """A cache whose keys and values have unit variance, with a few strong channels in the keys."""
    Hkv, D, nb = case["Hkv"], case["D"], case["page"] // 16
    strong = 1.0 + 3.0 * (torch.rand(D, generator=g, device="cuda") < 0.02)
    out = torch.empty(pages, Hkv, nb, 2, 9 * D, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (Hkv * case["page"] * 2 * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn(n, Hkv, nb, 2, 16, D, generator=g, device="cuda")
        x[:, :, :, 0] *= strong
        code, scale = _quantised(x)
        out[at:at + n, ..., :8 * D] = _nibbles(code).flatten(-2)
        out[at:at + n, ..., 8 * D:] = scale.view(torch.uint8).flatten(-2)
    return out


def _table(need, width, g, spare):
    """Block tables of rows with `need` pages each, drawn from a shuffled pool, -1 behind them; the pages left over."""
    R, total = len(need), sum(need)
    pool = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    need = torch.tensor(need, device="cuda")
    first = need.cumsum(0) - need
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j).clamp(max=total + spare - 1)
    return torch.where(j < need[:, None], pool[at], torch.full((R, width), -1, dtype=torch.int32, device="cuda")), pool[total:]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    s = dict(case)
    if case["op"] == "step":
        R, page = case["R"], case["page"]
        length = [r.randint(0, case["ctx"]) for _ in range(R)]
        new = [case["new"] if case["new"] == 1 else r.randint(case["new"] // 2, case["new"]) for _ in range(R)]
        ends = [r.random() < case["finished"] for _ in range(R)]
        new = [0 if e else n for n, e in zip(new, ends)]
        have = [-(-n // page) for n in length]
        most = -(-(case["ctx"] + case["new"]) // page)
        pages = R * most + 8
        s["tables"], left = _table(have, most, g, pages - sum(have))
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        s["free"][:left.numel()] = left
        s["count"] = _ints([left.numel()])
        s["length"], s["new_tokens"] = _ints(length), _ints(new)
        s["ends"] = torch.tensor(ends, device="cuda") if case["finished"] else None
        s["tokens"] = R * case["new"]
        return s
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "rope":
        T, rot = case["T"], case["rot"]
        wide = Hq * (2 if case["gated"] else 1)
        x = torch.randn(T, (wide + 2 * Hkv) * D, generator=g, device="cuda")
        x = (x * (1.0 + 4.0 * (torch.rand(x.shape[1], generator=g, device="cuda") < 0.01))).to(torch.bfloat16)
        # what one projection gives: queries (each with its gate behind it), keys, values
        s["q"] = x[:, :wide * D].view(T, Hq, -1)[:, :, :D]
        s["k"] = x[:, wide * D:(wide + Hkv) * D].view(T, Hkv, D)
        s["v"] = x[:, (wide + Hkv) * D:].view(T, Hkv, D)
        s["wq"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        s["wk"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        places = 32768
        angle = torch.arange(places, dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        s["rotary"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = (torch.arange(T, device="cuda") + r.randrange(places - T)).to(torch.int32)
        if case["cached"]:
            pages = -(-T // page) + 3
            s["cache"] = torch.zeros(pages, Hkv, page // 16, 2, 9 * D, dtype=torch.uint8, device="cuda")
            where = torch.randperm(pages, generator=g, device="cuda")
            t = torch.arange(T, device="cuda")
            s["slots"] = where[t // page] * page + t % page
        return s
    length, new = _requests(case)
    need = [-(-n // page) for n in length]
    s["tables"], _ = _table(need, max(need), g, 5)
    s["cache"] = _cache(sum(need) + 5, case, g)
    s["length"] = _ints(length)
    s["offsets"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
    T = sum(new)
    s["q"] = (torch.randn(T, Hq, D, generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    s["sink"] = torch.randn(Hq, generator=g, device="cuda") if case["sinks"] else None
    s["k_scale"], s["v_scale"] = 1.0, 0.75
    s["most"], s["most_new"] = max(length), max(new)
    return s


# ---------------------------------------------------------------- plain forms
def _step(s):
    page, R, T = s["page"], s["R"], s["tokens"]
    length, new, tables, free = s["length"].long(), s["new_tokens"].long(), s["tables"], s["free"]
    ends = s["ends"] if s["ends"] is not None else torch.zeros_like(length, dtype=torch.bool)
    have = (length + page - 1) // page
    # pages of the requests that end, onto the stack of free ones
    j = torch.arange(tables.shape[1], device="cuda")
    back = torch.where(ends, have, 0)
    top = s["count"].long() + back.sum()
    at = s["count"].long() + (back.cumsum(0) - back)[:, None] + j
    stack = torch.cat([free, free.new_zeros(1)])
    stack.scatter_(0, torch.where(j < back[:, None], at, free.numel()).flatten(), tables.flatten())
    free.copy_(stack[:-1])
    # pages for the new tokens, from its top
    length = torch.where(ends, 0, length)
    have = (length + page - 1) // page
    need = (length + new + page - 1) // page - have
    first = need.cumsum(0) - need
    taken = (need == 0) | (first + need <= top)
    got = torch.where(taken, need, 0)
    i = j - have[:, None]
    fresh = (i >= 0) & (i < got[:, None])
    tables.copy_(torch.where(fresh, free[(top - 1 - first[:, None] - i).clamp(0, free.numel() - 1)], tables))
    accepted = torch.where(taken, new, 0)
    offsets = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(T, device="cuda")
    r = (torch.searchsorted(offsets, t, right=True) - 1).clamp(max=R - 1)
    inside = t < offsets[-1]
    pos = torch.where(inside, length[r] + t - offsets[r], 0)
    slot = tables[r, (pos // page).clamp(max=tables.shape[1] - 1)].long() * page + pos % page
    return (offsets.int(), pos.int(), torch.where(inside & taken[r], slot, -1), (length + accepted).int(),
            (top - got.sum()).int(), accepted.int(), tables, free)


def _turned(y, table, rot, interleaved):
    c, n = table[:, None, :rot // 2], table[:, None, rot // 2:]
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([z, y[..., rot:]], -1)


def _normed(x, w, table, s):
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    return _turned(y, table, s["rot"], s["interleaved"])


def _store(s, kind, code, scale):
    D, page, Hkv = s["D"], s["page"], s["Hkv"]
    slot = s["slots"][:, None, None]
    head = torch.arange(Hkv, device="cuda")[:, None]
    block = ((slot // page * Hkv + head) * (page // 16) + slot % page // 16) * 2 + kind
    row = slot % 16
    flat = s["cache"].view(-1)
    flat[block * 9 * D + row * (D // 2) + torch.arange(D // 2, device="cuda")] = _nibbles(code)
    flat[block * 9 * D + 8 * D + row * (D // 16) + torch.arange(D // 16, device="cuda")] = scale.view(torch.uint8)


def _rope(s):
    table = s["rotary"][s["positions"].long()]
    q = _normed(s["q"].float(), s["wq"].float(), table, s).to(torch.bfloat16)
    # (in 64 bits: what is rounded to four bits lies next to their borders)
    k = _normed(s["k"].double(), s["wk"].double(), table.double(), s).float()
    if not s["cached"]:
        return q, k.to(torch.bfloat16)
    ck, sk = _quantised(k)
    cv, sv = _quantised(s["v"].float())
    _store(s, 0, ck, sk)
    _store(s, 1, cv, sv)
    return q, _values(ck, sk).to(torch.bfloat16), _values(cv, sv).to(torch.bfloat16)


def _attn(s):
    R, Hq, Hkv, D, page = s["R"], s["Hq"], s["Hkv"], s["D"], s["page"]
    L, N = s["most"], s["most_new"]
    G, nb = Hq // Hkv, -(-L // 16)
    length, offsets = s["length"].long(), s["offsets"].long()
    b = torch.arange(nb, device="cuda")
    blocks = s["cache"][s["tables"][:, b * 16 // page].clamp(min=0).long(), :, b % (page // 16)]  # [R, nb, Hkv, 2, 9 D]
    blocks = blocks.permute(0, 2, 3, 1, 4)
    byte = blocks[..., :8 * D].unflatten(-1, (16, D // 2))
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
    scale = blocks[..., 8 * D:].contiguous().view(torch.float8_e4m3fn).unflatten(-1, (16, D // 16))
    kv = _values(code, scale).flatten(3, 4)[..., :L, :]  # [R, Hkv, 2, L, D]
    new = offsets[1:] - offsets[:-1]
    i = torch.arange(N, device="cuda")
    row = (offsets[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(R, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, N * G, D)
    score = (q @ kv[:, :, 0].transpose(-1, -2)).view(R, Hkv, N, G, L) * (s["k_scale"] / math.sqrt(D))
    at = (length - new)[:, None] + i
    j = torch.arange(L, device="cuda")
    seen = j <= at[..., None]
    seen &= j > at[..., None] - (s["window"] or L + 1)
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, Hkv, 1, G, 1)
        top = torch.maximum(top, sink)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - top)
    out = (p.view(R, Hkv, N * G, L) @ kv[:, :, 1]).view(R, Hkv, N, G, D) / total * s["v_scale"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(offsets, t, right=True) - 1
    n = t - offsets[r]
    out = out[r, :, n].reshape(-1, Hq, D).to(torch.bfloat16)
    if not s["lse"]:
        return out
    return out, (top + torch.log(total)).squeeze(-1)[r, :, n].reshape(-1, Hq)


def run(s):
    op = s["op"]
    if not own:
        return {"step": _step, "rope": _rope, "attn": _attn}[op](s)
    import fp4_weight_moe_gb300 as m
    if op == "step":
        st = m.cache_step(s["length"], s["new_tokens"], s["tables"], s["free"], s["count"], s["page"], s["tokens"],
                          finished=s["ends"])
        return (st.offsets, st.positions, st.slots, st.lengths, st.free_count, st.accepted, s["tables"], s["free"])
    if op == "rope":
        more = dict(v=s["v"], cache=s["cache"], slots=s["slots"]) if s["cached"] else {}
        q, k = m.qk_norm_rope(s["q"], s["k"], s["positions"], s["rotary"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                              interleaved=s["interleaved"], **more)
        return (q, *m.fp4_cache_read(s["cache"], s["slots"])) if s["cached"] else (q, k)
    return m.fp4_attention(s["q"], s["cache"], s["tables"], s["length"], s["offsets"], window=s["window"],
                           sinks=s["sink"], k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=s["lse"])


# ----------------------------------------------------------------------- work
def work(case):
    if case["op"] == "step":
        R, page = case["R"], case["page"]
        T = R * case["new"]
        # lengths, new tokens and results per request; positions and slots; a table entry and a free page each
        return {"bytes": 20 * R + 12 * T + 8 * (T // page + R), "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rope":
        T, rot = case["T"], case["rot"]
        # queries in and out, keys in (values too where they are stored), angles and places
        one = 4 * Hq * D + 4 * rot + 4
        # keys and values in 4 bits, written and read back into 16
        one += (4 + 2 * 9 / 8 + 4) * Hkv * D + 16 if case["cached"] else 4 * Hkv * D
        return {"bytes": one * T, "flops": 10 * T * (Hq + Hkv) * D}
    pairs, keys = _visible(case)
    T = sum(_requests(case)[1])
    return {"bytes": keys * Hkv * D * 9 / 8 + 4 * T * Hq * D + (4 * T * Hq if case["lse"] else 0),
            "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------- exact
def _grid64(x):
    """Nearest E2M1 values of x in 64 bits, ties to the even code."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    half = (grid[1:] + grid[:-1]) / 2
    a = x.abs()
    up, down = torch.bucketize(a, half, right=True), torch.bucketize(a, half, right=False)
    return torch.where(x < 0, -1.0, 1.0) * grid[torch.where(up % 2 == 0, up, down)]


def _stored64(u):
    blocks = u.float().double().unflatten(-1, (-1, 16))
    s = torch.clamp(blocks.abs().amax(-1, keepdim=True) / 6, max=448.0).float().to(torch.float8_e4m3fn).double()
    return (torch.where(s > 0, _grid64(blocks / torch.where(s > 0, s, 1.0)), 0.0) * s).flatten(-2)


def _rope64(s, x, w):
    x, w, rot = x.double(), w.double(), s["rot"]
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["D"] + EPS) * w
    turn = torch.complex(*s["rotary"][s["positions"].long()].double()[:, None].chunk(2, -1))
    z = y.clone()
    if s["interleaved"]:
        z[..., :rot] = torch.view_as_real(torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    else:
        c = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        z[..., :rot // 2], z[..., rot // 2:rot] = c.real, c.imag
    return z


def _attn64(s):
    Hq, Hkv, D, page = s["Hq"], s["Hkv"], s["D"], s["page"]
    signed = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device="cuda")
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    offsets, lengths = s["offsets"].tolist(), s["length"].tolist()
    for r, L in enumerate(lengths):
        lo, hi = offsets[r], offsets[r + 1]
        if lo == hi:
            continue
        part = s["cache"][s["tables"][r, :-(-L // page)].long()]  # [pages, Hkv, page / 16, 2, 9 D]
        at = torch.arange(L - (hi - lo), L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        unseen = (j > at) | (j <= at - s["window"]) if s["window"] else j > at
        for h in range(Hkv):
            byte = part[:, h, ..., :8 * D].reshape(-1, 2, 16, D // 2)
            kv = signed[torch.stack([byte % 16, byte // 16], -1).long()].reshape(-1, 2, 16, D // 16, 16)
            kv = kv * part[:, h, ..., 8 * D:].reshape(-1, 2, 16, D // 16, 1).view(torch.float8_e4m3fn).double()
            k, v = kv.flatten(3).transpose(0, 1).reshape(2, -1, D)[:, :L]
            for i in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                x = s["q"][lo:hi, i].double() @ k.T * (s["k_scale"] / D ** 0.5)
                x[unseen] = -math.inf
                if s["sink"] is not None:
                    x = torch.cat([x, s["sink"][i].double().expand(hi - lo, 1)], 1)
                lse[lo:hi, i] = torch.logsumexp(x, 1)
                out[lo:hi, i] = torch.exp(x - lse[lo:hi, i, None])[:, :L] @ v * s["v_scale"]
    return out, lse


def exact(case, seed):
    if case["op"] == "step":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        q, k = _rope64(s, s["q"], s["wq"]), _rope64(s, s["k"], s["wk"])
        return (q, _stored64(k), _stored64(s["v"])) if case["cached"] else (q, k)
    if _visible(case)[0] * case["Hq"] * case["D"] > 6e11:  # (64-bit products are slow here)
        return None
    out, lse = _attn64(s)
    return (out, lse) if case["lse"] else out
