"""Cases of the key/value cache operators: what a serving step with block-sparse attention does beside its MoE layers.

  append   quantise the step's keys and values into the paged cache, refresh the blocks' bounds, and read
           the same tokens back
  read     read whole sequences back from the cache (a context handed over, or re-encoded)
  select   score every visible block of 64 tokens against a query's heads and list the best ones, with their scores
  attend   attention of a query's heads over the listed blocks only

A cache page holds 64 consecutive tokens of one sequence, for each key/value head: 64 key rows of `dim`
E4M3 codes, 64 value rows, 64 key scales and 64 value scales (one E8M0 byte a row).  `bounds` holds each
page's channel-wise largest and smallest key as whole numbers -63..63 in units of 2^bound_exp.  Tokens are
a flat list with a sequence number and a position each; a position of -1 is a padding entry.
"""
import math
import random

import torch

own = False

BLOCK = 64
DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    def c(name, op, batch, ctx, new, heads, group, dim, k=16, sink=1, local=2, ragged=False):
        return {"name": name, "op": op, "batch": batch, "ctx": ctx, "new": new, "heads": heads, "group": group,
                "dim": dim, "k": k, "sink": sink, "local": local, "ragged": ragged}
    return [
        # one new token of one sequence: the smallest call, all latency
        c("append_decode", "append", 1, 8192, 1, 4, 8, 128),
        # a prefill chunk of 8,192 tokens
        c("append_prefill", "append", 1, 16384, 8192, 4, 8, 128),
        # a mixed step: ragged chunks at odd positions, and a padding entry
        c("append_ragged", "append", 37, 2500, 333, 8, 4, 64, ragged=True),
        # ragged sequences of a small service read back
        c("read_ragged", "read", 5, 1001, 1001, 2, 16, 64, ragged=True),
        # one long context read back whole
        c("read_long", "read", 1, 131072, 131072, 4, 8, 128),
        # one token over a long context
        c("select_decode", "select", 1, 131072, 1, 4, 8, 128),
        # a decode batch over ragged contexts
        c("select_batch", "select", 64, 32768, 1, 4, 8, 128, k=32, ragged=True),
        # the second half of a 32k prompt as one chunk
        c("select_prefill", "select", 1, 32768, 8192, 4, 8, 128),
        # one token: its 16 blocks
        c("attend_decode", "attend", 1, 131072, 1, 4, 8, 128),
        # a decode batch over ragged contexts
        c("attend_batch", "attend", 64, 32768, 1, 4, 8, 128, k=32, ragged=True),
        # speculative-verify batches of 5 tokens a sequence, 16 query heads to a key/value head
        c("attend_verify", "attend", 12, 20000, 5, 2, 16, 64, k=24),
        # the second half of a 32k prompt as one chunk
        c("attend_prefill", "attend", 1, 32768, 8192, 4, 8, 128),
    ]


def draw(rng):
    def logint(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    while True:
        op = rng.choice(["append", "read", "select", "attend"])
        dim = rng.choice([64, 128])
        group = rng.choice([1, 2, 3, 4, 5, 6, 8, 8, 12, 16])
        heads = rng.choice([1, 2, 3, 4, 8])
        if group * heads > 64:
            continue
        if op in ("append", "read"):
            batch, ctx = logint(1, 64), logint(1, 65536)
            new = ctx if op == "read" else logint(1, min(ctx, 8192))
        elif rng.random() < 0.5:  # decoding: a few tokens for each sequence
            batch, ctx, new = logint(1, 96), logint(64, 100000), rng.choice([1, 1, 1, 2, 5, 8])
        else:  # prefill chunks
            batch, ctx = logint(1, 8), logint(64, 32768)
            new = logint(16, 8192)
        sink, local = rng.choice([0, 1, 1, 2]), rng.choice([1, 2, 3])
        case = {"op": op, "batch": batch, "ctx": ctx, "new": min(new, ctx), "heads": heads, "group": group, "dim": dim,
                "k": max(sink + local, rng.choice([4, 8, 15, 16, 16, 32, 48])), "sink": sink, "local": local,
                "ragged": rng.random() < 0.6}
        w = work(case)
        # no dearer than the largest listed case of its kind, and a state that is quickly made
        rows = sum(n for _, n in _lengths(case))
        tokens = sum(n for n, _ in _lengths(case))
        if (w["bytes"] <= 4e8 and w["flops"] <= 1.3e11 and tokens <= 2 ** 20
                and rows * case["heads"] * case["dim"] * min(case["k"], 1 + ctx // 64) <= 8192 * 4 * 128 * 16):
            return case


def _lengths(case):
    """(context length, new tokens) of each sequence; both follow from the case alone."""
    B, ctx, new = case["batch"], case["ctx"], case["new"]
    if not case["ragged"]:
        return [(ctx, min(new, ctx))] * B
    r = random.Random(B * 1000003 + ctx * 1009 + new * 17 + case["heads"])
    got = [(ctx, min(new, ctx))]
    for _ in range(B - 1):
        n = r.randint(1, ctx)
        got.append((n, n if case["op"] == "read" else min(n, r.randint(1, new))))
    return got


def work(case):
    H, G, D, k = case["heads"], case["group"], case["dim"], case["k"]
    lens = _lengths(case)
    T = sum(n for _, n in lens) + int(case["ragged"])
    row = 2 * D + 2  # a token's key and value codes with their scales, one head
    if case["op"] == "append":  # inputs in, codes out; the codes in again, values out
        return {"bytes": T * H * (4 * D + row) + T * H * (row + 4 * D), "flops": T * H * D * 6}
    if case["op"] == "read":
        return {"bytes": T * H * (row + 4 * D), "flops": T * H * D * 2}
    nb = [-(-L // BLOCK) for L, _ in lens]
    if case["op"] == "select":  # each block's bounds once, the queries, the lists
        seen = sum(n * H * (2 * D + 1) for n in nb)
        pairs = sum(n * b for (_, n), b in zip(lens, nb))
        return {"bytes": seen + T * H * (G * D * 2 + 8 * k), "flops": pairs * H * 4 * D}
    # attend: each listed block once while lists are disjoint, no more than the cache
    blocks = sum(min(b, n * min(k, b)) for (_, n), b in zip(lens, nb))
    pairs = sum(n * min(k, b) for (_, n), b in zip(lens, nb))
    return {"bytes": blocks * H * BLOCK * row + T * H * (4 * G * D + 4 * G + 4 * k), "flops": pairs * H * G * BLOCK * 4 * D}


# --------------------------------------------------------------------------- the plain form

def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(a, bits, frac):
    """Smallest e with a <= frac * 2^(bits + e), a >= 0 in 32 bits (frac in [1, 2)); -64 at least."""
    m, ex = torch.frexp(a)
    return torch.where(a > 0, ex - 1 - bits + (2 * m > frac).to(ex.dtype), -64).clamp_min(-64)


def _views(pages, D):
    n, H, _ = pages.shape
    return (pages[:, :, :BLOCK * D].view(n, H, BLOCK, D), pages[:, :, BLOCK * D:2 * BLOCK * D].view(n, H, BLOCK, D),
            pages[:, :, 2 * BLOCK * D:2 * BLOCK * D + BLOCK], pages[:, :, 2 * BLOCK * D + BLOCK:])


def _encode(x):
    """x [..., D] in 32 bits -> E4M3 codes and the row's E8M0 byte."""
    e = _exponent(x.abs().amax(-1), 8, 1.75)
    return (x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _decode(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * _pow2(scale.to(torch.int32) - 127)[..., None]


def _bounds_of(hi, lo):
    """Channel-wise extremes [..., D] -> (whole numbers [..., 2, D] that bound them, exponent [...])."""
    e = _exponent(torch.maximum(hi.abs(), lo.abs()).amax(-1), 5, 1.96875)
    s = _pow2(-e)[..., None]
    return torch.stack([torch.ceil(hi * s), torch.floor(lo * s)], -2).to(torch.int8), e.to(torch.int8)


def _where(st):
    """Page and slot of each token that is no padding, and which tokens those are."""
    t = torch.nonzero(st["pos"] >= 0)[:, 0]
    pos = st["pos"][t].long()
    return t, st["table"][st["seq"][t].long(), pos // BLOCK].long(), pos % BLOCK


def _plain_append(st):
    D = st["k"].shape[-1]
    kc, vc, ks, vs = _views(st["pages"], D)
    t, page, slot = _where(st)
    k, ke = _encode(st["k"][t].float())
    v, ve = _encode(st["v"][t].float())
    h = torch.arange(kc.shape[1], device=DEV)[None]
    at = (page[:, None], h, slot[:, None])
    kc[at], vc[at], ks[at], vs[at] = k, v, ke, ve
    # the touched blocks' extremes: of the new keys, and of the old bounds where the block had begun before
    new = _decode(k, ke)
    idx = page[:, None, None].expand_as(new)
    n = kc.shape[0]
    hi = torch.full((n, *new.shape[1:]), -math.inf, device=DEV).scatter_reduce(0, idx, new, "amax")
    lo = torch.full((n, *new.shape[1:]), math.inf, device=DEV).scatter_reduce(0, idx, new, "amin")
    first = torch.full((n,), BLOCK, device=DEV).scatter_reduce(0, page, slot, "amin")
    touched, old = (first < BLOCK), ((first > 0) & (first < BLOCK))[:, None]
    oe = st["bound_exp"].to(torch.int32)
    ob = st["bounds"].float() * _pow2(oe)[..., None, None]
    amax = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    e = _exponent(torch.where(touched[:, None], amax, 0.0), 5, 1.96875)
    e = torch.where(old, torch.maximum(e, oe), e)
    hi = torch.where(old[..., None], torch.maximum(hi, ob[:, :, 0]), hi)
    lo = torch.where(old[..., None], torch.minimum(lo, ob[:, :, 1]), lo)
    s = _pow2(-e)[..., None]
    b = torch.stack([torch.ceil(hi * s), torch.floor(lo * s)], 2)
    st["bounds"].copy_(torch.where(touched[:, None, None, None], b, st["bounds"].float()).to(torch.int8))
    st["bound_exp"].copy_(torch.where(touched[:, None], e, oe).to(torch.int8))
    return _plain_read(st) + [st["bounds"], st["bound_exp"]]


def _plain_read(st):
    kc, vc, ks, vs = _views(st["pages"], st["dim"])
    t, page, slot = _where(st)
    out = torch.zeros((2, st["pos"].numel(), kc.shape[1], st["dim"]), device=DEV)
    out[0, t] = _decode(kc[page, :, slot], ks[page, :, slot])
    out[1, t] = _decode(vc[page, :, slot], vs[page, :, slot])
    return list(out.to(torch.bfloat16))


def _plain_select(st):
    T, _, D = st["q"].shape
    H = st["bounds"].shape[1]
    q = st["q"].float().view(T, H, -1, D)
    e = _exponent(q.abs().amax((2, 3)), 6, 1.984375)
    c = torch.round(q * _pow2(-e)[..., None, None])  # whole numbers -127..127
    w = torch.cat([c.clamp_min(0).sum(2), -(-c).clamp_min(0).sum(2)], -1)
    table, seq, pos = st["table"], st["seq"].long(), st["pos"]
    at = table.clamp_min(0).long()
    # sums of whole numbers below 2^24: exact in 32 bits, in any order
    s = torch.einsum("thc,bnhc->tbhn", w, st["bounds"][at].flatten(-2).float())
    s = s[torch.arange(T, device=DEV), seq] * _pow2(st["bound_exp"][at[seq]]).transpose(1, 2) * _pow2(e)[..., None]
    n = torch.arange(table.shape[1], device=DEV)
    cur = torch.where(pos >= 0, pos // BLOCK, -1)[:, None]
    seen = ((n <= cur) & (table[seq] >= 0))[:, None]
    must = seen & ((n < st["sink"]) | (n > cur - st["local"]))[:, None]
    key = torch.where(must, math.inf, torch.where(seen, s, -math.inf))
    best = torch.sort(key, dim=-1, descending=True, stable=True)
    ids = torch.where(best.values > -math.inf, best.indices, 2 ** 30)[..., :st["top"]].sort(-1).values
    s = torch.where(ids < 2 ** 30, s.gather(-1, ids.clamp_max(s.shape[-1] - 1)), 0.0)
    ids = torch.where(ids < 2 ** 30, ids, -1).to(torch.int32)
    more = (0, st["top"] - ids.shape[-1])
    return [torch.nn.functional.pad(ids, more, value=-1), torch.nn.functional.pad(s, more)]


def _plain_attend(st):
    T, _, D = st["q"].shape
    kc, vc, ks, vs = _views(st["pages"], D)
    H = kc.shape[1]
    q = st["q"].float().view(T, H, -1, D)
    ids = st["ids"].long()
    page = st["table"][st["seq"].long()[:, None, None], ids.clamp_min(0)].long()
    h = torch.arange(H, device=DEV)[None, :, None]
    at = (page.clamp_min(0), h)
    pos = ids[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)
    seen = ((ids >= 0) & (page >= 0))[..., None] & (pos <= st["pos"][:, None, None, None])
    s = torch.einsum("thgd,thnsd->thgns", q, _decode(kc[at], ks[at])) * st["scale"]
    s = torch.where(seen[:, :, None], s, -math.inf)
    m = s.amax((-1, -2), keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    l = p.sum((-1, -2))
    o = torch.einsum("thgns,thnsd->thgd", p, _decode(vc[at], vs[at]))
    o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    lse = m[..., 0, 0] + torch.log(l)
    return [o.reshape(T, -1, D).to(torch.bfloat16), lse.reshape(T, -1)]


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    """Keys of a block share a topic, and so do a stretch of queries: a query has a few blocks to look for, and its
    neighbours look for mostly the same ones.  Values are unit normal.  Every tensor is made from the seed."""
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    H, G, D, op = case["heads"], case["group"], case["dim"], case["op"]
    lens = _lengths(case)
    B, N = len(lens), max(-(-L // BLOCK) for L, _ in lens)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    # physical pages in random order, as a served cache has them after a while
    nb = torch.tensor([-(-L // BLOCK) for L, _ in lens], device=DEV)
    used, spare = int(nb.sum()), 3
    order = torch.randperm(used + spare, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, N), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(N, device=DEV)[None] < nb[:, None]] = order[:used]
    seq, pos = _tokens(case, lens)
    topics = normal(32, H, D)
    n = used + spare
    pages = torch.zeros((n, H, 2 * BLOCK * D + 2 * BLOCK), dtype=torch.uint8, device=DEV)
    kc, vc, ks, vs = _views(pages, D)
    st = {"pages": pages, "table": table, "seq": seq, "pos": pos, "dim": D, "keep": {}}
    T = seq.numel()
    of = torch.randint(32, (n,), generator=g, device=DEV)
    keys = 0.6 * topics[of][:, :, None] + 0.8 * normal(n, H, BLOCK, D)
    kc[:], ks[:] = _encode(keys.to(torch.bfloat16).float())
    keys = _decode(kc.contiguous(), ks.contiguous())
    st["bounds"], st["bound_exp"] = _bounds_of(keys.amax(2), keys.amin(2))
    if op in ("append", "read", "attend"):
        vc[:], vs[:] = _encode(normal(n, H, BLOCK, D).to(torch.bfloat16).float())
    if op == "append":
        # one projection's output: queries, keys and values of a token side by side, taken as views of it
        qkv = normal(T, (G + 2) * H, D).to(torch.bfloat16)
        st["k"], st["v"] = qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]
    if op in ("select", "attend"):
        stretch = torch.randint(32, (T // 48 + 2,), generator=g, device=DEV)
        now = topics[stretch[(torch.arange(T, device=DEV) + 7 * seq) // 48 % stretch.numel()]]
        st["q"] = (0.6 * now[:, :, None] + 0.8 * normal(T, H, G, D)).reshape(T, H * G, D).to(torch.bfloat16)
        st["top"], st["sink"], st["local"] = case["k"], case["sink"], case["local"]
    if op == "attend":
        st["ids"], st["scale"] = _plain_select(st)[0], D ** -0.5
    return st


def _tokens(case, lens):
    """Flat sequence numbers and positions of the new tokens; ragged cases end with a padding entry."""
    n = torch.tensor([n for _, n in lens])
    L = torch.tensor([L for L, _ in lens])
    seq = torch.repeat_interleave(torch.arange(len(lens)), n)
    pos = torch.arange(int(n.sum())) - torch.repeat_interleave(n.cumsum(0) - n, n) + torch.repeat_interleave(L - n, n)
    if case["ragged"]:
        seq, pos = torch.cat([seq, seq[:1]]), torch.cat([pos, torch.tensor([-1])])
    return seq.to(torch.int32).to(DEV), pos.to(torch.int32).to(DEV)


# --------------------------------------------------------------------------- one pass

def run(st):
    if "ids" in st:
        return _own_attend(st) if own else _plain_attend(st)
    if "q" in st:
        return _own_select(st) if own else _plain_select(st)
    if "k" in st:
        return _own_append(st) if own else _plain_append(st)
    return _own_read(st) if own else _plain_read(st)


def _cache(st):
    from bit_routed_expert_gb300 import KvCache
    return KvCache(st["pages"], st["bounds"], st["bound_exp"])


def _own_append(st):
    from bit_routed_expert_gb300 import kv_append, kv_read
    cache = _cache(st)
    kv_append(cache, st["k"], st["v"], st["seq"], st["pos"], st["table"])
    k, v = kv_read(cache, st["seq"], st["pos"], st["table"])
    return [k, v, st["bounds"], st["bound_exp"]]


def _own_read(st):
    from bit_routed_expert_gb300 import kv_read
    return list(kv_read(_cache(st), st["seq"], st["pos"], st["table"]))


def _workspace(st, size, *args):
    """The workspace that a serving loop keeps from step to step."""
    if "ws" not in st["keep"]:
        st["keep"]["ws"] = torch.zeros(size(*args), dtype=torch.uint8, device=DEV)
    return st["keep"]["ws"]


def _own_select(st):
    from bit_routed_expert_gb300 import kv_select, kv_select_workspace
    T, Hq, D = st["q"].shape
    B, N = st["table"].shape
    ws = _workspace(st, kv_select_workspace, T, Hq, st["bounds"].shape[1], D, B, N, st["top"])
    return list(kv_select(st["q"], _cache(st), st["seq"], st["pos"], st["table"], st["top"], n_sink=st["sink"],
                          n_local=st["local"], ws=ws))


def _own_attend(st):
    from bit_routed_expert_gb300 import kv_attend, kv_attend_workspace
    T, Hq, D = st["q"].shape
    ws = _workspace(st, kv_attend_workspace, T, Hq, st["bounds"].shape[1], D, st["table"].shape[0], st["top"])
    return list(kv_attend(st["q"], _cache(st), st["seq"], st["pos"], st["table"], st["ids"], scale=st["scale"], ws=ws))


# --------------------------------------------------------------------------- from the definitions, in 64 bits

def _grid(x):
    """Nearest E4M3 value of x (|x| <= 448), ties to the even code."""
    _, ex = torch.frexp(x.abs())
    step = torch.exp2((ex - 1).clamp_min(-6).double() - 3)
    return torch.round(x / step) * step


def _least(a, top):
    """Smallest whole e >= -64 with a <= top * 2^e."""
    e = torch.ceil(torch.log2(a / top)).clamp_min(-64)
    e = torch.where(a > top * torch.exp2(e), e + 1, e)
    return torch.where((a <= top * torch.exp2(e - 1)) & (e > -64), e - 1, e)


def _stored(x):
    x = x.double()
    s = torch.exp2(_least(x.abs().amax(-1, keepdim=True), 448.0))
    return _grid(x / s) * s


def _cached(st):
    """Every page's keys and values [page, slot, head, dim] in 64 bits, bit by bit from the codes."""
    pages, D = st["pages"], st["dim"]
    got = []
    for first, sc in ((0, 2 * BLOCK * D), (BLOCK * D, 2 * BLOCK * D + BLOCK)):
        c = pages[:, :, first:first + BLOCK * D].reshape(pages.shape[0], -1, BLOCK, D).int()
        ex, man = (c >> 3) & 15, (c & 7).double()
        val = torch.where(ex > 0, (8 + man) * torch.exp2(ex.double() - 10), man * 2.0 ** -9)
        val = torch.where(c >= 128, -val, val)
        s = torch.exp2(pages[:, :, sc:sc + BLOCK].double() - 127)
        got.append((val * s[..., None]).transpose(1, 2))
    return got


def exact(case, seed):
    if case["op"] in ("read", "attend") and sum(L for L, _ in _lengths(case)) * case["heads"] * case["dim"] > 2 ** 30:
        return None  # more than the few seconds that this is given
    st = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "select": _exact_select, "attend": _exact_attend}[case["op"]](st)


def _exact_append(st):
    k, v = _stored(st["k"]), _stored(st["v"])
    pad = st["pos"] < 0
    bounds, bexp = st["bounds"].long(), st["bound_exp"].long()
    seq, pos, table = st["seq"].tolist(), st["pos"].tolist(), st["table"].tolist()
    runs = {}
    for t, (s, p) in enumerate(zip(seq, pos)):
        if p >= 0:
            runs.setdefault(table[s][p // BLOCK], []).append(t)
    for page, ts in runs.items():
        new = k[ts[0]:ts[-1] + 1]
        hi, lo, e = new.amax(0), new.amin(0), _least(new.abs().amax((0, 2)), 63.0)
        if pos[ts[0]] % BLOCK:
            old = bounds[page].double() * torch.exp2(bexp[page].double())[:, None, None]
            hi, lo = torch.maximum(hi, old[:, 0]), torch.minimum(lo, old[:, 1])
            e = torch.maximum(e, bexp[page].double())
        u = torch.exp2(e)[:, None]
        bounds[page] = torch.stack([torch.ceil(hi / u), torch.floor(lo / u)], 1).long()
        bexp[page] = e.long()
    k[pad], v[pad] = 0, 0
    return [k, v, bounds, bexp]


def _exact_read(st):
    k, v = _cached(st)
    out = torch.zeros((2, st["pos"].numel(), k.shape[2], k.shape[3]), dtype=torch.float64, device=DEV)
    ok = st["pos"] >= 0
    pos = st["pos"][ok].long()
    page = st["table"][st["seq"][ok].long(), pos // BLOCK].long()
    out[0, ok], out[1, ok] = k[page, pos % BLOCK], v[page, pos % BLOCK]
    return [out[0], out[1]]


def _exact_select(st):
    T, _, D = st["q"].shape
    H, N, top = st["bounds"].shape[1], st["table"].shape[1], st["top"]
    q = st["q"].double().view(T, H, -1, D)
    step = torch.exp2(_least(q.abs().amax((2, 3), keepdim=True), 127.0))
    c = torch.round(q / step)
    val = torch.zeros((T, H, top), dtype=torch.float64, device=DEV)
    out = torch.full((T, H, top), -1, dtype=torch.int64, device=DEV)
    bounds, unit = st["bounds"].double(), torch.exp2(st["bound_exp"].double())
    idx = torch.arange(N, device=DEV)
    seqs, pos = st["seq"].tolist(), st["pos"]
    t = 0
    while t < T:  # a stretch of tokens of one sequence
        t1 = t
        while t1 < T and seqs[t1] == seqs[t] and t1 - t < 256:
            t1 += 1
        row = st["table"][seqs[t]].long()
        hi, lo = bounds[row.clamp_min(0), :, 0], bounds[row.clamp_min(0), :, 1]
        score = torch.zeros((t1 - t, H, N), dtype=torch.float64, device=DEV)
        for g in range(c.shape[2]):  # the bound of q . k over the block, one head after the other
            x = c[t:t1, :, g]
            score += torch.einsum("thd,nhd->thn", x.clamp_min(0), hi) + torch.einsum("thd,nhd->thn", x.clamp_max(0), lo)
        score *= unit[row.clamp_min(0)].T * step[t:t1, :, 0]
        cur = torch.div(pos[t:t1], BLOCK, rounding_mode="floor")[:, None, None]
        ok = (idx <= cur) & (row >= 0)
        must = (idx < st["sink"]) | (idx > cur - st["local"])
        key = torch.where(ok & must, math.inf, score).masked_fill(~ok, -math.inf)
        by = torch.argsort(-key, dim=-1, stable=True)[..., :top]
        good = torch.gather(key, -1, by) > -math.inf
        ids = torch.where(good, by, N).sort(-1).values
        val[t:t1, :, :ids.shape[-1]] = torch.gather(score, -1, ids.clamp_max(N - 1)).masked_fill(ids == N, 0.0)
        out[t:t1, :, :ids.shape[-1]] = torch.where(ids < N, ids, -1)
        t = t1
    return [out, val]


def _exact_attend(st):
    T, Hq, D = st["q"].shape
    k, v = _cached(st)
    H, top = k.shape[2], st["ids"].shape[-1]
    q = st["q"].double().view(T, H, -1, D) * st["scale"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    step = max(1, 2 ** 27 // (H * top * BLOCK * D))
    h = torch.arange(H, device=DEV)[None, :, None]
    for t in range(0, T, step):
        ids, pos = st["ids"][t:t + step].long(), st["pos"][t:t + step]
        page = st["table"][st["seq"][t:t + step].long()[:, None, None], ids.clamp_min(0)].long()
        where = ids[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)
        ok = ((ids >= 0) & (page >= 0))[..., None] & (where <= pos[:, None, None, None])
        ok = ok.flatten(2)[:, :, None]
        kk = k.transpose(1, 2)[page.clamp_min(0), h].flatten(2, 3)
        vv = v.transpose(1, 2)[page.clamp_min(0), h].flatten(2, 3)
        s = torch.matmul(q[t:t + step], kk.transpose(-1, -2)).masked_fill(~ok, -math.inf)
        top_s = s.amax(-1, keepdim=True)
        w = torch.exp(s - top_s.masked_fill(top_s == -math.inf, 0.0))
        z = w.sum(-1, keepdim=True)
        o = torch.matmul(w, vv) / z.clamp_min(1e-300)
        out[t:t + step] = o.reshape(-1, Hq, D)
        lse[t:t + step] = (top_s + torch.log(z)).reshape(-1, Hq)
    return [out, lse]
