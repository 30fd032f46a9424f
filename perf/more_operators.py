"""Cases of the cache operators that a serving step with drafted tokens or several beams makes around its layers:

  rotate   rotary positions of a step's queries and keys: half and interleaved layouts, a part of the head, scaled
           frequencies; backward is the transposed rotation, which takes the outputs' gradients to the inputs'
  tree     attention over the whole cached context and, of the drafted tokens behind it, those on the token's own
           path through the tree of drafts; without a tree it is causal attention over all that is cached
  compact  keep the listed tokens of what was drafted (or of a whole context), move them together and bring
           the bounds of their blocks up to date; then read them back
  pages    a step of a beam search: every sequence continues another one, whose pages it shares; then each gets pages
           of its own for what it will write, with a copy of the shared block that it goes on in; that block read back

The cache is that of perf/operators.py: a page holds 64 consecutive tokens of one sequence, for each key/value
head 64 key rows of `dim` E4M3 codes, 64 value rows, 64 key scales and 64 value scales (E8M0 bytes).  Tokens are a
flat list with a sequence number and a position (the token's place in the cache) each; -1 is a padding entry.
"""
import math
import random

import torch

own = False

BLOCK = 64
DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    def rotate(name, tokens, heads, group, dim, rot, offset, inter, backward, scaling, far, pad=False):
        return {"name": name, "op": "rotate", "tokens": tokens, "heads": heads, "group": group, "dim": dim, "rot": rot,
                "offset": offset, "interleaved": inter, "backward": backward, "scaling": scaling, "far": far, "pad": pad}

    def tree(name, batch, ctx, nodes, heads, group, dim, drafts=True, ragged=False):
        return {"name": name, "op": "tree", "batch": batch, "ctx": ctx, "nodes": nodes, "heads": heads, "group": group,
                "dim": dim, "drafts": drafts, "ragged": ragged}

    def compact(name, batch, ctx, nodes, keep, heads, dim):
        return {"name": name, "op": "compact", "batch": batch, "ctx": ctx, "nodes": nodes, "keep": keep, "heads": heads,
                "dim": dim}

    def pages(name, batch, ctx, new, heads, dim):
        return {"name": name, "op": "pages", "batch": batch, "ctx": ctx, "new": new, "heads": heads, "dim": dim}

    return [
        # one decoded token far into a context: the smallest call, all latency
        rotate("rotate_decode", 1, 4, 8, 128, 128, 0, False, False, "ramp", 100000),
        # a prefill chunk of 8,192 tokens, half of the head rotated, pairs side by side
        rotate("rotate_prefill", 8192, 4, 8, 128, 64, 0, True, False, "none", 16384),
        # gradients of a packed batch with padding, the last channels of the head, scaled by wavelength
        rotate("rotate_backward", 5999, 2, 7, 64, 48, 16, False, True, "bands", 40000, pad=True),
        # one token of one sequence over everything that is cached
        tree("tree_token", 1, 8192, 1, 4, 8, 128, drafts=False),
        # 32 sequences with trees of 16 drafted tokens
        tree("tree_batch", 32, 16384, 16, 4, 8, 128, ragged=True),
        # ragged small trees, narrow heads, 16 query heads to a key/value head
        tree("tree_ragged", 12, 5000, 37, 2, 16, 64, ragged=True),
        # one long context with a tree of 64
        tree("tree_long", 1, 131072, 64, 4, 8, 128),
        # a whole prompt and the 4,096 tokens before it, causal
        tree("tree_prompt", 1, 8192, 4096, 4, 8, 128, drafts=False),
        # four sequences keep up to 8 of 32 drafted tokens
        compact("compact_drafts", 4, 4000, 32, 8, 4, 128),
        # eviction: a third of each context is kept
        compact("compact_context", 16, 0, 6000, 2000, 4, 128),
        # four beams
        pages("pages_beams", 4, 2001, 1, 4, 128),
        # 192 sequences in a pool of many pages
        pages("pages_many", 192, 16384, 64, 8, 64),
    ]


def draw(rng):
    def logint(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    while True:
        op = rng.choice(["rotate", "tree", "tree", "tree", "compact", "pages"])
        dim, heads = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16])
        if group * heads > 64:
            continue
        if op == "rotate":
            dim = rng.choice([64, 64, 80, 96, 128, 128, 192, 256])
            rot = 2 * rng.randint(1, dim // 2) if rng.random() < 0.3 else 8 * rng.randint(2, dim // 8)
            case = {"op": op, "tokens": logint(1, 8192), "heads": heads, "group": group, "dim": dim, "rot": rot,
                    "offset": rng.choice([0, 0, dim - rot, rng.randint(0, dim - rot)]), "interleaved": rng.random() < 0.5,
                    "backward": rng.random() < 0.4, "scaling": rng.choice(["none", "linear", "base", "ramp", "bands"]),
                    "far": logint(64, 1000000), "pad": rng.random() < 0.5}
        elif op == "tree":
            drafts = rng.random() < 0.7
            batch = logint(1, 64)
            case = {"op": op, "batch": batch, "ctx": logint(1, 100000), "nodes": logint(1, 190 if drafts else 4096),
                    "heads": heads, "group": group, "dim": dim, "drafts": drafts, "ragged": rng.random() < 0.6}
        elif op == "compact":
            nodes = logint(1, 8000)
            case = {"op": op, "batch": logint(1, 200), "ctx": logint(1, 8000) if nodes < 500 else 0, "nodes": nodes,
                    "keep": max(1, int(nodes * rng.uniform(0.05, 0.9))), "heads": heads, "dim": dim}
        else:
            case = {"op": op, "batch": logint(1, 256), "ctx": logint(1, 16384), "new": logint(1, 200), "heads": heads,
                    "dim": dim}
        if _fits(case):
            return case


def _fits(case):
    """No dearer than the largest listed cases, and a state that is quickly made."""
    w = work(case)
    if case["op"] == "rotate":
        return w["bytes"] <= 1.6e8
    if case["op"] == "tree":
        lens, M = _lengths(case), case["nodes"]
        cached = len(lens) * (case["ctx"] + M) * case["heads"] * case["dim"]
        scores = len(lens) * M * case["heads"] * case["group"] * (case["ctx"] + M)
        return cached <= 2 ** 28 and scores <= 2 ** 29 and w["flops"] <= 2.1e11 and w["bytes"] <= 4e8
    tokens = case["batch"] * (case["ctx"] + (case["nodes"] if case["op"] == "compact" else 0))
    return tokens * case["heads"] * case["dim"] <= 2 ** 28 and w["bytes"] <= 2e8


def _lengths(case):
    """(context, tokens behind it) of each sequence; both follow from the case alone."""
    B, ctx, new = case["batch"], case["ctx"], case["nodes"]
    if case["op"] == "tree" and not case["drafts"]:
        ctx = max(0, ctx - new)
    if not case.get("ragged", True):
        return [(ctx, new)] * B
    r = random.Random(B * 1000003 + ctx * 1009 + new * 17 + case["heads"])
    return [(ctx, new)] + [(r.randint(0, ctx), r.randint(1, new)) for _ in range(B - 1)]


def work(case):
    H, D = case["heads"], case["dim"]
    row = 2 * D + 2  # a token's key and value codes with their scales, one head
    if case["op"] == "rotate":  # rows in, rows out
        n = case["tokens"] * (case["group"] + 1) * H
        return {"bytes": 4 * n * D + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    if case["op"] == "tree":  # the context once, queries in, outputs and sums out
        G, lens = case["group"], _lengths(case)
        T, W = sum(n for _, n in lens), -(-case["nodes"] // 64)
        seen = sum(n * c + (n * (n + 1) // 2) for c, n in lens)
        return {"bytes": sum(c + n for c, n in lens) * H * row + T * H * G * (4 * D + 4) + T * 8 * (W + 1),
                "flops": seen * H * G * 4 * D}
    if case["op"] == "compact":  # kept rows read, written and read back, with keys read once more for the bounds
        kept = sum(min(n, case["keep"]) for _, n in _lengths(case))
        return {"bytes": kept * H * (2 * row + row + D + 4 * D), "flops": kept * H * D * 4}
    blocks = case["batch"] * -(-(case["ctx"] + case["new"]) // BLOCK)
    copies = case["batch"] * (case["ctx"] % BLOCK > 0)
    last = case["batch"] * min(BLOCK, case["ctx"])
    return {"bytes": blocks * 12 + 4 * copies * H * BLOCK * row + last * H * (row + 4 * D), "flops": last * H * D * 2}


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


def _plain_read(st, seq, pos):
    kc, vc, ks, vs = _views(st["pages"], st["dim"])
    t = torch.nonzero(pos >= 0)[:, 0]
    p = pos[t].long()
    page = st["table"][seq[t].long(), p // BLOCK].long()
    out = torch.zeros((2, pos.numel(), kc.shape[1], st["dim"]), device=DEV)
    out[0, t] = _decode(kc[page, :, p % BLOCK], ks[page, :, p % BLOCK])
    out[1, t] = _decode(vc[page, :, p % BLOCK], vs[page, :, p % BLOCK])
    return list(out.to(torch.bfloat16))


def _plain_rotate(st):
    live, R, at = st["pos"] >= 0, 2 * st["turns"].numel(), st["offset"]
    angle = st["pos"].clamp_min(0).double()[:, None] * st["freq"]
    c, s = ((f(angle) * st["gain"]).float()[:, None] for f in (torch.cos, torch.sin))
    if st["backward"]:
        s = -s

    def turned(x):
        y = x.float()
        part = y[..., at:at + R]
        if st["interleaved"]:
            a, b = part[..., 0::2], part[..., 1::2]
            part = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
        else:
            a, b = part[..., :R // 2], part[..., R // 2:]
            part = torch.cat([a * c - b * s, a * s + b * c], -1)
        y = torch.cat([y[..., :at], part, y[..., at + R:]], -1)
        return torch.where(live[:, None, None], y, 0.0).to(torch.bfloat16)

    return [turned(st["q"]), turned(st["k"])]


def _plain_tree(st):
    T, Hq, D = st["q"].shape
    kc, vc, ks, vs = _views(st["pages"], D)
    H, (B, N) = kc.shape[1], st["table"].shape
    at = st["table"].clamp_min(0).long()
    k, v = (_decode(c[at], s[at]).transpose(2, 3).reshape(B, N * BLOCK, H, D) for c, s in ((kc, ks), (vc, vs)))
    # the sequences' tokens side by side, padded to the longest
    t = torch.nonzero(st["pos"] >= 0)[:, 0]
    seq = st["seq"][t].long()
    rank = torch.arange(t.numel(), device=DEV) - torch.searchsorted(seq, seq)
    M = st["most"]
    q = torch.zeros((B, M, H, Hq // H, D), device=DEV)
    q[seq, rank] = st["q"][t].float().view(-1, H, Hq // H, D)
    x = torch.arange(N * BLOCK, device=DEV)
    pos = torch.full((B, M), -1, device=DEV)
    pos[seq, rank] = st["pos"][t].long()
    seen = x <= pos[..., None]
    if st["mask"] is not None:
        j = x - st["start"].long()[:, None]
        words = torch.zeros((B, M, st["mask"].shape[1]), dtype=torch.int64, device=DEV)
        words[seq, rank] = st["mask"][t]
        inside = (j >= 0) & (j < 64 * words.shape[-1])
        place = j.clamp(0, 64 * words.shape[-1] - 1)[:, None].expand(B, M, -1)
        bit = (torch.gather(words, 2, place // 64) >> (place % 64)) & 1
        seen &= (j < 0)[:, None] | (inside[:, None] & (bit > 0))
    s = torch.einsum("bmhgd,bxhd->bmhgx", q, k) * st["scale"]
    s.masked_fill_(~seen[:, :, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    z = p.sum(-1)
    o = torch.einsum("bmhgx,bxhd->bmhgd", p, v)
    o = torch.where(z[..., None] > 0, o / z[..., None], 0.0)
    lse = m[..., 0] + torch.log(z)
    out, lses = torch.zeros((T, Hq, D), device=DEV), torch.full((T, Hq), -math.inf, device=DEV)
    out[t], lses[t] = o[seq, rank].reshape(-1, Hq, D), lse[seq, rank].reshape(-1, Hq)
    return [out.to(torch.bfloat16), lses]


def _plain_compact(st):
    """Old rows are gathered before new ones are written; bounds from the keys that a touched block then has."""
    pages, D = st["pages"], st["dim"]
    views = _views(pages, D)
    B, A = st["nodes"].shape
    j = torch.arange(A, device=DEV)
    b, j = torch.nonzero(j < st["count"][:, None], as_tuple=True)
    src, dst = st["start"][b].long() + st["nodes"][b, j].long(), st["start"][b].long() + j
    table = st["table"].long()
    sp, dp = table[b, src // BLOCK], table[b, dst // BLOCK]
    moved = [x[sp, :, src % BLOCK] for x in views]
    h = torch.arange(pages.shape[1], device=DEV)
    views[0][dp[:, None], h, (dst % BLOCK)[:, None]], views[1][dp[:, None], h, (dst % BLOCK)[:, None]] = moved[:2]
    views[2][dp[:, None], h, (dst % BLOCK)[:, None]], views[3][dp[:, None], h, (dst % BLOCK)[:, None]] = moved[2:]
    length = torch.where(st["count"] >= 0, st["start"] + st["count"], st["start"])
    n = torch.arange(table.shape[1], device=DEV)
    touched = (n >= st["start"][:, None] // BLOCK) & (n * BLOCK < length[:, None]) & (st["count"] >= 0)[:, None]
    b, n = torch.nonzero(touched, as_tuple=True)
    page = table[b, n]
    keys = _decode(views[0][page], views[2][page])
    in_use = (n[:, None] * BLOCK + torch.arange(BLOCK, device=DEV) < length[b][:, None])[:, None, :, None]
    st["bounds"][page], st["bound_exp"][page] = _bounds_of(torch.where(in_use, keys, -math.inf).amax(2),
                                                           torch.where(in_use, keys, math.inf).amin(2))
    return [length] + _plain_read(st, st["seq"], st["pos"]) + [st["bounds"], st["bound_exp"]]


def _plain_pages(st):
    table, refs, length = st["table"], st["refs"], st["length"]
    B, N = table.shape
    n = torch.arange(N, device=DEV)
    # every sequence continues its parent: the parent's pages up to the length, one reference more each
    old = table.clone()
    table.copy_(torch.where(n < (-(-length // BLOCK))[:, None], old[st["parent"].long()], -1))
    refs += torch.bincount(table[table >= 0], minlength=refs.numel()).to(torch.int32)
    refs -= torch.bincount(old[old >= 0], minlength=refs.numel()).to(torch.int32)
    # pages for what comes: the lowest free ones, in the order of the sequences and blocks
    first, end = (length // BLOCK)[:, None], (-(-st["end"] // BLOCK))[:, None]
    page = table.clamp_min(0).long()
    release = (table >= 0) & (n >= end)
    shared = (table >= 0) & (n >= first) & (n < end) & (refs[page] > 1)
    need = shared | ((table < 0) & (n >= first) & (n < end))
    free = torch.nonzero(refs == 0)[:, 0]
    new = free[(need.flatten().cumsum(0) - 1).clamp_min(0).view(B, N)]
    copy = shared & (n == first) & (length % BLOCK > 0)[:, None]
    st["pages"][new[copy]] = st["pages"][page[copy]]
    st["bounds"][new[copy]] = st["bounds"][page[copy]]
    st["bound_exp"][new[copy]] = st["bound_exp"][page[copy]]
    refs -= torch.bincount(page[shared | release], minlength=refs.numel()).to(torch.int32)
    refs[new[need]] = 1
    table.copy_(torch.where(need, new, torch.where(release, -1, table)))
    return [table, refs] + _plain_read(st, st["seq"], st["pos"]) + [st["bounds"], st["bound_exp"]]


# --------------------------------------------------------------------------- inputs

def _frequencies(case):
    """(radians a position of each pair, the factor of cosine and sine), for contexts 8 times as long as the original
    2,048: positions divided; the base raised; a ramp over the pairs between 32 and 1 turns in the original context; or by
    wavelength between an original context and a quarter of it."""
    R, how, base, s, L = case["rot"], case["scaling"], 10000.0, 8.0, 2048.0
    if how == "base" and R > 2:
        base *= s ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if how == "linear":
        return [x / s for x in f], 1.0
    if how == "ramp":
        pair = [R * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), R // 2 - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(R // 2)]
        return [x / s * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(s) + 1.0
    if how == "bands":
        kept = [min(max((L * x / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0), 1.0) for x in f]
        return [(1 - w) * x / s + w * x for x, w in zip(f, kept)], 1.0
    return f, 1.0


def prepare(case, seed):
    """Queries, keys and values are normal; the cache's pages lie in random order; trees have random branches.  Every tensor
    is made from the seed."""
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    r = random.Random(int(seed) * 7919 + 5)
    H, D, op = case["heads"], case["dim"], case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    st = {"op": op, "dim": D, "keep": {}}
    if op == "rotate":
        T, G = case["tokens"], case["group"]
        f, gain = _frequencies(case)
        first = r.randint(0, max(0, case["far"] - T))
        pos = torch.arange(first, first + T, device=DEV)
        if case["pad"]:
            pos[torch.randint(T, (T // 50 + 1,), generator=g, device=DEV)] = -1
        # one projection's output: queries, keys and values of a token side by side
        qkv = normal(T, (G + 2) * H, D).to(torch.bfloat16)
        turns = [round(x / (2 * math.pi) * 2 ** 64) % 2 ** 64 for x in f]  # of a full turn, in units of 2^-64
        st |= {"q": qkv[:, :G * H], "k": qkv[:, G * H:(G + 1) * H], "pos": pos.to(torch.int32), "gain": gain,
               "freq": torch.tensor(f, dtype=torch.float64, device=DEV), "offset": case["offset"],
               "turns": torch.tensor([x - 2 ** 64 * (x >= 2 ** 63) for x in turns], device=DEV),
               "interleaved": case["interleaved"], "backward": case["backward"]}
        return st

    if op == "pages":
        # all sequences with pages of their own at first: the first pass brings the sharing
        B, L, end = case["batch"], case["ctx"], case["ctx"] + case["new"]
        N, nb = -(-end // BLOCK) + 1, -(-L // BLOCK)
        parents = max(1, B // 4)
        n = parents * nb + 2 * B * (-(-end // BLOCK) - L // BLOCK + 1) + 5
        table = torch.full((B, N), -1, dtype=torch.int32, device=DEV)
        table[:parents, :nb] = torch.randperm(n, generator=g, device=DEV)[:parents * nb].to(torch.int32).view(parents, nb)
        parent = whole([r.randrange(parents) for _ in range(B)])
        table = table[parent.long()]
        refs = torch.bincount(table[table >= 0], minlength=n).to(torch.int32)
        st |= {"parent": whole([r.randrange(B) for _ in range(B)]), "length": whole([L] * B), "end": whole([end] * B),
               "table": table.contiguous(), "refs": refs}
        lens, last = [(L, 0)] * B, (L - 1) // BLOCK * BLOCK
        st["seq"] = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(L - last)
        st["pos"] = torch.arange(last, L, device=DEV, dtype=torch.int32).repeat(B)
    else:
        lens = _lengths(case)
        nb = torch.tensor([-(-(c + m) // BLOCK) for c, m in lens], device=DEV)
        B, N, n = len(lens), int(nb.max()), int(nb.sum()) + 3
        order = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, N), -1, dtype=torch.int32, device=DEV)
        table[torch.arange(N, device=DEV)[None] < nb[:, None]] = order[:n - 3]
        st["table"], st["start"] = table, whole([c for c, _ in lens])
    pages = torch.zeros((n, H, 2 * BLOCK * D + 2 * BLOCK), dtype=torch.uint8, device=DEV)
    kc, vc, ks, vs = _views(pages, D)
    kc[:], ks[:] = _encode(normal(n, H, BLOCK, D).to(torch.bfloat16).float())
    vc[:], vs[:] = _encode(normal(n, H, BLOCK, D).to(torch.bfloat16).float())
    keys = _decode(kc.contiguous(), ks.contiguous())
    st["pages"], (st["bounds"], st["bound_exp"]) = pages, _bounds_of(keys.amax(2), keys.amin(2))

    if op == "compact":
        count, nodes = [], []
        much = random.Random(case["batch"] * 31 + case["nodes"])  # how much is kept follows from the case alone
        for i, (_, m) in enumerate(lens):
            kept = min(m, case["keep"]) if i == 0 else much.randint(0, min(m, case["keep"]))
            nodes.append(sorted(r.sample(range(m), kept)) + [-1] * (case["keep"] - kept))
            count.append(-1 if i % 17 == 16 else kept)
        st["count"], st["nodes"] = whole(count), whole(nodes)
        got = [(i, c + j) for i, ((c, _), k) in enumerate(zip(lens, count)) for j in range(max(k, 0))] or [(0, -1)]
        st["seq"], st["pos"] = whole([s for s, _ in got]), whole([p for _, p in got])
    if op == "tree":
        G, drafts = case["group"], case["drafts"]
        seq = [i for i, (_, m) in enumerate(lens) for _ in range(m)]
        pos = [c + j for c, m in lens for j in range(m)]
        masks, W = [], -(-case["nodes"] // 64)
        for _, m in lens if drafts else []:
            tree = []
            for j in range(m):
                parent = r.randint(max(-1, j - 9), j - 1)
                tree.append((tree[parent] if parent >= 0 else 0) | 1 << j)
            masks += tree
        if case["ragged"]:  # a padding entry at the end
            seq, pos, masks = seq + [0], pos + [-1], masks + [0]
        cut = [[(m >> 64 * w) % 2 ** 64 for w in range(W)] for m in masks]
        st["mask"] = torch.tensor([[x - 2 ** 64 * (x >= 2 ** 63) for x in m] for m in cut], device=DEV) if drafts else None
        st["seq"], st["pos"], st["most"], st["scale"] = whole(seq), whole(pos), max(m for _, m in lens), D ** -0.5
        # a query looks for a few keys, as in earnest: it is like one of its own sequence's
        like = torch.randint(n, (len(seq),), generator=g, device=DEV)
        st["q"] = (0.8 * keys[like, :, 0][:, :, None] + normal(len(seq), H, G, D)).reshape(-1, H * G, D).to(torch.bfloat16)
    return st


# --------------------------------------------------------------------------- one pass

def run(st):
    return (_own if own else _plain)[st["op"]](st)


_plain = {"rotate": _plain_rotate, "tree": _plain_tree, "compact": _plain_compact, "pages": _plain_pages}


def _cache(st):
    from bit_routed_expert_gb300 import KvCache
    return KvCache(st["pages"], st["bounds"], st["bound_exp"])


def _own_rotate(st):
    from bit_routed_expert_gb300 import kv_rotate
    return list(kv_rotate(st["q"], st["k"], st["pos"], st["turns"], gain=st["gain"], offset=st["offset"],
                          interleaved=st["interleaved"], backward=st["backward"]))


def _own_tree(st):
    from bit_routed_expert_gb300 import kv_attend_tree, kv_attend_tree_workspace
    if "ws" not in st["keep"]:  # the workspace that a serving loop keeps from step to step
        T, Hq, D = st["q"].shape
        size = kv_attend_tree_workspace(T, Hq, st["bounds"].shape[1], D)
        st["keep"]["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return list(kv_attend_tree(st["q"], _cache(st), st["seq"], st["pos"], st["table"], start=st["start"], mask=st["mask"],
                               scale=st["scale"], ws=st["keep"]["ws"]))


def _own_compact(st):
    from bit_routed_expert_gb300 import kv_compact, kv_read
    cache = _cache(st)
    length = kv_compact(cache, st["table"], st["start"], st["nodes"], st["count"])
    k, v = kv_read(cache, st["seq"], st["pos"], st["table"])
    return [length, k, v, st["bounds"], st["bound_exp"]]


def _own_pages(st):
    from bit_routed_expert_gb300 import kv_fork, kv_read, kv_resize, kv_resize_workspace
    cache = _cache(st)
    if "ws" not in st["keep"]:
        size = kv_resize_workspace(cache.n_pages, *st["table"].shape)
        st["keep"]["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    kv_fork(cache, st["refs"], st["table"], st["parent"], st["length"])
    kv_resize(cache, st["refs"], st["table"], st["length"], st["end"], ws=st["keep"]["ws"])
    k, v = kv_read(cache, st["seq"], st["pos"], st["table"])
    return [st["table"], st["refs"], k, v, st["bounds"], st["bound_exp"]]


_own = {"rotate": _own_rotate, "tree": _own_tree, "compact": _own_compact, "pages": _own_pages}


# --------------------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "tree": _exact_tree, "compact": _exact_compact, "pages": _exact_pages}[case["op"]](st)


def _exact_rotate(st):
    """Angles by whole numbers: position times turns, what is beyond a full turn dropped."""
    turn = (st["pos"].long()[:, None] * st["turns"][None]).double() * 2.0 ** -64
    turn = torch.exp(2j * math.pi * (-turn if st["backward"] else turn)) * st["gain"]
    at, R = st["offset"], 2 * st["turns"].numel()
    out = []
    for x in (st["q"], st["k"]):
        y = x.double().clone()
        one, two = (slice(at, at + R, 2), slice(at + 1, at + R, 2)) if st["interleaved"] else \
            (slice(at, at + R // 2), slice(at + R // 2, at + R))
        z = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * turn[:, None]
        y[..., one], y[..., two] = z.real, z.imag
        y[st["pos"] < 0] = 0
        out.append(y)
    return out


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


def _exact_tree(st):
    T, Hq, D = st["q"].shape
    H = st["pages"].shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    seq, pos = st["seq"].tolist(), st["pos"].tolist()
    words = None if st["mask"] is None else st["mask"].tolist()
    k, v = (x.to(torch.float32) for x in _cached(st))  # (exact: a code times a power of two)
    t = 0
    while t < T:  # a stretch of tokens of one sequence
        t1 = t
        while t1 < T and seq[t1] == seq[t] and t1 - t < 128:
            t1 += 1
        top = max(pos[t:t1]) + 1
        if top > 0:
            row = st["table"][seq[t]].long()[:-(-top // BLOCK)]
            x = torch.arange(top, device=DEV)
            ok = torch.stack([x <= p for p in pos[t:t1]])
            if words is not None:
                c = int(st["start"][seq[t]])
                for i in range(t, t1):
                    bits = sum((w % 2 ** 64) << 64 * n for n, w in enumerate(words[i]))
                    behind = torch.tensor([bits >> j & 1 for j in range(max(0, top - c))], dtype=torch.bool, device=DEV)
                    ok[i - t, c:] &= behind
            for h in range(H):
                qq = st["q"][t:t1].double().view(t1 - t, H, -1, D)[:, h] * st["scale"]
                kk, vv = (y[row, :, h].double().reshape(-1, D)[:top] for y in (k, v))
                s = (qq @ kk.T).masked_fill(~ok[:, None], -math.inf)
                m = s.amax(-1, keepdim=True)
                w = torch.exp(s - m.masked_fill(m == -math.inf, 0.0))
                z = w.sum(-1, keepdim=True)
                G = qq.shape[1]
                out[t:t1, h * G:(h + 1) * G] = (w @ vv) / z.clamp_min(1e-300)
                lse[t:t1, h * G:(h + 1) * G] = (m + torch.log(z))[..., 0]
        t = t1
    return [out, lse]


def _least(a, top):
    """Smallest whole e >= -64 with a <= top * 2^e."""
    e = torch.ceil(torch.log2(a / top)).clamp_min(-64)
    e = torch.where(a > top * torch.exp2(e), e + 1, e)
    return torch.where((a <= top * torch.exp2(e - 1)) & (e > -64), e - 1, e)


def _exact_compact(st):
    start, count = st["start"].tolist(), st["count"].tolist()
    nodes, table = st["nodes"].tolist(), st["table"].tolist()
    k, v = _cached(st)
    bounds, bexp = st["bounds"].clone(), st["bound_exp"].clone()
    length, rows = [], []
    for b, n in enumerate(count):
        length.append(start[b] + max(n, 0))
        src = [start[b] + x for x in nodes[b][:max(n, 0)]]
        at = [(table[b][p // BLOCK], p % BLOCK) for p in src]
        rows.append(torch.tensor(at, dtype=torch.int64, device=DEV).view(-1, 2))
        if n < 0 or length[b] == start[b] // BLOCK * BLOCK:
            continue
        first = start[b] // BLOCK * BLOCK
        kept = torch.tensor([(table[b][p // BLOCK], p % BLOCK) for p in list(range(first, start[b])) + src],
                            device=DEV)
        for i, part in enumerate(kept.split(BLOCK)):
            keys = k[part[:, 0], part[:, 1]]
            e = _least(keys.abs().amax((0, 2)), 63.0)
            u, page = torch.exp2(e)[:, None], table[b][first // BLOCK + i]
            bounds[page] = torch.stack([torch.ceil(keys.amax(0) / u), torch.floor(keys.amin(0) / u)], 1).to(torch.int8)
            bexp[page] = e.to(torch.int8)
    at = torch.cat(rows)
    if not at.numel():
        zero = torch.zeros((1, *k.shape[2:]), dtype=torch.float64, device=DEV)
        return [torch.tensor(length, dtype=torch.int32, device=DEV), zero, zero, bounds, bexp]
    return [torch.tensor(length, dtype=torch.int32, device=DEV), k[at[:, 0], at[:, 1]], v[at[:, 0], at[:, 1]], bounds, bexp]


def _exact_pages(st):
    table, refs, parent = st["table"].tolist(), st["refs"].tolist(), st["parent"].tolist()
    length, end = st["length"].tolist(), st["end"].tolist()
    k, v = _cached(st)
    B, N = len(table), len(table[0])
    forked = [table[p][:-(-n // BLOCK)] + [-1] * (N - -(-n // BLOCK)) for p, n in zip(parent, length)]
    for was, now in zip(table, forked):
        for p in was:
            refs[p] -= p >= 0
        for p in now:
            refs[p] += p >= 0
    free, then = [i for i, n in enumerate(refs) if n == 0], list(refs)
    copied, taken = {}, 0
    for b, row in enumerate(forked):
        for n in range(length[b] // BLOCK, N):
            p = row[n]
            if n >= -(-end[b] // BLOCK):
                row[n] = -1
                then[p] -= p >= 0
            elif p < 0 or refs[p] > 1:
                row[n] = free[taken]
                then[row[n]], taken = 1, taken + 1
                then[p] -= p >= 0
                if p >= 0 and n == length[b] // BLOCK and length[b] % BLOCK:
                    copied[row[n]] = p
    new, old = (torch.tensor(list(x), dtype=torch.int64, device=DEV) for x in (copied.keys(), copied.values()))
    bounds, bexp = st["bounds"].clone(), st["bound_exp"].clone()
    bounds[new], bexp[new] = bounds[old], bexp[old]
    where = torch.arange(k.shape[0], device=DEV)
    where[new] = old  # a copied page holds what its original holds
    after = torch.tensor(forked, dtype=torch.int32, device=DEV)
    at = where[after[st["seq"].long(), st["pos"].long() // BLOCK].long()]
    slot = st["pos"].long() % BLOCK
    return [after, torch.tensor(then, dtype=torch.int32, device=DEV), k[at, slot], v[at, slot], bounds, bexp]
