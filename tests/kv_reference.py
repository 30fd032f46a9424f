"""The key/value cache calls restated from their definitions in include/bre.h, in 64 bits on the
CPU, token by token; and small ragged batches to run them on."""
import math
from dataclasses import dataclass

import torch

BLOCK = 64
MAX = 448.0 * 2.0 ** 119


def least_exp(a: float, top: float) -> int:
    """Least e >= -64 with a <= top * 2^e."""
    e = -64
    if a > 0:
        e = max(-64, math.frexp(a / top)[1] - 2)
    while a > math.ldexp(top, e):
        e += 1
    return e


def e4m3_code(x: float) -> int:
    """Nearest E4M3 code of |x| <= 448, ties to even; NaN 0x7F."""
    if x != x:
        return 0x7F
    sign = 0x80 if math.copysign(1.0, x) < 0 else 0
    a = abs(x)
    e = max(-6, math.frexp(a)[1] - 1) if a else -6
    n = round(math.ldexp(a, 3 - e))       # Python rounds halves to even
    if n == 16:
        e, n = e + 1, 8
    return sign | (n if n < 8 else ((e + 7) << 3) | (n - 8))


def e4m3_value(c: int) -> float:
    ex, man = (c >> 3) & 15, c & 7
    if (c & 0x7F) == 0x7F:
        return math.nan
    v = math.ldexp(8 + man, ex - 10) if ex else math.ldexp(man, -9)
    return -v if c & 0x80 else v


VALUES = torch.tensor([e4m3_value(c) for c in range(256)], dtype=torch.float64)


def store_row(row: torch.Tensor):
    """[D] -> (codes uint8 [D], scale byte)."""
    if bool(row.isnan().any()):
        return torch.zeros(len(row), dtype=torch.uint8), 255
    x = [v if v != v else max(-MAX, min(MAX, v)) for v in row.double().tolist()]
    e = least_exp(max(abs(v) for v in x), 448.0)
    return torch.tensor([e4m3_code(math.ldexp(v, -e)) for v in x], dtype=torch.uint8), e + 127


def views(pages: torch.Tensor, D: int):
    n, H, _ = pages.shape
    return (pages[:, :, :BLOCK * D].view(n, H, BLOCK, D), pages[:, :, BLOCK * D:2 * BLOCK * D].view(n, H, BLOCK, D),
            pages[:, :, 2 * BLOCK * D:2 * BLOCK * D + BLOCK], pages[:, :, 2 * BLOCK * D + BLOCK:])


def page_of(table, n_pages, s, b):
    """(page or -1, whether the lookup is an error)."""
    if not (0 <= s < table.shape[0] and 0 <= b < table.shape[1]):
        return -1, True
    p = int(table[s, b])
    return (-1, True) if p >= n_pages else (max(p, -1), False)


def append(pages, bounds, bexp, k, v, seq, pos, table):
    """Updates pages, bounds and bexp (CPU tensors) in place; whether an error bit is due."""
    D, H, err = k.shape[2], k.shape[1], False
    kc, vc, ks, vs = views(pages, D)
    t, T = 0, len(seq)
    while t < T:
        t1 = t + 1
        if pos[t] >= 0:
            b = pos[t] // BLOCK
            while t1 < T and seq[t1] == seq[t] and pos[t1] >= 0 and pos[t1] // BLOCK == b:
                t1 += 1
            pg, bad = page_of(table, pages.shape[0], seq[t], b)
            err |= bad or pg < 0
            for h in range(H if pg >= 0 else 0):
                new = []
                for i in range(t, t1):
                    slot = pos[i] % BLOCK
                    kc[pg, h, slot], ks[pg, h, slot] = store_row(k[i, h])
                    vc[pg, h, slot], vs[pg, h, slot] = store_row(v[i, h])
                    new.append(VALUES[kc[pg, h, slot].long()] * 2.0 ** (int(ks[pg, h, slot]) - 127))
                new = torch.stack(new)
                hi, lo, e = new.amax(0), new.amin(0), least_exp(float(new.abs().max()), 63.0)
                if pos[t] % BLOCK:
                    oe = int(bexp[pg, h])
                    hi = torch.maximum(hi, bounds[pg, h, 0].double() * 2.0 ** oe)
                    lo = torch.minimum(lo, bounds[pg, h, 1].double() * 2.0 ** oe)
                    e = max(e, oe)
                bounds[pg, h, 0] = torch.ceil(hi * 2.0 ** -e).to(torch.int8)
                bounds[pg, h, 1] = torch.floor(lo * 2.0 ** -e).to(torch.int8)
                bexp[pg, h] = e
        t = t1
    return err


def values(pages, D):
    """Stored keys and values [page, head, slot, D] in 64 bits."""
    kc, vc, ks, vs = views(pages, D)
    scale = [torch.where(x == 255, math.nan, 2.0 ** (x.double() - 127))[..., None] for x in (ks, vs)]
    return VALUES[kc.long()] * scale[0], VALUES[vc.long()] * scale[1]


def select(q, bounds, bexp, seq, pos, table, k, n_sink, n_local):
    """(ids [T, H, k], scores in 64 bits, whether an error bit is due)."""
    T, Hq, D = q.shape
    H = bounds.shape[1]
    ids = torch.full((T, H, k), -1, dtype=torch.int32)
    scores = torch.zeros((T, H, k), dtype=torch.float64)
    err = False
    for t in range(T):
        if pos[t] < 0:
            continue
        cur = pos[t] // BLOCK
        if not 0 <= seq[t] < table.shape[0]:
            err = True
            continue
        err |= cur >= table.shape[1]
        blocks = []
        for b in range(min(cur + 1, table.shape[1])):
            pg, bad = page_of(table, bounds.shape[0], seq[t], b)
            err |= bad
            if pg >= 0:
                blocks.append((b, pg))
        if not blocks:
            continue
        at = torch.tensor([p for _, p in blocks])
        for h in range(H):
            x = q[t].double().view(H, -1, D)[h]
            x = torch.where(x.isnan(), x, x.clamp(-MAX, MAX))
            e = least_exp(float(x.nan_to_num(0.0).abs().max()), 127.0)
            c = torch.round(x * 2.0 ** -e).nan_to_num(0.0)
            s = (bounds[at, h, 0].double() @ c.clamp_min(0).sum(0) + bounds[at, h, 1].double() @ c.clamp_max(0).sum(0))
            s = s * 2.0 ** bexp[at, h].double() * 2.0 ** e
            order = sorted(range(len(blocks)), key=lambda i: (
                not (blocks[i][0] < n_sink or blocks[i][0] > cur - n_local), -float(s[i]), i)
                if not (blocks[i][0] < n_sink or blocks[i][0] > cur - n_local) else (False, 0.0, i))
            for j, i in enumerate(sorted(order[:k])):
                ids[t, h, j] = blocks[i][0]
                scores[t, h, j] = s[i]
    return ids, scores, err


def attend(q, pages, seq, pos, table, ids, scale):
    """(out, lse, bound of the weights' effect on out, bound of the logits' error, error bit):
    out and lse in 64 bits, and for each row sum_x p_x |v_x| and max_x scale * sum |q||k|."""
    T, Hq, D = q.shape
    kk, vv = values(pages, D)
    H = kk.shape[1]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    mass = torch.zeros((T, Hq, D), dtype=torch.float64)
    size = torch.zeros((T, Hq), dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    err = False
    for t in range(T):
        if pos[t] < 0:
            continue
        for h in range(H):
            ks, vs = [], []
            for b in ids[t, h].tolist():
                if b < 0 or b * BLOCK > pos[t]:
                    continue
                pg, bad = page_of(table, pages.shape[0], seq[t], b)
                err |= bad
                if pg >= 0:
                    n = min(BLOCK, pos[t] - b * BLOCK + 1)
                    ks.append(kk[pg, h, :n])
                    vs.append(vv[pg, h, :n])
            if not ks:
                continue
            ks, vs = torch.cat(ks), torch.cat(vs)
            x = q[t, h * G:(h + 1) * G].double()
            s = x @ ks.T * scale
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - m)
            z = p.sum(1, keepdim=True)
            r = slice(h * G, (h + 1) * G)
            out[t, r], mass[t, r] = p @ vs / z, p @ vs.abs() / z
            lse[t, r] = (m + torch.log(z))[:, 0] if not bool(vs.isnan().any()) else math.nan   # a NaN value row too
            size[t, r] = (x.abs() @ ks.abs().T).amax(1) * abs(scale)
    return out, lse, mass, size, err


@dataclass
class Batch:
    seq: list
    pos: list
    table: torch.Tensor
    n_pages: int

    def on(self, dev):
        return (torch.tensor(self.seq, dtype=torch.int32, device=dev), torch.tensor(self.pos, dtype=torch.int32, device=dev),
                self.table.to(dev))


def batch(lens, new, seed=0, spare=2, pad=(), blocks=None):
    """Sequences of lens[b] tokens of which the last new[b] are in the call; pages in random order;
    `pad`: indexes at which padding entries are put in."""
    g = torch.Generator().manual_seed(seed)
    nb = [-(-n // BLOCK) for n in lens]
    N = max(max(nb), 1) if blocks is None else blocks
    order = torch.randperm(sum(nb) + spare, generator=g).tolist()
    table = torch.full((len(lens), N), -1, dtype=torch.int32)
    for b, n in enumerate(nb):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    seq = [b for b, n in enumerate(new) for _ in range(n)]
    pos = [p for b, n in enumerate(new) for p in range(lens[b] - n, lens[b])]
    for i in pad:
        seq.insert(i, 0)
        pos.insert(i, -1)
    return Batch(seq, pos, table, sum(nb) + spare)


def rows(seed, *shape, gain=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * gain).to(torch.bfloat16)


def filled(b: Batch, lens, H, D, seed=0):
    """CPU pages, bounds and exponents that hold every token of the batch's sequences (stored by torch's
    own E4M3 cast, whose bytes test_kv_cache.py compares with store_row)."""
    k = rows(seed + 1, b.n_pages, H, BLOCK, D).double() * (1 + (torch.arange(D) % 7 == 0) * 3.0)
    v = rows(seed + 2, b.n_pages, H, BLOCK, D).double()
    pages = torch.zeros((b.n_pages, H, 2 * BLOCK * (D + 1)), dtype=torch.uint8)
    kc, vc, ks, vs = views(pages, D)
    for c, sc, x in ((kc, ks, k), (vc, vs, v)):
        a = x.abs().amax(-1)
        e = torch.ceil(torch.log2(a / 448.0)).clamp_min(-64)
        e = torch.where(a > 448.0 * 2.0 ** e, e + 1, e)
        c[:] = (x * 2.0 ** -e[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        sc[:] = (e + 127).to(torch.uint8)
    kk, _ = values(pages, D)
    a = kk.abs().amax((2, 3))
    e = torch.ceil(torch.log2(a / 63.0)).clamp_min(-64)
    e = torch.where(a > 63.0 * 2.0 ** e, e + 1, e)
    s = 2.0 ** -e[..., None]
    bounds = torch.stack([torch.ceil(kk.amax(2) * s), torch.floor(kk.amin(2) * s)], 2).to(torch.int8)
    return pages, bounds, e.to(torch.int8)
