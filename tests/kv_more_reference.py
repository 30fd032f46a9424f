"""Rotary positions, tree attention and the page calls restated from include/bre.h on the CPU, in 64 bits and whole numbers."""
import math

import torch

import kv_reference as R

BLOCK = R.BLOCK


def rotate(x, pos, turns, gain, offset, interleaved, backward):
    """(result in 64 bits, |a| + |b| of each rotated channel's pair, times the gain)."""
    P = len(turns)
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    for i in range(P):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + P + i)
        angle = torch.tensor([2 * math.pi * math.ldexp((max(int(p), 0) * int(turns[i])) % 2 ** 64, -64) for p in pos],
                             dtype=torch.float64)
        c, s = (torch.cos(angle) * gain)[:, None], (torch.sin(angle) * gain * (-1 if backward else 1))[:, None]
        u, v = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * c - v * s, u * s + v * c
        size[..., a] = size[..., b] = (u.abs() + v.abs()) * abs(gain)
    y[pos < 0], size[pos < 0] = 0.0, 0.0
    return y, size


def turns_of(f):
    """Frequencies (radians a position) as whole numbers of 2^-64 turns."""
    return [round(x / (2 * math.pi) * 2 ** 64) % 2 ** 64 for x in f]


def as_int64(words):
    return torch.tensor([w - 2 ** 64 * (w >= 2 ** 63) for w in words], dtype=torch.int64)


def mask_tensor(masks, words):
    """[T][words] int64 from Python's whole numbers."""
    return torch.stack([as_int64([(m >> 64 * w) % 2 ** 64 for w in range(words)]) for m in masks]) if masks else \
        torch.zeros((0, words), dtype=torch.int64)


def tree(g, nodes):
    """Random ancestor masks of a tree whose nodes follow their parents."""
    got = []
    for j in range(nodes):
        parent = int(torch.randint(max(-1, j - 6), j, (1,), generator=g)) if j else -1
        got.append((got[parent] if parent >= 0 else 0) | 1 << j)
    return got


def attend_tree(q, pages, seq, pos, table, start, masks, scale, words=None):
    """(out, lse, sum p |v|, largest scale sum |q||k|, largest scale max|q| sum|k|, error bit); masks: whole numbers or None."""
    T, Hq, D = q.shape
    kk, vv = R.values(pages, D)
    H = kk.shape[1]
    G = Hq // H
    out, mass = torch.zeros((T, Hq, D), dtype=torch.float64), torch.zeros((T, Hq, D), dtype=torch.float64)
    size, peak = torch.zeros((T, Hq), dtype=torch.float64), torch.zeros((T, Hq), dtype=torch.float64)
    lse, err = torch.full((T, Hq), -math.inf, dtype=torch.float64), False
    for t in range(T):
        if pos[t] < 0:
            continue
        at = []
        err |= pos[t] // BLOCK >= table.shape[1]
        for b in range(min(pos[t] // BLOCK + 1, table.shape[1])):
            pg, bad = R.page_of(table, pages.shape[0], seq[t], b)
            err |= bad
            for x in range(b * BLOCK, min((b + 1) * BLOCK, pos[t] + 1) if pg >= 0 else 0):
                c = max(int(start[seq[t]]), 0) if masks is not None else 0
                if masks is None or x < c or (x - c < 64 * words and masks[t] >> (x - c) & 1):
                    at.append((pg, x % BLOCK))
        if not at:
            continue
        at = torch.tensor(at)
        for h in range(H):
            k, v = kk[at[:, 0], h, at[:, 1]], vv[at[:, 0], h, at[:, 1]]
            r = slice(h * G, (h + 1) * G)
            x = q[t, r].double()
            s = x @ k.T * scale
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - m)
            z = p.sum(1, keepdim=True)
            out[t, r], mass[t, r] = p @ v / z, p @ v.abs() / z
            lse[t, r] = (m + torch.log(z))[:, 0]
            size[t, r] = (x.abs() @ k.abs().T).amax(1) * abs(scale)
            peak[t, r] = x.abs().amax(1) * float(k.abs().sum(1).max()) * abs(scale)
            if bool(k.isnan().any() | v.isnan().any()):
                out[t, r], lse[t, r] = math.nan, math.nan
            odd = ~torch.isfinite(x).all(1)
            out[t, r][odd], lse[t, r][odd] = math.nan, math.nan
    return out, lse, mass, size, peak, err


def compact(pages, bounds, bexp, table, start, nodes, count):
    """Updates the CPU tensors in place; (lengths, whether an error bit is due)."""
    D, (B, N), err, length = bounds.shape[3], table.shape, False, []
    old = pages.clone()
    views, was = R.views(pages, D), R.views(old, D)
    for b in range(B):
        c, n = int(start[b]), int(count[b])
        length.append(c)
        if n < 0:
            continue
        keep = [int(x) for x in nodes[b][:n]] if n <= nodes.shape[1] else [-1]
        ok = c >= 0 and keep == sorted(set(keep)) and (not keep or keep[0] >= 0) and c + n <= N * BLOCK
        at = [c + x for x in keep] + list(range(c // BLOCK * BLOCK, c + n)) if ok else []
        ok = ok and all(R.page_of(table, pages.shape[0], b, x // BLOCK) >= (0, False) and
                        R.page_of(table, pages.shape[0], b, x // BLOCK)[0] >= 0 for x in at)
        if not ok:
            err = True
            continue
        length[-1] = c + n
        for j, x in enumerate(keep):
            sp, dp = int(table[b, (c + x) // BLOCK]), int(table[b, (c + j) // BLOCK])
            for v, w in zip(views, was):
                v[dp, :, (c + j) % BLOCK] = w[sp, :, (c + x) % BLOCK]
        for blk in range(c // BLOCK, -(-(c + n) // BLOCK)):
            page, m = int(table[b, blk]), min(BLOCK, c + n - blk * BLOCK)
            kk, _ = R.values(pages[page:page + 1], D)
            kk = kk[0, :, :m].nan_to_num(0.0)
            for h in range(kk.shape[0]):
                e = R.least_exp(float(kk[h].abs().max()), 63.0)
                bounds[page, h, 0] = torch.ceil(kk[h].amax(0) * 2.0 ** -e).to(torch.int8)
                bounds[page, h, 1] = torch.floor(kk[h].amin(0) * 2.0 ** -e).to(torch.int8)
                bexp[page, h] = e
    return length, err


def count_refs(table, n_pages):
    flat = table.flatten()
    return torch.bincount(flat[(flat >= 0) & (flat < n_pages)].long(), minlength=n_pages).to(torch.int32)


def fork(refs, table, parent, length):
    old, (B, N), err = table.clone(), table.shape, False
    for b in range(B):
        p, n = int(parent[b]), -(-max(int(length[b]), 0) // BLOCK)
        if p >= B:
            err = True
            continue
        for c in range(N):
            now = int(old[p, c]) if p >= 0 and c < n else -1
            if now >= len(refs):
                err, now = True, -1
            was = int(old[b, c])
            table[b, c] = max(now, -1) if max(now, -1) != was else was
            if max(now, -1) != was:
                if now >= 0:
                    refs[now] += 1
                if 0 <= was < len(refs):
                    refs[was] -= 1
    return err


def resize(pages, bounds, bexp, refs, table, start, end):
    """In place; the error bits due: (page, full)."""
    (B, N), n_pages = table.shape, len(refs)
    free, before = [i for i in range(n_pages) if int(refs[i]) == 0], refs.clone()
    page_err = full = False
    copies = []
    for b in range(B):
        if int(end[b]) < 0:
            continue
        first, last = max(int(start[b]), 0) // BLOCK, -(-int(end[b]) // BLOCK)
        page_err |= last > N
        last = min(last, N)
        for c in range(first, last):
            old = int(table[b, c])
            page_err |= old >= n_pages
            lives = 0 <= old < n_pages
            if lives and int(before[old]) <= 1:
                continue
            if not free:
                full = True
                continue
            new = free.pop(0)
            if lives:
                refs[old] -= 1
                if c == first and int(start[b]) % BLOCK > 0:
                    copies.append((new, old))
            table[b, c], refs[new] = new, 1
        for c in range(last, N):
            old = int(table[b, c])
            if 0 <= old < n_pages:
                refs[old] -= 1
            table[b, c] = min(old, -1) if old < 0 else -1
    for new, old in copies:
        pages[new], bounds[new], bexp[new] = pages[old], bounds[old], bexp[old]
    return page_err, full
