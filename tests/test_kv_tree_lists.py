"""kv_attend_tree over lists longer than the 512 tokens that its plan takes at a time, whose sequences begin and end where such a
round does, and whose contexts differ in length: every row of every output.

The definition is formed in 64 bits with PyTorch's elementary operations on the device, a sequence and kv head at a time.
Tolerances as in test_kv_tree.py.
"""
import math
import random

import pytest
import torch

import kv_more_reference as M
import kv_reference as R
from bit_routed_expert_gb300 import KvCache, kv_attend_tree, kv_attend_tree_workspace

pytestmark = pytest.mark.gpu


def filled(dev, lens, H, D, seed):
    """A cache of random codes (no NaN) and scales around 2^-6, and a table in random order."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    blocks = [-(-n // R.BLOCK) for n in lens]
    n = sum(blocks) + 3
    pages = torch.randint(0, 256, (n, H, 128 * (D + 1)), generator=g, device=dev, dtype=torch.uint8)
    for at in (slice(0, 64 * D), slice(64 * D, 128 * D)):
        c = pages[:, :, at]
        c[(c & 0x7F) == 0x7F] = 0x35
    pages[:, :, 128 * D:] = 119 + pages[:, :, 128 * D:] % 4
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), max(blocks) + 1), -1, dtype=torch.int32)
    for b, k in enumerate(blocks):
        table[b, :k] = torch.tensor([order.pop() for _ in range(k)], dtype=torch.int32)
    cache = KvCache(pages, torch.zeros((n, H, 2, D), dtype=torch.int8, device=dev), torch.zeros((n, H), dtype=torch.int8, device=dev))
    return cache, table


def definition(q, cache, table, runs, start, bits, scale):
    """(out, lse, sum p |v|, error of a logit) of all rows; runs: (sequence, first token of the list, tokens, first position)."""
    T, Hq, D = q.shape
    H = cache.pages.shape[1]
    G, dev = Hq // H, q.device
    value = R.VALUES.to(dev)
    kc, vc, ks, vs = R.views(cache.pages, D)
    out, mass = torch.zeros((2, T, Hq, D), dtype=torch.float64, device=dev)
    lse, off = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev), torch.zeros((T, Hq), dtype=torch.float64, device=dev)
    for b, t0, n, p0 in runs:
        L = p0 + n
        pg = table[b, :-(-L // R.BLOCK)].long().to(dev)
        x = torch.arange(L, device=dev)
        seen = x <= p0 + torch.arange(n, device=dev)[:, None]
        if bits is not None:
            own = torch.zeros((n, L), dtype=torch.bool, device=dev)
            own[:, start[b]:] = bits[t0:t0 + n, :L - start[b]].to(dev)
            seen &= (x < start[b]) | own
        hidden = ~seen.repeat_interleave(G, 0)
        for h in range(H):
            k = (value[kc[pg, h].long()] * 2.0 ** (ks[pg, h].double() - 127)[..., None]).reshape(-1, D)[:L]
            v = (value[vc[pg, h].long()] * 2.0 ** (vs[pg, h].double() - 127)[..., None]).reshape(-1, D)[:L]
            y = q[t0:t0 + n, h * G:(h + 1) * G].reshape(n * G, D).double()
            s = (y @ k.T * scale).masked_fill_(hidden, -math.inf)
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - m)
            z = p.sum(1, keepdim=True)
            size = (y.abs() @ k.abs().T).masked_fill_(hidden, 0.0).amax(1) * scale
            peak = y.abs().amax(1) * float(k.abs().sum(1).max()) * scale
            at = (slice(t0, t0 + n), slice(h * G, (h + 1) * G))
            out[at], mass[at] = (p @ v / z).view(n, G, D), (p @ v.abs() / z).view(n, G, D)
            lse[at] = (m + torch.log(z)).view(n, G)
            off[at] = (D * 2.0 ** -23 * size + 2.0 ** -19 * peak + 2.0 ** -20).view(n, G)
    return out, lse, mass, off


def check(dev, parts, H, G, D, drafts=False, seed=1):
    """parts: (cached tokens, new tokens) of a sequence each, or (-1, entries) for padding."""
    lens = [c + n for c, n in parts if c >= 0]
    cache, table = filled(dev, lens, H, D, seed)
    seq, pos, runs, start = [], [], [], []
    for c, n in parts:
        if c >= 0:
            runs.append((len(start), len(seq), n, c))
            start.append(c)
        seq += [len(start) - 1] * n
        pos += list(range(c, c + n)) if c >= 0 else [-1] * n
    T = len(seq)
    q = R.rows(seed + 5, T, H * G, D, gain=0.5).to(dev)
    i32 = dict(dtype=torch.int32, device=dev)
    kw, bits = {}, None
    if drafts:
        most = max(n for _, n in parts)
        g = torch.Generator().manual_seed(seed)
        masks = [m for c, n in parts for m in (M.tree(g, n) if c >= 0 else [0] * n)]
        bits = torch.tensor([[m >> j & 1 for j in range(most)] for m in masks], dtype=torch.bool)
        kw = dict(start=torch.tensor(start, **i32), mask=M.mask_tensor(masks, -(-most // 64)).to(dev))
    scale = D ** -0.5
    want, wl, mass, d = definition(q, cache, table, runs, start, bits, scale)
    err = torch.zeros(1, **i32)
    ws = torch.full((kv_attend_tree_workspace(T, H * G, H, D),), 255, dtype=torch.uint8, device=dev)
    out, lse = torch.full((T, H * G, D), math.nan, dtype=torch.bfloat16, device=dev), torch.full((T, H * G), math.nan, device=dev)
    kv_attend_tree(q, cache, torch.tensor(seq, **i32), torch.tensor(pos, **i32), table.to(dev), ws=ws, out=out, lse=lse, dev_err=err, **kw)
    assert int(err) == 0
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * d)[..., None] * mass + 1e-30
    bad = ~((out.double() - want).abs() <= tol).all(-1) | ~((lse == wl) | ((lse.double() - wl).abs() <= d + 2.0 ** -22 * wl.abs()))
    assert not bool(bad.any()), f"rows (token, head) {bad.nonzero()[:8].tolist()}, {int(bad.sum())} in all"


@pytest.mark.parametrize("parts,H,G,D", [([(0, 2048)] * 2, 4, 8, 64), ([(0, 512)] * 8, 4, 8, 128), ([(8192, 1024)] * 2, 8, 8, 64),
                                         ([(16384, 512), (0, 512), (8000, 512), (100, 512)], 4, 8, 64),
                                         ([(9000, 512), (-1, 100), (70, 3)], 4, 8, 128), ([(-1, 512), (9000, 600)], 2, 16, 64),
                                         ([(5000, 500), (300, 12), (7, 600)], 2, 3, 128)])
def test_prompts(cuda_dev, parts, H, G, D):
    check(cuda_dev, parts, H, G, D)


@pytest.mark.parametrize("seed,H,G,D,many,most", [(6, 8, 8, 64, 100, 4000), (1, 8, 8, 64, 100, 4000), (3, 4, 8, 128, 64, 8000)])
def test_drafts_behind_contexts_of_any_length(cuda_dev, seed, H, G, D, many, most):
    """Sixteen drafts each, so that every 32nd sequence begins a round."""
    rng = random.Random(seed)
    check(cuda_dev, [(rng.randint(1, most), 16) for _ in range(many)], H, G, D, drafts=True)


def test_long_contexts_before_short_ones(cuda_dev):
    check(cuda_dev, [(8192, 16)] * 32 + [(1024, 16)] * 32, 4, 8, 64, drafts=True)
