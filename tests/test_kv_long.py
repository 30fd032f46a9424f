"""kv_append and kv_read over so many tokens that a CTA goes through many of them: whole chunks of 64 tokens with several
runs each, and a capped grid.  The calls over few tokens are compared with the definitions in test_kv_cache.py; here the
same tokens in one call and in many must give the same bits."""
import math

import pytest
import torch

import kv_reference as R
from bit_routed_expert_gb300 import kv_append, kv_read
from test_kv_cache import blank, err_word, on

pytestmark = pytest.mark.gpu


def ragged(total, seqs, seed, padding):
    """About `total` tokens of `seqs` sequences: chunks of any length at any position, padding entries among them."""
    r = torch.Generator().manual_seed(seed)
    new = (torch.rand(seqs, generator=r) * 2 * total / seqs).long().clamp_min(1).tolist()
    lens = [n + int(torch.randint(0, 200, (1,), generator=r)) for n in new]
    T = sum(new)
    pad = sorted(torch.randint(0, T, (padding,), generator=r).tolist() + [0, 0, T // 2, T // 2 + 1, T // 2 + 2])
    return R.batch(lens, new, seed=seed, pad=pad)


def special(x, seed):
    """NaN, infinite, zero and tiny rows here and there."""
    T, H, D = x.shape
    g = torch.Generator().manual_seed(seed)
    at = torch.randint(0, T * H, (64,), generator=g)
    flat = x.view(T * H, D)
    flat[at[:16], 3] = math.nan
    flat[at[16:32], 5] = math.inf
    flat[at[32:48]] = 0.0
    flat[at[48:]] *= 2.0 ** -60
    return x


# T * H in 152 * 4 * (2 .. 64 and more): chunks of 2, 16, 64 and 64 tokens
@pytest.mark.parametrize("D,H,total,seqs,padding", [(128, 1, 2000, 3, 9), (64, 3, 5000, 40, 50), (64, 8, 6400, 37, 60),
                                                    (128, 4, 10500, 5, 300), (64, 8, 5200, 1500, 100)])
def test_append_in_one_call_and_in_many(cuda_dev, D, H, total, seqs, padding):
    b = ragged(total, seqs, seed=total + seqs, padding=padding)
    T = len(b.seq)
    k, v = special(R.rows(1, T, H, D), 3), special(R.rows(2, T, H, D), 4)
    old = blank(b, H, D)
    one, many = on(cuda_dev, *old), on(cuda_dev, *old)
    # blocks begun before the call have bounds of their own
    for c in (one, many):
        c.bounds.clamp_(-63, 63)
    seq, pos, table = b.on(cuda_dev)
    k, v = k.to(cuda_dev), v.to(cuda_dev)
    e = err_word(cuda_dev)
    kv_append(one, k, v, seq, pos, table, dev_err=e)
    step = max(1, 600 // H)     # one token a CTA
    for i in range(0, T, step):
        kv_append(many, k[i:i + step], v[i:i + step], seq[i:i + step], pos[i:i + step], table, dev_err=e)
    assert int(e) == 0
    assert torch.equal(one.pages, many.pages)
    assert torch.equal(one.bound_exp, many.bound_exp)
    assert torch.equal(one.bounds, many.bounds)
    assert not torch.equal(one.pages.cpu(), old[0])
    # and what was stored is what is read: each row within half a step of E4M3 of its own scale
    ko, vo = kv_read(one, seq, pos, table)
    for got, x in ((ko, k), (vo, v)):
        got, x = got.cpu().double(), x.cpu().double()
        nan = x.isnan().any(-1, keepdim=True)
        pad = torch.tensor(b.pos)[:, None, None] < 0
        x = torch.where(pad, 0.0, x.clamp(-R.MAX, R.MAX))
        e8 = torch.ceil(torch.log2(x.nan_to_num(0.0).abs().amax(-1, keepdim=True) / 448.0)).clamp_min(-64)
        tol = torch.maximum(2.0 ** -4 * x.abs(), torch.exp2(e8 - 10))
        ok = torch.where(nan & ~pad, got.isnan(), (got - x).abs() <= tol)
        assert bool(ok.all())


@pytest.mark.parametrize("D,H,T", [(128, 4, 40007), (64, 8, 40007), (128, 4, 90001)])
def test_read_more_rows_than_the_grid_has(cuda_dev, D, H, T):
    lens = [700, 65]
    b = R.batch(lens, lens)
    pages, bounds, bexp = R.filled(b, lens, H, D)
    R.views(pages, D)[2][int(b.table[0, 1]), 0, 7] = 255     # a NaN row
    R.views(pages, D)[0][int(b.table[0, 1]), 0, 7] = 0
    c = on(cuda_dev, pages, bounds, bexp)
    g = torch.Generator().manual_seed(T)
    at = torch.randint(0, len(b.seq), (T,), generator=g)
    seq, pos = torch.tensor(b.seq)[at], torch.tensor(b.pos)[at]
    pos[torch.randint(0, T, (50,), generator=g)] = -1
    e = err_word(cuda_dev)
    ko, vo = kv_read(c, seq.int().to(cuda_dev), pos.int().to(cuda_dev), b.table.to(cuda_dev), dev_err=e)
    kk, vv = (x.float().to(cuda_dev) for x in R.values(pages, D))
    page = b.table[seq, pos.clamp_min(0) // 64].long().to(cuda_dev)
    slot, real = (pos.clamp_min(0) % 64).to(cuda_dev), (pos >= 0).to(cuda_dev)[:, None, None]
    assert int(e) == 0
    for got, x in ((ko, kk), (vo, vv)):
        want = torch.where(real, x[page, :, slot], 0.0).to(torch.bfloat16)
        assert torch.equal(got.nan_to_num(nan=7e30), want.nan_to_num(nan=7e30))
