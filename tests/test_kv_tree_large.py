"""kv_attend_tree where logits are large: keys that stand for infinities among ordinary ones, up to 2^119.  What such a token's
logit does is certain: it takes all of the weight, or has none.  By both kernels (wide tables lead to the tiles).

An output may be off as in test_kv_tree.py, the logits' error being that of the ordinary tokens.
"""
import pytest
import torch

import kv_more_reference as M
import kv_reference as R
import test_kv_tree as base
from bit_routed_expert_gb300 import kv_attend_tree

pytestmark = pytest.mark.gpu

EXPONENTS = [14, 20, 24, 25, 26, 27, 28, 29, 30, 31, 40, 64, 90, 110, 119]


def attend(dev, b, pages, q, wide, scale, **kw):
    if wide:
        b = R.Batch(b.seq, b.pos, torch.cat([b.table, torch.full((len(b.table), 5000), -1, dtype=torch.int32)], 1), b.n_pages)
    seq, pos, table = b.on(dev)
    out, lse = kv_attend_tree(q.to(dev), base.on(dev, pages, pages.shape[1], q.shape[2]), seq, pos, table, scale=scale, **kw)
    return out.cpu().double(), lse.cpu().double()


def without(q, pages, b, gone, scale):
    """The definition over all tokens x <= pos but those of `gone`; and the tolerance of an output."""
    D, n = q.shape[2], max(b.pos) + 1
    masks = [(1 << n) - 1 & ~sum(1 << x for x in gone)] * len(b.pos)
    want, wl, mass, size, peak, _ = M.attend_tree(q, pages, b.seq, b.pos, b.table, [0], masks, scale, -(-n // 64))
    d = D * 2.0 ** -23 * size + 2.0 ** -19 * peak + 2.0 ** -20
    return want, wl, 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * d)[..., None] * mass + 1e-30, d


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ctx,T,x", [(200, 40, 70), (200, 40, 203), (130, 170, 127), (0, 1, 0), (640, 2, 640)])
def test_one_large_key(cuda_dev, wide, ctx, T, x):
    D = 64
    b = R.batch([ctx + T], [T], seed=2)
    pages, _, _ = R.filled(b, [ctx + T], 1, D, seed=3)
    kc, vc, ks, vs = R.views(pages, D)
    pg, at = int(b.table[0, x // 64]), x % 64
    kc[pg, 0, at], kc[pg, 0, at, 0] = 0, 0x38   # 1 in channel 0
    q = R.rows(4, T, 1, D, gain=0.5)
    q[:, 0, 0] = (torch.rand(T, generator=torch.Generator().manual_seed(1)) + 0.5).to(torch.bfloat16)
    q[1::3, 0, 0] *= -1
    sees, wins = torch.tensor(b.pos) >= x, q[:, 0, 0] > 0
    rest, rest_lse, tol, d = without(q, pages, b, [x], 1.0)
    v = R.VALUES[vc[pg, 0, at].long()] * 2.0 ** (int(vs[pg, 0, at]) - 127)
    for e in EXPONENTS:
        ks[pg, 0, at] = 127 + e
        out, lse = attend(cuda_dev, b, pages, q, wide, 1.0)
        one = sees & wins
        assert bool(((out[one, 0] - v).abs() <= (2.0 ** -8 + 2.0 ** -10) * v.abs()).all()), e
        assert bool(((lse[one, 0] - q[one, 0, 0].double() * 2.0 ** e).abs() <= 2.0 ** (e - 17) * 2).all()), e
        few = ~one & (rest_lse[:, 0] > -float("inf"))   # (a token that sees only the large key has all of its weight there)
        assert bool(((out - rest).abs() <= tol)[few].all()), e
        assert bool(((lse - rest_lse).abs() <= d + 2.0 ** -22 * rest_lse.abs())[few].all()), e


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T", [3, 150])
def test_ordinary_keys_behind_a_block_of_large_negative_logits(cuda_dev, wide, T):
    """The maximum rises from -2^e to some hundreds of either sign."""
    D, ctx = 64, 400
    b = R.batch([ctx + T], [T], seed=2)
    pages, _, _ = R.filled(b, [ctx + T], 1, D, seed=3)
    kc, _, ks, _ = R.views(pages, D)
    first = int(b.table[0, 0])
    kc[first], kc[first, :, :, 0] = 0, 0xB8   # -1
    for gain, shift in ((1.0, 0.0), (30.0, 0.0), (8.0, 60.0), (8.0, -60.0)):
        q = R.rows(4, T, 1, D, gain=gain)
        q[:, 0, 0] = 1.0
        q[:, 0, 1] = shift
        k = pages.clone()
        R.views(k, D)[0][:, :, :, 1] &= 0x7F   # (one sign: all ordinary logits of a row move by much the same)
        rest, rest_lse, tol, d = without(q, k, b, range(64), 1.0)
        for e in EXPONENTS:
            if 2.0 ** e < 100 * float(rest_lse.abs().max()):
                continue
            R.views(k, D)[2][first] = 127 + e
            out, lse = attend(cuda_dev, b, k, q, wide, 1.0)
            assert bool(((out - rest).abs() <= tol).all()), (gain, shift, e)
            assert bool(((lse - rest_lse).abs() <= d + 2.0 ** -22 * rest_lse.abs()).all()), (gain, shift, e)


@pytest.mark.parametrize("wide", [False, True])
def test_products_beyond_fp32_whose_logits_are_not(cuda_dev, wide):
    """Codes' products times the keys' scale pass 2^128; times the scale of the logits they are some tens."""
    D, T, ctx = 64, 30, 300
    b = R.batch([ctx + T], [T], seed=5)
    pages, _, _ = R.filled(b, [ctx + T], 1, D, seed=6)
    ks = R.views(pages, D)[2]
    ks[:] = 127 + 117
    q = R.rows(7, T, 1, D).to(torch.bfloat16)
    base.check(cuda_dev, b, pages, q, None, None, scale=2.0 ** -124) if not wide else None
    rest, rest_lse, tol, d = without(q, pages, b, [], 2.0 ** -124)
    out, lse = attend(cuda_dev, b, pages, q, wide, 2.0 ** -124)
    assert bool(((out - rest).abs() <= tol).all()) and bool(((lse - rest_lse).abs() <= d + 2.0 ** -22 * rest_lse.abs()).all())
