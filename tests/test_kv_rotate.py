"""kv_rotate on the GPU against its definition in 64 bits.

An output is off by half a BF16 step of itself (2^-8, torch.finfo(bfloat16).eps / 2) and by what FP32 costs before that,
relative to gain (|a| + |b|): the angle's 2^-25 of half a turn and its cut to 2^-31 of it (2^-23.3), cosine and sine to two
of their last places (2^-23), the gain and the products (3 * 2^-24): less than 2^-21 together.
"""
import math

import pytest
import torch

import kv_more_reference as M
import kv_reference as R
from bit_routed_expert_gb300 import StepGraph, kv_rotate, rope_turns

pytestmark = pytest.mark.gpu


def check(dev, T, Hq, Hk, D, P, offset, inter, backward, pos=None, gain=1.0, seed=0, x=None, in_place=False):
    turns, _ = rope_turns(2 * P)
    g = torch.Generator().manual_seed(seed)
    if pos is None:
        pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, dtype=torch.int32)
        pos[torch.randperm(T, generator=g)[:T // 5]] = -1
    qkv = R.rows(seed + 1, T, Hq + 2 * Hk, D) if x is None else x   # queries, keys and values side by side
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    on = qkv.to(dev)
    dq, dk = on[:, :Hq], on[:, Hq:Hq + Hk]
    out = dict(q_out=dq, k_out=dk) if in_place else {}
    got = kv_rotate(dq, dk if Hk else None, pos.to(dev), turns.to(dev), gain=gain, offset=offset, interleaved=inter, backward=backward,
                    **(out if Hk else {n: out[n] for n in out if n == "q_out"}))
    if in_place:
        assert got[0] is dq and torch.equal(on[:, Hq + Hk:].cpu(), qkv[:, Hq + Hk:])
    else:
        assert torch.equal(on.cpu().view(torch.int16), qkv.view(torch.int16))
    g32 = float(torch.tensor(gain, dtype=torch.float32))
    for y, z in ((q, got[0]), (k, got[1])):
        if z is None:
            assert Hk == 0
            continue
        want, size = M.rotate(y, pos, [int(t) % 2 ** 64 for t in turns], g32, offset, inter, backward)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -21 * size + 2.0 ** -133   # BF16's least step is 2^-133
        off = (z.cpu().double() - want).abs()
        assert bool((off <= tol).all()), float((off / tol).max())
        still = torch.ones(D, dtype=torch.bool)
        still[offset:offset + 2 * P] = False
        live = pos >= 0
        assert torch.equal(z.cpu()[live][..., still], y[live][..., still])
    return got


SHAPES = [(64, 32, 0), (64, 24, 16), (128, 64, 0), (128, 32, 0), (128, 32, 64), (80, 20, 0), (96, 1, 5), (64, 31, 1), (64, 3, 50),
          (256, 128, 0), (256, 1, 254), (192, 36, 24), (8, 4, 0), (128, 10, 4), (64, 12, 8)]


@pytest.mark.parametrize("D,P,offset", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_layouts(cuda_dev, D, P, offset, inter, backward):
    check(cuda_dev, 23, 6, 2, D, P, offset, inter, backward, gain=1.25, seed=D + P)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 0), (1, 32, 4), (1, 64, 8), (2, 7, 3), (700, 5, 1), (1300, 12, 2), (3001, 2, 2), (610, 33, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_token_and_head_counts(cuda_dev, T, Hq, Hk, in_place):
    check(cuda_dev, T, Hq, Hk, 64, 32, 0, False, False, seed=T, in_place=in_place)
    check(cuda_dev, T, Hq, Hk, 64, 12, 8, True, False, seed=T, in_place=in_place)


def test_positions_at_the_ends(cuda_dev):
    pos = torch.tensor([0, 1, 2 ** 31 - 1, 2 ** 30, -1, -2 ** 31, 65535, 65536], dtype=torch.int32)
    for inter in (False, True):
        check(cuda_dev, 8, 2, 1, 64, 32, 0, inter, False, pos=pos)


def test_no_tokens(cuda_dev):
    q, k = kv_rotate(torch.empty((0, 4, 64), dtype=torch.bfloat16, device=cuda_dev), torch.empty((0, 2, 64), dtype=torch.bfloat16, device=cuda_dev),
                     torch.empty(0, dtype=torch.int32, device=cuda_dev), torch.zeros(8, dtype=torch.int64, device=cuda_dev))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


def test_infinities_and_nan_stay_in_their_pairs(cuda_dev):
    x = R.rows(3, 4, 3, 64)
    x[0, 0, 3], x[1, 1, 40], x[2, 0, 60] = math.inf, math.nan, -math.inf
    turns, _ = rope_turns(48)
    pos = torch.tensor([5, 6, 7, -1], dtype=torch.int32)
    q, _ = kv_rotate(x.to(cuda_dev), None, pos.to(cuda_dev), turns.to(cuda_dev))
    bad = ~torch.isfinite(q.cpu().float())
    want = torch.zeros_like(bad)
    want[0, 0, [3, 27]] = want[1, 1, [16, 40]] = want[2, 0, 60] = True
    assert torch.equal(bad, want) and float(q[3].abs().max()) == 0


def test_bases_and_strides_that_are_not_aligned(cuda_dev):
    """Rows that start on 2, 4 and 8 bytes: narrower pieces, the same numbers."""
    turns, _ = rope_turns(64)
    pos = torch.arange(9, dtype=torch.int32)
    x = R.rows(8, 9, 4, 64)
    want, _ = kv_rotate(x.to(cuda_dev), None, pos.to(cuda_dev), turns.to(cuda_dev))
    for shift, pad in ((1, 0), (2, 0), (4, 0), (0, 1), (0, 2), (0, 6), (3, 5)):
        wide = torch.zeros(9 * (256 + pad) + shift, dtype=torch.bfloat16, device=cuda_dev)
        v = wide[shift:].view(9, 256 + pad)[:, :256].view(9, 4, 64) if pad == 0 else \
            wide[shift:].view(9, 256 + pad)[:, :256].unflatten(1, (4, 64))
        v.copy_(x)
        out, _ = kv_rotate(v, None, pos.to(cuda_dev), turns.to(cuda_dev), q_out=v)
        assert torch.equal(out, want)


def test_gradient_of_a_sum_by_differences(cuda_dev):
    """backward(w) is the gradient of sum(w * rotate(x)): the map is linear, so <w, rotate(x)> = <backward(w), x> up to the
    rounding of both sides' BF16 outputs (2^-8 of each term's size)."""
    turns, gain = rope_turns(48, scaling="ramp", factor=8.0, length=2048.0)
    pos = torch.arange(1000, 1064, dtype=torch.int32).to(cuda_dev)
    x, w = R.rows(1, 64, 4, 64).to(cuda_dev), R.rows(2, 64, 4, 64).to(cuda_dev)
    for inter in (False, True):
        kw = dict(gain=gain, offset=16, interleaved=inter)
        y, _ = kv_rotate(x, None, pos, turns.to(cuda_dev), **kw)
        v, _ = kv_rotate(w, None, pos, turns.to(cuda_dev), backward=True, **kw)
        one, two = (w.double() * y.double()), (v.double() * x.double())
        assert abs(float(one.sum() - two.sum())) <= 2.0 ** -8 * float(one.abs().sum() + two.abs().sum())
        # rounding errors of both signs: their sum over 16,384 terms is far below the bound above
        assert abs(float(one.sum() - two.sum())) <= 2.0 ** -8 * 8 * float((one ** 2).sum() + (two ** 2).sum()) ** 0.5


def test_streams_and_graphs(cuda_dev):
    turns = rope_turns(64, device=cuda_dev)[0]
    x, pos = R.rows(1, 40, 6, 64).to(cuda_dev), torch.arange(40, dtype=torch.int32, device=cuda_dev)
    want, _ = kv_rotate(x, None, pos, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = kv_rotate(x, None, pos, turns, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    g = StepGraph(lambda: kv_rotate(x, None, pos, turns, q_out=out))
    pos += 1
    g.replay()
    assert torch.equal(out, kv_rotate(x, None, pos, turns)[0])
