"""kv_attend_tree on the GPU against its definition in 64 bits.

An output may be off by half a BF16 step of itself (2^-8) and, relative to sum p |v|, by the FP16 rounding of the
weights (2^-11) and twice the error of a logit.  A logit is a sum of D products in FP32 whatever their order (D * 2^-23 of
scale sum |q||k|) of queries that are off by 2^-19 of their largest at most (of scale max|q| sum|k|); 2^-20 more covers the
exponential's argument and result.
"""
import math

import pytest
import torch

import kv_more_reference as M
import kv_reference as R
from bit_routed_expert_gb300 import KvCache, StepGraph, kv_attend, kv_attend_tree, kv_attend_tree_workspace
from bit_routed_expert_gb300._lib import BRE_DEVERR_PAGE

pytestmark = pytest.mark.gpu


def on(dev, pages, H, D):
    n = pages.shape[0]
    return KvCache(pages.to(dev), torch.zeros((n, H, 2, D), dtype=torch.int8, device=dev), torch.zeros((n, H), dtype=torch.int8, device=dev))


def check(dev, b, pages, q, start, masks, words=1, scale=None, **kw):
    T, Hq, D = q.shape
    H = pages.shape[1]
    scale = D ** -0.5 if scale is None else scale
    want, wl, mass, size, peak, err = M.attend_tree(q, pages, b.seq, b.pos, b.table, start, masks, scale, words)
    d = D * 2.0 ** -23 * size + 2.0 ** -19 * peak + 2.0 ** -20
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * d)[..., None] * mass + 1e-30
    e = torch.zeros(1, dtype=torch.int32, device=dev)
    args = {} if masks is None else dict(start=torch.tensor(start, dtype=torch.int32, device=dev), mask=M.mask_tensor(masks, words).to(dev))
    # what lies in the workspace and in the outputs before must not matter
    ws = torch.full((kv_attend_tree_workspace(T, Hq, H, D),), 255, dtype=torch.uint8, device=dev)
    out, lse = torch.full((T, Hq, D), math.nan, dtype=torch.bfloat16, device=dev), torch.full((T, Hq), math.nan, device=dev)
    seq, pos, table = b.on(dev)
    got = kv_attend_tree(q.to(dev), on(dev, pages, H, D), seq, pos, table, scale=scale, ws=ws, out=out, lse=lse, dev_err=e, **args, **kw)
    assert got[0] is out and got[1] is lse
    out, lse = out.cpu().double(), lse.cpu().double()
    assert int(e) == (BRE_DEVERR_PAGE if err else 0)
    nan, empty = wl.isnan(), wl == -math.inf
    assert torch.equal(lse.isnan(), nan) and torch.equal(out.isnan().any(-1), nan) and torch.equal(out.isnan().all(-1), nan)
    assert torch.equal(lse == -math.inf, empty) and float(out[empty].abs().sum()) == 0
    assert bool(((out - want).abs() <= tol)[~nan].all()), float(((out - want).abs() / tol)[~nan].max())
    off, some = (lse - wl).abs(), ~nan & ~empty
    assert bool((off <= d + 2.0 ** -22 * wl.abs())[some].all()), float((off / d)[some].max())
    return out, lse


def trees(ctx, nodes, seed=0, pad=(), spare=2):
    """Sequences with ctx[b] tokens cached and nodes[b] drafted behind them."""
    lens = [c + n for c, n in zip(ctx, nodes)]
    b = R.batch(lens, nodes, seed=seed, spare=spare)
    g = torch.Generator().manual_seed(seed + 9)
    masks = [m for n in nodes for m in M.tree(g, n)]
    for i in pad:
        b.seq.insert(i, 0), b.pos.insert(i, -1), masks.insert(i, 0)
    return b, lens, masks


HEADS = [(64, 1, 1), (128, 2, 8), (64, 2, 16), (128, 1, 5), (64, 3, 3), (128, 4, 1), (128, 1, 12)]
TREES = [([0], [1]), ([63], [1]), ([64], [1]), ([100], [28]), ([100], [29]), ([128], [64]), ([500], [7]), ([1], [130]), ([70, 0, 300, 64], [5, 9, 1, 16]),
         ([200] * 9, [3] * 9), ([1000, 3], [40, 33]), ([190], [65])]


@pytest.mark.parametrize("D,H,G", HEADS)
@pytest.mark.parametrize("ctx,nodes", TREES)
def test_trees(cuda_dev, D, H, G, ctx, nodes):
    b, lens, masks = trees(ctx, nodes, seed=len(ctx) + nodes[0], pad=(0, 2) if nodes[0] > 1 else ())
    pages, _, _ = R.filled(b, lens, H, D, seed=3)
    q = R.rows(5, len(b.seq), H * G, D, gain=1.5)
    check(cuda_dev, b, pages, q, ctx, masks, words=-(-max(nodes) // 64))


@pytest.mark.parametrize("D,H,G", HEADS)
@pytest.mark.parametrize("lens,new", [([1], [1]), ([64], [64]), ([65], [1]), ([300], [300]), ([130, 63, 64, 1], [130, 63, 64, 1]),
                                      ([500, 70], [100, 1]), ([1025], [2])])
def test_causal(cuda_dev, D, H, G, lens, new):
    b = R.batch(lens, new, pad=(1,))
    pages, _, _ = R.filled(b, lens, H, D, seed=4)
    check(cuda_dev, b, pages, R.rows(6, len(b.seq), H * G, D), None, None)


def test_long_context_is_split(cuda_dev):
    """One sequence over the whole GPU: parts of different sizes, joined."""
    D, H, G = 64, 1, 4
    for ctx, nodes in ((20000, 1), (9000, 40)):
        b, lens, masks = trees([ctx], [nodes], seed=1)
        pages, _, _ = R.filled(b, lens, H, D, seed=5)
        check(cuda_dev, b, pages, R.rows(7, nodes, H * G, D, gain=3.0), [ctx], masks)


def test_masks_of_any_kind(cuda_dev):
    """Empty rows, no own bit, bits beyond the own position and beyond the words, a context that starts inside a block,
    behind the token, below 0."""
    D, H, G, ctx = 64, 2, 2, 70
    b, lens, _ = trees([ctx], [100])
    pages, _, _ = R.filled(b, lens, H, D, seed=6)
    q = R.rows(8, 100, H * G, D)
    g = torch.Generator().manual_seed(2)
    some = [int(x) for x in torch.randint(0, 2 ** 62, (100,), generator=g)]
    for start, masks, words in (([ctx], [0] * 100, 2), ([0], [0] * 100, 2), ([0], [1 << j for j in range(100)], 2),
                                ([ctx], [2 ** 128 - 1] * 100, 2), ([ctx], [2 ** 64 - 1] * 100, 1), ([130], some, 1), ([169], some, 1),
                                ([170], some, 3), ([10 ** 6], some, 1), ([2 ** 31 - 1], some, 1), ([-5], some, 2), ([-2 ** 31], some, 1),
                                ([1], some, 1), ([63], some, 1), ([64], [x << 60 for x in some], 2)):
        check(cuda_dev, b, pages, q, start, masks, words)


def test_neighbours_of_one_tile_differ(cuda_dev):
    """A row's keys may be another's unseen ones: large keys and values that only one token sees."""
    D, H, G = 64, 1, 4
    b, lens, _ = trees([60], [32])
    pages, _, _ = R.filled(b, lens, H, D, seed=7)
    kc, vc, ks, vs = R.views(pages, D)
    for j in range(32):
        pg, at = int(b.table[0, (60 + j) // 64]), (60 + j) % 64
        ks[pg, :, at] = 127 - 8 + j // 4
        vs[pg, :, at] = 127 - 8 + j
    check(cuda_dev, b, pages, R.rows(9, 32, G, D, gain=0.1), [60], [1 << j for j in range(32)])
    check(cuda_dev, b, pages, R.rows(9, 32, G, D, gain=0.1), [0], [1 << j for j in range(32)])


@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_any_size(cuda_dev, D):
    """Keys and values from 2^-60 to 2^60 beside one another, rows of zeros, infinities stored as the largest value."""
    H, G = 1, 8
    b, lens, masks = trees([200], [9])
    for seed in range(4):
        pages, _, _ = R.filled(b, lens, H, D, seed=seed)
        kc, vc, ks, vs = R.views(pages, D)
        g = torch.Generator().manual_seed(seed)
        if seed < 2:
            vs[:] = torch.randint(127 - 60, 127 + 60, vs.shape, generator=g).to(torch.uint8)
            ks[:] = torch.randint(127 - 60, 127 - 5, ks.shape, generator=g).to(torch.uint8)
        if seed == 2:
            vs[:, :, 5], vc[:, :, 5] = 246, 0x7E
        if seed == 3:
            vs[:], kc[:, :, ::3], ks[:, :, ::3] = 63, 0, 63
        check(cuda_dev, b, pages, R.rows(9, len(b.seq), G, D), [200], masks, scale=0.05)


def test_nan_rows(cuda_dev):
    """Only rows that see a NaN key or value are NaN; so are rows whose query holds a NaN or an infinity."""
    D, H, G = 64, 1, 2
    b, lens, masks = trees([64], [20])
    pages, _, _ = R.filled(b, lens, H, D, seed=8)
    kc, vc, ks, vs = R.views(pages, D)
    for j, (c, s) in ((4, (kc, ks)), (11, (vc, vs))):
        pg, at = int(b.table[0, (64 + j) // 64]), (64 + j) % 64
        c[pg, :, at], s[pg, :, at] = 0, 255
    q = R.rows(3, 20, G, D)
    q[2, 0, 5], q[3, 1, 7], q[6, 0, 0] = math.nan, math.inf, -math.inf
    check(cuda_dev, b, pages, q, [64], masks)
    check(cuda_dev, b, pages, q, [0], [0] * 10 + [1] * 10)


def test_unwritten_slots_do_not_matter(cuda_dev):
    """Slots that no row sees hold anything at all: NaN codes, NaN scales."""
    D, H, G = 128, 1, 4
    b, lens, _ = trees([10], [60])
    pages, _, _ = R.filled(b, lens, H, D, seed=9)
    masks = [1 << j & 0x0F0F0F0F0F0F0F0F for j in range(60)]
    seen = {x for x in range(10)} | {10 + j for j in range(60) if masks[j]}
    q = R.rows(4, 60, G, D)
    for byte in (0x7F, 0xFF, 0x00):
        kc, vc, ks, vs = R.views(pages, D)
        for x in range(128):
            if x not in seen:
                pg = int(b.table[0, x // 64])
                kc[pg, :, x % 64], vc[pg, :, x % 64], ks[pg, :, x % 64], vs[pg, :, x % 64] = 0x7F, 0xFF, byte, byte
        check(cuda_dev, b, pages, q, [10], masks)


def test_holes_and_outside_the_cache(cuda_dev):
    D, H, G = 64, 2, 2
    b, lens, masks = trees([300, 100, 40], [6, 6, 6])
    pages, _, _ = R.filled(b, lens, H, D, seed=1)
    q = R.rows(2, 18, H * G, D)
    b.table[0, 1] = -1
    b.table[1, 0] = -7
    check(cuda_dev, b, pages, q, [300, 100, 40], masks)
    b.table[2, 0] = b.n_pages
    check(cuda_dev, b, pages, q, [300, 100, 40], masks)
    N = b.table.shape[1]
    for seq, p in (([-1, 0], [5, 5]), ([3, 2 ** 31 - 1], [5, 5]), ([0, 0], [64 * N, 5]), ([2, 0], [2 ** 31 - 1, 5]), ([0, 0], [64 * N - 1, 64 * N])):
        check(cuda_dev, R.Batch(seq, p, b.table, b.n_pages), pages, q[:2], None, None)


def test_sequences_in_pieces_and_out_of_order(cuda_dev):
    """A sequence's tokens strewn over the list, and the same token twice."""
    D, H, G = 64, 1, 4
    b, lens, masks = trees([100, 30], [8, 8])
    pages, _, _ = R.filled(b, lens, H, D, seed=2)
    g = torch.Generator().manual_seed(4)
    order = torch.randperm(16, generator=g).tolist() + [3, 3, 12]
    n = R.Batch([b.seq[i] for i in order], [b.pos[i] for i in order], b.table, b.n_pages)
    check(cuda_dev, n, pages, R.rows(5, 19, G, D), [100, 30], [masks[i] for i in order])


def test_slices_of_a_projection_and_no_lse(cuda_dev):
    D, H, G = 128, 2, 2
    b, lens, masks = trees([90], [7])
    pages, _, _ = R.filled(b, lens, H, D)
    qkv = R.rows(5, 7, H * (G + 2), D)
    wide = qkv.to(cuda_dev)
    seq, pos, table = b.on(cuda_dev)
    kw = dict(start=torch.tensor([90], dtype=torch.int32, device=cuda_dev), mask=M.mask_tensor(masks, 1).to(cuda_dev))
    c = on(cuda_dev, pages, H, D)
    one, _ = kv_attend_tree(wide[:, :H * G], c, seq, pos, table, **kw)
    two, _ = kv_attend_tree(wide[:, :H * G].contiguous(), c, seq, pos, table, **kw)
    assert torch.equal(one, two)


def test_agrees_with_attention_over_all_blocks(cuda_dev):
    """kv_attend with every block listed answers the same question."""
    D, H, G, n = 128, 2, 8, 700
    b = R.batch([n], [3])
    pages, _, _ = R.filled(b, [n], H, D)
    q = R.rows(5, 3, H * G, D).to(cuda_dev)
    c = on(cuda_dev, pages, H, D)
    seq, pos, table = b.on(cuda_dev)
    ids = torch.arange(11, dtype=torch.int32, device=cuda_dev).expand(3, H, 11).contiguous()
    one, l1 = kv_attend(q, c, seq, pos, table, ids)
    two, l2 = kv_attend_tree(q, c, seq, pos, table)
    assert float((one.float() - two.float()).abs().max()) <= 2 * 2.0 ** -8 * float(one.float().abs().max())
    assert float((l1 - l2).abs().max()) <= 2.0 ** -18 * float(l1.abs().max())


def test_the_same_bits_every_time_and_on_other_streams(cuda_dev):
    D, H, G = 128, 4, 8
    b, lens, masks = trees([3000, 700, 64], [16, 5, 1])
    pages, _, _ = R.filled(b, lens, H, D)
    q = R.rows(5, 22, H * G, D).to(cuda_dev)
    c = on(cuda_dev, pages, H, D)
    seq, pos, table = b.on(cuda_dev)
    kw = dict(start=torch.tensor([3000, 700, 64], dtype=torch.int32, device=cuda_dev), mask=M.mask_tensor(masks, 1).to(cuda_dev))
    want, wl = kv_attend_tree(q, c, seq, pos, table, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(30):
        out, lse = kv_attend_tree(q, c, seq, pos, table, stream=side if i % 3 == 2 else None, **kw)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    g = StepGraph(lambda: kv_attend_tree(q, c, seq, pos, table, out=out, lse=lse, **kw))
    for _ in range(3):
        out.zero_(), lse.zero_()
        g.replay()
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_no_tokens(cuda_dev):
    D, H = 64, 2
    b, lens, _ = trees([10], [1])
    pages, _, _ = R.filled(b, lens, H, D)
    seq, pos, table = R.Batch([], [], b.table, b.n_pages).on(cuda_dev)
    out, lse = kv_attend_tree(torch.empty((0, 4, D), dtype=torch.bfloat16, device=cuda_dev), on(cuda_dev, pages, H, D), seq, pos, table)
    assert out.shape == (0, 4, D) and lse.shape == (0, 4)
