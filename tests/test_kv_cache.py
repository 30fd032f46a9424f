"""The key/value cache calls on the GPU against their definitions in 64 bits (kv_reference.py).

Stored bytes, bounds, block lists and scores are equal bit for bit.  Attention: an output may be
off by half a BF16 step of itself (2^-8, torch.finfo(bfloat16).eps / 2), plus, relative to
sum p |v|, the FP16 rounding of the weights (2^-11) and twice the error of a logit.  A logit is a
sum of D products in FP32, whatever their order: off by at most D * 2^-23 of scale * sum |q||k|;
2^-20 more covers the exponential's argument and result.
"""
import math

import pytest
import torch

import kv_reference as R
from bit_routed_expert_gb300 import (BreError, KvCache, StepGraph, _lib, kv_append, kv_attend, kv_attend_workspace, kv_read,
                                     kv_select, kv_select_workspace)
from bit_routed_expert_gb300._lib import BRE_DEVERR_PAGE

pytestmark = pytest.mark.gpu


def err_word(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def on(dev, pages, bounds, bexp):
    return KvCache(pages.to(dev), bounds.to(dev), bexp.to(dev))


def same_cache(c, pages, bounds, bexp):
    assert torch.equal(c.pages.cpu(), pages)
    assert torch.equal(c.bounds.cpu(), bounds)
    assert torch.equal(c.bound_exp.cpu(), bexp)


def copies_for_tiles(T, H, G):
    """How often a call's tokens have to be repeated for select and attend to go by tiles of many tokens, not token
    by token (their launchers' rules); every copy then lies differently in its tiles."""
    return -(-max(2048, 16384 // G + 1) // (T * H))


def repeated(b, copies):
    return R.Batch(b.seq * copies, b.pos * copies, b.table, b.n_pages)


def blank(b, H, D):
    g = torch.Generator().manual_seed(5)   # what was in memory before must not matter
    return (torch.randint(0, 256, (b.n_pages, H, 128 * (D + 1)), generator=g, dtype=torch.uint8),
            torch.randint(-128, 128, (b.n_pages, H, 2, D), generator=g).to(torch.int8),
            torch.randint(-64, 100, (b.n_pages, H), generator=g).to(torch.int8))


# ------------------------------------------------------------------ append and read

LENS = [([1], [1]), ([64], [64]), ([65], [1]), ([130, 63, 64, 1], [130, 63, 64, 1]), ([200, 77, 300], [5, 77, 131]),
        ([70] * 9, [1] * 9), ([129, 128, 127], [2, 1, 3])]


@pytest.mark.parametrize("D,H", [(64, 1), (128, 2), (64, 3)])
@pytest.mark.parametrize("lens,new", LENS)
def test_append_and_read(cuda_dev, D, H, lens, new):
    b = R.batch(lens, new, pad=(0, 2))
    pages, bounds, bexp = R.filled(b, lens, H, D)
    T = len(b.seq)
    k, v = R.rows(1, T, H, D, gain=2.0), R.rows(2, T, H, D, gain=0.01)
    c = on(cuda_dev, pages, bounds, bexp)
    seq, pos, table = b.on(cuda_dev)
    e = err_word(cuda_dev)
    kv_append(c, k.to(cuda_dev), v.to(cuda_dev), seq, pos, table, dev_err=e)
    ko, vo = kv_read(c, seq, pos, table, dev_err=e)
    assert not R.append(pages, bounds, bexp, k, v, b.seq, b.pos, b.table)
    same_cache(c, pages, bounds, bexp)
    assert int(e) == 0
    kk, vv = R.values(pages, D)
    for t, (s, p) in enumerate(zip(b.seq, b.pos)):
        want = [x[int(b.table[s, p // 64]), :, p % 64] if p >= 0 else torch.zeros(H, D) for x in (kk, vv)]
        assert torch.equal(ko[t].cpu().double(), want[0].double()) and torch.equal(vo[t].cpu().double(), want[1].double())


def test_append_into_fresh_memory_and_in_steps(cuda_dev):
    """Nothing is read of a page before it is written, and any cut of the tokens into calls gives the same."""
    D, H, lens = 128, 2, [150, 67]
    b = R.batch(lens, lens)
    k, v = R.rows(3, 217, H, D), R.rows(4, 217, H, D)
    pages, bounds, bexp = blank(b, H, D)
    c = on(cuda_dev, pages, bounds, bexp)
    for cut in ([0, 217], [0, 1, 3, 64, 100, 149, 150, 151, 216, 217]):
        for i, j in zip(cut, cut[1:]):
            n = R.Batch(b.seq[i:j], b.pos[i:j], b.table, b.n_pages).on(cuda_dev)
            kv_append(c, k[i:j].to(cuda_dev), v[i:j].to(cuda_dev), *n)
        if len(cut) == 2:
            R.append(pages, bounds, bexp, k, v, b.seq, b.pos, b.table)
        same_cache(c, pages, bounds, bexp)


def special_rows(D):
    x = R.rows(7, 12, 1, D)
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 1e-38
    x[3] *= 2.0 ** -60
    x[4, 0, 5] = math.inf
    x[5, 0, 6] = -math.inf
    x[6, 0, 7] = math.nan
    x[7] = math.nan
    x[8, 0, 0] = 3.3e38
    x[9] = 448.0
    x[10, 0, 3] = 450.0
    x[11] = torch.finfo(torch.bfloat16).max
    return x


@pytest.mark.parametrize("D", [64, 128])
def test_append_special_values(cuda_dev, D):
    """Each in a page of its own, so that a block's bounds meet it too."""
    x = special_rows(D)
    b = R.batch([1] * 12, [1] * 12)
    pages, bounds, bexp = blank(b, 1, D)
    c = on(cuda_dev, pages, bounds, bexp)
    seq, pos, table = b.on(cuda_dev)
    kv_append(c, x.to(cuda_dev), x.flip(0).contiguous().to(cuda_dev), seq, pos, table)
    R.append(pages, bounds, bexp, x, x.flip(0), b.seq, b.pos, b.table)
    same_cache(c, pages, bounds, bexp)
    ko, _ = kv_read(c, seq, pos, table)
    kk, _ = R.values(pages, D)
    want = torch.stack([kk[int(b.table[s, 0]), :, 0] for s in b.seq])
    assert torch.equal(ko.cpu().double().nan_to_num(nan=7e300), want.nan_to_num(nan=7e300))


def test_append_slices_of_a_projection(cuda_dev):
    D, H, T = 64, 3, 70
    b = R.batch([T], [T])
    qkv = R.rows(5, T, 4 * H, D)
    pages, bounds, bexp = blank(b, H, D)
    c = on(cuda_dev, pages, bounds, bexp)
    x = qkv.to(cuda_dev)
    kv_append(c, x[:, H:2 * H], x[:, 3 * H:], *b.on(cuda_dev))
    R.append(pages, bounds, bexp, qkv[:, H:2 * H], qkv[:, 3 * H:], b.seq, b.pos, b.table)
    same_cache(c, pages, bounds, bexp)


def test_rewritten_positions_only_widen_the_bounds(cuda_dev):
    """A verify batch that was rejected: positions 5.. are written again."""
    D, H = 64, 1
    b = R.batch([20], [20])
    pages, bounds, bexp = blank(b, H, D)
    c = on(cuda_dev, pages, bounds, bexp)
    for a, z, gain in ((0, 20, 1.0), (5, 12, 0.5), (12, 13, 8.0)):
        k = R.rows(a, z - a, H, D, gain=gain)
        n = R.Batch(b.seq[a:z], b.pos[a:z], b.table, b.n_pages)
        kv_append(c, k.to(cuda_dev), k.to(cuda_dev), *n.on(cuda_dev))
        R.append(pages, bounds, bexp, k, k, n.seq, n.pos, n.table)
    same_cache(c, pages, bounds, bexp)


def test_append_and_read_outside_the_cache(cuda_dev):
    """A sequence, block or page out of range, or no page: the bit, and nothing else is touched."""
    D, H = 64, 2
    b = R.batch([100, 100], [3, 3])
    b.table[1, 1] = -1
    pages, bounds, bexp = R.filled(b, [100, 100], H, D)
    for seq, pos in (([2], [5]), ([-1], [5]), ([0], [64 * b.table.shape[1]]), ([1], [70]), ([0, 0], [2 ** 31 - 1, 3])):
        c = on(cuda_dev, pages, bounds, bexp)
        n = R.Batch(seq, pos, b.table, b.n_pages)
        k = R.rows(1, len(seq), H, D)
        want = [x.clone() for x in (pages, bounds, bexp)]
        assert R.append(*want, k, k, seq, pos, b.table)
        e = err_word(cuda_dev)
        kv_append(c, k.to(cuda_dev), k.to(cuda_dev), *n.on(cuda_dev), dev_err=e)
        same_cache(c, *want)
        assert int(e) == BRE_DEVERR_PAGE
        e.zero_()
        ko, vo = kv_read(c, *n.on(cuda_dev), dev_err=e)
        assert int(e) == BRE_DEVERR_PAGE and float(ko[0].abs().max()) == 0 and float(vo[0].abs().max()) == 0
    table = b.table.clone()
    table[0, 0] = b.n_pages
    c = on(cuda_dev, pages, bounds, bexp)
    e = err_word(cuda_dev)
    k = R.rows(1, 1, H, D).to(cuda_dev)
    kv_append(c, k, k, *R.Batch([0], [3], table, 0).on(cuda_dev), dev_err=e)
    same_cache(c, pages, bounds, bexp)
    assert int(e) == BRE_DEVERR_PAGE


# ------------------------------------------------------------------ select

def check_select(dev, b, cache, q, k, sink, local):
    """Token by token, and in tiles."""
    pages, bounds, bexp = cache
    c = on(dev, pages, bounds, bexp)
    want, ws, err = R.select(q, bounds, bexp, b.seq, b.pos, b.table, k, sink, local)
    T, H = len(b.seq), bounds.shape[1]
    for copies in (1, copies_for_tiles(T, H, q.shape[1] // H)):
        e = err_word(dev)
        ids, scores = kv_select(q.to(dev).repeat(copies, 1, 1), c, *repeated(b, copies).on(dev), k, n_sink=sink,
                                n_local=local, dev_err=e)
        for i, s in zip(ids.cpu().split(T), scores.cpu().split(T)):
            assert torch.equal(i, want)
            assert torch.equal(s, ws.float())
        assert int(e) == (BRE_DEVERR_PAGE if err else 0)


SELECT = [([1], [1], 1, 4, 1, 1), ([64], [2], 2, 1, 0, 0), ([4000], [1], 4, 8, 1, 2), ([4000], [40], 4, 8, 1, 2),
          ([2000, 90, 64, 700], [1, 1, 1, 1], 8, 5, 1, 1), ([2000, 90, 64, 700], [33, 17, 3, 60], 8, 5, 2, 1),
          ([700], [700], 3, 4, 0, 1), ([3000], [20], 16, 32, 0, 0), ([3000, 1], [1, 1], 16, 32, 3, 29),
          ([100, 200], [100, 200], 5, 16, 1, 1), ([6000] * 3, [5] * 3, 2, 47, 1, 2)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,new,G,k,sink,local", SELECT)
def test_select(cuda_dev, D, lens, new, G, k, sink, local):
    H = 2
    b = R.batch(lens, new, pad=(1,))
    q = R.rows(11, len(b.seq), H * G, D)
    check_select(cuda_dev, b, R.filled(b, lens, H, D), q, k, sink, local)


@pytest.mark.parametrize("T", [1, 40])
def test_select_ties_take_the_lowest_block(cuda_dev, T):
    """Zero queries score every block 0; blocks that share a page score the same."""
    D, H, G = 64, 1, 4
    lens = [3000]
    b = R.batch(lens, [T])
    cache = R.filled(b, lens, H, D)
    check_select(cuda_dev, b, cache, torch.zeros(T, G, D, dtype=torch.bfloat16), 7, 0, 1)
    b.table[0] = b.table[0, torch.arange(b.table.shape[1]) % 3]
    check_select(cuda_dev, b, cache, R.rows(3, T, G, D), 20, 1, 1)


@pytest.mark.parametrize("T", [1, 40])
def test_select_long_contexts(cuda_dev, T):
    """Up to 20,000 blocks, in shared pages (a block's score depends on its page alone)."""
    D, H, G = 64, 1, 2
    b = R.batch([2560], [1])
    cache = R.filled(b, [2560], H, D)
    g = torch.Generator().manual_seed(1)
    for blocks in (2047, 2048, 2049, 5000, 20000):
        n = R.Batch([0] * T, list(range(64 * blocks - T, 64 * blocks)),
                    torch.randint(0, b.n_pages, (1, blocks), generator=g).to(torch.int32), b.n_pages)
        check_select(cuda_dev, n, cache, R.rows(blocks, T, G, D)[:, :], 16, 1, 2)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("k", [33, 150, 200, 256])
def test_select_many(cuda_dev, T, k):
    """Lists longer than a warp, than a prefill tile's shared memory, and than the blocks there are."""
    D, H, G = 64, 1, 2
    b = R.batch([2560], [1])
    cache = R.filled(b, [2560], H, D)
    g = torch.Generator().manual_seed(k)
    for blocks in (100, 700, 1300):
        n = R.Batch([0] * T, list(range(64 * blocks - T, 64 * blocks)),
                    torch.randint(0, b.n_pages, (1, blocks), generator=g).to(torch.int32), b.n_pages)
        check_select(cuda_dev, n, cache, R.rows(blocks, T, G, D), k, 3, 20)


def test_select_longest_table(cuda_dev):
    """131,072 blocks: the whole of eight CTAs' shared memory."""
    D, H, G, blocks = 64, 1, 1, 131072
    b = R.batch([2560], [1])
    cache = R.filled(b, [2560], H, D)
    g = torch.Generator().manual_seed(1)
    n = R.Batch([0], [64 * blocks - 1], torch.randint(0, b.n_pages, (1, blocks), generator=g).to(torch.int32), b.n_pages)
    for k in (16, 256):
        check_select(cuda_dev, n, cache, R.rows(5, 1, G, D), k, 1, 2)


@pytest.mark.parametrize("T", [1, 40])
def test_select_blocks_without_pages(cuda_dev, T):
    D, H, G = 128, 2, 2
    lens = [1500, 900]
    b = R.batch(lens, [T, T])
    cache = R.filled(b, lens, H, D)
    q = R.rows(2, 2 * T, H * G, D)
    b.table[0, 2:9] = -1
    b.table[1, :] = -1
    check_select(cuda_dev, b, cache, q, 12, 4, 2)
    b.table[1, 3] = b.n_pages          # outside: the bit, and not taken
    check_select(cuda_dev, b, cache, q, 12, 4, 2)


@pytest.mark.parametrize("T", [2, 40])
def test_select_sequences_and_positions_out_of_range(cuda_dev, T):
    D, H, G = 64, 1, 1
    lens = [500]
    b = R.batch(lens, [T])
    cache = R.filled(b, lens, H, D)
    b.seq[0], b.pos[1] = 1, 64 * 30
    check_select(cuda_dev, b, cache, R.rows(2, T, H * G, D), 4, 1, 1)


@pytest.mark.parametrize("T", [1, 40])
def test_select_special_queries(cuda_dev, T):
    D, H, G = 64, 1, 4
    lens = [1000]
    b = R.batch(lens, [T])
    q = R.rows(2, T, G, D)
    q[0, 0, 3], q[0, 1, 4], q[0, 2] = math.nan, 1e-30, 0.0
    q[T - 1, 3] = math.nan
    check_select(cuda_dev, b, R.filled(b, lens, H, D), q, 6, 1, 1)
    q[0, 2, 9] = -math.inf
    check_select(cuda_dev, b, R.filled(b, lens, H, D), q, 6, 1, 1)


def test_select_query_slices_and_one_workspace(cuda_dev):
    """One workspace, zeroed once, for calls of different sizes; queries as slices of wider rows."""
    D, H, G = 64, 2, 4
    ws = torch.zeros(max(kv_select_workspace(T, H * G, H, D, 4, 64, 16) for T in (1, 4, 400)), dtype=torch.uint8,
                     device=cuda_dev)
    for lens, new in (([4000], [1]), ([4000, 1000, 30, 2000], [1] * 4), ([3000], [400]), ([4000], [1])):
        b = R.batch(lens, new, blocks=64)
        cache = R.filled(b, lens, H, D)
        wide = R.rows(4, len(b.seq), H * G + 3, D)
        c = on(cuda_dev, *cache)
        ids, _ = kv_select(wide.to(cuda_dev)[:, 3:], c, *b.on(cuda_dev), 9, ws=ws)
        assert torch.equal(ids.cpu(), R.select(wide[:, 3:], *cache[1:], b.seq, b.pos, b.table, 9, 1, 2)[0])


# ------------------------------------------------------------------ attend

def check_attend(dev, b, pages, q, ids, scale=None):
    """Token by token, and in tiles."""
    T, H = len(b.seq), pages.shape[1]
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    c = on(dev, pages, torch.zeros((b.n_pages, H, 2, D), dtype=torch.int8),
           torch.zeros((b.n_pages, H), dtype=torch.int8))
    want, wl, mass, size, err = R.attend(q, pages, b.seq, b.pos, b.table, ids, scale)
    d = (D * 2.0 ** -23 * size + 2.0 ** -20)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * d)[..., None] * mass + 1e-30
    empty = wl == -math.inf
    for copies in (1, copies_for_tiles(T, H, q.shape[1] // H)):
        e = err_word(dev)
        outs, lses = kv_attend(q.to(dev).repeat(copies, 1, 1), c, *repeated(b, copies).on(dev),
                               ids.to(dev).repeat(copies, 1, 1), scale=scale, dev_err=e)
        assert int(e) == (BRE_DEVERR_PAGE if err else 0)
        for out, lse in zip(outs.cpu().double().split(T), lses.cpu().double().split(T)):
            assert bool((out - want).abs().le(tol).all()), float(((out - want).abs() / tol).max())
            assert torch.equal(lse == -math.inf, empty) and float(out[empty].abs().sum()) == 0
            off = (lse - wl)[~empty].abs()
            assert bool((off <= d[~empty] + 2.0 ** -22 * wl[~empty].abs()).all()), float(off.max())


def some_ids(b, H, k, seed=0):
    """Ascending lists of visible blocks, the own block always among them; neighbours mostly alike."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.full((len(b.seq), H, k), -1, dtype=torch.int32)
    base = {}
    for t, (s, p) in enumerate(zip(b.seq, b.pos)):
        if p < 0:
            continue
        n = p // 64 + 1
        for h in range(H):
            if (s, h) not in base or t % 5 == 0:
                base[s, h] = torch.randperm(n, generator=g).tolist()
            take = sorted(set([n - 1] + [x for x in base[s, h] if x < n][:k - 1]))
            ids[t, h, :len(take)] = torch.tensor(take)
    return ids


ATTEND = [([1], [1], 1, 1), ([64], [1], 4, 1), ([65], [3], 8, 4), ([3000], [1], 8, 16), ([3000], [1], 16, 40),
          ([2000, 90, 64, 700, 1], [1, 1, 1, 1, 1], 8, 5), ([1000] * 3, [5] * 3, 16, 9), ([300], [300], 8, 2),
          ([500], [150], 3, 6), ([500, 70, 130], [90, 70, 41], 4, 8), ([260], [260], 1, 5), ([400], [100], 16, 7),
          ([900], [70], 12, 15)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,new,G,k", ATTEND)
def test_attend(cuda_dev, D, lens, new, G, k):
    H = 2
    b = R.batch(lens, new, pad=(1,))
    pages, _, _ = R.filled(b, lens, H, D)
    check_attend(cuda_dev, b, pages, R.rows(21, len(b.seq), H * G, D), some_ids(b, H, k))


@pytest.mark.parametrize("T", [1, 70])
def test_attend_lists_of_every_kind(cuda_dev, T):
    """Empty lists, holes, any order, blocks listed twice, blocks past the token, blocks without a
    page, and with a page or a block number out of range."""
    D, H, G, k = 64, 2, 4, 10
    lens = [1000]
    b = R.batch(lens, [T])
    pages, _, _ = R.filled(b, lens, H, D)
    q = R.rows(1, T, H * G, D)
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(-3, 15, (T, H, k), generator=g).to(torch.int32)
    ids[0, 0] = -1
    ids[T - 1, 1] = torch.tensor([-1, 9, 9, -5, 2, 0, 15, 15, 3, -1])
    check_attend(cuda_dev, b, pages, q, ids)
    b.table[0, 4], b.table[0, 9] = -1, -7
    check_attend(cuda_dev, b, pages, q, ids)
    ids[0, 1, 3] = 13
    b.table[0, 13] = b.n_pages + 5
    check_attend(cuda_dev, b, pages, q, ids)
    b.table[0, 13] = 0
    ids[0, 1, 2], ids[0, 1, 4] = 2 ** 31 - 1, 14
    b.pos[0] = 64 * 40
    ids[0, 0, 1] = 30
    check_attend(cuda_dev, b, pages, q, ids)


def test_attend_sequences_out_of_range(cuda_dev):
    D, H, G = 64, 1, 2
    b = R.batch([300, 300], [2, 2])
    pages, _, _ = R.filled(b, [300, 300], H, D)
    b.seq[1], b.seq[2] = -1, 2
    check_attend(cuda_dev, b, pages, R.rows(1, 4, H * G, D), some_ids(R.batch([300, 300], [2, 2]), H, 3))


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-3])
def test_attend_scales(cuda_dev, T, scale):
    D, H, G = 128, 1, 8
    lens = [700]
    b = R.batch(lens, [T])
    pages, _, _ = R.filled(b, lens, H, D)
    check_attend(cuda_dev, b, pages, R.rows(3, T, H * G, D), some_ids(b, H, 6), scale=scale)


@pytest.mark.parametrize("T", [1, 40])
def test_attend_rows_of_very_different_size(cuda_dev, T):
    """Values of one token 2^40 times another's, keys of all zeros, queries near the ends of the range."""
    D, H, G = 64, 1, 4
    lens = [400]
    b = R.batch(lens, [T])
    pages, _, _ = R.filled(b, lens, H, D)
    kc, vc, ks, vs = R.views(pages, D)
    g = torch.Generator().manual_seed(8)
    vs += torch.randint(-40, 40, vs.shape, generator=g).to(torch.uint8)
    kc[:, :, 5] = 0
    vs[:, :, 6], vc[:, :, 6] = 63, 0
    ks[:, :, 7] = 63
    q = R.rows(1, T, G, D)
    q[:, 1] *= 1e-30
    q[:, 2] = 0.0
    check_attend(cuda_dev, b, pages, q, some_ids(b, H, 5))
    ks -= 60
    q[:, 0] *= 2.0 ** 60
    q[:, 1:] *= 0.01
    check_attend(cuda_dev, b, pages, q, some_ids(b, H, 5))


@pytest.mark.parametrize("T", [1, 40])
def test_attend_nan_stays_in_its_rows(cuda_dev, T):
    """A NaN key or value row spoils the rows that see its token, and no others."""
    D, H, G = 64, 2, 2
    lens = [400]
    b = R.batch(lens, [T])
    pages, _, _ = R.filled(b, lens, H, D)
    q = R.rows(1, T, H * G, D)
    q[0, 1] = math.nan
    ids = some_ids(b, H, 7)
    clean, _, _, _, _ = R.attend(q, pages, b.seq, b.pos, b.table, ids, 0.125)
    kc, vc, ks, vs = R.views(pages, D)
    kc[int(b.table[0, 1]), 0, 3], ks[int(b.table[0, 1]), 0, 3] = 0, 255
    last = lens[0] - 1
    for x in (kc, vc, ks, vs):     # never written, never seen
        x[int(b.table[0, last // 64]), :, last % 64 + 1:] = 0xFF
    vc[int(b.table[0, 2]), 1, 4], vs[int(b.table[0, 2]), 1, 4] = 0, 255
    c = on(cuda_dev, pages, torch.zeros((b.n_pages, H, 2, D), dtype=torch.int8), torch.zeros((b.n_pages, H), dtype=torch.int8))
    want, wl, _, _, _ = R.attend(q, pages, b.seq, b.pos, b.table, ids, 0.125)
    ok = ~want.isnan()
    for copies in (1, copies_for_tiles(T, H, G)):
        outs, lses = kv_attend(q.to(cuda_dev).repeat(copies, 1, 1), c, *repeated(b, copies).on(cuda_dev),
                               ids.to(cuda_dev).repeat(copies, 1, 1), scale=0.125)
        for out, lse in zip(outs.cpu().double().split(T), lses.cpu().double().split(T)):
            assert torch.equal(out.isnan(), want.isnan()) and torch.equal(lse.isnan(), wl.isnan())
            assert float((out - want)[ok].abs().max()) <= 2.0 ** -7 * float(clean[ok].abs().max())


def test_attend_query_slices_workspace_and_repeats(cuda_dev):
    """One workspace for calls of different sizes; the same call gives the same bits."""
    D, H, G = 128, 2, 4
    sizes = (([2000], [1]), ([1000, 300], [1, 1]), ([2200], [2100]), ([2000], [1]))
    ws = torch.zeros(max(kv_attend_workspace(T, H * G, H, D, 2, 12) for T in (1, 2, 2100)), dtype=torch.uint8,
                     device=cuda_dev)
    for lens, new in sizes:
        b = R.batch(lens, new)
        pages, _, _ = R.filled(b, lens, H, D)
        wide = R.rows(4, len(b.seq), H * G + 2, D)
        c = on(cuda_dev, pages, torch.zeros((b.n_pages, H, 2, D), dtype=torch.int8),
               torch.zeros((b.n_pages, H), dtype=torch.int8))
        first = None
        for _ in range(3):
            out, lse = kv_attend(wide.to(cuda_dev)[:, 2:], c, *b.on(cuda_dev), some_ids(b, H, 12).to(cuda_dev), ws=ws)
            first = first or (out, lse)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        want, _, mass, size, _ = R.attend(wide[:, 2:], pages, b.seq, b.pos, b.table, some_ids(b, H, 12), D ** -0.5)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * (D * 2.0 ** -23 * size + 2.0 ** -20))[..., None] * mass
        assert bool(((first[0].cpu().double() - want).abs() <= tol).all())


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("T", [1, 40])
def test_pages_past_four_gigabytes(cuda_dev, T):
    """The pages in use are the last of a cache of 5 GB."""
    D, H, G, n = 128, 8, 2, 38000
    lens = [500]
    b = R.batch(lens, [T])
    pages, bounds, bexp = R.filled(b, lens, H, D)
    c = KvCache.empty(n, H, D, cuda_dev)
    m = b.n_pages
    c.pages[-m:], c.bounds[-m:], c.bound_exp[-m:] = pages.to(cuda_dev), bounds.to(cuda_dev), bexp.to(cuda_dev)
    far = R.Batch(b.seq, b.pos, torch.where(b.table >= 0, b.table + (n - m), b.table), n)
    k, v, q = R.rows(1, T, H, D), R.rows(2, T, H, D), R.rows(3, T, H * G, D)
    on_dev = far.on(cuda_dev)
    kv_append(c, k.to(cuda_dev), v.to(cuda_dev), *on_dev)
    R.append(pages, bounds, bexp, k, v, b.seq, b.pos, b.table)
    assert torch.equal(c.pages[-m:].cpu(), pages) and torch.equal(c.bounds[-m:].cpu(), bounds)
    ko, vo = kv_read(c, *on_dev)
    kk, vv = R.values(pages, D)
    at = [int(b.table[s, p // 64]) for s, p in zip(b.seq, b.pos)]
    assert torch.equal(ko.cpu().double(), torch.stack([kk[a, :, p % 64] for a, p in zip(at, b.pos)]))
    assert torch.equal(vo.cpu().double(), torch.stack([vv[a, :, p % 64] for a, p in zip(at, b.pos)]))
    want_ids = R.select(q, bounds, bexp, b.seq, b.pos, b.table, 4, 1, 2)[0]
    want, _, mass, size, _ = R.attend(q, pages, b.seq, b.pos, b.table, want_ids, D ** -0.5)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * (D * 2.0 ** -23 * size + 2.0 ** -20))[..., None] * mass
    for copies in (1, copies_for_tiles(T, H, G)):
        on_dev = repeated(far, copies).on(cuda_dev)
        ids, _ = kv_select(q.to(cuda_dev).repeat(copies, 1, 1), c, *on_dev, 4)
        out, _ = kv_attend(q.to(cuda_dev).repeat(copies, 1, 1), c, *on_dev, ids)
        assert all(torch.equal(i, want_ids) for i in ids.cpu().split(T))
        assert all(bool(((o - want).abs() <= tol).all()) for o in out.cpu().double().split(T))


@pytest.mark.parametrize("T,G", [(1, 4), (70, 4), (1100, 8)])
def test_a_step_on_another_stream_and_in_a_graph(cuda_dev, T, G):
    """append, select and attend of one step: on a side stream, and captured and replayed on new inputs."""
    D, H, k = 64, 2, 6
    lens = [1200]
    b = R.batch(lens, [T])
    pages, bounds, bexp = R.filled(b, lens, H, D)
    c = on(cuda_dev, pages, bounds, bexp)
    seq, pos, table = b.on(cuda_dev)
    kvq = [R.rows(i, T, n, D).to(cuda_dev) for i, n in ((1, H), (2, H), (3, H * G))]
    B, N = table.shape
    sws = torch.zeros(kv_select_workspace(T, H * G, H, D, B, N, k), dtype=torch.uint8, device=cuda_dev)
    aws = torch.zeros(kv_attend_workspace(T, H * G, H, D, B, k), dtype=torch.uint8, device=cuda_dev)
    ids, scores = (torch.empty((T, H, k), dtype=d, device=cuda_dev) for d in (torch.int32, torch.float32))
    out, lse = torch.empty((T, H * G, D), dtype=torch.bfloat16, device=cuda_dev), torch.empty((T, H * G), device=cuda_dev)

    def step():
        kv_append(c, kvq[0], kvq[1], seq, pos, table)
        kv_select(kvq[2], c, seq, pos, table, k, ws=sws, ids=ids, scores=scores)
        kv_attend(kvq[2], c, seq, pos, table, ids, ws=aws, out=out, lse=lse)

    def expect():
        p, bo, be = pages.clone(), bounds.clone(), bexp.clone()
        kc, vc, q = (x.cpu() for x in kvq)
        R.append(p, bo, be, kc, vc, b.seq, b.pos, b.table)
        want_ids = R.select(q, bo, be, b.seq, b.pos, b.table, k, 1, 2)[0]
        assert torch.equal(ids.cpu(), want_ids)
        want, _, mass, size, _ = R.attend(q, p, b.seq, b.pos, b.table, want_ids, D ** -0.5)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * (D * 2.0 ** -23 * size + 2.0 ** -20))[..., None] * mass
        assert bool(((out.cpu().double() - want).abs() <= tol).all())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    expect()
    c.bounds.copy_(bounds.to(cuda_dev)), c.bound_exp.copy_(bexp.to(cuda_dev))
    graph = StepGraph(step)
    for i in (10, 20):
        c.bounds.copy_(bounds.to(cuda_dev)), c.bound_exp.copy_(bexp.to(cuda_dev))
        for x, s in zip(kvq, (i, i + 1, i + 2)):
            x.copy_(R.rows(s, *x.shape))
        graph.replay()
        torch.cuda.synchronize()
        expect()


def test_binding_refuses(cuda_dev):
    c = KvCache.empty(3, 2, 64, cuda_dev)
    b = R.batch([100], [2])
    seq, pos, table = b.on(cuda_dev)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=cuda_dev)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=cuda_dev)
    ids = torch.zeros((2, 2, 4), dtype=torch.int32, device=cuda_dev)
    for bad in (k[:, :1], k.float(), k.half(), k[:1], torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=cuda_dev)[:, ::2],
                k.cpu()):
        with pytest.raises(ValueError):
            kv_append(c, bad, k, seq, pos, table)
    for args in ((seq.long(), pos, table), (seq, pos[:1], table), (seq, pos, table.long())):
        with pytest.raises(ValueError):
            kv_read(c, *args)
    if kv_select_workspace(2, 4, 2, 64, 1, 2, 4):
        with pytest.raises(BreError, match="workspace"):
            kv_select(q, c, seq, pos, table, 4, ws=torch.zeros(0, dtype=torch.uint8, device=cuda_dev))
    with pytest.raises(BreError):
        kv_select(q, c, seq, pos, table, 2, n_sink=2, n_local=1)
    with pytest.raises(ValueError):
        kv_attend(q, c, seq, pos, table, ids[:, :1])
    with pytest.raises(ValueError):
        kv_attend(q, c, seq, pos, table, ids, out=torch.zeros((2, 4, 32), dtype=torch.bfloat16, device=cuda_dev))
    with pytest.raises(BreError, match="unsupported"):
        kv_attend(torch.zeros((2, 34, 64), dtype=torch.bfloat16, device=cuda_dev), c, seq, pos, table, ids)
    none = [torch.zeros(0, dtype=torch.int32, device=cuda_dev)] * 2
    out, lse = kv_attend(q[:0], c, *none, table, ids[:0])
    assert out.shape == (0, 4, 64) and kv_read(c, *none, table)[0].shape == (0, 2, 64)


def test_attend_wait_budget_runs_out_then_the_next_call_is_clean(cuda_dev):
    """The tile kernel's waits with a budget of one cycle: the call returns and sets the bit; the next call, with
    the default budget, gives the bits of the one before."""
    D, H, G, k = 64, 2, 8, 6
    b = R.batch([1200], [1100])
    pages, bounds, bexp = R.filled(b, [1200], H, D)
    c = on(cuda_dev, pages, bounds, bexp)
    q, ids, tokens = R.rows(3, 1100, H * G, D).to(cuda_dev), some_ids(b, H, k).to(cuda_dev), b.on(cuda_dev)
    e = err_word(cuda_dev)
    out, lse = kv_attend(q, c, *tokens, ids, dev_err=e)
    assert int(e) == 0
    L = _lib.load()
    try:
        assert L.bre_set_ffn_wait_limit(1) == _lib.BRE_OK
        kv_attend(q, c, *tokens, ids, dev_err=e)
        torch.cuda.synchronize()
    finally:
        assert L.bre_set_ffn_wait_limit(0) == _lib.BRE_OK
    assert int(e) == _lib.BRE_DEVERR_TIMEOUT
    e.zero_()
    again, lse2 = kv_attend(q, c, *tokens, ids, dev_err=e)
    assert int(e) == 0 and torch.equal(again, out) and torch.equal(lse2, lse)
