"""kv_compact, kv_fork and kv_resize on the GPU: every byte and number equals the definition's (kv_more_reference.py)."""
import pytest
import torch

import kv_more_reference as M
import kv_reference as R
from bit_routed_expert_gb300 import (KvCache, StepGraph, kv_append, kv_attend_tree, kv_compact, kv_fork, kv_read, kv_resize,
                                     kv_resize_workspace)
from bit_routed_expert_gb300._lib import BRE_DEVERR_FULL, BRE_DEVERR_PAGE

pytestmark = pytest.mark.gpu


def whole(dev, x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def same(c, pages, bounds, bexp):
    assert torch.equal(c.pages.cpu(), pages) and torch.equal(c.bounds.cpu(), bounds) and torch.equal(c.bound_exp.cpu(), bexp)


# ------------------------------------------------------------------ compaction

def check_compact(dev, b, lens, H, D, start, nodes, count, seed=0, change=None):
    pages, bounds, bexp = R.filled(b, lens, H, D, seed=seed)
    if change:
        change(pages)
    A = max((len(n) for n in nodes), default=0)
    table = [n + [-1] * (A - len(n)) for n in nodes]
    nd = torch.tensor(table, dtype=torch.int32).view(len(nodes), A)
    c = KvCache(pages.to(dev), bounds.to(dev), bexp.to(dev))
    e = whole(dev, [0])
    got = kv_compact(c, b.table.to(dev), whole(dev, start), nd.to(dev), whole(dev, count), dev_err=e)
    want, err = M.compact(pages, bounds, bexp, b.table, start, nd, count)
    assert got.tolist() == want
    assert int(e) == (BRE_DEVERR_PAGE if err else 0)
    same(c, pages, bounds, bexp)


@pytest.mark.parametrize("D,H", [(64, 1), (128, 2), (64, 3)])
@pytest.mark.parametrize("ctx,kept", [([0], [[0]]), ([0], [[]]), ([5], [[]]), ([64], [[]]), ([64], [[3]]), ([63], [[0, 1]]), ([63], [[1, 4]]),
                                      ([100], [[2, 5, 6, 31]]), ([0], [list(range(0, 300, 3))]), ([70], [list(range(1, 400, 2))]),
                                      ([0], [list(range(200))]), ([10, 64, 0, 127, 30], [[1], [0, 70], [5, 6, 7], [], [60, 61]])])
def test_compact(cuda_dev, D, H, ctx, kept):
    lens = [c + (max(k) + 2 if k else 3) for c, k in zip(ctx, kept)]
    b = R.batch(lens, lens)
    check_compact(cuda_dev, b, lens, H, D, ctx, kept, [len(k) for k in kept], seed=D)


def test_compact_takes_fewer_than_listed_and_leaves_sequences(cuda_dev):
    lens = [100, 100, 100]
    b = R.batch(lens, lens)
    kept = [[1, 3, 5], [2, 4, 6], [7, 8, 9]]
    check_compact(cuda_dev, b, lens, 2, 64, [40, 40, 40], kept, [2, -1, 0])


def test_compact_refuses_lists_that_do_not_hold(cuda_dev):
    """Each beside a sequence that is moved; nothing of the refused one changes."""
    lens = [200, 200]
    for start, kept, count in ((10, [3, 3], 2), (10, [5, 4], 2), (10, [-1, 4], 2), (10, [0, 400], 2), (-3, [1, 2], 2), (10, [1, 2], 3),
                               (2 ** 31 - 5, [1, 2], 2), (10, [1, 2 ** 31 - 1], 2), (190, [2 ** 31 - 1, 4], 2), (255, [0, 1], 2), (10, [1, 2], 2 ** 31 - 1)):
        b = R.batch(lens, lens)
        check_compact(cuda_dev, b, lens, 1, 64, [start, 10], [kept, [4, 5]], [count, 2])
    for hole in (0, 1, 2):
        b = R.batch(lens, lens)
        b.table[0, hole] = -1 if hole < 2 else b.n_pages
        check_compact(cuda_dev, b, lens, 1, 64, [60, 10], [[10, 100], [4, 5]], [2, 2])


def test_compact_of_special_rows(cuda_dev):
    """NaN rows, zeros, rows of very different scales; what the dropped rows held leaves the bounds."""
    lens = [150]

    def change(pages):
        kc, vc, ks, vs = R.views(pages, 64)
        ks[:, :, 5::9], kc[:, :, 5::9] = 255, 0
        kc[:, :, 3::7], ks[:, :, 3::7] = 0, 63
        ks[:, :, 1::11] = 127 + 100
        ks[:, :, 2::5] = 127 - 60
        vs[:, :, ::13], vc[:, :, ::13] = 255, 0
    for kept in (list(range(0, 80, 2)), [2, 3, 5, 9], [4], []):
        b = R.batch(lens, lens)
        check_compact(cuda_dev, b, lens, 2, 64, [50], [kept], [len(kept)], change=change)


def test_compact_equals_appending_the_kept_tokens(cuda_dev):
    D, H, ctx, n = 64, 2, 30, 90
    b = R.batch([ctx + n], [ctx + n])
    k, v = R.rows(1, ctx + n, H, D).to(cuda_dev), R.rows(2, ctx + n, H, D).to(cuda_dev)
    keep = list(range(1, n, 4))
    caches = [KvCache.empty(b.n_pages, H, D, cuda_dev) for _ in range(2)]
    seq, pos, table = b.on(cuda_dev)
    kv_append(caches[0], k, v, seq, pos, table)
    length = kv_compact(caches[0], table, whole(cuda_dev, [ctx]), whole(cuda_dev, [keep]), whole(cuda_dev, [len(keep)]))
    assert length.tolist() == [ctx + len(keep)]
    at = torch.tensor(list(range(ctx)) + [ctx + x for x in keep], device=cuda_dev)
    m = len(at)
    kv_append(caches[1], k[at], v[at], seq[:m], pos[:m], table)
    for x, y in zip(kv_read(caches[0], seq[:m], pos[:m], table), kv_read(caches[1], seq[:m], pos[:m], table)):
        assert torch.equal(x, y)
    used = b.table[0, :-(-m // 64)].long().to(cuda_dev)
    assert torch.equal(caches[0].bounds[used], caches[1].bounds[used])
    assert torch.equal(caches[0].bound_exp[used], caches[1].bound_exp[used])


# ------------------------------------------------------------------ forks and resizes

def pool(lens, N, n_pages, seed=0, share=()):
    """(table, refs) of sequences with pages of their own, but for `share`: (row, row whose first blocks it names, how many)."""
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), N), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for c in range(-(-n // 64)):
            table[b, c] = order.pop()
    for row, of, n in share:
        table[row, :n] = table[of, :n]
    return table, M.count_refs(table, n_pages)


def dummy(n_pages, H, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, 256, (n_pages, H, 128 * (D + 1)), generator=g, dtype=torch.uint8),
            torch.randint(-128, 128, (n_pages, H, 2, D), generator=g).to(torch.int8), torch.randint(-64, 100, (n_pages, H), generator=g).to(torch.int8))


def check_fork(dev, table, refs, parent, length):
    n = len(refs)
    c = KvCache(*[x.to(dev) for x in dummy(n, 1, 64)])
    t, r, e = table.to(dev), refs.to(dev), whole(dev, [0])
    kv_fork(c, r, t, whole(dev, parent), whole(dev, length), dev_err=e)
    err = M.fork(refs, table, parent, length)
    assert torch.equal(t.cpu(), table) and torch.equal(r.cpu(), refs)
    assert int(e) == (BRE_DEVERR_PAGE if err else 0)
    same(c, *dummy(n, 1, 64))


FORKS = [([100], 3, [0], [100]), ([100], 3, [0], [64]), ([100], 3, [-1], [100]), ([100, 0], 2, [0, 0], [100, 65]), ([100, 300], 7, [1, 0], [300, 100]),
         ([100, 300, 64], 7, [1, 2, 0], [128, 64, 63]), ([100, 300, 64], 7, [0, 1, 2], [10 ** 6] * 3), ([640] * 9, 40, [3] * 9, [601] * 9),
         ([640] * 9, 40, [8, 7, 6, 5, 4, 3, 2, 1, 0], [0, 1, 63, 64, 65, 639, 640, 641, -4])]


@pytest.mark.parametrize("lens,N,parent,length", FORKS)
def test_fork(cuda_dev, lens, N, parent, length):
    table, refs = pool(lens, N, 130)
    check_fork(cuda_dev, table, refs, parent, length)


def test_fork_of_many_rows(cuda_dev):
    """More rows than a CTA's threads, and tables whose columns no longer fit 48 KB."""
    g = torch.Generator().manual_seed(3)
    for B, N in ((700, 70), (2000, 33), (13000, 5), (49152, 2)):
        table = torch.randint(-1, 500, (B, N), generator=g).to(torch.int32)
        parent = torch.randint(0, B, (B,), generator=g)
        length = torch.randint(0, 64 * N + 1, (B,), generator=g)
        refs = M.count_refs(table, 500)
        c = KvCache(*[x.to(cuda_dev) for x in dummy(500, 1, 64)])
        t, r = table.to(cuda_dev), refs.to(cuda_dev)
        kv_fork(c, r, t, parent.to(torch.int32).to(cuda_dev), length.to(torch.int32).to(cuda_dev))
        want = torch.where(torch.arange(N) < (-(-length // 64))[:, None], table[parent], -1)
        assert torch.equal(t.cpu(), want) and torch.equal(r.cpu(), M.count_refs(want, 500))


def test_fork_outside_the_cache(cuda_dev):
    table, refs = pool([200, 200], 5, 20)
    table[0, 1], table[1, 2], table[1, 3] = 20, 2 ** 31 - 1, -9
    refs = M.count_refs(table, 20)
    check_fork(cuda_dev, table.clone(), refs.clone(), [1, 0], [320, 320])
    check_fork(cuda_dev, table.clone(), refs.clone(), [2, 1], [320, 320])
    check_fork(cuda_dev, table.clone(), refs.clone(), [2 ** 31 - 1, -2 ** 31], [320, 320])


def check_resize(dev, table, refs, start, end, H=1, D=64, ws=None):
    n, (B, N) = len(refs), table.shape
    held = dummy(n, H, D)
    c = KvCache(*[x.to(dev) for x in held])
    t, r, e = table.to(dev), refs.to(dev), whole(dev, [0])
    ws = torch.full((kv_resize_workspace(n, B, N),), 255, dtype=torch.uint8, device=dev)   # its contents must not matter
    kv_resize(c, r, t, whole(dev, start), whole(dev, end), ws=ws, dev_err=e)
    page_err, full = M.resize(*held, refs, table, start, end)
    assert torch.equal(t.cpu(), table) and torch.equal(r.cpu(), refs)
    assert int(e) == (BRE_DEVERR_PAGE if page_err else 0) | (BRE_DEVERR_FULL if full else 0)
    same(c, *held)


RESIZES = [([100], 4, [], [100], [101]), ([100], 4, [], [100], [129]), ([100], 4, [], [100], [256]), ([100], 4, [], [0], [0]), ([100], 4, [], [64], [64]),
           ([128], 4, [], [128], [128]), ([100], 4, [], [100], [-1]), ([0], 4, [], [0], [1]), ([0], 4, [], [0], [64]), ([100], 4, [], [-7], [200]),
           ([100, 100], 4, [(1, 0, 2)], [100, 100], [101, 101]), ([100, 100], 4, [(1, 0, 2)], [100, 100], [101, -1]),
           ([128, 128], 4, [(1, 0, 2)], [128, 128], [130, 128]), ([200, 200], 6, [(1, 0, 4)], [70, 64], [300, 384]),
           ([200] * 5, 9, [(1, 0, 4), (2, 0, 3), (4, 3, 1)], [150, 100, 200, 10, 0], [576, 200, 150, 64, 0]),
           ([300, 0, 20, 500], 70, [], [300, 0, 20, 500], [4000, 2000, 64, 0]), ([300], 5, [], [300], [10 ** 6]), ([300], 5, [], [400], [100])]


@pytest.mark.parametrize("lens,N,share,start,end", RESIZES)
@pytest.mark.parametrize("H,D", [(1, 64), (3, 128)])
def test_resize(cuda_dev, lens, N, share, start, end, H, D):
    table, refs = pool(lens, N, 150, share=share)
    check_resize(cuda_dev, table, refs, start, end, H, D)


def test_resize_runs_out_of_pages(cuda_dev):
    """The first blocks in the order of rows get what there is; the others, shared ones too, stay as they were."""
    for n in (8, 9, 10, 12):
        table, refs = pool([200, 200], 8, n if n > 8 else 8, share=[(1, 0, 4)])
        check_resize(cuda_dev, table, refs, [200, 200], [300, 400])
    table, refs = pool([200, 200], 8, 8)
    check_resize(cuda_dev, table, refs, [200, 100], [260, 100])   # what this call gives back is free for the next one
    check_resize(cuda_dev, table, refs, [200, 100], [260, 100])


def test_resize_of_many_rows_and_pages(cuda_dev):
    g = torch.Generator().manual_seed(5)
    for B, N, n in ((300, 40, 5000), (5, 1500, 70000), (1, 1, 300000), (1500, 3, 9000), (40, 65, 2500)):
        lens = torch.randint(0, 64 * N // 3 + 1, (B,), generator=g).tolist()
        table, _ = pool(lens, N, n, seed=B)
        for b in range(0, B, 3):   # some rows go on in another one's pages
            of = int(torch.randint(0, B, (1,), generator=g))
            table[b] = table[of]
            lens[b] = lens[of]
        refs = M.count_refs(table, n)
        if n == 300000:
            refs[:299000] = 1   # a pool that is almost full
        end = [int(x + torch.randint(-70, 200, (1,), generator=g)) for x in lens]
        check_resize(cuda_dev, table, refs, lens, end)


def test_resize_outside_the_cache(cuda_dev):
    table, refs = pool([300, 300], 6, 30)
    table[0, 3], table[0, 5], table[1, 4] = 30, 2 ** 31 - 1, -8
    refs = M.count_refs(table, 30)
    check_resize(cuda_dev, table, refs, [130, 130], [320, 200])


def test_beams_as_a_whole(cuda_dev):
    """Steps of a beam search through one graph: fork, resize, append, attend.  Every beam's cache is what a cache of its own
    would hold, and every page is named as often as refs says."""
    D, H, G, B, ctx, steps = 64, 2, 4, 5, 61, 9
    n_pages, N = 40, 3
    c = KvCache.empty(n_pages, H, D, cuda_dev)
    table, refs = torch.full((B, N), -1, dtype=torch.int32, device=cuda_dev), torch.zeros(n_pages, dtype=torch.int32, device=cuda_dev)
    err = whole(cuda_dev, [0])
    k, v = R.rows(1, ctx + steps * B, H, D).to(cuda_dev), R.rows(2, ctx + steps * B, H, D).to(cuda_dev)
    one = whole(cuda_dev, [0] * B)
    kv_resize(c, refs, table, one, whole(cuda_dev, [ctx] + [-1] * (B - 1)), dev_err=err)
    kv_append(c, k[:ctx], v[:ctx], whole(cuda_dev, [0] * ctx), torch.arange(ctx, dtype=torch.int32, device=cuda_dev), table, dev_err=err)
    parent, length, seq = whole(cuda_dev, [0] * B), whole(cuda_dev, [ctx] * B), torch.arange(B, dtype=torch.int32, device=cuda_dev)
    kn, vn, q = k[:B].clone(), v[:B].clone(), R.rows(3, B, H * G, D).to(cuda_dev)
    end = length + 1
    out = torch.empty((B, H * G, D), dtype=torch.bfloat16, device=cuda_dev)

    def step():
        kv_fork(c, refs, table, parent, length, dev_err=err)
        kv_resize(c, refs, table, length, end, dev_err=err)
        kv_append(c, kn, vn, seq, length, table, dev_err=err)
        kv_attend_tree(q, c, seq, length, table, out=out, dev_err=err)

    keep = [x.clone() for x in (c.pages, c.bounds, c.bound_exp, table, refs)]
    graph = StepGraph(step)
    for x, y in zip((c.pages, c.bounds, c.bound_exp, table, refs), keep):   # what the warm-up did
        x.copy_(y)
    paths = [list(range(ctx))] * B
    g = torch.Generator().manual_seed(1)
    for s in range(steps):
        p = torch.randint(0, B, (B,), generator=g) if s else torch.zeros(B, dtype=torch.int64)
        parent.copy_(p.to(torch.int32))
        length.fill_(ctx + s)
        end.fill_(ctx + s + 1)
        new = ctx + s * B
        kn.copy_(k[new:new + B])
        vn.copy_(v[new:new + B])
        graph.replay()
        paths = [paths[int(p[b])] + [new + b] for b in range(B)]
        assert torch.equal(refs.cpu(), M.count_refs(table.cpu(), n_pages))
        assert int(err) == 0
        L = ctx + s + 1
        own = KvCache.empty(B * N, H, D, cuda_dev)
        flat = torch.arange(B * N, dtype=torch.int32, device=cuda_dev).view(B, N)
        seqs, poss = seq.repeat_interleave(L), torch.arange(L, dtype=torch.int32, device=cuda_dev).repeat(B)
        at = torch.tensor(sum(paths, []), device=cuda_dev)
        kv_append(own, k[at], v[at], seqs, poss, flat)
        for x, y in zip(kv_read(c, seqs, poss, table), kv_read(own, seqs, poss, flat)):
            assert torch.equal(x, y)
        assert torch.equal(out, kv_attend_tree(q, own, seq, length, flat)[0])
    # everything given back
    kv_fork(c, refs, table, whole(cuda_dev, [-1] * B), length, dev_err=err)
    assert int(refs.abs().sum()) == 0 and int((table + 1).abs().sum()) == 0
