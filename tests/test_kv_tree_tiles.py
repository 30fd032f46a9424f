"""kv_attend_tree's tile kernel at the sizes of test_kv_tree.py, where most calls are small enough for the other one, and what only
it does: lists of many tokens, waits that run out.

Which kernel a call takes goes by the width of the table too, so that wide ones (whose blocks behind the sequences have no
pages) lead to the tiles.
"""
import pytest
import torch

import kv_more_reference as M
import kv_reference as R
import test_kv_tree as base
from bit_routed_expert_gb300 import _lib, kv_attend_tree, kv_attend_tree_workspace

pytestmark = pytest.mark.gpu

WIDE = 5000


@pytest.fixture(autouse=True)
def wide_tables(monkeypatch):
    narrow = R.batch

    def batch(*a, **kw):
        b = narrow(*a, **kw)
        b.table = torch.cat([b.table, torch.full((len(b.table), WIDE), -1, dtype=torch.int32)], 1)
        return b

    monkeypatch.setattr(R, "batch", batch)


test_trees, test_causal, test_long_context_is_split = base.test_trees, base.test_causal, base.test_long_context_is_split
test_masks_of_any_kind, test_neighbours_of_one_tile_differ = base.test_masks_of_any_kind, base.test_neighbours_of_one_tile_differ
test_scales_of_any_size, test_nan_rows = base.test_scales_of_any_size, base.test_nan_rows
test_unwritten_slots_do_not_matter = base.test_unwritten_slots_do_not_matter
test_sequences_in_pieces_and_out_of_order = base.test_sequences_in_pieces_and_out_of_order
test_slices_of_a_projection_and_no_lse = base.test_slices_of_a_projection_and_no_lse
test_the_same_bits_every_time_and_on_other_streams = base.test_the_same_bits_every_time_and_on_other_streams


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 40.0])
def test_scales_of_the_logits(cuda_dev, scale):
    """A negative scale turns the order round; with 0 every weight is the same; 40: weights of 0 and 1."""
    D, H, G, ctx = 64, 2, 4, 300
    b, lens, masks = base.trees([ctx], [40], seed=4)
    pages, _, _ = R.filled(b, lens, H, D, seed=12)
    base.check(cuda_dev, b, pages, R.rows(13, 40, H * G, D), [ctx], masks, scale=scale)


def test_maxima_that_rise_along_the_context(cuda_dev):
    """Every block's keys are twice the last one's, and then within blocks: the maximum that the weights are held against is
    replaced in either half of a block, by small and by large steps."""
    D, H, G, ctx = 128, 1, 8, 1500
    b, lens, masks = base.trees([ctx], [20], seed=6)
    for gain in (0.05, 1.0, 8.0):
        pages, _, _ = R.filled(b, lens, H, D, seed=14)
        _, _, ks, _ = R.views(pages, D)
        for x in range(ctx):
            ks[int(b.table[0, x // 64]), :, x % 64] = 127 - 14 + x // 128 + (x % 64 >= 40) * 3 + (x % 64 >= 20) * 2
        q = R.rows(15, 20, G, D).abs() * gain   # (with keys of both signs: rows that rise and rows that fall)
        base.check(cuda_dev, b, pages, q.to(torch.bfloat16), [ctx], masks)
        kc, _, _, _ = R.views(pages, D)
        kc &= 0x7F   # all rise
        base.check(cuda_dev, b, pages, q.to(torch.bfloat16), [ctx], masks)


def subset(b, at):
    return R.Batch([b.seq[i] for i in at], [b.pos[i] for i in at], b.table, b.n_pages)


@pytest.mark.parametrize("lens,D,H,G,pad", [([700, 520], 64, 1, 2, (3, 511, 512, 1000)), ([41] * 60, 128, 1, 3, ()), ([1100], 64, 2, 1, (0,)),
                                            ([33] * 560, 64, 1, 1, (7, 17000))])
def test_lists_longer_than_a_cta(cuda_dev, lens, D, H, G, pad):
    """All tokens of their sequences; the reference, which goes token by token, for some of them, first and last ones among
    them."""
    b = R.batch(lens, lens, seed=8, pad=pad)
    pages, _, _ = R.filled(b, lens, H, D, seed=9)
    T = len(b.seq)
    q = R.rows(10, T, H * G, D)
    seq, pos, table = b.on(cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    ws = torch.full((kv_attend_tree_workspace(T, H * G, H, D),), 255, dtype=torch.uint8, device=cuda_dev)
    out, lse = kv_attend_tree(q.to(cuda_dev), base.on(cuda_dev, pages, H, D), seq, pos, table, ws=ws, dev_err=err)
    assert int(err) == 0
    g = torch.Generator().manual_seed(1)
    at = sorted({0, 1, 31, 32, 511, 512, 513, 1023, 1024, T - 2, T - 1, *torch.randint(0, T, (60,), generator=g).tolist(), *pad})
    sub = subset(b, at)
    want, wl, mass, size, peak, _ = M.attend_tree(q[at], pages, sub.seq, sub.pos, sub.table, None, None, D ** -0.5)
    d = D * 2.0 ** -23 * size + 2.0 ** -19 * peak + 2.0 ** -20   # (see test_kv_tree.py)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * d)[..., None] * mass + 1e-30
    assert bool(((out.cpu()[at].double() - want).abs() <= tol).all())
    some = wl > -float("inf")
    got = lse.cpu()[at].double()
    assert torch.equal(got > -float("inf"), some)
    assert bool(((got - wl).abs() <= d + 2.0 ** -22 * wl.abs())[some].all())


def test_waits_that_run_out(cuda_dev):
    """With a budget of one cycle the kernel gives up, says so and ends; the next call, on the same workspace, is a clean one."""
    L = _lib.load()
    D, H, G, ctx = 128, 2, 8, 3000
    b, lens, masks = base.trees([ctx, 500], [20, 30], seed=3)
    pages, _, _ = R.filled(b, lens, H, D, seed=4)
    q = R.rows(11, len(b.seq), H * G, D).to(cuda_dev)
    seq, pos, table = b.on(cuda_dev)
    c, err = base.on(cuda_dev, pages, H, D), torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    args = dict(start=torch.tensor([ctx, 500], dtype=torch.int32, device=cuda_dev), mask=M.mask_tensor(masks, 1).to(cuda_dev),
                ws=torch.zeros(kv_attend_tree_workspace(len(b.seq), H * G, H, D), dtype=torch.uint8, device=cuda_dev), dev_err=err)
    want, want_lse = kv_attend_tree(q, c, seq, pos, table, **args)
    torch.cuda.synchronize()
    assert int(err) == 0
    try:
        assert L.bre_set_ffn_wait_limit(1) == _lib.BRE_OK
        kv_attend_tree(q, c, seq, pos, table, **args)
        torch.cuda.synchronize()
    finally:
        assert L.bre_set_ffn_wait_limit(0) == _lib.BRE_OK
    assert int(err) == _lib.BRE_DEVERR_TIMEOUT
    err.zero_()
    again, again_lse = kv_attend_tree(q, c, seq, pos, table, **args)
    assert int(err) == 0 and torch.equal(again, want) and torch.equal(again_lse, want_lse)
