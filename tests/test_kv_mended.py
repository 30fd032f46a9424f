"""Cases of the key/value cache calls that answered wrongly once, against the definitions in 64 bits."""
import copy
import pickle

import pytest
import torch

import kv_reference as R
from bit_routed_expert_gb300 import KvCache, kv_append, kv_attend, kv_read, kv_select
from test_kv_cache import check_attend, check_select, on, some_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sink,local,k", [(0, 1, 7), (1, 2, 16), (0, 3, 40)])
@pytest.mark.parametrize("blocks", [511, 512, 513, 514, 515, 1025])
def test_select_last_piece_holds_only_forced_blocks(cuda_dev, blocks, sink, local, k):
    """The kernels select from pieces of 512 blocks; where the last piece has none but local blocks, which are taken
    anyway, its selection ends at once and the list held so far is passed on as it is."""
    D, H, G, T = 64, 1, 2, 40
    b = R.batch([2560], [1])
    cache = R.filled(b, [2560], H, D)
    g = torch.Generator().manual_seed(blocks)
    n = R.Batch([0] * T, list(range(64 * blocks - T, 64 * blocks)),
                torch.randint(0, b.n_pages, (1, blocks), generator=g).to(torch.int32), b.n_pages)
    check_select(cuda_dev, n, cache, R.rows(blocks, T, G, D), k, sink, local)


def own(c):
    return c.pages.cpu(), c.bounds.cpu(), c.bound_exp.cpu()


def test_a_cache_that_grew_and_a_copy_use_their_own_tensors(cuda_dev):
    """append, read, select and attend after the fields were assigned, and on a deep copy and an unpickled cache."""
    D, H, G = 64, 2, 2
    b = R.batch([100], [30])
    small = R.filled(b, [100], H, D)
    old = on(cuda_dev, *small)
    held = [old.pages, old.bounds, old.bound_exp]
    c = on(cuda_dev, *small)
    c.pages, c.bounds, c.bound_exp = (torch.cat([x, x.flip(0)]) for x in held)
    assert c.n_pages == 2 * b.n_pages
    table = torch.where(b.table >= 0, b.table + b.n_pages, b.table)   # pages that only the larger cache has
    n = R.Batch(b.seq, b.pos, table, 2 * b.n_pages)
    k, v, q = R.rows(1, 30, H, D), R.rows(2, 30, H, D), R.rows(3, 30, H * G, D)
    for other in (copy.deepcopy(c), pickle.loads(pickle.dumps(c)), c):
        want, before = own(other), own(c)
        e = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        kv_append(other, k.to(cuda_dev), v.to(cuda_dev), *n.on(cuda_dev), dev_err=e)
        assert not R.append(*want, k, v, n.seq, n.pos, table)
        assert all(torch.equal(x, y) for x, y in zip(own(other), want)) and int(e) == 0
        if other is not c:
            assert all(torch.equal(x, y) for x, y in zip(own(c), before))
        kk, _ = R.values(want[0], D)
        got, _ = kv_read(other, *n.on(cuda_dev))
        assert torch.equal(got.cpu().double(), torch.stack([kk[int(table[0, p // 64]), :, p % 64] for p in n.pos]))
        ids, _ = kv_select(q.to(cuda_dev), other, *n.on(cuda_dev), 3)
        assert torch.equal(ids.cpu(), R.select(q, *want[1:], n.seq, n.pos, table, 3, 1, 2)[0])
        out, _ = kv_attend(q.to(cuda_dev), other, *n.on(cuda_dev), ids)
        o, _, mass, size, _ = R.attend(q, want[0], n.seq, n.pos, table, ids.cpu(), D ** -0.5)
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * (D * 2.0 ** -23 * size + 2.0 ** -20))[..., None] * mass
        assert bool(((out.cpu().double() - o).abs() <= tol).all())
    assert all(torch.equal(x.cpu(), y) for x, y in zip(held, small))


def test_fields_that_do_not_belong_together_are_refused(cuda_dev):
    """A cache half way through its growth."""
    c = KvCache.empty(3, 2, 64, cuda_dev)
    c.pages = torch.cat([c.pages, c.pages])
    tokens = R.batch([3], [3]).on(cuda_dev)
    with pytest.raises(ValueError, match="belong together"):
        kv_read(c, *tokens)
    c.pages = c.pages[:3].cpu()
    with pytest.raises(ValueError, match="CUDA"):
        kv_read(c, *tokens)


def test_new_outputs_of_a_call_on_another_stream_are_allocated_there(cuda_dev):
    """Memory that the current stream has just given back may still be read by what runs there."""
    D, H, G, T = 64, 2, 4, 8192
    b = R.batch([T], [T])
    c = on(cuda_dev, *R.filled(b, [T], H, D))
    tokens = b.on(cuda_dev)
    q = R.rows(3, T, H * G, D).to(cuda_dev)
    ids = torch.zeros((T, H, 2), dtype=torch.int32, device=cuda_dev)
    first = [*kv_read(c, *tokens), *kv_select(q, c, *tokens, 8), *kv_attend(q, c, *tokens, ids)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made = []
    for call in (lambda: kv_read(c, *tokens, stream=side), lambda: kv_select(q, c, *tokens, 8, stream=side),
                 lambda: kv_attend(q, c, *tokens, ids, stream=side)):
        free = [torch.empty_like(x) for x in first[len(made):len(made) + 2]]
        places = [x.data_ptr() for x in free]
        del free
        out = call()
        assert not {x.data_ptr() for x in out} & set(places)
        made += out
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(made, first))
    # given back while the current stream still works: not handed out again before it is done
    torch.cuda._sleep(200_000_000)
    places = {x.data_ptr() for x in made}
    shapes = [(x.shape, x.dtype) for x in made]
    del made, out
    with torch.cuda.stream(side):
        assert not {torch.empty(s, dtype=d, device=cuda_dev).data_ptr() for s, d in shapes} & places
    torch.cuda.synchronize()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("up", [14, 15, 16, 24, 40, 100])
def test_attend_beside_a_key_of_another_size(cuda_dev, up, D):
    """One key of every block is 2^up times the others: for the rows that see it, orthogonal to their queries; the
    tokens before it in the last block do not see it.  The other keys count in full either way."""
    H, G, T, slot = 2, 4, 40, 15
    lens = [400]
    b = R.batch(lens, [T])
    pages, _, _ = R.filled(b, lens, H, D)
    kc, _, ks, _ = R.views(pages, D)
    kc[:, :, slot, 1:] = 0
    kc[:, :, slot, 0] = 0x7E
    ks[:, :, slot] += up
    q = R.rows(21, T, H * G, D)
    q[:, :, 0] = 0.0
    check_attend(cuda_dev, b, pages, q, some_ids(b, H, 5))
    ks -= 60   # and all keys small, the queries large
    q *= 2.0 ** 60
    check_attend(cuda_dev, b, pages, q, some_ids(b, H, 5))


@pytest.mark.parametrize("where", ["first", "last", "everywhere"])
@pytest.mark.parametrize("big", [50, 80, 110, 119])
def test_attend_beside_a_value_of_another_size(cuda_dev, big, where):
    """Value rows of zeros (the least scale, 2^-64) and a few whose scale is 2^big, up to that of infinities, which
    saturate: every token counts in the sum of the weights whatever its value's scale."""
    D, H, G, T = 64, 2, 4, 40
    lens = [400]
    b = R.batch(lens, [T])
    pages, _, _ = R.filled(b, lens, H, D)
    _, vc, _, vs = R.views(pages, D)
    g = torch.Generator().manual_seed(big)
    zero = torch.rand(vs.shape, generator=g) < 0.5
    vc[zero], vs[zero] = 0, 63
    block = {"first": [0], "last": [5], "everywhere": range(7)}[where]
    for i in block:
        vs[int(b.table[0, i]), :, ::9] = 127 + big
    ids = torch.arange(6, dtype=torch.int32).expand(T, H, 6).contiguous()
    check_attend(cuda_dev, b, pages, R.rows(21, T, H * G, D), ids)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("shift", [50, 90, 119])
def test_select_compares_scores_beyond_the_range(cuda_dev, T, shift):
    """Keys so large (infinities are stored as 448 * 2^119) that a score without the query's factor is beyond FP32: the
    blocks still compare as whole numbers do, and with small queries the scores themselves are within the range."""
    D, H, G = 64, 1, 4
    lens = [1000]
    b = R.batch(lens, [T])
    pages, bounds, bexp = R.filled(b, lens, H, D)
    bexp += shift
    q = R.rows(2, T, G, D)
    check_select(cuda_dev, b, (pages, bounds, bexp), q * 2.0 ** -shift, 6, 1, 1)
    q[:, :, :D // 2] = 0.0
    check_select(cuda_dev, b, (pages, bounds, bexp), q * 2.0 ** -50, 6, 0, 1)


@pytest.mark.parametrize("D,H", [(64, 3), (128, 1)])
@pytest.mark.parametrize("before,between,behind", [(0, 0, 4000), (4000, 0, 0), (1300, 1, 1300), (70, 130, 1025), (33, 257, 31)])
def test_append_among_long_padding(cuda_dev, D, H, before, between, behind):
    """Padding before, between the tokens of (and between) blocks, and behind; chunks that are all padding."""
    lens, new = [150, 70], [90, 70]
    b = R.batch(lens, new)
    seq, pos = [0] * before, [-1] * before
    for i, (s, p) in enumerate(zip(b.seq, b.pos)):
        gap = between if i % 37 == 5 else 0
        seq += [s] + [1] * gap
        pos += [p] + [-1] * gap
    n = R.Batch(seq + [0] * behind, pos + [-1] * behind, b.table, b.n_pages)
    T = len(n.seq)
    pages, bounds, bexp = R.filled(b, lens, H, D)
    k, v = R.rows(1, T, H, D), R.rows(2, T, H, D)
    c = on(cuda_dev, pages, bounds, bexp)
    kv_append(c, k.to(cuda_dev), v.to(cuda_dev), *n.on(cuda_dev))
    real = [i for i in range(T) if n.pos[i] >= 0]   # padding between a block's tokens changes nothing
    assert not R.append(pages, bounds, bexp, k[real], v[real], b.seq, b.pos, b.table)
    assert all(torch.equal(x, y) for x, y in zip(own(c), (pages, bounds, bexp)))


def test_writing_slot_0_again_starts_the_bounds_anew(cuda_dev):
    """The bounds are then those of that call's keys alone (a page is used again; a rejected block is decoded again); a
    later slot written again widens them."""
    D, H = 64, 2
    b = R.batch([20], [20])
    pages, bounds, bexp = R.filled(b, [20], H, D)
    c = on(cuda_dev, pages, bounds, bexp)
    for a, z, gain in ((0, 20, 8.0), (0, 3, 0.5), (3, 6, 2.0)):
        k = R.rows(a + z, z - a, H, D, gain=gain)
        n = R.Batch(b.seq[a:z], b.pos[a:z], b.table, b.n_pages)
        kv_append(c, k.to(cuda_dev), k.to(cuda_dev), *n.on(cuda_dev))
        R.append(pages, bounds, bexp, k, k, n.seq, n.pos, n.table)
        assert all(torch.equal(x, y) for x, y in zip(own(c), (pages, bounds, bexp)))
    kk = R.values(pages, D)[0][int(b.table[0, 0])]
    hi = bounds[int(b.table[0, 0]), :, 0].double() * 2.0 ** bexp[int(b.table[0, 0])].double()[:, None]
    assert bool((kk[:, :6].amax(1) <= hi).all()) and not bool((kk[:, :20].amax(1) <= hi).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("codes", ["zeros", "minus zeros", "one code", "mixed"])
def test_attend_beside_keys_of_the_least_scale(cuda_dev, codes, D):
    """Key rows of zeros have the least scale and are exact beside anything; others of that scale count where the queries
    are as large as these keys are small."""
    H, G, T = 2, 4, 40
    lens = [400]
    b = R.batch(lens, [T])
    pages, _, _ = R.filled(b, lens, H, D)
    kc, _, ks, _ = R.views(pages, D)
    row = torch.zeros(64, D, dtype=torch.uint8)
    if codes == "minus zeros":
        row[:] = 0x80
    elif codes == "one code":
        row[:, D - 1] = 0x7E
    elif codes == "mixed":
        row[20, 0], row[50, 5] = 0x38, 0xB8
    for i, x in enumerate((0, 7, 20, 31, 32, 50, 63)):
        kc[:, :, x], ks[:, :, x] = row[x], 63
    q = R.rows(21, T, H * G, D)
    check_attend(cuda_dev, b, pages, q, some_ids(b, H, 5))
    q[:, :, :D // 2] = 0.0
    kc[:, :, :, D // 2:D - 1] &= 0x80   # only the last channel meets the queries: the small rows' logits are theirs
    near = torch.tensor([x not in (0, 7, 20, 31, 32, 50, 63) for x in range(64)])
    kc[:, :, near, D - 1] = 0
    check_attend(cuda_dev, b, pages, q * 2.0 ** 55, some_ids(b, H, 5))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [1, 7, 20])
def test_bounds_hold_beside_a_key_of_another_size(cuda_dev, D, step):
    """An infinity (stored as 448 * 2^119) among keys of 2^-34: the other channels' bounds are 1 and -1 of its unit, not 0."""
    H = 2
    b = R.batch([20], [20])
    pages, bounds, bexp = R.filled(b, [20], H, D)
    c = on(cuda_dev, pages, bounds, bexp)
    k = R.rows(3, 20, H, D, gain=2.0 ** -34)
    k[9, 1, 5], k[11, 0, 6] = float("inf"), float("-inf")
    k[:, :, 7], k[:, :, 8], k[:, :, 9] = k[:, :, 7].abs(), -k[:, :, 8].abs(), 0.0
    for i in range(0, 20, step):
        n = R.Batch(b.seq[i:i + step], b.pos[i:i + step], b.table, b.n_pages)
        kv_append(c, k[i:i + step].to(cuda_dev), k[i:i + step].to(cuda_dev), *n.on(cuda_dev))
        R.append(pages, bounds, bexp, k[i:i + step], k[i:i + step], n.seq, n.pos, n.table)
    assert all(torch.equal(x, y) for x, y in zip(own(c), (pages, bounds, bexp)))
    kk, u = R.values(pages, D)[0][int(b.table[0, 0])], 2.0 ** bexp[int(b.table[0, 0])].double()[:, None]
    assert bool((kk[:, :20].amax(1) <= bounds[int(b.table[0, 0]), :, 0] * u).all())
    assert bool((kk[:, :20].amin(1) >= bounds[int(b.table[0, 0]), :, 1] * u).all())
