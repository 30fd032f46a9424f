"""The 64-bit reference of the key/value cache calls against closed forms (CPU)."""
import math

import pytest
import torch

import kv_reference as R


def test_e4m3_codes_match_the_library_cast():
    g = torch.Generator().manual_seed(3)
    x = torch.cat([torch.randn(4000, generator=g) * 2.0 ** torch.randint(-12, 8, (4000,), generator=g),
                   R.VALUES[:127].float(), R.VALUES[128:255].float(),
                   torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 27.0, 29.0, 448.0])]).clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8)
    assert [R.e4m3_code(float(v)) for v in x.double()] == want.tolist()
    fin = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    assert torch.equal(R.VALUES[fin.long()].float(), fin.view(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("top", [448.0, 127.0, 63.0])
def test_least_exp(top):
    for a in (0.0, 1e-30, 2.0 ** -64 * top, 0.3, top, math.nextafter(top, 1e9), 1.0, 1e38):
        e = R.least_exp(a, top)
        assert a <= math.ldexp(top, e) and (e == -64 or a > math.ldexp(top, e - 1))


def test_stored_row_is_within_half_a_step():
    for seed in range(5):
        x = R.rows(seed, 128, gain=10.0 ** (seed - 2))
        codes, byte = R.store_row(x)
        y = R.VALUES[codes.long()] * 2.0 ** (byte - 127)
        step = torch.maximum(x.double().abs() * 2.0 ** -4, torch.tensor(2.0 ** (byte - 127 - 10), dtype=torch.float64))
        assert bool(((y - x.double()).abs() <= step).all())
        assert float(y.abs().max()) <= 448 * 2.0 ** (byte - 127)


def test_bounds_hold_and_grow_in_steps_as_at_once():
    D, H = 64, 2
    k, v = R.rows(1, 40, H, D, gain=3.0), R.rows(2, 40, H, D)
    table = torch.zeros((1, 1), dtype=torch.int32)

    def run(cuts):
        pages = torch.zeros((1, H, 128 * (D + 1)), dtype=torch.uint8)
        bounds, bexp = torch.zeros((1, H, 2, D), dtype=torch.int8), torch.zeros((1, H), dtype=torch.int8)
        for a, b in zip(cuts, cuts[1:]):
            assert not R.append(pages, bounds, bexp, k[a:b], v[a:b], [0] * (b - a), list(range(a, b)), table)
        return pages, bounds, bexp

    one, many = run([0, 40]), run([0, 1, 2, 17, 40])
    assert all(torch.equal(x, y) for x, y in zip(one, many))
    kk, _ = R.values(one[0], D)
    hi, lo = (one[1].double() * 2.0 ** one[2].double()[..., None, None]).unbind(2)
    assert bool((kk[:, :, :40].amax(2) <= hi).all()) and bool((kk[:, :, :40].amin(2) >= lo).all())


def test_score_bounds_the_summed_logits():
    D, H, G = 64, 2, 3
    lens = [400]
    b = R.batch(lens, [5])
    pages, bounds, bexp = R.filled(b, lens, H, D)
    q = R.rows(9, 5, H * G, D)
    ids, scores, err = R.select(q, bounds, bexp, b.seq, b.pos, b.table, 16, 1, 1)
    assert not err and ids.shape == (5, H, 16)
    kk, _ = R.values(pages, D)
    for t in range(5):
        for h in range(H):
            for j, blk in enumerate(ids[t, h].tolist()):
                if blk < 0:
                    continue
                x = q[t].double().view(H, G, D)[h]
                dots = (x @ kk[int(b.table[0, blk]), h].T).sum(0)
                slack = float(x.abs().max()) / 64 * 0.5 * G * float(kk.abs().max()) * D   # q's rounding
                assert float(dots.max()) <= float(scores[t, h, j]) + slack


def test_attention_over_everything_is_plain_attention():
    D, H, G = 64, 1, 2
    lens = [130]
    b = R.batch(lens, [3], pad=(1,))
    pages, _, _ = R.filled(b, lens, H, D)
    q = R.rows(4, 4, G, D)
    ids = torch.arange(3, dtype=torch.int32).expand(4, H, 3).contiguous()
    out, lse, _, _, err = R.attend(q, pages, b.seq, b.pos, b.table, ids, 0.125)
    kk, vv = R.values(pages, D)
    kk, vv = kk[b.table[0].long(), 0].reshape(-1, D), vv[b.table[0].long(), 0].reshape(-1, D)
    assert not err and float(out[1].abs().max()) == 0 and float(lse[1].max()) == -math.inf
    for t in (0, 2, 3):
        s = q[t].double() @ kk[:b.pos[t] + 1].T * 0.125
        torch.testing.assert_close(out[t], torch.softmax(s, -1) @ vv[:b.pos[t] + 1])
        torch.testing.assert_close(lse[t], torch.logsumexp(s, -1))
