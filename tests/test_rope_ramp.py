"""The two ramps of rope_turns (no GPU): what they share, and where the one that may end behind the last pair differs.
64-bit arithmetic on both sides, as in test_kv_more_args.py."""
import math

import pytest

import kv_more_reference as M
from bit_routed_expert_gb300 import rope_turns


def definition(R, base, s, low, high, L, most):
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    p = lambda n: R * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    a, b = max(math.floor(p(high)), 0), min(math.ceil(p(low)), most)
    r = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(R // 2)]
    return [x / s * y + x * (1 - y) for x, y in zip(f, r)]


CASES = [(128, 10000.0, 4.0, 131072.0), (128, 10000.0, 2.0, 65536.0), (64, 10000.0, 8.0, 2.0 ** 20), (4, 10000.0, 16.0, 2048.0), (128, 10000.0, 16.0, 4096.0),
         (64, 500000.0, 8.0, 8192.0), (2, 10000.0, 4.0, 100.0)]


@pytest.mark.parametrize("R,base,s,L", CASES)
@pytest.mark.parametrize("scaling", ["ramp", "ramp_past"])
def test_values(R, base, s, L, scaling):
    turns, gain = rope_turns(R, base, scaling, s, length=L)
    want = M.turns_of(definition(R, base, s, 1.0, 32.0, L, R - 1 if scaling == "ramp_past" else R // 2 - 1))
    for x, w in zip(turns.tolist(), want):
        assert abs((x - w + 2 ** 63) % 2 ** 64 - 2 ** 63) <= max(w, 2 ** 40) * 2.0 ** -46 + 1
    assert gain == pytest.approx(0.1 * math.log(s) + 1, rel=2.0 ** -23)


def test_they_differ_only_where_the_last_pair_turns_in_the_length():
    for R, base, s, L in CASES:
        one, two = (rope_turns(R, base, how, s, length=L)[0] for how in ("ramp", "ramp_past"))
        beyond = math.ceil(R * math.log(L / (2 * math.pi)) / (2 * math.log(base))) > R // 2 - 1 and R > 2
        assert bool((one != two).any()) == beyond
