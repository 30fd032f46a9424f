"""What the calls that go through ctypes do with numbers outside 32 bits: refuse them, like the binding of the other kv_* calls (no GPU)."""
from ctypes import ArgumentError

import pytest

from bit_routed_expert_gb300 import kv_attend_tree_workspace, kv_resize_workspace, rope_turns

BIG = 2 ** 32


@pytest.mark.parametrize("n", [BIG, BIG + 64, -BIG, 2 ** 31, 2 ** 70])
def test_refused(n):
    with pytest.raises(ValueError, match="32 bits"):
        rope_turns(n)
    for at in range(4):
        with pytest.raises(ValueError, match="32 bits"):
            kv_attend_tree_workspace(*(n if i == at else x for i, x in enumerate((5, 8, 2, 64))))
    for at in range(3):
        with pytest.raises(ValueError, match="32 bits"):
            kv_resize_workspace(*(n if i == at else x for i, x in enumerate((100, 3, 7))))


def test_whole_numbers_only():
    for bad in (64.0, "64", None):
        with pytest.raises((ValueError, TypeError, ArgumentError)):
            rope_turns(bad)
        with pytest.raises((ValueError, TypeError, ArgumentError)):
            kv_resize_workspace(bad, 3, 7)
