"""Limits of the key/value cache calls that are checked before any launch (no GPU; addresses are made up)."""
import ctypes as C

import pytest

from bit_routed_expert_gb300 import _lib
from bit_routed_expert_gb300._lib import BRE_ERR_UNSUPPORTED, BRE_OK, BreKvCache

P = C.c_void_p(1 << 20)


def attend(N, T):
    c = BreKvCache(1 << 20, 1 << 20, 1 << 20, 4, 2, 64)
    return _lib.load().kv_attend(C.byref(c), P, 256, 4, P, P, T, P, 1, N, P, 4, 1.0, P, None, None, 0, None, None)


@pytest.mark.parametrize("N", [2 ** 25 - 1, 2 ** 25, 2 ** 31 - 1])
def test_attend_block_numbers_fit_their_25_bits(N):
    """The tile kernel tells blocks apart by 25 bits less one value: block 2^25 - 2 must lie outside the table, or a list's
    entry 2^25 - 1 would be read as it."""
    assert attend(N, 3) == BRE_ERR_UNSUPPORTED
    assert attend(2 ** 25 - 2, 0) == BRE_OK


def test_no_call_needs_a_workspace():
    """The arguments stay for callers that pass one: 0 bytes for every size, and what is passed is not looked at."""
    L = _lib.load()
    for T in (0, 1, 5, 8192, 1 << 20):
        for G in (1, 16):
            assert L.kv_select_workspace(T, 4 * G, 4, 128, 64, 131072, 256) == 0
            assert L.kv_attend_workspace(T, 4 * G, 4, 128, 64, 256) == 0
