"""kv_rotate refuses outputs that lie over what other threads still read or write (no GPU)."""
import ctypes as C

import pytest

from bit_routed_expert_gb300 import _lib
from bit_routed_expert_gb300._lib import BRE_ERR_ARG

BASE, FAR = 1 << 20, 1 << 30


def rotate(q=0, q_out=FAR, k=FAR * 2, k_out=FAR * 3, qs=512, qos=512, ks=512, kos=512, Hq=4, Hk=2, T=3):
    """Rows of four and two heads of 64; places in elements behind BASE."""
    at = lambda x: None if x is None else C.c_void_p(BASE + 2 * x)  # noqa: E731
    P = C.c_void_p(BASE)
    return _lib.load().kv_rotate(at(q), qs, Hq, at(k), ks, Hk, 64, P, T, P, 16, 1.0, 0, 0, 0, at(q_out), qos, at(k_out), kos, None)


@pytest.mark.parametrize("kw", [
    dict(q_out=0, qos=256), dict(q_out=0, qs=256),                            # its input with another stride
    dict(q_out=64), dict(q_out=255), dict(q=64, q_out=0), dict(q_out=512), dict(q_out=1024 + 255), dict(q=512, q_out=0),
    dict(q_out=1), dict(q=1, q_out=0), dict(k=0, k_out=FAR, q=FAR * 2, q_out=127),   # half a row, one channel, a row on
    dict(q=0, k=256, q_out=256, k_out=0), dict(q=0, k=256, q_out=0, k_out=0), dict(q=0, k=256, k_out=128), dict(q_out=FAR, k_out=FAR),
    dict(q_out=FAR, k_out=FAR + 255), dict(k=FAR + 100), dict(q_out=2 * FAR - 255), dict(q_out=0, qos=256, T=2), dict(q_out=100, T=1),
    dict(q_out=700, qos=600), dict(k=100, q_out=255 + 100 - 355, q=FAR, T=1), dict(k=600, ks=128, q_out=400, T=1)])
def test_refused(kw):
    assert rotate(**kw) == BRE_ERR_ARG

