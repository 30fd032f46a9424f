"""What the key/value cache calls refuse before any launch (no GPU), by status through the C ABI."""
import ctypes as C

import pytest
import torch

from bit_routed_expert_gb300 import KvCache, _lib
from bit_routed_expert_gb300._lib import BRE_ERR_ARG, BRE_ERR_UNSUPPORTED, BRE_ERR_WORKSPACE, BRE_OK, BreKvCache

P = C.c_void_p(1 << 20)     # stands for a device pointer: nothing here is launched
ODD = C.c_void_p((1 << 20) + 2)


def cache(**kw):
    f = dict(pages=1 << 20, bounds=1 << 20, bound_exp=1 << 20, n_pages=4, n_kv_heads=2, head_dim=64)
    f.update(kw)
    return BreKvCache(*[f[n] for n in ("pages", "bounds", "bound_exp", "n_pages", "n_kv_heads", "head_dim")])


def append(c=None, k=P, v=P, ks=128, vs=128, seq=P, pos=P, T=3, table=P, B=1, N=1):
    c = cache() if c is None else c
    return _lib.load().kv_append(C.byref(c), k, v, ks, vs, seq, pos, T, table, B, N, None, None)


def read(c=None, T=3, k=P, v=P):
    c = cache() if c is None else c
    return _lib.load().kv_read(C.byref(c), P, P, T, P, 1, 1, k, v, None, None)


def select(c=None, q=P, qs=256, Hq=4, T=3, B=1, N=1, k=4, sink=1, local=1, ids=P, ws=None, wsb=0):
    c = cache() if c is None else c
    return _lib.load().kv_select(C.byref(c), q, qs, Hq, P, P, T, P, B, N, k, sink, local, ids, None, ws, wsb, None,
                                 None)


def attend(c=None, q=P, qs=256, Hq=4, T=3, ids=P, k=4, scale=1.0, out=P, ws=None, wsb=0):
    c = cache() if c is None else c
    return _lib.load().kv_attend(C.byref(c), q, qs, Hq, P, P, T, P, 1, 1, ids, k, scale, out, None, ws, wsb, None, None)


BAD_CACHES = [({"pages": 0}, BRE_ERR_ARG), ({"bounds": 0}, BRE_ERR_ARG), ({"bound_exp": 0}, BRE_ERR_ARG),
              ({"n_pages": 0}, BRE_ERR_ARG), ({"n_kv_heads": 0}, BRE_ERR_ARG), ({"n_pages": -1}, BRE_ERR_ARG),
              ({"head_dim": 96}, BRE_ERR_UNSUPPORTED), ({"head_dim": 0}, BRE_ERR_UNSUPPORTED),
              ({"head_dim": 256}, BRE_ERR_UNSUPPORTED), ({"n_kv_heads": 65536}, BRE_ERR_UNSUPPORTED), ({"pages": (1 << 20) + 8}, BRE_ERR_ARG),
              ({"bounds": (1 << 20) + 4}, BRE_ERR_ARG)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refused(kw, status):
    c = cache(**kw)
    assert append(c) == read(c) == select(c) == attend(c) == status


def test_no_tokens_is_no_work():
    assert append(T=0, seq=None, pos=None) == read(T=0) == select(T=0) == attend(T=0) == BRE_OK


def test_append_refuses():
    assert append(k=None) == append(v=None) == append(seq=None) == append(pos=None) == append(table=None) == BRE_ERR_ARG
    assert append(k=ODD) == append(v=ODD) == append(ks=120) == append(vs=120) == append(ks=132) == BRE_ERR_ARG
    assert append(T=-1) == append(B=0) == append(N=0) == append(seq=ODD) == BRE_ERR_ARG
    assert append(T=2 ** 30) == BRE_ERR_UNSUPPORTED


def test_read_refuses():
    assert read(k=None, v=None) == read(k=ODD) == read(v=ODD) == BRE_ERR_ARG


def test_select_refuses():
    assert select(q=None) == select(q=ODD) == select(qs=248) == select(qs=260) == select(ids=None) == BRE_ERR_ARG
    assert select(Hq=3, qs=192) == select(Hq=0) == select(k=0) == BRE_ERR_ARG
    assert select(sink=-1) == select(local=-1) == select(sink=3, local=2) == select(sink=5, local=0) == BRE_ERR_ARG
    assert select(Hq=34, qs=34 * 64) == select(k=257) == select(N=131073) == BRE_ERR_UNSUPPORTED
    need = _lib.load().kv_select_workspace(3, 4, 2, 64, 1, 1, 4)
    if need:
        assert select() == select(ws=P, wsb=need - 1) == select(ws=C.c_void_p((1 << 20) + 16), wsb=need)
        assert select() == BRE_ERR_WORKSPACE


def test_attend_refuses():
    assert attend(q=None) == attend(q=ODD) == attend(qs=248) == attend(ids=None) == attend(out=None) == BRE_ERR_ARG
    assert attend(out=ODD) == attend(Hq=3, qs=192) == attend(k=0) == BRE_ERR_ARG
    assert attend(scale=float("nan")) == attend(scale=float("inf")) == BRE_ERR_ARG
    assert attend(Hq=34, qs=34 * 64) == attend(k=257) == BRE_ERR_UNSUPPORTED
    need = _lib.load().kv_attend_workspace(3, 4, 2, 64, 1, 4)
    if need:
        assert attend() == attend(ws=P, wsb=need - 1) == BRE_ERR_WORKSPACE


def test_workspace_sizes():
    L = _lib.load()
    assert L.kv_select_workspace(0, 4, 2, 64, 1, 1, 4) == L.kv_attend_workspace(0, 4, 2, 64, 1, 4) == 0
    for T in (1, 7, 100, 8192):
        assert L.kv_select_workspace(T, 32, 4, 128, 1, 2048, 16) <= L.kv_select_workspace(T + 1, 32, 4, 128, 1, 2048, 16)
        assert L.kv_attend_workspace(T, 32, 4, 128, 1, 16) <= L.kv_attend_workspace(T + 1, 32, 4, 128, 1, 16)


def test_python_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        KvCache.empty(2, 2, 64, "cpu")
    with pytest.raises(ValueError, match="belong together"):
        KvCache(torch.zeros((2, 2, 100), dtype=torch.uint8), torch.zeros((2, 2, 2, 64), dtype=torch.int8),
                torch.zeros((2, 2), dtype=torch.int8))
    with pytest.raises(ValueError, match="int8"):
        KvCache(torch.zeros((2, 2, 128 * 65), dtype=torch.uint8), torch.zeros((2, 2, 2, 64), dtype=torch.uint8),
                torch.zeros((2, 2), dtype=torch.int8))
