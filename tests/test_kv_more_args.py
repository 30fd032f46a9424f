"""What rotary positions, tree attention and the page calls refuse before any launch, and their host-side parts (no GPU)."""
import ctypes as C
import math
from unittest import mock

import pytest
import torch

import kv_more_reference as M
from bit_routed_expert_gb300 import (KvCache, _lib, kv_attend_tree, kv_compact, kv_fork, kv_resize, kv_rotate, rope_turns)
from bit_routed_expert_gb300._lib import (BRE_ERR_ARG, BRE_ERR_UNSUPPORTED, BRE_ERR_WORKSPACE, BRE_OK, BreError, BreKvCache)

P = C.c_void_p(1 << 20)     # stands for a device pointer: nothing here is launched
ODD = C.c_void_p((1 << 20) + 2)
BYTE = C.c_void_p((1 << 20) + 1)


def cache(**kw):
    f = dict(pages=1 << 20, bounds=1 << 20, bound_exp=1 << 20, n_pages=4, n_kv_heads=2, head_dim=64)
    f.update(kw)
    return BreKvCache(*[f[n] for n in ("pages", "bounds", "bound_exp", "n_pages", "n_kv_heads", "head_dim")])


def tree(c=None, q=P, qs=256, Hq=4, seq=P, pos=P, T=3, table=P, B=1, N=1, start=P, mask=P, words=1, scale=1.0, out=P, lse=None,
         ws=P, wsb=1 << 40):
    c = cache() if c is None else c
    return _lib.load().kv_attend_tree(C.byref(c), q, qs, Hq, seq, pos, T, table, B, N, start, mask, words, scale, out, lse, ws, wsb,
                                      None, None)


def rotate(q=P, qs=256, Hq=4, k=P, ks=128, Hk=2, D=64, pos=P, T=3, turns=P, pairs=16, gain=1.0, offset=0, q_out=P, qos=256, k_out=P,
           kos=128):
    return _lib.load().kv_rotate(q, qs, Hq, k, ks, Hk, D, pos, T, turns, pairs, gain, offset, 0, 0, q_out, qos, k_out, kos, None)


def compact(c=None, table=P, B=1, N=1, start=P, nodes=P, A=4, count=P, length=None):
    c = cache() if c is None else c
    return _lib.load().kv_compact(C.byref(c), table, B, N, start, nodes, A, count, length, None, None)


def fork(c=None, refs=P, table=P, B=1, N=1, parent=P, length=P):
    c = cache() if c is None else c
    return _lib.load().kv_fork(C.byref(c), refs, table, B, N, parent, length, None, None)


def resize(c=None, refs=P, table=P, B=1, N=1, start=P, end=P, ws=P, wsb=1 << 40):
    c = cache() if c is None else c
    return _lib.load().kv_resize(C.byref(c), refs, table, B, N, start, end, ws, wsb, None, None)


BAD_CACHES = [({"pages": 0}, BRE_ERR_ARG), ({"bounds": 0}, BRE_ERR_ARG), ({"bound_exp": 0}, BRE_ERR_ARG), ({"n_pages": 0}, BRE_ERR_ARG),
              ({"n_kv_heads": -1}, BRE_ERR_ARG), ({"head_dim": 96}, BRE_ERR_UNSUPPORTED), ({"pages": (1 << 20) + 8}, BRE_ERR_ARG)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refused(kw, status):
    c = cache(**kw)
    assert tree(c) == compact(c) == fork(c) == resize(c) == status


def test_no_tokens_is_no_work():
    assert tree(T=0, seq=None, pos=None) == rotate(T=0, q=None, q_out=None) == BRE_OK


def test_tree_refuses():
    assert tree(q=None) == tree(q=ODD) == tree(qs=248) == tree(qs=260) == tree(out=None) == tree(out=ODD) == tree(lse=ODD) == BRE_ERR_ARG
    assert tree(seq=None) == tree(pos=None) == tree(table=None) == tree(T=-1) == tree(B=0) == tree(N=0) == BRE_ERR_ARG
    assert tree(Hq=3, qs=192) == tree(Hq=0) == tree(scale=math.nan) == tree(scale=math.inf) == BRE_ERR_ARG
    assert tree(start=None) == tree(words=0) == tree(words=-1) == tree(mask=C.c_void_p((1 << 20) + 4)) == tree(start=ODD) == BRE_ERR_ARG
    assert tree(Hq=34, qs=34 * 64) == tree(words=1025) == BRE_ERR_UNSUPPORTED
    assert tree(cache(n_pages=2 ** 30)) == tree(T=2 ** 27, Hq=32, qs=2048) == BRE_ERR_UNSUPPORTED   # 32-bit rows of pages, of queries
    need = _lib.load().kv_attend_tree_workspace(3, 4, 2, 64)
    if need:
        assert tree(ws=None, wsb=0) == tree(wsb=need - 1) == tree(ws=C.c_void_p((1 << 20) + 16)) == BRE_ERR_WORKSPACE


def test_rotate_refuses():
    assert rotate(q=None) == rotate(q_out=None) == rotate(q=BYTE) == rotate(k_out=None) == rotate(k=None) == rotate(Hk=0) == BRE_ERR_ARG
    assert rotate(qs=255) == rotate(qos=255) == rotate(ks=127) == rotate(kos=127) == rotate(Hq=0) == rotate(T=-1) == BRE_ERR_ARG
    assert rotate(pairs=0) == rotate(pairs=33) == rotate(offset=-1) == rotate(offset=33) == rotate(pairs=2 ** 31 - 1) == BRE_ERR_ARG
    assert rotate(turns=None) == rotate(turns=ODD) == rotate(pos=None) == rotate(pos=ODD) == rotate(gain=math.nan) == BRE_ERR_ARG
    assert rotate(D=68, qs=272, qos=272) == rotate(D=264, qs=2000, qos=2000, ks=2000, kos=2000) == BRE_ERR_UNSUPPORTED
    assert rotate(D=0) == BRE_ERR_ARG


def test_page_calls_refuse():
    for f in (compact, fork, resize):
        assert f(table=None) == f(B=0) == f(N=0) == f(table=ODD) == BRE_ERR_ARG
    assert compact(start=None) == compact(nodes=None) == compact(count=None) == compact(A=-1) == compact(length=ODD) == BRE_ERR_ARG
    apart = [C.c_void_p((1 << 20) + (i << 16)) for i in range(3)]
    for i in range(3):   # a length that is one of the lists, or begins inside of it
        lists = dict(zip(("start", "count", "nodes"), apart))
        assert compact(length=apart[i], B=3, **lists) == compact(length=C.c_void_p(apart[i].value + 8), B=3, **lists) == BRE_ERR_ARG
    assert fork(refs=None) == fork(parent=None) == fork(length=None) == fork(refs=ODD) == BRE_ERR_ARG
    assert resize(refs=None) == resize(start=None) == resize(end=None) == resize(start=ODD) == BRE_ERR_ARG
    assert fork(B=49153) == fork(B=40000, N=60000) == resize(B=40000, N=60000) == BRE_ERR_UNSUPPORTED
    need = _lib.load().kv_resize_workspace(4, 3, 5)
    assert resize(B=3, N=5, wsb=need - 1) == resize(ws=None) == resize(ws=C.c_void_p((1 << 20) + 8)) == BRE_ERR_WORKSPACE


def test_workspaces_grow_with_the_sizes():
    L = _lib.load()
    assert L.kv_resize_workspace(0, 1, 1) == L.kv_attend_tree_workspace(0, 8, 2, 64) == 0
    sizes = [L.kv_attend_tree_workspace(T, 32, 2, 64) for T in (1, 7, 500, 2 ** 20, 2 ** 30, 2 ** 31 - 1)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] > 2 ** 40
    sizes = [L.kv_resize_workspace(n, b, N) for n, b, N in ((4, 1, 1), (400, 1, 1), (400, 7, 1), (400, 7, 900), (10 ** 6, 7, 900))]
    assert sizes == sorted(sizes) and sizes[0] > 0


# ------------------------------------------------------------------ frequencies

def frequencies(R, theta=10000.0, how=None, s=1.0, low=1.0, high=32.0, L=0.0):
    base = theta * s ** (R / (R - 2)) if how == "base" and R > 2 else theta
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if how == "linear":
        return [x / s for x in f]
    if how == "ramp":
        p = lambda n: R * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        a, b = max(math.floor(p(high)), 0), min(math.ceil(p(low)), R // 2 - 1)
        r = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(R // 2)]
        return [x / s * y + x * (1 - y) for x, y in zip(f, r)]
    if how == "bands":
        w = [min(max((L * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
        return [(1 - y) * x / s + y * x for x, y in zip(f, w)]
    return f


@pytest.mark.parametrize("R", [2, 4, 48, 64, 128, 254])
@pytest.mark.parametrize("how,s,L", [(None, 1.0, 0.0), ("linear", 8.0, 0.0), ("base", 4.0, 0.0), ("ramp", 16.0, 2048.0),
                                     ("ramp", 1.0, 100.0), ("bands", 8.0, 8192.0)])
def test_frequencies(R, how, s, L):
    """64-bit arithmetic on both sides: pow, log and the products are off by a few of 2^-53 each, and log's error is
    multiplied by ln(theta') < 16 in a power."""
    high = 4.0 if how == "bands" else 32.0
    turns, gain = rope_turns(R, 10000.0, how, s, length=L)
    want = M.turns_of(frequencies(R, 10000.0, how, s, 1.0, high, L))
    assert turns.dtype == torch.int64 and len(turns) == R // 2
    for x, w in zip(turns.tolist(), want):
        off = (x - w + 2 ** 63) % 2 ** 64 - 2 ** 63
        assert abs(off) <= max(w, 2 ** 40) * 2.0 ** -46 + 1
    assert gain == pytest.approx(0.1 * math.log(s) + 1 if how == "ramp" and s > 1 else 1.0, rel=2.0 ** -23)


def test_frequencies_refused():
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=-2), dict(rot_dim=64, theta=1.0), dict(rot_dim=64, theta=math.inf),
               dict(rot_dim=64, scaling="linear", factor=0.0), dict(rot_dim=64, scaling="ramp", factor=2.0, length=0.0),
               dict(rot_dim=64, scaling="bands", factor=2.0, length=100.0, low=4.0, high=4.0),
               dict(rot_dim=64, scaling="base", factor=math.nan)):
        with pytest.raises(BreError):
            rope_turns(**kw)
    with pytest.raises(ValueError, match="scaling"):
        rope_turns(64, scaling="other")


# ------------------------------------------------------------------ the Python face

def fake(device, *shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device=device)


def fake_call(name, **where):
    """One call whose tensors are all on cuda:0 but for those named in `where`."""
    at = lambda n: where.get(n, "cuda:0")  # noqa: E731
    with mock.patch("torch.cuda.is_available", lambda: False), torch._subclasses.fake_tensor.FakeTensorMode():
        c = KvCache(fake("cuda:0", 3, 2, 128 * 65, dtype=torch.uint8), fake("cuda:0", 3, 2, 2, 64, dtype=torch.int8),
                    fake("cuda:0", 3, 2, dtype=torch.int8))
        table, err, refs = fake(at("table"), 2, 3), fake(at("dev_err"), 1), fake(at("refs"), 3)
        one, two = fake(at("one"), 2), fake(at("two"), 2)
        rows = lambda n, h: fake(at(n), 5, h, 64, dtype=torch.bfloat16)  # noqa: E731
        if name == "tree":
            kv_attend_tree(rows("q", 4), c, fake(at("seq"), 5), fake(at("pos"), 5), table, one, fake(at("mask"), 5, 1, dtype=torch.int64),
                           ws=fake(at("ws"), 0, dtype=torch.uint8), out=rows("out", 4), dev_err=err)
        elif name == "compact":
            kv_compact(c, table, one, fake(at("nodes"), 2, 4), two, length=fake(at("length"), 2), dev_err=err)
        elif name == "fork":
            kv_fork(c, refs, table, one, two, dev_err=err)
        elif name == "resize":
            kv_resize(c, refs, table, one, two, ws=fake(at("ws"), 0, dtype=torch.uint8), dev_err=err)
        else:
            kv_rotate(rows("q", 4), rows("k", 2), fake(at("pos"), 5), fake(at("turns"), 16, dtype=torch.int64), q_out=rows("q_out", 4),
                      k_out=rows("k_out", 2))


ARGUMENTS = {"tree": ["q", "seq", "pos", "table", "one", "mask", "ws", "out", "dev_err"],
             "compact": ["table", "one", "nodes", "two", "length", "dev_err"], "fork": ["refs", "table", "one", "two", "dev_err"],
             "resize": ["refs", "table", "one", "two", "ws", "dev_err"], "rotate": ["k", "pos", "turns", "q_out", "k_out"]}


@pytest.mark.parametrize("name", list(ARGUMENTS))
def test_tensors_on_another_device_are_refused(name):
    for arg in ARGUMENTS[name]:
        for device in ("cuda:1", "cpu"):
            with pytest.raises(ValueError, match="device"):
                fake_call(name, **{arg: device})


def test_rotate_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        kv_rotate(torch.zeros(2, 2, 64, dtype=torch.bfloat16), None, torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.int64))


# ------------------------------------------------------------------ the reference against closed forms

def test_reference_rotation_keeps_lengths_and_products():
    """Products of a rotated query and key depend on the distance only; backward undoes forward."""
    turns = [int(x) % 2 ** 64 for x in M.turns_of(frequencies(32))]
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(1, 1, 40, generator=g).double(), torch.randn(1, 1, 40, generator=g).double()
    for inter in (False, True):
        got = []
        for a, b in ((100, 90), (10 ** 9 + 10, 10 ** 9)):
            x, _ = M.rotate(q, torch.tensor([a]), turns, 1.0, 8, inter, False)
            y, _ = M.rotate(k, torch.tensor([b]), turns, 1.0, 8, inter, False)
            got.append(float((x * y).sum()))
            back, _ = M.rotate(x, torch.tensor([a]), turns, 1.0, 8, inter, True)
            assert float((back - q).abs().max()) < 1e-12
        assert abs(got[0] - got[1]) < 1e-9
