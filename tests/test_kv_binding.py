"""The Python face of the key/value cache calls on the host (no GPU): what reaches the library, what is refused."""
import copy
import pickle
from unittest import mock

import pytest
import torch

from bit_routed_expert_gb300 import KvCache, _lib, kv_append, kv_attend, kv_read, kv_select


class Recorder:
    """Stands for the native binding: which tensors a call could see of its cache."""

    def __init__(self):
        self.seen = None

    def check(self, cache):
        pass

    def _call(self, cache, *args):
        self.seen = cache.pages, cache.bounds, cache.bound_exp
        return 0, None, None

    read = select = attend = _call

    def append(self, cache, *args):
        self._call(cache)
        return 0


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(_lib, "load_kv", lambda: r)
    return r


def fields(n):
    return (torch.zeros((n, 2, 128 * 65), dtype=torch.uint8), torch.zeros((n, 2, 2, 64), dtype=torch.int8),
            torch.zeros((n, 2), dtype=torch.int8))


def calls(c):
    yield lambda: kv_append(c, 0, 0, 0, 0, 0)
    yield lambda: kv_read(c, 0, 0, 0)
    yield lambda: kv_select(0, c, 0, 0, 0, 4)
    yield lambda: kv_attend(0, c, 0, 0, 0, 0)


def sees(recorder, c):
    for call in calls(c):
        recorder.seen = None
        call()
        if not (recorder.seen[0] is c.pages and recorder.seen[1] is c.bounds and recorder.seen[2] is c.bound_exp):
            return False
    return True


def test_calls_take_the_cache_as_it_is(recorder):
    """After its fields were assigned (it grew), copied deep and flat, and pickled."""
    c = KvCache(*fields(3))
    assert sees(recorder, c) and (c.n_pages, c.n_kv_heads, c.head_dim) == (3, 2, 64)
    c.pages, c.bounds, c.bound_exp = fields(5)
    assert sees(recorder, c) and c.n_pages == 5
    for other in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert sees(recorder, other)
        assert other.pages.data_ptr() != c.pages.data_ptr() and other.bounds.data_ptr() != c.bounds.data_ptr()
    assert sees(recorder, copy.copy(c)) and copy.copy(c).pages is c.pages


def test_no_cache_is_refused():
    binding = _lib.load_kv()
    for bad in (None, 0, 1 << 20, object(), torch.zeros(3)):
        with pytest.raises(ValueError, match="not a cache"):
            binding.check(bad)
        with pytest.raises(ValueError, match="not a cache"):
            binding.read(bad, 0, 0, 0, None, None, None, None)


def fake(device, *shape, dtype=torch.int32):
    """A tensor that says that it is on `device`, without memory."""
    return torch.empty(shape, dtype=dtype, device=device)


def fake_call(name, cache_devices=("cuda:0",) * 3, **where):
    """One call whose tensors are all on cuda:0 but for those named in `where`."""
    at = lambda n: where.get(n, "cuda:0")  # noqa: E731
    # (a fake tensor would begin with a real one on its device, where there are devices)
    with mock.patch("torch.cuda.is_available", lambda: False), torch._subclasses.fake_tensor.FakeTensorMode():
        d = cache_devices
        c = KvCache(fake(d[0], 3, 2, 128 * 65, dtype=torch.uint8), fake(d[1], 3, 2, 2, 64, dtype=torch.int8),
                    fake(d[2], 3, 2, dtype=torch.int8))
        tokens = fake(at("seq"), 5), fake(at("pos"), 5), fake(at("table"), 1, 3)
        rows = lambda n, h: fake(at(n), 5, h, 64, dtype=torch.bfloat16)  # noqa: E731
        err = fake(at("dev_err"), 1)
        ids = fake(at("ids"), 5, 2, 4)
        if name == "append":
            kv_append(c, rows("k", 2), rows("v", 2), *tokens, dev_err=err)
        elif name == "read":
            kv_read(c, *tokens, k_out=rows("k_out", 2), v_out=rows("v_out", 2), dev_err=err)
        elif name == "select":
            kv_select(rows("q", 4), c, *tokens, 4, ids=ids, scores=fake(at("scores"), 5, 2, 4, dtype=torch.float32),
                      ws=fake(at("ws"), 0, dtype=torch.uint8), dev_err=err)
        else:
            kv_attend(rows("q", 4), c, *tokens, ids, out=rows("out", 4), ws=fake(at("ws"), 0, dtype=torch.uint8),
                      lse=fake(at("lse"), 5, 4, dtype=torch.float32), dev_err=err)


ARGUMENTS = {"append": ["k", "v"], "read": ["k_out", "v_out"], "select": ["q", "ids", "scores", "ws"],
             "attend": ["q", "ids", "out", "lse", "ws"]}


@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
@pytest.mark.parametrize("name", list(ARGUMENTS))
def test_tensors_on_another_device_are_refused(name, device):
    """Before anything looks at an address: a launch would take one device's pointers to another."""
    for arg in ARGUMENTS[name] + ["seq", "pos", "table", "dev_err"]:
        with pytest.raises(ValueError, match="device of the cache's pages, cuda:0: there is one on " + device):
            fake_call(name, **{arg: device})


def test_a_cache_on_two_devices_is_refused():
    for i in range(1, 3):
        d = ["cuda:0"] * 3
        d[i] = "cuda:1"
        with pytest.raises(ValueError, match="device of the cache's pages"):
            fake_call("append", cache_devices=d)


@pytest.mark.parametrize("kw", [{"k": 2 ** 32 + 4}, {"n_sink": 2 ** 32}, {"n_local": 2 ** 32 + 1}, {"k": -2 ** 31 - 1},
                                {"k": 2 ** 64 + 4}, {"n_sink": -2 ** 63 - 1}])
def test_numbers_outside_32_bits_are_refused(kw):
    """Not cut to the 32 bits that the library takes, where 2^32 + 4 would be 4."""
    with torch._subclasses.fake_tensor.FakeTensorMode(), mock.patch("torch.cuda.is_available", lambda: False):
        c = KvCache(fake("cuda:0", 3, 2, 128 * 65, dtype=torch.uint8), fake("cuda:0", 3, 2, 2, 64, dtype=torch.int8),
                    fake("cuda:0", 3, 2, dtype=torch.int8))
        tokens = fake("cuda:0", 5), fake("cuda:0", 5), fake("cuda:0", 1, 3)
        args = {"k": 4, "n_sink": 1, "n_local": 1, **kw}
        with pytest.raises(ValueError, match=next(iter(kw)) + " is outside 32 bits"):
            kv_select(fake("cuda:0", 5, 4, 64, dtype=torch.bfloat16), c, *tokens, args.pop("k"), **args)
        with pytest.raises(ValueError, match="k must be a whole number"):
            kv_select(fake("cuda:0", 5, 4, 64, dtype=torch.bfloat16), c, *tokens, 4.0)


@pytest.mark.parametrize("T,B,N,name", [(2 ** 32 + 1, 1, 3, "T"), (5, 2 ** 32 + 1, 3, "B"), (5, 1, 2 ** 32 + 3, "N")])
def test_sizes_outside_32_bits_are_refused(T, B, N, name):
    with torch._subclasses.fake_tensor.FakeTensorMode(), mock.patch("torch.cuda.is_available", lambda: False):
        c = KvCache(fake("cuda:0", 3, 2, 128 * 65, dtype=torch.uint8), fake("cuda:0", 3, 2, 2, 64, dtype=torch.int8),
                    fake("cuda:0", 3, 2, dtype=torch.int8))
        with pytest.raises(ValueError, match=name + " is outside 32 bits"):
            kv_read(c, fake("cuda:0", T), fake("cuda:0", T), fake("cuda:0", B, N))
        with pytest.raises(ValueError, match="n_pages is outside 32 bits"):
            KvCache(fake("cuda:0", 2 ** 32 + 3, 2, 128 * 65, dtype=torch.uint8),
                    fake("cuda:0", 2 ** 32 + 3, 2, 2, 64, dtype=torch.int8), fake("cuda:0", 2 ** 32 + 3, 2, dtype=torch.int8))


def test_a_binding_of_another_version_is_built_again(monkeypatch, tmp_path):
    """Not loaded: it reads PyTorch's own structures."""
    from bit_routed_expert_gb300 import build
    right = build.binding_is_current() and open(build.BUILT_FOR).read()
    assert right and torch.__version__ in right
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_kv.so"))
    monkeypatch.setattr(build, "BUILT_FOR", str(tmp_path / "_kv.built_for"))
    monkeypatch.setattr(_lib, "_kv", None)

    def built(*a, **kw):
        raise RuntimeError("built again")

    monkeypatch.setattr(build, "build", built)
    for so, version in ((False, None), (True, None), (True, right + "x"), (True, "torch 1.0"), (False, right)):
        for name, there in (("_kv.so", so), ("_kv.built_for", version)):
            (tmp_path / name).unlink(missing_ok=True)
            if there:
                (tmp_path / name).write_text(there if isinstance(there, str) else "")
        assert not build.binding_is_current()
        with pytest.raises(RuntimeError, match="built again"):
            _lib.load_kv()
    (tmp_path / "_kv.so").write_text("")
    assert build.binding_is_current()
