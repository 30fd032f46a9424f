"""The Python face of the key/value cache calls on the host (no GPU): what reaches the library, what is refused."""
import copy
import pickle

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
