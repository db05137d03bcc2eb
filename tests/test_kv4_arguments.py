"""Whole numbers that 32 bits do not hold are refused by KV4Cache before anything is called."""
import os
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rt():
    from accelerator_decode_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from accelerator_decode_gb300 import runtime
    return runtime


@pytest.fixture()
def cache(rt, monkeypatch):
    """A cache object without a device; every call to the library is a failure of the test."""
    c = object.__new__(rt.KV4Cache)
    c.index, c.device = -1, torch.device("cpu")           # get_device() of a CPU tensor
    c.n_slots, c.capacity, c.track, c.num_q_heads, c.num_kv_heads, c.head_dim = 4, 100, True, 2, 1, 64
    c._ta, c._tb, c._pa, c._pb, c.h = rt._g4.g4_kv4_tensor(), rt._g4.g4_kv4_tensor(), None, None, None
    c._stream = lambda stream: 0

    def called(name):
        def f(*a):
            raise AssertionError(f"{name} was called with {a}")
        return f

    monkeypatch.setattr(rt._g4, "lib", types.SimpleNamespace(**{
        n: called(n) for n in ("g4_kv4_append", "g4_kv4_read", "g4_kv4_account", "g4_kv4_attend", "g4_kv4_evict",
                               "g4_kv4_create")}))
    return c


LONG = [2 ** 31, 2 ** 32, 2 ** 32 + 1, -2 ** 31 - 1, 2 ** 64 + 5]


@pytest.mark.parametrize("v", LONG)
def test_long_numbers_are_refused(rt, cache, v):
    s = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 1, 2, 64)
    for call in (lambda: cache.attend(q, s, s, window=v), lambda: cache.evict(s, s, v), lambda: cache.evict(s, s, 5, v),
                 lambda: cache.read(s, s, v), lambda: cache.account(s, s, v)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


@pytest.mark.parametrize("v", LONG)
@pytest.mark.parametrize("name", ["n_slots", "capacity", "num_q_heads", "num_kv_heads", "head_dim", "max_q_len", "page_size"])
def test_long_sizes_are_refused(rt, cache, name, v):
    good = dict(n_slots=4, capacity=100, num_q_heads=2, num_kv_heads=1, head_dim=64)
    with pytest.raises(ValueError, match="32 bits"):
        rt.KV4Cache(**{**good, name: v}, device=0)


def test_numbers_that_are_not_whole_are_refused(rt, cache):
    s = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        cache.evict(s, s, 5.5)
    with pytest.raises(TypeError):
        cache.attend(torch.zeros(2, 1, 2, 64), s, s, window=2.0)
