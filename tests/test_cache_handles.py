"""CPU checks of the handles that the paged cache's calls take, with a stand-in for the compiled marshaller."""
import copy
import gc
import pickle

import pytest
import torch

import ring_attn_gb300 as ra

COPIES = [copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x)), copy.copy]


@pytest.fixture
def calls(monkeypatch):
    """The arguments of every marshalled call; nothing is launched."""
    seen = []

    class Ext:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or (0, None, None)

    monkeypatch.setattr(ra, "_EXT", Ext())
    return seen


def handle():
    """A KVCache without device tensors."""
    cache = ra.KVCache.__new__(ra.KVCache)
    cache._call, cache.device, cache.scale = (0, -1, 1, 64), torch.device("cpu"), 0.125
    return cache


def addresses(x):
    """Every address that an argument names, as a tensor or as a number."""
    if isinstance(x, torch.Tensor):
        return {x.data_ptr()}
    if isinstance(x, (tuple, list)):
        return set().union(*map(addresses, x))
    return {x} if isinstance(x, int) else set()


@pytest.mark.parametrize("duplicate", COPIES)
@pytest.mark.parametrize("name", ["append", "read", "fwd"])
def test_a_copied_cu_seqlens_names_its_own_arrays(calls, duplicate, name):
    first = ra.CuSeqlens([0, 3, 10], "cpu")
    before = {first.dev.data_ptr(), first.host.data_ptr()}
    cu = duplicate(first)
    if duplicate is not copy.copy:
        assert not before & {cu.dev.data_ptr(), cu.host.data_ptr()}
    args = {"append": (None, None, handle(), None, None, cu), "read": (handle(), None, None, cu),
            "fwd": (None, handle(), None, None, cu)}[name]
    getattr(ra, "ring_attn_cache_" + name)(*args)
    got = set().union(*map(addresses, calls[-1][1]))
    assert {cu.dev.data_ptr(), cu.host.data_ptr()} <= got
    if duplicate is not copy.copy:
        assert not before & got  # a call on the copy names nothing of the first
    del first
    gc.collect()
    assert cu.host.tolist() == [0, 3, 10]


def test_a_cu_seqlens_with_other_arrays(calls):
    """The calls take the arrays that the object holds when they are made, as the varlen calls do."""
    cu, other = ra.CuSeqlens([0, 3, 10], "cpu"), ra.CuSeqlens([0, 4, 9], "cpu")
    cu.dev, cu.host = other.dev, other.host
    ra.ring_attn_cache_read(handle(), None, None, cu)
    assert {other.dev.data_ptr(), other.host.data_ptr()} <= set().union(*map(addresses, calls[-1][1]))


def test_a_kv_cache_keeps_the_tensors_that_it_describes(monkeypatch):
    """Replacing one would leave its description, addresses included, to memory that nobody holds."""
    u8, f8 = torch.zeros(2, 1, 16, 32, dtype=torch.uint8), torch.zeros(2, 1, 16, 4, dtype=torch.uint8).view(torch.float8_e4m3fn)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    cache = ra.KVCache(u8, f8, u8.clone(), f8.clone())
    monkeypatch.undo()
    for name in ("k", "k_scale", "v", "v_scale"):
        x = getattr(cache, name)
        with pytest.raises(AttributeError):
            setattr(cache, name, x.clone())
        assert getattr(cache, name) is x and getattr(cache._c, name).data == x.data_ptr()


@pytest.mark.parametrize("duplicate", COPIES)
def test_a_copied_kv_cache_describes_its_own_tensors(monkeypatch, duplicate):
    monkeypatch.setattr(ra.torch.Tensor, "is_cuda", property(lambda self: True))
    both = torch.arange(2 * 16 * 64, dtype=torch.int32).to(torch.uint8).view(2, 1, 16, 64)  # keys and values in one allocation
    scales = [torch.full((2, 1, 16, 4), x, dtype=torch.uint8).view(torch.float8_e4m3fn) for x in (7, 8)]
    first = ra.KVCache(both[..., :32], scales[0], both[..., 32:], scales[1])
    made = duplicate(first)
    assert made is not first and made._c is not first._c and made._call[1:] == first._call[1:]
    for name in ("k", "k_scale", "v", "v_scale"):
        x, y, t = getattr(first, name), getattr(made, name), getattr(made._c, name)
        assert t.data == y.data_ptr() and list(t.stride) == list(y.stride()) == list(x.stride())
        assert (x.data_ptr() == y.data_ptr()) == (duplicate is copy.copy)
        assert x.dtype == y.dtype and torch.equal(x.view(torch.uint8), y.view(torch.uint8))
