"""Host-side tests of the 4-bit operators' Python objects: what a changed field of a cache or a weight leads to. The tensors are
CPU ones whose missing device is let through, so that the descriptors can be looked at without a GPU; no call is made."""

import copy
import pickle

import pytest
import torch

from ternary_weight_only_tern_b200 import api


@pytest.fixture
def on_cpu(monkeypatch):
    """The binding's check of a tensor without its device."""
    def need(t, dtype, name, ndim=2):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(name)
        if t.dim() != ndim or not t.is_contiguous():
            raise ValueError(name)
    monkeypatch.setattr(api, "_need", need)


def pool(pages=3, heads=2, blocks=4, D=64):
    return torch.zeros((pages, heads, blocks, 18 * D), dtype=torch.uint8)


def described(cache):
    c = cache._c
    return c.pool, c.pages, c.page, c.kv_heads, c.head_dim


def test_another_pool_takes_the_place_of_the_first(on_cpu):
    cache = api.PagedCache(pool())
    cache._ws[(1, 1, 4, 9, 0, 0)] = 123                  # a size that was asked for
    for p, sizes in ((pool(pages=7), (7, 64, 2, 64)), (pool(heads=5, blocks=1, D=128), (3, 16, 5, 128))):
        cache.pool = p
        assert described(cache) == (p.data_ptr(), *sizes)
        assert (cache.pages, cache.page, cache.kv_heads, cache.head_dim) == sizes
        assert cache.pool is p and cache.nbytes() == p.numel() and not cache._ws
        assert cache._ref._obj is cache._c               # the reference that calls pass


def test_a_pool_that_cannot_be_one_is_refused_and_changes_nothing(on_cpu):
    p = pool()
    cache = api.PagedCache(p)
    before = described(cache)
    for bad, error in ((pool(D=96), ValueError), (pool()[:0], ValueError), (pool().half(), TypeError), (pool()[0], ValueError),
                       (pool(D=128)[..., ::2], ValueError), (None, TypeError)):
        with pytest.raises(error):
            cache.pool = bad
        assert described(cache) == before and cache.pool is p


@pytest.mark.parametrize("name", ["pages", "page", "kv_heads", "head_dim", "_c"])
def test_the_sizes_are_the_pools(on_cpu, name):
    cache = api.PagedCache(pool())
    with pytest.raises(AttributeError, match=name):
        setattr(cache, name, 4)
    assert cache.kv_heads == 2
    cache.layer = 7                                      # a user's own
    assert cache.layer == 7


def test_a_copy_of_a_cache_describes_its_own_pool(on_cpu):
    cache = api.PagedCache(pool())
    for twin in (copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        assert twin.pool.data_ptr() != cache.pool.data_ptr() and twin._c.pool == twin.pool.data_ptr()


def weight(N=40, K=256, group=64, offset=True):
    strips = -(-N // 16)
    half = lambda: torch.zeros((strips, K // group, 16), dtype=torch.float16)  # noqa: E731
    return api.NibWeight(N, K, group, torch.zeros((strips, K // 128, 256), dtype=torch.int32), half(), half() if offset else None)


def test_a_changed_field_reaches_the_descriptor(on_cpu):
    w = weight()
    first = w.c_struct()
    assert w.c_struct() is first                         # remembered
    w.codes = torch.ones_like(w.codes)
    assert w.c_struct().codes == w.codes.data_ptr()
    w.mu = None
    assert not w.c_struct().mu
    w.static = True
    assert w.c_struct().flags == 1
    w.N = 48                                             # as many strips
    assert w.c_struct().N == 48


@pytest.mark.parametrize("name,value,error", [
    ("N", 49, ValueError), ("K", 384, ValueError), ("K", 200, ValueError), ("group", 128, ValueError), ("group", 16, ValueError), ("N", 0, ValueError),
    ("codes", torch.zeros((2, 2, 256), dtype=torch.int32), ValueError), ("codes", torch.zeros((3, 2, 256), dtype=torch.uint8), TypeError),
    ("scale", torch.zeros((3, 2, 16), dtype=torch.float16), ValueError), ("scale", None, TypeError),
    ("scale", torch.zeros((3, 16, 4), dtype=torch.float16).transpose(1, 2), ValueError),
    ("mu", torch.zeros((3, 4, 16), dtype=torch.float32), TypeError)])
def test_a_field_that_does_not_fit_is_refused_at_the_next_use(on_cpu, name, value, error):
    """Sizes and tensors are assigned one after another, so they are held to each other when the weight is used."""
    w = weight()
    w.c_struct()
    good = getattr(w, name)
    setattr(w, name, value)
    for _ in range(2):
        with pytest.raises(error):
            w.c_struct()
    setattr(w, name, good)
    w.c_struct()


def test_a_weight_made_of_right_shapes_is_checked_again_once_changed(on_cpu):
    w = api._nib_empty(40, 256, 64, True, torch.zeros(1))
    w.c_struct()
    w.N = 64
    with pytest.raises(ValueError, match="codes"):
        w.c_struct()


def other_weight():
    t = torch.zeros
    return api.TernWeight(16, 128, t((16, 8), dtype=torch.int32), t((16, 1), dtype=torch.float16), t(0, dtype=torch.int32),
                          t(16, dtype=torch.int32), t((0, 8), dtype=torch.int32), t((0, 1), dtype=torch.float16))


@pytest.mark.parametrize("w", [None, 3, torch.zeros((16, 128), dtype=torch.float16), other_weight()], ids=["None", "number", "dense", "ternary"])
def test_what_is_no_nib_weight_is_refused_by_name(w):
    x = torch.zeros((1, 128), dtype=torch.float16)
    for call in (lambda: api.nib_linear(x, w), lambda: api.nib_dequant(w), lambda: api.nib_workspace_bytes(w, 1)):
        with pytest.raises(TypeError, match="NibWeight"):
            call()


@pytest.mark.parametrize("cache", [None, pool(), weight], ids=["None", "pool", "function"])
def test_what_is_no_cache_is_refused_by_name(cache):
    x, i = torch.zeros((1, 1, 2, 64), dtype=torch.float16), torch.zeros((1, 1), dtype=torch.int32)
    for call in (lambda: api.cache_append(cache, x, x, i, i[0]), lambda: api.cache_read(cache, i, i[0], 1),
                 lambda: api.cache_attention(x, cache, i, i[0])):
        with pytest.raises(TypeError, match="PagedCache"):
            call()


@pytest.mark.parametrize("t", [None, [1, 2], 3.0])
def test_what_is_no_tensor_is_refused_as_one(on_cpu, t):
    cache, i = api.PagedCache(pool()), torch.zeros((1, 1), dtype=torch.int32)
    for call in (lambda: api.nib_fit(t), lambda: api.nib_pack(t, t), lambda: api.nib_linear(t, weight()), lambda: api.cache_append(cache, t, t, i, i[0]),
                 lambda: api.cache_read(cache, t, i[0], 1), lambda: api.cache_attention(t, cache, i, i[0])):
        with pytest.raises(TypeError):
            call()
