"""Host-side validation of the 4-bit operators: every refusal here comes before a launch, so no GPU is touched;
and the binding's own checks."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import nib_oracle as no
from ternary_weight_only_tern_b200 import _lib, api

S = _lib.STATUS
F = 1 << 20              # an aligned non-null address that is never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from ternary_weight_only_tern_b200 import build
        build.build()
    return _lib.load()


def nib(N=64, K=256, group=128, flags=0, codes=F, scale=F, mu=None):
    return _lib.TernNibWeightC(N, K, group, flags, codes, scale, mu)


def kv(pool=F, pages=4, page=64, heads=2, D=128):
    return _lib.TernCacheC(pool, pages, page, heads, D)


BAD_NIB = [(dict(N=0), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=200), "SHAPE"), (dict(group=16), "SHAPE"),
           (dict(group=256), "SHAPE"), (dict(N=(1 << 22) + 1), "SHAPE"), (dict(K=(1 << 20) + 128), "SHAPE"),
           (dict(codes=None), "NULL"), (dict(scale=None), "NULL"), (dict(codes=F + 4), "ALIGN"),
           (dict(scale=F + 2), "ALIGN"), (dict(mu=F + 8), "ALIGN")]


@pytest.mark.parametrize("kw,err", BAD_NIB)
def test_a_bad_weight_is_refused_everywhere(lib, kw, err):
    w = ctypes.byref(nib(**kw))
    e = S["TERN_ERR_" + err]
    assert lib.tern_nib_linear(w, F, 1, F * 4, None, 0, None) == e
    assert lib.tern_nib_dequant(w, F * 4, None) == e
    assert lib.tern_nib_linear_workspace_bytes(w, 1) == 0


def test_nib_linear_refusals(lib):
    call = lambda x=F, M=1, y=F * 4, ws=None, wsb=0, w=nib(): lib.tern_nib_linear(  # noqa: E731
        ctypes.byref(w) if w is not None else None, x, M, y, ws, wsb, None)
    assert call(w=None) == S["TERN_ERR_NULL"]
    assert call(M=0, x=None, y=None) == S["TERN_OK"]
    assert call(M=-1) == S["TERN_ERR_SHAPE"]
    assert call(M=(1 << 31) + 1) == S["TERN_ERR_SHAPE"]
    assert call(x=None) == S["TERN_ERR_NULL"]
    assert call(y=None) == S["TERN_ERR_NULL"]
    assert call(x=F + 2) == S["TERN_ERR_ALIGN"]
    assert call(y=F * 4 + 8) == S["TERN_ERR_ALIGN"]
    assert call(y=F) == S["TERN_ERR_SHAPE"]                      # x and y overlap
    assert call(ws=F * 8 + 4, wsb=1 << 20) == S["TERN_ERR_ALIGN"]
    for M in (1, 5, 16, 17, 64, 100, 4096):
        for N, K in ((64, 256), (4096, 4096), (12288, 4096), (4096, 12288)):
            w = nib(N=N, K=K)
            need = lib.tern_nib_linear_workspace_bytes(ctypes.byref(w), M)
            assert need % 256 == 0
            if need:
                assert call(w=w, M=M, y=F * 4096) == S["TERN_ERR_WORKSPACE"]
                assert call(w=w, M=M, y=F * 4096, ws=F * 8, wsb=need - 1) == S["TERN_ERR_WORKSPACE"]


def test_nib_fit_and_pack_refusals(lib):
    fit = lambda W=F, N=4, K=256, g=128, off=1, c=F * 2, s=F * 3, m=F * 4: lib.tern_nib_fit(W, N, K, g, off, c, s, m, None)  # noqa: E731
    assert fit(K=200) == S["TERN_ERR_SHAPE"]
    assert fit(N=0) == S["TERN_ERR_SHAPE"]
    assert fit(g=48) == S["TERN_ERR_SHAPE"]
    assert fit(m=None) == S["TERN_ERR_NULL"]
    assert fit(W=None) == S["TERN_ERR_NULL"]
    assert fit(c=F + 8) == S["TERN_ERR_ALIGN"]
    pack = lambda c=F, s=F, m=None, N=4, K=256, g=64, oc=F * 2, os_=F * 3, om=None: lib.tern_nib_pack(c, s, m, N, K, g, oc, os_, om, None)  # noqa: E731
    assert pack(K=100) == S["TERN_ERR_SHAPE"]
    assert pack(m=F) == S["TERN_ERR_NULL"]
    assert pack(om=F) == S["TERN_ERR_NULL"]
    assert pack(c=None) == S["TERN_ERR_NULL"]
    assert pack(s=F + 2) == S["TERN_ERR_ALIGN"]


BAD_CACHE = [(dict(pages=0), "SHAPE"), (dict(page=0), "SHAPE"), (dict(page=24), "SHAPE"), (dict(page=65552), "SHAPE"),
             (dict(heads=0), "SHAPE"), (dict(D=96), "SHAPE"), (dict(pool=None), "NULL"), (dict(pool=F + 8), "ALIGN")]


@pytest.mark.parametrize("kw,err", BAD_CACHE)
def test_a_bad_cache_is_refused_everywhere(lib, kw, err):
    c, e = ctypes.byref(kv(**kw)), S["TERN_ERR_" + err]
    assert lib.tern_cache_append(c, F, F, 1, 1, F, 4, F, None, None) == e
    assert lib.tern_cache_read(c, F, F, 1, 1, F, 4, F, None, None) == e
    heads = kw.get("heads", 2) or 2
    assert lib.tern_cache_attention(c, F, 1, 1, heads, F, 4, F, None, 1.0, 0, 0, F * 2, None, 0, None) == e
    assert lib.tern_cache_attention_workspace_bytes(c, 1, 1, heads, 1 << 20, 0, 0) == 0


@pytest.mark.parametrize("name", ["tern_cache_append", "tern_cache_read"])
def test_append_and_read_refusals(lib, name):
    c = kv()
    call = lambda k=F, v=F, B=2, T=3, table=F, width=4, start=F: getattr(lib, name)(  # noqa: E731
        ctypes.byref(c), k, v, B, T, table, width, start, None, None)
    assert getattr(lib, name)(None, F, F, 1, 1, F, 4, F, None, None) == S["TERN_ERR_NULL"]
    assert call(B=0, k=None) == S["TERN_OK"]
    assert call(T=0, v=None) == S["TERN_OK"]
    for kw in (dict(B=-1), dict(T=-1), dict(width=-1), dict(B=65536), dict(T=(1 << 24) + 1), dict(width=(1 << 24) + 1)):
        assert call(**kw) == S["TERN_ERR_SHAPE"], kw
    for kw in (dict(k=None), dict(v=None), dict(table=None), dict(start=None)):
        assert call(**kw) == S["TERN_ERR_NULL"], kw
    for kw in (dict(k=F + 2), dict(v=F + 8)):
        assert call(**kw) == S["TERN_ERR_ALIGN"], kw


def test_attention_refusals(lib):
    c = kv()
    call = lambda q=F, B=2, T=3, H=8, table=F, width=400, lens=F, scale=0.1, window=0, sinks=0, o=F * 2, ws=F * 4, wsb=1 << 40: \
        lib.tern_cache_attention(ctypes.byref(c), q, B, T, H, table, width, lens, None, scale, window, sinks, o, ws, wsb, None)  # noqa: E731
    assert call(B=0, q=None) == S["TERN_OK"]
    assert call(T=0, o=None) == S["TERN_OK"]
    for kw in (dict(B=-1), dict(T=65), dict(T=-1), dict(H=0), dict(H=7), dict(width=-1), dict(window=-1), dict(sinks=-1),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.1e4), dict(o=F + 256)):
        assert call(**kw) == S["TERN_ERR_SHAPE"], kw
    for kw in (dict(q=None), dict(o=None), dict(lens=None), dict(table=None)):
        assert call(**kw) == S["TERN_ERR_NULL"], kw
    for kw in (dict(q=F + 2), dict(o=F * 2 + 8), dict(ws=F * 4 + 4)):
        assert call(**kw) == S["TERN_ERR_ALIGN"], kw
    size = lambda width, window=0, sinks=0: lib.tern_cache_attention_workspace_bytes(  # noqa: E731
        ctypes.byref(c), 2, 3, 8, width, window, sinks)
    need = size(400)
    assert size(400, -1) == size(400, 0, -1) == size(-1) == 0
    assert size(4) == size(400, 100) == size(400, 1, 5) == 0           # no sequence can be long
    assert size(400, 2**63 - 1, 2**63 - 1) == size(400, 100, 10**6) == need
    if need:
        assert call(ws=None) == S["TERN_ERR_WORKSPACE"]
        assert call(wsb=need - 1) == S["TERN_ERR_WORKSPACE"]


def test_the_binding_checks_its_arguments():
    """On CPU tensors: what is refused for its device, type, shape or order before the library is called."""
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    with pytest.raises(TypeError):
        api.nib_fit(h(16, 128))
    with pytest.raises(TypeError):
        api.nib_linear(h(1, 128), None)
    with pytest.raises(TypeError):
        api.PagedCache(torch.zeros((1, 1, 1, 18 * 64), dtype=torch.uint8))
    with pytest.raises(ValueError, match="group"):
        api.NibWeight(16, 128, 48, h(1), h(1))
    with pytest.raises(ValueError, match="128"):
        api.NibWeight(16, 100, 32, h(1), h(1))
    with pytest.raises(ValueError, match="multiple of 16"):
        api.PagedCache.empty(2, 24, 1, 64)


def test_oracle_layouts_hold_every_code_once():
    """The oracle's own words give back each code (a planted wrong nibble order does not)."""
    rng = np.random.default_rng(0)
    c = rng.integers(0, 16, size=(32, 256), dtype=np.uint8)
    w = no.nib_words(c)
    def code(r, k, order=lambda i: i // 2 + 4 * (i % 2)):  # noqa: E306
        kk = k % 128
        word = ((r % 16 // 8 * 8 + r % 8) * 4 + kk % 32 // 8) * 4 + kk // 32
        return w[r // 16, k // 128, word] >> np.uint32(4 * order(kk % 8)) & 15
    places = [(int(r), int(k)) for r, k in zip(rng.integers(0, 32, 400), rng.integers(0, 256, 400))]
    assert all(code(r, k) == c[r, k] for r, k in places)
    assert any(code(r, k, lambda i: i) != c[r, k] for r, k in places)


def test_oracle_fit_meets_the_formula_and_halves_the_step():
    """Every weight within half a step of its value (and what fp16's rounding of step and offset adds)."""
    rng = np.random.default_rng(1)
    W = (rng.standard_normal((8, 256)) * 0.05).astype(np.float16)
    for offset in (False, True):
        c, s, mu = no.nib_fit(W, 64, offset)
        err = np.abs(no.nib_values(c, s, mu) - W.astype(np.float64)).reshape(8, 4, 64)
        step = s.astype(np.float64)[..., None]
        assert (err <= 0.5 * step + 16 * step * 2.0**-11 + np.abs(W).max() * 2.0**-11).all()
        assert c.min() >= 0 and c.max() <= 15 and len(np.unique(c)) == (16 if offset else 15)


def test_the_most_tokens_of_a_call(lib):
    w = ctypes.byref(nib(N=16, K=128))
    call = lambda M: lib.tern_nib_linear(w, None, M, F, None, 0, None)  # noqa: E731
    assert call(1 << 22) == S["TERN_ERR_NULL"]                   # of a size that is taken
    assert call((1 << 22) + 1) == S["TERN_ERR_SHAPE"]
