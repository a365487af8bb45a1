"""GPU tests of the 4-bit cache beside those of test_cache_gpu.py, whose oracle, inputs and tolerance they use: the two paths of the
attention (a CTA per segment where none can be long, an even split with a join where some can), what lies around their
buffers, and a pool that takes the place of another."""

import numpy as np
import pytest
import torch

from oracle import nib_oracle as no
from ternary_weight_only_tern_b200 import api
from test_cache_gpu import check_attention, cuda, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T,G", [(64, 1, 4), (128, 1, 2), (128, 3, 4)])
def test_short_segments_over_several_waves_of_ctas(D, T, G):
    """Many more CTAs than the SMs hold at once, most of them of one to three blocks, whose lens and tables the SM has seen
    before: every launch of them gives the same bits, and no bounded wait runs out."""
    rng = np.random.default_rng(D + T)
    lens = [int(n) for n in rng.integers(0, 70, 400)]
    cache, table, K, V, _, _ = make(rng, lens, 16, 8, D, width=6)
    q = rng.standard_normal((400, T, 8 * G, D)).astype(np.float16)
    args = cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32))
    assert cache.workspace_bytes(400, T, 8 * G, 6) == 0                  # nothing is split
    first = api.cache_attention(*args)
    again = [api.cache_attention(*args) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in again)
    check_attention(first.cpu().numpy(), q, K, V, lens, [T] * 400, D**-0.5, 0, 0)
    from ternary_weight_only_tern_b200 import _lib
    assert _lib.load().tern_device_status(api._stream()) == 0


def test_a_cache_goes_on_in_a_larger_pool():
    """A pool replaced by a larger one that begins with the same pages: appends go there and the first is left alone."""
    rng = np.random.default_rng(31)
    lens = [40, 25]
    cache, table, K, V, _, _ = make(rng, lens, 16, 2, 64, spare=0, width=4)
    old = cache.pool
    kept = old.clone()
    q = rng.standard_normal((2, 1, 4, 64)).astype(np.float16)
    api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32)))
    cache.pool = torch.cat([old, torch.zeros_like(old)])
    for b, n in enumerate(lens):
        table[b, -(-n // 16)] = len(old) + b
    k, v = (rng.standard_normal((2, 10, 2, 64)).astype(np.float16) for _ in range(2))
    api.cache_append(cache, cuda(k), cuda(v), cuda(table), cuda(np.array(lens, np.int32)))
    assert torch.equal(old, kept)
    for b in range(2):
        K[b], V[b] = (np.concatenate([X[b], no.cache_values(*no.cache_quantise(x[b]))]) for X, x in ((K, k), (V, v)))
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32) + 10)).cpu().numpy()
    check_attention(o, q, K, V, [50, 35], [1, 1], 0.125, 0, 0)


def first_token_above(n, powers, D, scale, rng):
    """K, V of n tokens, one kv head, and a query of 4 heads: token 0 lies about `powers` powers of two above the others and its V is
    zero, so that the others, all about alike, are the whole result."""
    q = rng.standard_normal(D)
    k = rng.standard_normal((1, n, 1, D)) * 0.1
    k[0, 0, 0] = q * powers * np.log(2) / (scale * (q @ q))
    v = 4 + rng.standard_normal((1, n, 1, D))
    v[0, 0] = 0
    return k.astype(np.float16), v.astype(np.float16), np.repeat(q[None, None, None], 4, 2).astype(np.float16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,powers", [(9, 14), (9, 19), (30, 14), (30, 17), (30, 19), (30, 26), (30, 30), (600, 14), (600, 19), (600, 26), (5000, 19), (5000, 26),
                                      (131072, 19), (131072, 26)])
def test_tokens_far_below_the_first_one_keep_their_bits(n, powers, D):
    """Tolerance: a probability counts 2^7 at the maximum, so one of at least 2^-21 of it is a normal fp16 number and rounded by
    2^-11 of itself, as are V and the result; below that each is off by up to 2^-25 2^-7 of the maximum's. A score is off by at most
    D 2^-22 |q| |k| scale. (At 2^7 less, those of 2^-26 would all be zeros, and so would the result.)"""
    rng = np.random.default_rng(n + powers)
    scale, page = D**-0.5, 64
    k, v, q = first_token_above(n, powers, D, scale, rng)
    cache = api.PagedCache.empty(-(-n // page), page, 1, D)
    table = np.arange(-(-n // page), dtype=np.int32)[None]
    api.cache_append(cache, cuda(k), cuda(v), cuda(table), cuda(np.zeros(1, np.int32)))
    K, V = (no.cache_values(*no.cache_quantise(x[0])) for x in (k, v))
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array([n], np.int32))).cpu().numpy().astype(np.float64)[0, 0]
    s = scale * (K[:, 0] @ q[0, 0, 0].astype(np.float64))
    p = np.exp(s - s[0])
    low = np.count_nonzero(p < 2.0**-21)
    assert p[1:].max() < 2.0**(2 - powers)
    p /= p.sum()
    ref, mass = p @ V[:, 0], p @ np.abs(V[:, 0])
    qk = np.linalg.norm(q[0, 0, 0].astype(np.float64)) * np.linalg.norm(K[:, 0], axis=-1).max()
    tol = 2.0**-11 * np.abs(ref) + 2.0**-25 + (2 * 2.0**-11 + 2 * D * 2.0**-22 * qk * scale) * mass + low * 2.0**-32 * np.abs(V).max()
    err = np.abs(o - ref)
    assert (err <= tol).all(), f"{np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("scale", [128**-0.5, -(128**-0.5), 1e4, -7.0])
@pytest.mark.parametrize("n", [40, 700, 6000])
def test_scores_of_any_size_leave_a_result(n, scale):
    """Queries and keys near the ends of fp16's range: scores to base 2 of up to 1e9 (1e14 with the largest scale), whose last bits
    count far more than 1. One token is above all others by much more than a score's error (D 2^-22 |q| |k| scale: 2^-15 of the
    largest score), so each query's result is that token's V, rounded to fp16 for the product and so exact here."""
    rng = np.random.default_rng(n)
    D, heads, page = 128, 24, 64
    u = np.where(rng.random(D) < 0.5, -1.0, 1.0)
    c = rng.permutation(np.linspace(-1, 1, n))           # of the key along u; steps of at least 2^-12
    k = (c[:, None] * u * 60000.0).astype(np.float16)
    v = rng.integers(-50, 50, (n, D)).astype(np.float16)
    q = (np.where(np.arange(heads) % 2, 1.0, -1.0)[:, None] * np.ldexp(1000.0, -(np.arange(heads) // 2))[:, None] * u).astype(np.float16)
    cache = api.PagedCache.empty(-(-n // page), page, 1, D)
    table = np.arange(-(-n // page), dtype=np.int32)[None]
    api.cache_append(cache, cuda(k[None, :, None]), cuda(v[None, :, None]), cuda(table), cuda(np.zeros(1, np.int32)))
    K, V = (no.cache_values(*no.cache_quantise(x)) for x in (k, v))
    s = scale * (q.astype(np.float64) @ K.T)
    best = s.argmax(1)
    two = np.sort(s, 1)[:, -2:]
    error = D * 2.0**-22 * np.linalg.norm(q.astype(np.float64), axis=1) * np.linalg.norm(K, axis=1).max() * abs(scale)
    clear = two[:, 1] - two[:, 0] > 2 * error + 40       # the second token's share is below e^-40
    assert clear.sum() >= 8 and np.abs(s).max() > 3e8 / 1.5
    o = api.cache_attention(cuda(q[None, None]), cache, cuda(table), cuda(np.array([n], np.int32)), scale=scale).cpu().numpy()[0, 0]
    assert np.isfinite(o).all()
    assert np.array_equal(o[clear], V.astype(np.float16)[best[clear]])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hk,G,T,longest,width,split", [(3, 2, 4, 1, 9000, None, True), (2, 1, 3, 5, 9000, None, True), (3, 2, 2, 64, 3000, None, True),
                                                          (150, 8, 2, 1, 200, 60, True), (60, 5, 3, 7, 200, 60, True), (40, 3, 4, 1, 200, None, False),
                                                          (9, 3, 5, 6, 200, None, False)])
def test_attention_writes_its_rows_and_workspace_alone(B, Hk, G, T, longest, width, split, D):
    """Fewer and more segments than CTAs, split ones and such with a CTA of their own: a workspace of just the stated bytes (all NaN before)
    and the output lie between guard bytes, which stay as they are, as do the output's rows behind a sequence's queries."""
    rng = np.random.default_rng(B + T + D)
    lens = [longest] + [int(n) for n in rng.integers(0, longest, B - 1)]
    counts = [T] + [int(n) for n in rng.integers(0, T + 1, B - 1)]
    cache, table, K, V, _, _ = make(rng, lens, 32, Hk, D, width=width)
    H, W = Hk * G, table.shape[1]
    need = cache.workspace_bytes(B, T, H, W)
    assert (need > 0) == split
    q = rng.standard_normal((B, T, H, D)).astype(np.float16)
    n = q.size
    buf = torch.full((n + 256,), 7.5, dtype=torch.float16, device="cuda")
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    ws[256:256 + need] = 0xFF
    out = buf[128:128 + n].view(B, T, H, D)
    api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32)), counts=cuda(np.array(counts, np.int32)), out=out,
                        workspace=ws[256:256 + need])
    assert (buf[:128] == 7.5).all() and (buf[128 + n:] == 7.5).all()
    assert (ws[:256] == 0x5A).all() and (ws[256 + need:] == 0x5A).all()
    assert not split or (ws[256:256 + need] != 0xFF).any()       # (the workspace given is the one used)
    o = out.cpu().numpy()
    assert all((o[b, counts[b]:] == 7.5).all() for b in range(B))
    check_attention(o, q, K, V, lens, counts, D**-0.5, 0, 0)


@pytest.mark.parametrize("D", [64, 128])
def test_two_tokens_in_one_place(D):
    """Two sequences that share their pages append to the same tokens: where they are equal (a common beginning) nothing is lost, where
    they are not every code, step and zero is that of one of them, and no other token changes."""
    rng = np.random.default_rng(D)
    T, Hk, page = 24, 2, 16
    k, v = (rng.standard_normal((2, T, Hk, D)).astype(np.float16) for _ in range(2))
    same = 10
    k[1, :same], v[1, :same] = k[0, :same], v[0, :same]
    table, start = cuda(np.array([[1, 2], [1, 2]], np.int32)), cuda(np.full(2, 3, np.int32))
    caches = [api.PagedCache(torch.full((4, Hk, 1, 18 * D), 0x33, dtype=torch.uint8, device="cuda")) for _ in range(3)]
    for b in range(2):
        api.cache_append(caches[b], cuda(k[b:b + 1]), cuda(v[b:b + 1]), table[:1], start[:1])
    for _ in range(10):
        api.cache_append(caches[2], cuda(k), cuda(v), table, start)
        one, two, both = (c.pool.view(torch.int16) for c in caches)
        assert ((both == one) | (both == two)).all()       # (half words: a token's codes are whole ones)
        got = api.cache_read(caches[2], table, start, same)
        want = api.cache_read(caches[0], table, start, same)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_values_at_the_end_of_fp16s_range():
    """A range of -65504 .. 65504 has a step of 8733.9, rounded to 8736: its top is 65536, finite in K's scores (which are in fp32) and
    infinite where it is turned into fp16."""
    D, n = 64, 20
    k = np.zeros((1, n, 1, D), np.float16)
    k[0, 4, 0, 0], k[0, 4, 0, 1] = 65504, -65504
    v = np.ones((1, n, 1, D), np.float16)
    v[0, 4] = 2
    cache = api.PagedCache.empty(2, 16, 1, D)
    table, zero = cuda(np.array([[1, 0]], np.int32)), cuda(np.zeros(1, np.int32))
    api.cache_append(cache, cuda(k), cuda(v), table, zero)
    K = no.cache_values(*no.cache_quantise(k[0]))
    got = api.cache_read(cache, table, zero, n)[0][0].cpu().numpy()
    with np.errstate(over="ignore"):
        assert K[4, 0, 0] == 65536 and np.array_equal(got, K.astype(np.float16)) and np.isinf(got[4, 0, 0])
    q = np.zeros((1, 1, 2, D), np.float16)
    q[0, 0, 0, 0], q[0, 0, 1, 0] = 1, -1                   # all for token 4, and all for the others
    o = api.cache_attention(cuda(q), cache, table, zero + n).cpu().numpy()[0, 0]
    assert (o[0] == 2).all() and (o[1] == 1).all()
    api.cache_append(cache, cuda(v), cuda(k), table, zero)      # as V: the row that sees it all is infinite or NaN there, and there alone
    o = api.cache_attention(cuda(q), cache, table, zero + n).cpu().numpy()[0, 0]
    assert not np.isfinite(o[:, 0]).any() and np.isfinite(o[:, 1:]).all()
