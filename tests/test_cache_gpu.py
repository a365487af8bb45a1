"""GPU parity of the 4-bit KV cache (tern_cache_append, tern_cache_read, tern_cache_attention) against the CPU
oracle.

Append and read are compared bit for bit. Tolerance of attention, against float64 over the cache's exact values:
the probabilities and V are rounded to fp16 before their product (2^-11 each, of sum p |v|), a probability
below fp16's normal range is off by up to 2^-25 (n tokens of the largest |v|, over a sum of at least 1), the result is
rounded (2^-11 |o|), and a score is off by at most D 2^-22 |q| |k| scale, which moves every probability by
that share twice (its own and the sum's)."""

import copy

import numpy as np
import pytest
import torch

from oracle import nib_oracle as no
from ternary_weight_only_tern_b200 import api

pytestmark = pytest.mark.gpu


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make(rng, lens, page, Hk, D, spare=2, width=None):
    """A cache with `lens` tokens per sequence in shuffled pages: (cache, table, K, V float64 lists, k, v fp16)."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    width = width or max(max(need), 1)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = api.PagedCache.empty(pages, page, Hk, D)
    T = max(max(lens), 1)
    k, v = ((rng.standard_normal((len(lens), T, Hk, D)) * rng.uniform(0.3, 2, (1, 1, Hk, D))).astype(np.float16) for _ in range(2))
    api.cache_append(cache, cuda(k), cuda(v), cuda(table), cuda(np.zeros(len(lens), np.int32)), cuda(np.array(lens, np.int32)))
    K, V = ([no.cache_values(*no.cache_quantise(x[b, :n])) for b, n in enumerate(lens)] for x in (k, v))
    return cache, table, K, V, k, v


def check_attention(o, q, K, V, lens, counts, scale, window, sinks, present=None):
    B, T, H, D = q.shape
    for b in range(B):
        ref, mass = no.attention(q[b], K[b], V[b], lens[b], counts[b], scale, window, sinks,
                                 present[b] if present is not None else None)
        c = counts[b]
        n = max(len(K[b]), 1)
        qk = np.linalg.norm(q[b, :c].astype(np.float64), axis=-1).max(initial=0) * (np.linalg.norm(K[b], axis=-1).max() if len(K[b]) else 0)
        top = np.abs(V[b]).max() if len(V[b]) else 0
        tol = 2.0**-11 * np.abs(ref) + 2.0**-25 + (2 * 2.0**-11 + 2 * D * 2.0**-22 * qk * scale) * mass + n * 2.0**-25 * top
        err = np.abs(o[b, :c].astype(np.float64) - ref[:c])
        assert np.isfinite(o[b, :c]).all()
        assert (err <= tol[:c]).all(), f"sequence {b}: {np.max(err / tol[:c]):.3g} of the tolerance"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,Hk", [(16, 1), (32, 3), (64, 8), (48, 2)])
def test_append_lays_out_by_the_definition(page, Hk, D):
    rng = np.random.default_rng(page + D)
    lens = [page * 2, 5, 0, page + 17]
    cache, table, K, V, k, v = make(rng, lens, page, Hk, D)
    pool = cache.pool.cpu().numpy()
    for b, n in enumerate(lens):
        for first in range(0, n - 15, 16):               # whole blocks
            t = slice(first, first + 16)
            kc, ks, kz = no.cache_quantise(k[b, t].transpose(1, 0, 2))
            vc, vs, vz = no.cache_quantise(v[b, t].transpose(1, 0, 2))
            assert np.array_equal(pool[table[b, first // page], :, first % page // 16], no.cache_units(kc, ks, kz, vc, vs, vz))
    got = api.cache_read(cache, cuda(table), cuda(np.zeros(4, np.int32)), k.shape[1], cuda(np.array(lens, np.int32)))
    for b, n in enumerate(lens):
        for x, ref in zip(got, (K[b], V[b])):
            x = x[b].cpu().numpy()
            assert np.array_equal(x[:n], ref.astype(np.float16)) and not x[n:].any()


@pytest.mark.parametrize("D", [64, 128])
def test_append_piece_by_piece_gives_the_same_cache(D):
    """One call, or calls of 1, 3, 16, 20 ... tokens that begin and end inside a block: the same bytes, and nothing else touched."""
    rng = np.random.default_rng(D)
    lens = [77, 130]
    cache, table, K, V, k, v = make(rng, lens, 32, 2, D)
    other = api.PagedCache(torch.full_like(cache.pool, 0xA5))
    at = np.zeros(2, np.int32)
    steps = [1, 3, 16, 20, 1, 1, 33, 2, 60]
    for n in steps:
        counts = np.minimum(n, np.array(lens, np.int32) - at).astype(np.int32)
        kk, vv = (np.zeros((2, n, 2, D), np.float16) for _ in range(2))
        for b in range(2):
            kk[b, :counts[b]], vv[b, :counts[b]] = k[b, at[b]:at[b] + counts[b]], v[b, at[b]:at[b] + counts[b]]
            kk[b, counts[b]:] = np.nan                   # rows behind a sequence's tokens
        api.cache_append(other, cuda(kk), cuda(vv), cuda(table), cuda(at), cuda(counts))
        at = at + counts
    assert (at == lens).all()
    a, o = cache.pool.cpu().numpy(), other.pool.cpu().numpy()
    used = {(table[b, t // 32], t % 32 // 16) for b, n in enumerate(lens) for t in range(n - n % 16)}
    for page in range(len(a)):
        for blk in range(2):
            if (page, blk) in used:
                assert np.array_equal(a[page, :, blk], o[page, :, blk])
    untouched = set(range(len(a))) - set(table[table >= 0].tolist())
    assert all((o[p] == 0xA5).all() for p in untouched)
    got = api.cache_read(other, cuda(table), cuda(np.array([3, 5], np.int32)), 70)
    assert np.array_equal(got[0][0].cpu().numpy(), K[0][3:73].astype(np.float16))
    assert np.array_equal(got[1][1].cpu().numpy(), V[1][5:75].astype(np.float16))


def test_bad_pages_and_places_are_skipped():
    rng = np.random.default_rng(1)
    cache = api.PagedCache.empty(3, 16, 1, 64)
    table = cuda(np.array([[0, 7, 2], [-1, -5, 2**31 - 1]], np.int32))
    k = cuda(rng.standard_normal((2, 60, 1, 64)).astype(np.float16))
    api.cache_append(cache, k, k, table, cuda(np.array([-4, 20], np.int32)))     # before token 0, past the table, no pages
    assert not cache.pool[1].any()
    K, V = api.cache_read(cache, table, cuda(np.array([-4, 0], np.int32)), 60, cuda(np.array([1000, -3], np.int32)))
    x = K[0, :, 0].cpu().numpy()
    ref = no.cache_values(*no.cache_quantise(k[0, :, 0].cpu().numpy())).astype(np.float16)
    assert not x[:4].any() and np.array_equal(x[4:20], ref[4:20]) and not x[20:36].any()
    assert np.array_equal(x[36:52], ref[36:52]) and not x[52:].any() and not K[1].any()
    q = cuda(rng.standard_normal((2, 1, 2, 64)).astype(np.float16))
    o = api.cache_attention(q, cache, table, cuda(np.array([48, 48], np.int32))).cpu().numpy()
    assert not o[1].any()                                                            # no page at all: zeros
    Kf = no.cache_values(*no.cache_quantise(k[0, 4:52, 0].cpu().numpy()))[:, None]
    here = np.repeat([True, False, True], 16)
    check_attention(o[:1], q[:1].cpu().numpy(), [Kf], [Kf], [48], [1], 0.125, 0, 0, [here])
    api.cache_attention(q, cache, table, cuda(np.array([2**31 - 1, -2**31], np.int32)))   # far past the table
    torch.cuda.synchronize()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G,T", [(1, 1, 1), (8, 4, 1), (2, 8, 1), (2, 3, 1), (1, 4, 5), (2, 5, 4), (1, 16, 1), (2, 2, 17), (1, 1, 64)])
def test_attention_over_ragged_lengths(Hk, G, T, D):
    rng = np.random.default_rng(Hk * 100 + G * 10 + T)
    lens = [1, 2, 15, 16, 17, 63, 0, 200, 1027]
    cache, table, K, V, _, _ = make(rng, lens, 32, Hk, D)
    q = rng.standard_normal((len(lens), T, Hk * G, D)).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32))).cpu().numpy()
    check_attention(o, q, K, V, lens, [T] * len(lens), D**-0.5, 0, 0)
    assert not o[6].any()


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (17, 3), (100, 16), (100, 33), (64, 500), (2000, 5), (5, 1)])
@pytest.mark.parametrize("T", [1, 6])
def test_attention_with_a_window_and_sinks(window, sinks, T):
    rng = np.random.default_rng(window + sinks + T)
    lens = [3, 40, 333, 700]
    cache, table, K, V, _, _ = make(rng, lens, 16, 2, 128)
    q = rng.standard_normal((4, T, 6, 128)).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32)), window=window, sinks=sinks).cpu().numpy()
    check_attention(o, q, K, V, lens, [T] * 4, 128**-0.5, window, sinks)


@pytest.mark.parametrize("window", [1000, 2**31 - 60, 2**31 - 1, 2**40])
def test_queries_before_token_zero_and_windows_past_every_length(window):
    """Sequences with fewer cached tokens than queries: the first queries see nothing, the others all there is."""
    rng = np.random.default_rng(7)
    lens, T = [5, 64, 40, 0, 200], 64
    cache, table, K, V, _, _ = make(rng, lens, 32, 2, 64)
    q = rng.standard_normal((5, T, 4, 64)).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32)), window=window).cpu().numpy()
    check_attention(o, q, K, V, lens, [T] * 5, 64**-0.5, 0, 0)
    assert not o[0, :59].any() and not o[3].any() and not o[2, :24].any()


def test_a_copied_cache_is_a_cache_of_its_own():
    rng = np.random.default_rng(8)
    cache, table, K, V, k, v = make(rng, [50], 32, 2, 64)
    q = cuda(rng.standard_normal((1, 1, 4, 64)).astype(np.float16))
    where, lens = cuda(table), cuda(np.array([50], np.int32))
    o = api.cache_attention(q, cache, where, lens)
    twin = copy.deepcopy(cache)
    assert twin.pool.data_ptr() != cache.pool.data_ptr()
    cache.pool.zero_()
    assert torch.equal(api.cache_attention(q, twin, where, lens), o)


def test_attention_of_a_padded_batch_leaves_the_rest():
    rng = np.random.default_rng(8)
    lens, counts = [50, 7, 300, 20], [3, 0, 5, 1]
    cache, table, K, V, _, _ = make(rng, lens, 64, 2, 64)
    q = rng.standard_normal((4, 5, 4, 64)).astype(np.float16)
    for b, c in enumerate(counts):
        q[b, c:] = np.nan
    out = torch.full((4, 5, 4, 64), 3.25, dtype=torch.float16, device="cuda")
    api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32)), counts=cuda(np.array(counts, np.int32)), out=out)
    o = out.cpu().numpy()
    check_attention(o, q, K, V, lens, counts, 0.125, 0, 0)
    for b, c in enumerate(counts):
        assert (o[b, c:] == 3.25).all()


@pytest.mark.parametrize("D", [64, 128])
def test_attention_over_long_lengths(D):
    rng = np.random.default_rng(D)
    lens = [20011, 64, 5000]
    cache, table, K, V, _, _ = make(rng, lens, 128, 2, D)
    q = (rng.standard_normal((3, 2, 8, D)) * 2).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32))).cpu().numpy()
    check_attention(o, q, K, V, lens, [2] * 3, D**-0.5, 0, 0)


def test_pages_past_four_gigabytes():
    """A pool of 4.6 GB with a sequence in its first and last pages: byte offsets past 32 bits in all three operators."""
    rng = np.random.default_rng(12)
    pages, page, Hk, D = 31500, 128, 8, 128
    cache = api.PagedCache(torch.empty((pages, Hk, page // 16, 18 * D), dtype=torch.uint8, device="cuda"))
    table = np.array([[pages - 1, 0, pages - 2]], np.int32)
    n = 300
    k, v = (rng.standard_normal((1, n, Hk, D)).astype(np.float16) for _ in range(2))
    zero = cuda(np.zeros(1, np.int32))
    api.cache_append(cache, cuda(k), cuda(v), cuda(table), zero)
    K, V = (no.cache_values(*no.cache_quantise(x[0])) for x in (k, v))
    got = api.cache_read(cache, cuda(table), zero, n)
    assert np.array_equal(got[0][0].cpu().numpy(), K.astype(np.float16)) and np.array_equal(got[1][0].cpu().numpy(), V.astype(np.float16))
    q = rng.standard_normal((1, 2, 16, D)).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array([n], np.int32))).cpu().numpy()
    check_attention(o, q, [K], [V], [n], [2], D**-0.5, 0, 0)


@pytest.mark.parametrize("B", [129, 700])
def test_batches_past_one_scan(B):
    """More sequences than a CTA has threads, most of them empty or tiny, one long among them."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 20, B)]
    lens[B - 3] = 1500
    cache, table, K, V, _, _ = make(rng, lens, 16, 1, 64)
    q = rng.standard_normal((B, 1, 2, 64)).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32)), window=1000, sinks=3).cpu().numpy()
    check_attention(o, q, K, V, lens, [1] * B, 0.125, 1000, 3)


def test_many_heads_and_tiles():
    """Every (sequence, head, tile) counts: more of them than CTAs, rows that do not fill a tile."""
    rng = np.random.default_rng(33)
    lens = [100, 37, 260]
    cache, table, K, V, _, _ = make(rng, lens, 48, 40, 64)
    q = rng.standard_normal((3, 7, 200, 64)).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32))).cpu().numpy()
    check_attention(o, q, K, V, lens, [7] * 3, 0.125, 0, 0)


def test_empty_calls():
    cache = api.PagedCache.empty(2, 16, 2, 64)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f16 = lambda *s: torch.ones(s, dtype=torch.float16, device="cuda")  # noqa: E731
    api.cache_append(cache, f16(0, 3, 2, 64), f16(0, 3, 2, 64), i32(0, 4), i32(0))
    api.cache_append(cache, f16(2, 0, 2, 64), f16(2, 0, 2, 64), i32(2, 4), i32(2))
    api.cache_append(cache, f16(1, 3, 2, 64), f16(1, 3, 2, 64), i32(1, 0), i32(1))        # a table without columns
    assert not cache.pool.any()
    assert not api.cache_read(cache, i32(1, 0), i32(1), 3)[0].any()
    assert api.cache_attention(f16(0, 1, 4, 64), cache, i32(0, 4), i32(0)).shape == (0, 1, 4, 64)
    assert not api.cache_attention(f16(2, 1, 4, 64), cache, i32(2, 0), i32(2) + 5).any()
    with pytest.raises(ValueError, match="shape"):
        api.cache_attention(f16(1, 1, 3, 64), cache, i32(1, 4), i32(1))
    with pytest.raises(ValueError, match="rows"):
        api.cache_attention(f16(2, 1, 4, 64), cache, i32(1, 4), i32(2))
    with pytest.raises(ValueError, match="entries"):
        api.cache_append(cache, f16(2, 1, 2, 64), f16(2, 1, 2, 64), i32(2, 4), i32(1))
    with pytest.raises(TypeError, match="int32"):
        api.cache_read(cache, i32(1, 4), torch.zeros(1, dtype=torch.int64, device="cuda"), 3)
    with pytest.raises(ValueError, match="contiguous"):
        api.cache_attention(f16(1, 1, 64, 4).transpose(2, 3), cache, i32(1, 4), i32(1))


def test_many_short_sequences():
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(0, 90, 300)]
    cache, table, K, V, _, _ = make(rng, lens, 16, 2, 64, width=40)
    q = rng.standard_normal((300, 1, 4, 64)).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32))).cpu().numpy()
    check_attention(o, q, K, V, lens, [1] * 300, 0.125, 0, 0)


def test_sharp_and_far_scores():
    """Scores of hundreds either way: one token takes all, and the running maximum moves late."""
    rng = np.random.default_rng(2)
    cache, table, K, V, _, _ = make(rng, [600], 64, 1, 128)
    q = np.zeros((1, 1, 8, 128), np.float16)
    for i, t in enumerate((0, 1, 17, 300, 585, 598, 599, 450)):
        q[0, 0, i] = (K[0][t, 0] * 8).astype(np.float16)
    lens = cuda(np.array([600], np.int32))
    o = api.cache_attention(cuda(q), cache, cuda(table), lens).cpu().numpy()
    check_attention(o, q, K, V, [600], [1], 128**-0.5, 0, 0)
    o = api.cache_attention(cuda(q), cache, cuda(table), lens, scale=-0.5).cpu().numpy()
    check_attention(o, -q, K, V, [600], [1], 0.5, 0, 0)
    o = api.cache_attention(cuda(q), cache, cuda(table), lens, scale=0.0).cpu().numpy()
    check_attention(o, q, K, V, [600], [1], 0.0, 0, 0)


@pytest.mark.parametrize("T", [1, 4])
def test_what_is_not_seen_does_not_reach_a_result(T):
    """NaN and infinities behind the last token, outside the window, and in tokens that later queries alone see."""
    rng = np.random.default_rng(T)
    lens = [301, 90]
    cache, table, K, V, k, v = make(rng, lens, 32, 2, 128, spare=3)
    pool = cache.pool.clone()
    bad = cuda(np.full((2, 1, 2, 128), np.nan, np.float16))
    for place in ([301, 90], [310, 95], [100, 20], [163, 0]):                # behind the end, and outside the window
        api.cache_append(cache, bad, bad, cuda(table), cuda(np.array(place, np.int32)))
    bad = bad.clone().fill_(float("inf"))
    api.cache_append(cache, bad, bad, cuda(table), cuda(np.array([303, 92], np.int32)))
    spare = sorted(set(range(cache.pages)) - set(table[table >= 0].tolist()))
    cache.pool[spare] = 0xFF
    q = rng.standard_normal((2, T, 4, 128)).astype(np.float16)
    o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32)), window=40, sinks=0).cpu().numpy()
    check_attention(o, q, K, V, lens, [T] * 2, 128**-0.5, 40, 0)
    if T > 1:
        cache.pool.copy_(pool)
        api.cache_append(cache, bad, bad, cuda(table), cuda(np.array([299, 89], np.int32)))   # the last queries' own
        o = api.cache_attention(cuda(q), cache, cuda(table), cuda(np.array(lens, np.int32)), window=40).cpu().numpy()
        # sequence 0's queries sit at 297 .. 300, sequence 1's at 86 .. 89
        for b, c in ((0, 2), (1, 3)):
            full = [x[b] for x in (K, V)]
            ref, mass = no.attention(q[b], full[0], full[1], lens[b], T, 128**-0.5, 40, 0)
            assert np.isfinite(o[b, :c]).all()
            assert (np.abs(o[b, :c] - ref[:c]) <= 4 * 2.0**-11 * (mass[:c] + np.abs(ref[:c])) + 1e-4 * mass[:c]).all()
            assert np.isnan(o[b, c:]).all()


def test_streams_graphs_and_repeats_agree_to_the_bit():
    rng = np.random.default_rng(6)
    lens = [900, 33, 2500, 1]
    cache, table, K, V, _, _ = make(rng, lens, 64, 4, 128)
    q, tab, n = cuda(rng.standard_normal((4, 1, 16, 128)).astype(np.float16)), cuda(table), cuda(np.array(lens, np.int32))
    first = api.cache_attention(q, cache, tab, n)
    torch.cuda.synchronize()
    outs = []
    for st in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(st):
            outs += [api.cache_attention(q, cache, tab, n) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    ws = torch.full((max(1, cache.workspace_bytes(4, 1, 16, table.shape[1])),), 0xFF, dtype=torch.uint8, device="cuda")
    qg, lg = torch.zeros_like(q), torch.ones_like(n)
    graphs = []
    for _ in range(2):                                   # two graphs, one workspace, one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = api.cache_attention(qg, cache, tab, lg, workspace=ws)
        graphs.append((g, o))
    qg.copy_(q)
    lg.copy_(n)
    for _ in range(2):
        for g, o in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for _, o in graphs)
    del graphs


@pytest.mark.parametrize("static", [False, True])
def test_a_decode_step_of_all_of_them(static):
    """Projection in 4 bits, append, attention over the cache, output projection and head in ternary and 4 bits, captured
    once and replayed for three tokens, each checked against float64 from the values that the step before rounded."""
    rng = np.random.default_rng(9)
    B, Hk, G, D, hidden = 3, 2, 2, 128, 512
    mk = lambda n, k: api.nib_fit(cuda((rng.standard_normal((n, k)) * k**-0.5).astype(np.float16)))  # noqa: E731
    wq, wk, wv, head = mk(Hk * G * D, hidden), mk(Hk * D, hidden), mk(Hk * D, hidden), mk(1003, hidden)
    t1, s1, mu, _, _ = api.fit(cuda((rng.standard_normal((hidden, Hk * G * D)) * (Hk * G * D)**-0.5).astype(np.float16)))
    wo = api.TernWeight.from_trits(t1, s1, mu=mu)
    for w in (wq, wk, wv, wo, head):
        w.static = static
    lens0 = [40, 5, 64]
    cache, table, K, V, _, _ = make(rng, lens0, 16, Hk, D, spare=0, width=8)
    extra = api.PagedCache(torch.cat([cache.pool, torch.zeros_like(cache.pool[:3])]))
    for b in range(B):
        table[b, -(-lens0[b] // 16)] = cache.pages + b   # room for the new tokens
    tab = cuda(table)
    x = torch.zeros((B, hidden), dtype=torch.float16, device="cuda")
    start = cuda(np.array(lens0, np.int32))
    lens = start + 1
    bufs = {}

    def step():
        q, k, v = api.nib_linear(x, wq), api.nib_linear(x, wk), api.nib_linear(x, wv)
        api.cache_append(extra, k.view(B, 1, Hk, D), v.view(B, 1, Hk, D), tab, start)
        o = api.cache_attention(q.view(B, 1, Hk * G, D), extra, tab, lens)
        y = api.linear(o.view(B, -1), wo)
        bufs.update(q=q, k=k, v=v, o=o, y=y, logits=api.nib_linear(y, head))
        start.add_(1)
        lens.add_(1)

    side = torch.cuda.Stream()
    before = extra.pool.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    extra.pool.copy_(before)
    start.copy_(cuda(np.array(lens0, np.int32)))
    lens.copy_(start + 1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    n = list(lens0)
    W = {k: api.nib_dequant(w).cpu().numpy().astype(np.float64) for k, w in dict(q=wq, k=wk, v=wv, logits=head).items()}
    parts = [np.repeat(a.cpu().numpy().astype(np.float64), 128, 1) for a in (s1, mu)]
    W["y"] = parts[0] * t1.cpu().numpy() + parts[1]
    for _ in range(3):
        xs = rng.standard_normal((B, hidden)).astype(np.float16)
        x.copy_(cuda(xs))
        g.replay()
        torch.cuda.synchronize()
        h = {k: t.cpu().numpy() for k, t in bufs.items()}
        near = lambda a, r: np.abs(a - r).max() <= 2.0**-9 * np.abs(r).max()  # noqa: E731
        for k in "qkv":
            assert near(h[k], xs.astype(np.float64) @ W[k].T), k
        for b in range(B):
            K[b] = np.concatenate([K[b], no.cache_values(*no.cache_quantise(h["k"][b].reshape(1, Hk, D)))])
            V[b] = np.concatenate([V[b], no.cache_values(*no.cache_quantise(h["v"][b].reshape(1, Hk, D)))])
            n[b] += 1
        check_attention(h["o"], h["q"].reshape(B, 1, Hk * G, D), K, V, n, [1] * B, D**-0.5, 0, 0)
        assert near(h["y"], h["o"].reshape(B, -1).astype(np.float64) @ W["y"].T)
        assert near(h["logits"], h["y"].astype(np.float64) @ W["logits"].T)
    del g
