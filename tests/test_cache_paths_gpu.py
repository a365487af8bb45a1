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
