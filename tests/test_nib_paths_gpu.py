"""GPU tests of the 4-bit linear beside those of test_nib_gpu.py, whose inputs they use: what each of its two paths makes of
the weights, and what lies around their buffers."""

import numpy as np
import pytest
import torch

from oracle import nib_oracle as no
from ternary_weight_only_tern_b200 import api
from test_nib_gpu import check_product, draw, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 9, 16, 17, 65, 300])
@pytest.mark.parametrize("N,K,group,offset", [(200, 2560, 32, True), (515, 1152, 64, False), (272, 9728, 128, True)])
def test_the_weights_enter_as_stated(M, N, K, group, offset):
    """Up to 16 tokens as they are, past them rounded to fp16: each against the product of those weights. Tolerance without any part for
    a rounding of the weights: 2 K 2^-23 sum |w x| for the fp32 sums, half a step of the result (2^-25 below its normal range)."""
    rng = np.random.default_rng(M + N)
    c, s, mu = draw(rng, N, K, group, offset)
    x = rng.standard_normal((M, K), dtype=np.float32).astype(np.float16)
    y = api.nib_linear(torch.from_numpy(x).cuda(), weight(c, s, mu)).cpu().numpy().astype(np.float64)
    W = no.nib_values(c, s, mu)
    if M > 16:
        W = W.astype(np.float16).astype(np.float64)
    ref, mass = x.astype(np.float64) @ W.T, np.abs(x.astype(np.float64)) @ np.abs(W).T
    tol = 2.0**-11 * np.abs(ref) + 2.0**-25 + 2 * K * 2.0**-23 * mass
    assert (np.abs(y - ref) <= tol).all()


@pytest.mark.parametrize("M", [1, 16, 17, 40])
def test_weights_past_the_range_of_fp16(M):
    """mu + s (c - 8) = 70008 in one row: 16 tokens and fewer give its product, more tokens what an infinite weight gives, and the
    other rows know nothing of it."""
    N, K = 33, 256
    c = np.full((N, K), 8, np.uint8)
    s, mu = np.ones((N, K // 128), np.float16), np.zeros((N, K // 128), np.float16)
    c[5, 7], s[5, 0], mu[5, 0] = 15, 1000, 63008           # 63008 + 7 1000
    w = weight(c, s, mu)
    x = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    x[:, 7] = 2.0**-12
    y = api.nib_linear(x, w).cpu().numpy()
    assert np.isinf(api.nib_dequant(w).cpu().numpy()[5, 7])
    row = y[:, 5].astype(np.float64)
    assert (np.delete(y, 5, 1) == 0).all()
    if M > 16:
        assert not np.isfinite(row).any()
    else:
        assert (np.abs(row - 70008 * 2.0**-12) <= 2.0**-11 * 17.1).all()


@pytest.mark.parametrize("M,N,K,group", [(16, 515, 12288, 128), (9, 37, 20480, 32), (2, 50, 65536, 64), (24, 1000, 2560, 64), (40, 130, 9728, 32),
                                         (300, 260, 4096, 64), (200, 1001, 2560, 128)])
def test_sums_of_slices_stay_in_their_workspace(M, N, K, group):
    """Calls that cut K into slices, on both paths: a workspace of just the stated bytes (all NaN before) and the output lie between guard
    bytes, which stay as they are, and the result is that of a call with buffers of its own."""
    rng = np.random.default_rng(M + N)
    c, s, mu = draw(rng, N, K, group, True)
    w = weight(c, s, mu)
    need = api.nib_workspace_bytes(w, M)
    assert need >= 2 * M * N * 4
    x = torch.from_numpy(rng.standard_normal((M, K), dtype=np.float32).astype(np.float16)).cuda()
    buf = torch.full((M * N + 256,), 7.5, dtype=torch.float16, device="cuda")
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    ws[256:256 + need] = 0xFF
    out = buf[128:128 + M * N].view(M, N)
    api.nib_linear(x, w, out=out, workspace=ws[256:256 + need])
    assert (buf[:128] == 7.5).all() and (buf[128 + M * N:] == 7.5).all()
    assert (ws[:256] == 0x5A).all() and (ws[256 + need:] == 0x5A).all()
    assert (ws[256:256 + need] != 0xFF).any()              # (the workspace given is the one used)
    check_product(out.cpu().numpy(), x.cpu().numpy(), no.nib_values(c, s, mu))
    assert torch.equal(api.nib_linear(x, w), out)
