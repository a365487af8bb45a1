"""GPU parity of the 4-bit weights (tern_nib_fit, tern_nib_pack, tern_nib_dequant, tern_nib_linear) against
the CPU oracle.

The fit, the packing and the way back are compared bit for bit. Tolerance of the product: fp32 sums of K exact
products, of which each addition is off by at most 2^-23 of the largest partial sum, so 2 K 2^-23 sum |w x|; past
16 tokens the weights are rounded to fp16 first, half a step of each, 2^-11 sum |w x|; one rounding of the
result, 2^-11 |y| (2^-25 below fp16's normal range). The norm of all errors is held to two such roundings."""

import copy

import numpy as np
import pytest
import torch

from oracle import nib_oracle as no
from ternary_weight_only_tern_b200 import _lib, api

pytestmark = pytest.mark.gpu


def draw(rng, N, K, group, offset):
    c = rng.integers(0, 16, size=(N, K), dtype=np.uint8)
    s = rng.uniform(0.005, 0.02, size=(N, K // group)).astype(np.float16)
    mu = rng.uniform(-0.01, 0.01, size=(N, K // group)).astype(np.float16) if offset else None
    return c, s, mu


def weight(c, s, mu, **kw):
    w = api.nib_pack(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(),
                     torch.from_numpy(mu).cuda() if mu is not None else None)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def check_product(y, x, W):
    ref = x.astype(np.float64) @ W.T
    mass = np.abs(x.astype(np.float64)) @ np.abs(W).T
    K, M = W.shape[1], len(x)
    tol = 2.0**-11 * np.abs(ref) + 2.0**-25 + (2 * K * 2.0**-23 + (2.0**-11 if M > 16 else 0)) * mass
    err = np.abs(y.astype(np.float64) - ref)
    assert np.isfinite(y).all()
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3g} of the tolerance"
    assert np.linalg.norm(err) <= 2 * 2.0**-11 * np.linalg.norm(ref)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 128), (16, 256), (37, 640), (100, 2560)])
def test_pack_lays_out_by_the_definition(N, K, group):
    c, s, mu = draw(np.random.default_rng(N + group), N, K, group, True)
    w = weight(c, s, mu)
    assert np.array_equal(w.codes.cpu().numpy().view(np.uint32), no.nib_words(c))
    assert np.array_equal(w.scale.cpu().numpy(), no.nib_scale_layout(s))
    assert np.array_equal(w.mu.cpu().numpy(), no.nib_scale_layout(mu))
    back = api.nib_dequant(w).cpu().numpy()
    assert np.array_equal(back, no.nib_values(c, s, mu).astype(np.float16))


def test_pack_reports_a_bad_code():
    c, s, _ = draw(np.random.default_rng(0), 20, 256, 128, False)
    c[17, 200] = 16
    with pytest.raises(_lib.TernError, match="TERN_ERR_BAD_CODE"):
        weight(c, s, None)


@pytest.mark.parametrize("offset", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 128), (45, 512), (300, 2560)])
def test_fit_bit_exact(N, K, group, offset):
    rng = np.random.default_rng(7 * N + group)
    W = (rng.standard_normal((N, K)) * 0.02 + rng.uniform(-0.01, 0.01, (N, 1))).astype(np.float16)
    W[0, :group] = 0.25                                  # a constant group
    W[-1, -group:] = 0                                   # and an empty one
    if N > 2:
        W[1] = np.round(W[1].astype(np.float32) * 512) / 512   # quotients on and next to ties
        W[2, ::2] *= np.float16(1e-4)                    # subnormal steps
    c, s, mu = no.nib_fit(W, group, offset)
    w = api.nib_fit(torch.from_numpy(W).cuda(), group=group, offset=offset)
    assert np.array_equal(w.scale.cpu().numpy(), no.nib_scale_layout(s))
    assert np.array_equal(w.codes.cpu().numpy().view(np.uint32), no.nib_words(c))
    if offset:
        assert np.array_equal(w.mu.cpu().numpy(), no.nib_scale_layout(mu))
    else:
        assert w.mu is None


def test_fit_ties_everywhere():
    """Steps that are powers of two and weights on multiples of half a step: every quotient a tie or whole."""
    rng = np.random.default_rng(3)
    W = (rng.integers(-14, 15, size=(64, 256)) / 64).astype(np.float16)
    W[:, ::32] = 7 / 32
    W[:, 1::32] = -7 / 32
    for offset in (False, True):
        c, s, mu = no.nib_fit(W, 32, offset)
        w = api.nib_fit(torch.from_numpy(W).cuda(), group=32, offset=offset)
        assert np.array_equal(w.codes.cpu().numpy().view(np.uint32), no.nib_words(c))


def test_fit_of_non_finite_weights_marks_the_group():
    W = np.ones((2, 256), np.float16)
    W[0, 3] = np.inf
    W[1, 200] = np.nan
    back = api.nib_dequant(api.nib_fit(torch.from_numpy(W).cuda())).cpu().numpy()
    assert not np.isfinite(back[0, :128]).any() and not np.isfinite(back[1, 128:]).any()
    assert (back[0, 128:] == 1).all() and (back[1, :128] == 1).all()


@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 16, 17, 31, 33, 64, 65, 100, 129, 300])
@pytest.mark.parametrize("N,K,group,offset", [(1, 128, 128, True), (77, 384, 32, True), (1024, 2560, 128, False),
                                              (515, 1152, 64, True), (272, 9728, 128, True), (4099, 256, 32, False)])
def test_linear_matches_oracle(M, N, K, group, offset):
    rng = np.random.default_rng(M * 31 + N)
    c, s, mu = draw(rng, N, K, group, offset)
    w = weight(c, s, mu)
    x = rng.standard_normal((M, K), dtype=np.float32).astype(np.float16)
    y = api.nib_linear(torch.from_numpy(x).cuda(), w).cpu().numpy()
    check_product(y, x, no.nib_values(c, s, mu))


@pytest.mark.parametrize("M", [1, 7, 16, 40, 200])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_exact_case_bit_exact(M, group):
    """Whole activations and steps that are powers of two: every sum is exact, both sides round once."""
    rng = np.random.default_rng(M)
    N, K = 130, 1280
    c = rng.integers(0, 16, size=(N, K), dtype=np.uint8)
    s = np.ldexp(1.0, -rng.integers(4, 7, size=(N, K // group))).astype(np.float16)
    mu = (np.ldexp(1.0, -rng.integers(4, 7, size=(N, K // group))) * rng.integers(-1, 2, size=(N, K // group))).astype(np.float16)
    x = rng.integers(-2, 3, size=(M, K)).astype(np.float16)
    y = api.nib_linear(torch.from_numpy(x).cuda(), weight(c, s, mu)).cpu().numpy()
    assert np.array_equal(y, (x.astype(np.float64) @ no.nib_values(c, s, mu).T).astype(np.float16))


@pytest.mark.parametrize("M,N,K,group", [(1, 12288, 4096, 128), (16, 4096, 12288, 64), (48, 9728, 2560, 32), (2048, 4096, 4096, 128)])
def test_linear_full_sizes_on_sampled_rows(M, N, K, group):
    rng = np.random.default_rng(N)
    c, s, mu = draw(rng, N, K, group, True)
    x = rng.standard_normal((M, K), dtype=np.float32).astype(np.float16)
    y = api.nib_linear(torch.from_numpy(x).cuda(), weight(c, s, mu)).cpu().numpy()
    rows = np.concatenate([rng.choice(N, 200, replace=False), [0, N - 1]])
    check_product(y[:, rows], x, no.nib_values(c[rows], s[rows], mu[rows]))


@pytest.mark.parametrize("M,N,K,group", [(600, 4864, 512, 32), (600, 4864, 384, 64), (1000, 1000, 1024, 128), (257, 2100, 640, 32),
                                         (128, 515, 2560, 64), (112, 4099, 256, 128), (2049, 300, 128, 32)])
def test_linear_of_many_tokens_on_sampled_rows(M, N, K, group):
    """Tiles of 128 and 256 rows, of 112 to 256 tokens, ragged both ways, with and without slices of K."""
    rng = np.random.default_rng(N + M)
    c, s, mu = draw(rng, N, K, group, True)
    x = rng.standard_normal((M, K), dtype=np.float32).astype(np.float16)
    y = api.nib_linear(torch.from_numpy(x).cuda(), weight(c, s, mu)).cpu().numpy()
    rows = np.unique(np.concatenate([rng.choice(N, 150, replace=False), [0, N - 1]]))
    check_product(y[:, rows], x, no.nib_values(c[rows], s[rows], mu[rows]))


@pytest.mark.parametrize("M", [1, 8, 16, 40])
def test_activations_of_one_sign_lose_nothing(M):
    """A large common part of x: the decoding's excess, 72 times the sum of x, has to come off exactly enough."""
    rng = np.random.default_rng(M)
    c, s, mu = draw(rng, 300, 4096, 32, False)
    x = (rng.standard_normal((M, 4096)) * 0.25 + 20).astype(np.float16)
    y = api.nib_linear(torch.from_numpy(x).cuda(), weight(c, s, mu)).cpu().numpy()
    check_product(y, x, no.nib_values(c, s, mu))


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_linear_writes_its_rows_alone(M):
    """Outputs and workspace between guard words, a weight of 16 rows more than the last strip needs."""
    rng = np.random.default_rng(M)
    N, K = 201, 512
    c, s, mu = draw(rng, N, K, 128, True)
    w = weight(c, s, mu)
    buf = torch.full((M * N + 256,), 7.5, dtype=torch.float16, device="cuda")
    need = api.nib_workspace_bytes(w, M)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    x = rng.standard_normal((M, K), dtype=np.float32).astype(np.float16)
    out = buf[128:128 + M * N].view(M, N)
    api.nib_linear(torch.from_numpy(x).cuda(), w, out=out, workspace=ws[256:256 + need])
    torch.cuda.synchronize()
    check_product(out.cpu().numpy(), x, no.nib_values(c, s, mu))
    assert (buf[:128] == 7.5).all() and (buf[128 + M * N:] == 7.5).all()
    assert (ws[:256] == 0x5A).all() and (ws[256 + need:] == 0x5A).all()


@pytest.mark.parametrize("M", [1, 3, 20])
def test_non_finite_activations_stay_in_their_token(M):
    rng = np.random.default_rng(5)
    c, s, mu = draw(rng, 64, 512, 64, True)
    x = rng.standard_normal((M, 512), dtype=np.float32).astype(np.float16)
    x[0, 100] = np.inf
    y = api.nib_linear(torch.from_numpy(x).cuda(), weight(c, s, mu)).cpu().numpy()
    assert not np.isfinite(y[0]).any()
    if M > 1:
        check_product(np.concatenate([y[1:], y[1:]])[:max(M - 1, 1)], x[1:], no.nib_values(c, s, mu))


@pytest.mark.parametrize("M", [1, 6, 24, 200])
def test_linear_repeats_to_the_bit_on_any_stream_and_in_a_graph(M):
    rng = np.random.default_rng(M)
    c, s, mu = draw(rng, 1000, 2560, 128, True)
    w = weight(c, s, mu, static=True)
    x = torch.from_numpy(rng.standard_normal((M, 2560), dtype=np.float32).astype(np.float16)).cuda()
    first = api.nib_linear(x, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for st in streams:                                   # two at a time, each with its own workspace
        with torch.cuda.stream(st):
            outs += [api.nib_linear(x, w) for _ in range(3)]
    torch.cuda.synchronize()
    ws = torch.empty(max(1, api.nib_workspace_bytes(w, M)), dtype=torch.uint8, device="cuda")
    xg, yg = torch.zeros_like(x), torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.nib_linear(xg, w, out=yg, workspace=ws)
        yy = api.nib_linear(xg, w, workspace=ws)
    xg.copy_(x)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, first) and torch.equal(yy, first)
    assert all(torch.equal(o, first) for o in outs)
    del g


def test_a_copied_weight_is_a_weight_of_its_own():
    rng = np.random.default_rng(4)
    w = weight(*draw(rng, 48, 256, 64, True))
    x = torch.from_numpy(rng.standard_normal((2, 256), dtype=np.float32).astype(np.float16)).cuda()
    y = api.nib_linear(x, w)
    twin = copy.deepcopy(w)
    assert twin.codes.data_ptr() != w.codes.data_ptr()
    w.codes.zero_()
    assert torch.equal(api.nib_linear(x, twin), y)
    assert not torch.equal(api.nib_linear(x, w), y)


def test_no_tokens():
    c, s, mu = draw(np.random.default_rng(0), 32, 256, 128, False)
    assert api.nib_linear(torch.empty((0, 256), dtype=torch.float16, device="cuda"), weight(c, s, mu)).shape == (0, 32)
