"""CPU oracle of the 4-bit operators: weights (fit, layout, product) and the KV cache (layout, quantising,
attention), plain numpy restatements of their definitions. Test infrastructure: shares no code with the
CUDA library."""

from __future__ import annotations

import numpy as np


def nib_fit(W: np.ndarray, group: int, offset: bool):
    """fp16 W [N, K] -> codes uint8 [N, K], s fp16 [N, K/group], mu fp16 or None; fp32, each operation rounded."""
    w = W.astype(np.float32).reshape(W.shape[0], -1, group)
    f = np.float32
    with np.errstate(all="ignore"):
        if offset:
            lo, hi = w.min(-1), w.max(-1)
            s = ((hi - lo) / f(15)).astype(np.float16)
            mu = (lo + f(8) * s.astype(f)).astype(np.float16)
        else:
            s = (np.abs(w).max(-1) / f(7)).astype(np.float16)
            mu = np.zeros_like(s)
        s32 = s.astype(f)[..., None]
        t = np.rint((w - mu.astype(f)[..., None]) / s32) + f(8)
    c = np.where(s32 > 0, np.clip(t, 0, 15), 8).astype(np.uint8)
    return c.reshape(W.shape), s, mu if offset else None


def nib_values(codes, s, mu=None) -> np.ndarray:
    """float64 W of row-major codes."""
    N, K = codes.shape
    w = (codes.astype(np.float64) - 8).reshape(N, s.shape[1], -1) * s.astype(np.float64)[..., None]
    if mu is not None:
        w = w + mu.astype(np.float64)[..., None]
    return w.reshape(N, K)


def nib_words(codes: np.ndarray) -> np.ndarray:
    """Row-major codes [N, K] -> the strip layout's words uint32 [ceil(N/16), K/128, 256], by its definition."""
    N, K = codes.shape
    strips = -(-N // 16)
    c = np.full((strips * 16, K), 8, np.uint32)
    c[:N] = codes
    out = np.zeros((strips, K // 128, 256), np.uint32)
    for h in range(2):
        for g in range(8):
            for q in range(4):
                for j in range(4):
                    for p in range(8):
                        col = 32 * j + 8 * q + 2 * (p % 4) + p // 4
                        out[:, :, ((h * 8 + g) * 4 + q) * 4 + j] |= c[8 * h + g::16, col::128] << np.uint32(4 * p)
    return out


def nib_scale_layout(s: np.ndarray) -> np.ndarray:
    """fp16 [N, G] -> [ceil(N/16), G, 16]."""
    N, G = s.shape
    strips = -(-N // 16)
    p = np.zeros((strips * 16, G), s.dtype)
    p[:N] = s
    out = np.empty((strips, G, 16), s.dtype)
    for r in range(16):
        out[:, :, 2 * (r % 8) + r // 8] = p[r::16]
    return out


def cache_quantise(x: np.ndarray):
    """fp16 x [..., D] -> codes [..., D] uint8, s and z fp16 [..., D/64]; fp32, each operation rounded."""
    f = np.float32
    g = x.astype(f).reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        s, z = ((hi - lo) / f(15)).astype(np.float16), lo.astype(np.float16)
        s32 = s.astype(f)[..., None]
        t = np.rint((g - z.astype(f)[..., None]) / s32)
    c = np.where(s32 > 0, np.clip(t, 0, 15), 0).astype(np.uint8)
    return c.reshape(x.shape), s, z


def cache_values(c, s, z) -> np.ndarray:
    g = c.astype(np.float64).reshape(*c.shape[:-1], c.shape[-1] // 64, 64)
    return (z.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * g).reshape(c.shape)


def cache_units(kc, ks, kz, vc, vs, vz) -> np.ndarray:
    """16 tokens of n blocks (codes [n, 16, D], scales [n, 16, D/64]) -> uint8 [n, 18 D], by the definition."""
    n, _, D = kc.shape
    W = D // 32
    out = np.zeros((n, 18 * D), np.uint8)
    words = np.zeros((2, n, 2 * D), np.uint32)
    for h in range(2):
        for g in range(8):
            for q in range(4):
                for j in range(W):
                    at = ((h * 8 + g) * 4 + q) * W + j
                    for p in range(8):
                        words[0, :, at] |= kc[:, 8 * h + g, 32 * j + 8 * q + 2 * (p % 4) + p // 4].astype(np.uint32) << np.uint32(4 * p)
                    for p in range(4):
                        d = 16 * (2 * j + p // 2) + 8 * (p % 2) + g
                        words[1, :, at] |= vc[:, 8 * h + 2 * q, d].astype(np.uint32) << np.uint32(4 * p)
                        words[1, :, at] |= vc[:, 8 * h + 2 * q + 1, d].astype(np.uint32) << np.uint32(16 + 4 * p)
    out[:, :8 * D] = words[0].view(np.uint8).reshape(n, -1)
    out[:, 8 * D:16 * D] = words[1].view(np.uint8).reshape(n, -1)
    k = np.stack([ks, kz], -1).astype(np.float16)                        # [n, 16, D/64, 2]
    out[:, 16 * D:17 * D] = np.ascontiguousarray(k).view(np.uint8).reshape(n, -1)
    v = np.zeros((n, 4, D // 64, 2, 4), np.float16)
    for q in range(4):
        for i, t in enumerate((2 * q, 2 * q + 1, 2 * q + 8, 2 * q + 9)):
            v[:, q, :, 0, i] = vs[:, t]
            v[:, q, :, 1, i] = vz[:, t]
    out[:, 17 * D:] = v.view(np.uint8).reshape(n, -1)
    return out


def attention(q, K, V, length, count, scale, window=0, sinks=0, present=None):
    """One sequence: q [T, H, D], K and V float64 [L, Hk, D] of its tokens; (o, bound) float64 [T, H, D] of its first
    `count` queries. present [L]: tokens that have a page. bound: sum_j p_j |v_j|, for tolerances."""
    T, H, D = q.shape
    G = H // K.shape[1]
    o, a = np.zeros((T, H, D)), np.zeros((T, H, D))
    j = np.arange(len(K))
    for i in range(count):
        pos = length - count + i
        see = (j <= pos) & (j < length)
        if window > 0:
            see &= (j > pos - window) | (j < sinks)
        if present is not None:
            see &= present
        if not see.any():
            continue
        for h in range(H):
            s = scale * (K[see, h // G] @ q[i, h].astype(np.float64))
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h] = p @ V[see, h // G]
            a[i, h] = p @ np.abs(V[see, h // G])
    return o, a
