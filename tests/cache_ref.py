"""Plain statements of the paged 4-bit cache for its tests: the pool's bytes
taken apart with numpy, the codec's oracle for codes and meta, and attention in
64 bits from the stored values. Nothing here uses the library's kernels."""
from __future__ import annotations

import numpy as np
import torch

import oracle

GOLDEN = 0x9E3779B97F4A7C15


def diagonal_seed(seed, per_vector, index, d):
    """The state whose first sign words are the diagonal of (layer, kv, head) `index`."""
    return (seed + (index * (d // 64) * GOLDEN if per_vector else 0)) % 2 ** 64


def signs(seed, per_vector, layers, heads, d, first_layer=0):
    """+-1 diagonals, float64 [layers, 2, heads, d]."""
    out = np.empty((layers, 2, heads, d))
    for l in range(layers):
        for kv in range(2):
            for h in range(heads):
                i = ((first_layer + l) * 2 + kv) * heads + h
                w = oracle.sign_words(diagonal_seed(seed, per_vector, i, d), d)
                bits = (w[np.arange(d) // 64] >> (np.arange(d) % 64).astype(np.uint64)) & np.uint64(1)
                out[l, kv, h] = 1.0 - 2.0 * bits.astype(np.float64)
    return out


def hadamard(d):
    i = np.arange(d)
    return 1.0 - 2.0 * (np.bitwise_count(i[:, None] & i[None, :]) % 2)


def block_bytes(d, g, page):
    return page * (d // 2 + d // g * 4)


def places(slots, page):
    slots = np.asarray(slots)
    return slots // page, slots % page // 16, slots % 16


def split_pool(pool, d, g, page):
    """uint8 [L, P, 2, H, block] -> codes in channel order [L, P, 2, H, tiles, 16, d/2]
    and meta uint16 [..., 16, d/g, 2] (scale, zero)."""
    cb, mb = d // 2, d // g * 4
    t = pool.reshape(*pool.shape[:4], page // 16, 16 * (cb + mb))
    stored = t[..., :16 * cb].reshape(*t.shape[:-1], 16, cb)
    meta = np.ascontiguousarray(t[..., 16 * cb:]).view("<u2").reshape(*t.shape[:-1], 16, d // g, 2)
    codes = np.empty_like(stored)
    j = np.arange(cb)
    codes[:, :, 0] = stored[:, :, 0][..., (j // 4 % 4) * (cb // 4) + j // 16 * 4 + j % 4]
    codes[:, :, 1] = stored[:, :, 1][..., (j // 2 % 8) * (cb // 8) + j // 16 * 2 + j % 2]
    return codes, meta


def rows_of(pool, slots, d, g, page):
    """Codes [L, 2, H, N, d/2] and meta bytes [L, 2, H, N, d/g*4] of the slots."""
    codes, meta = split_pool(pool, d, g, page)
    p, t, i = places(slots, page)
    c = np.moveaxis(codes[:, p, :, :, t, i], 0, 3)
    m = np.ascontiguousarray(np.moveaxis(meta[:, p, :, :, t, i], 0, 3)).view(np.uint8)
    return c, m.reshape(*c.shape[:-1], d // g * 4)


def grid_values(codes, meta, g):
    """Transformed values in 64 bits from codes [..., d/2] and meta bytes [..., d/g*4]."""
    q = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2 // g, g).astype(np.float64)
    h = np.ascontiguousarray(meta).view(np.float16).astype(np.float64)
    y = (h[..., 1::2, None] + q * h[..., 0::2, None]) * 8.0
    return y.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def values(pool, slots, sg, d, g, page):
    """Stored vectors in 64 bits [L, 2, H, N, d]."""
    c, m = rows_of(pool, slots, d, g, page)
    return grid_values(c, m, g) @ hadamard(d) / d * sg[:, :, :, None]


def spreads(codes, meta, g):
    """sum over channels of 8 s |n - 8| / d per stored vector: how far one relative unit of
    a weight's rounding moves a channel of the output, at most."""
    q = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2 // g, g).astype(np.float64)
    s = np.ascontiguousarray(meta).view(np.float16).astype(np.float64)[..., 0::2, None]
    return (8 * s * np.abs(q - 8)).sum((-1, -2)) / (2 * codes.shape[-1])


def attend(x, q, qpk, scale, limits, spread):
    """x [L, 2, H, N, d], q [L, m, H*qpk, d] (64 bits), limits: (lo, hi) per query,
    spread [L, 2, H, N] -> out [L, m, H*qpk, d], lse, and the bound's parts: sum p (|v| +
    spread) per channel and the largest sum |q k| over keys (the size that score
    roundings are relative to)."""
    L, _, H, N, d = x.shape
    m = q.shape[1]
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    mag, size = np.zeros(q.shape), np.zeros(q.shape[:3])
    had = hadamard(d)
    for l in range(L):
        for j in range(H * qpk):
            k, v = x[l, 0, j // qpk], x[l, 1, j // qpk]
            yk, yq = np.abs(k @ had), np.abs(q[l, :, j] @ had)  # the signs drop out of the sizes
            for i, (lo, hi) in enumerate(limits):
                if hi <= lo:
                    continue
                s = scale * (k[lo:hi] @ q[l, i, j])
                top = s.max()
                p = np.exp(s - top)
                out[l, i, j] = p @ v[lo:hi] / p.sum()
                lse[l, i, j] = top + np.log(p.sum())
                mag[l, i, j] = p @ (np.abs(v[lo:hi]) + spread[l, 1, j // qpk, lo:hi, None]) / p.sum()
                size[l, i, j] = (yk[lo:hi].max(0) * yq[i]).sum() * scale / d
    return out, lse, mag, size


def bf16(x):
    """float array -> torch bf16 tensor whose values fp16 holds too."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
