"""The 4-bit key/value cache and the attention over it in float64 numpy, for
the tests: the format's own roundings made one by one, everything else in 64
bits."""
from __future__ import annotations

import numpy as np

SHIFT = np.array([4 * (j // 2) + 16 * (j % 2) for j in range(8)], dtype=np.uint32)


def f32(x):
    with np.errstate(over="ignore"):
        return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def bf16(x, down=False):
    """float32 values rounded to bf16 (to nearest even, or down), as float64. Infinities and NaN stay."""
    x32 = np.asarray(x, dtype=np.float64).astype(np.float32)
    u = x32.view(np.uint32).astype(np.uint64)
    if down:
        up = (u >> np.uint64(31) == 1) & (u & np.uint64(0xFFFF) != 0)   # negative: away from zero
        r = u + np.where(up, np.uint64(0x10000), np.uint64(0))
    else:
        r = u + np.uint64(0x7FFF) + ((u >> np.uint64(16)) & np.uint64(1))
    r = (r & np.uint64(0xFFFF0000)).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x32), r, x32).astype(np.float64)


def store(x, dtype):
    return bf16(f32(x)) if dtype == "bf16" else f32(x)


def quantize(x, group):
    """Codes [..., hd], steps and offsets [..., hd / group] of x [..., hd] (values of the storage type)."""
    with np.errstate(all="ignore"):
        v = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, group)
        lo, hi = v.min(-1), v.max(-1)
        z = bf16(f32(lo - 16 * f32(f32(hi - lo) / 15)), down=True)
        s = bf16(f32(f32(hi - z) / 31))
        bad = ~(np.isfinite(s) & np.isfinite(z))
        m = f32(16 * s + z)
        q = np.rint(f32(v - m[..., None]) / s[..., None])
        c = np.where((s[..., None] > 0) & ~bad[..., None], np.clip(q, 0, 15), 0)
    c = np.where(np.isnan(c), 0, c).astype(np.int64).reshape(x.shape)
    return c, np.where(bad, np.nan, s), np.where(bad, np.nan, z)


def values(c, s, z, dtype):
    g = c.shape[-1] // s.shape[-1]
    with np.errstate(invalid="ignore"):
        return store((16 + c) * np.repeat(s, g, -1) + np.repeat(z, g, -1), dtype)


def pack(c):
    """uint32 words [..., hd / 8] of codes [..., hd]."""
    w = np.asarray(c, dtype=np.uint32).reshape(*c.shape[:-1], -1, 8)
    return np.bitwise_or.reduce(w << SHIFT, axis=-1)


def unpack(words):
    w = np.asarray(words).view(np.uint32)[..., None]
    return ((w >> SHIFT) & 15).astype(np.int64).reshape(*words.shape[:-1], -1)


def attention(q, k, v, lens, dtype):
    """q [B, n, H, hd], k, v [B, L, n_kv, hd] in float64, lens [B]: the outputs and, for every one of them, how far a
    kernel may be off.

    Terms of the bound, with u the storage type's half step (bf16 2^-8, float32 2^-24), e = 2^-24 and
    A = sum_i p_i |v_i| (p normalised):
    * bf16: P is rounded to bf16 for its product with V: u A;
    * the output's rounding: u |o|;
    * float32 sums: a score is a sum of hd products, off by (hd + 4) e sum |q k| scale (the products, the sum in any
      order, the scale), which moves p by that much relatively, in the numerator and in the row sum; so do the
      exponentials' own 4 e (on arguments of the size of the score's terms, so counted with it) and the sums over
      L keys, L e each: 2 ((hd + 8) S + L + 16) e A, S = 1 + max_i sum |q k_i| scale.
    """
    B, n, H, hd = q.shape
    share = H // k.shape[2]
    out, tol = np.zeros_like(q), np.zeros_like(q)
    u, e = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24), 2.0 ** -24
    for b in range(B):
        L = int(lens[b])
        if L <= 0:
            continue
        for h in range(H):
            kk, vv = k[b, :L, h // share], v[b, :L, h // share]
            with np.errstate(invalid="ignore"):
                s = q[b, :, h] @ kk.T / np.sqrt(hd)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o, a = p @ vv, p @ np.abs(vv)
                size = 1 + (np.abs(q[b, :, h]) @ np.abs(kk).T / np.sqrt(hd)).max(-1, keepdims=True)
            out[b, :, h] = o
            tol[b, :, h] = u * np.abs(o) + (u if dtype == "bf16" else 0) * a + 2 * ((hd + 8) * size + L + 16) * e * a + 1e-37
    return out, tol
