"""Float64 oracle of the softmax-attention layer beside the mixer: norms of queries and keys
with the position rotation and its gradient, the 8-bit cache, and attention over it.

Plain definitions in numpy, one sequence, head or block at a time; no code is shared with the
HIP path. The cache is held here in token order: codes as float64 values of e4m3 and one scale
per (block, head).
"""
from __future__ import annotations

import numpy as np

BLOCK = 64
LARGEST = 248.0 * 2.0 ** 120  # from here on a code would stand for 2^128, an infinity


def _split(n, rot, interleaved):
    if interleaved:
        return n[..., 0:rot:2], n[..., 1:rot:2]
    return n[..., : rot // 2], n[..., rot // 2 : rot]


def _join(n, a, b, rot, interleaved):
    y = n.copy()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a, b
    else:
        y[..., : rot // 2], y[..., rot // 2 : rot] = a, b
    return y


def rotate(n, positions, inv_freq, interleaved=False, back=False):
    """n [..., H, d] by positions [...] * inv_freq; back: by the negative angle."""
    rot = 2 * len(inv_freq)
    ang = np.asarray(positions, np.float64)[..., None, None] * np.asarray(inv_freq, np.float64)
    cs, sn = np.cos(ang), np.sin(ang) * (-1.0 if back else 1.0)
    a, b = _split(n, rot, interleaved)
    return _join(n, a * cs - b * sn, b * cs + a * sn, rot, interleaved)


def norm_rope(x, weight, positions, inv_freq, eps=1e-6, interleaved=False, norm=True):
    """x [..., H, d] -> rows normed over d, times weight (None: ones), rotated."""
    x = np.asarray(x, np.float64)
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) if norm else x.copy()
    if weight is not None:
        n = n * np.asarray(weight, np.float64)
    return rotate(n, positions, inv_freq, interleaved)


def norm_rope_backward(x, dy, weight, positions, inv_freq, eps=1e-6, interleaved=False, norm=True):
    """(dx, dweight) of norm_rope."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    d = x.shape[-1]
    w = np.ones(d) if weight is None else np.asarray(weight, np.float64)
    dn = rotate(dy, positions, inv_freq, interleaved, back=True)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) if norm else np.ones_like(x[..., :1])
    dw = (dn * x * r).reshape(-1, d).sum(0)
    u = w * dn
    back = r * r / d * np.sum(u * x, -1, keepdims=True) if norm else 0.0
    return r * (u - x * back), dw


# ------------------------------------------------------------------ e4m3 and block scales

def round_e4m3(x):
    """Nearest e4m3 value, ties to even; |x| <= 448, NaN stays."""
    x = np.asarray(x, np.float64)
    mag = np.where((x == 0) | np.isnan(x), 1.0, np.abs(x))
    step = np.exp2(np.maximum(np.floor(np.log2(mag)), -6) - 3)
    return np.rint(x / step) * step


def block_scale(amax):
    """Smallest power of two s >= 2^-64 with amax <= 448 s."""
    s = 2.0 ** -64
    while amax > 448 * s:
        s *= 2
    return s


class Cache:
    """k, v [P, Hk, 64, d] code values, k_scale, v_scale [P, Hk]."""

    def __init__(self, P, Hk, d):
        self.k, self.v = np.zeros((P, Hk, BLOCK, d)), np.zeros((P, Hk, BLOCK, d))
        self.k_scale, self.v_scale = np.zeros((P, Hk)), np.zeros((P, Hk))


def append(cache, block_row, total, k, v):
    """The last rows of a sequence of `total` tokens into the cache, one call's worth: k, v
    [n, Hk, d] (k normed and rotated), block_row: the sequence's row of the block table. The
    rows before position 0 hold no token."""
    n, Hk, _ = k.shape
    P = cache.k.shape[0]
    start = total - n
    first = max(start, 0)
    for b in range(first // BLOCK, -(-total // BLOCK) if total > 0 else 0):
        if b >= len(block_row) or not 0 <= block_row[b] < P:
            continue
        p0, p1 = max(first, b * BLOCK), min(total, (b + 1) * BLOCK)
        if p0 >= p1:
            continue
        slot, o0, o1 = block_row[b], p0 - b * BLOCK, p1 - b * BLOCK
        for h in range(Hk):
            kn, vn = k[p0 - start:p1 - start, h], v[p0 - start:p1 - start, h]
            fine = (np.abs(kn) < LARGEST).all(-1) & (np.abs(vn) < LARGEST).all(-1)
            for held, scale, x, mark in ((cache.k, cache.k_scale, kn, np.nan),
                                         (cache.v, cache.v_scale, vn, 0.0)):
                s = block_scale(np.abs(x[fine]).max() if fine.any() else 0.0)
                if o0 > 0:
                    old = scale[slot, h]
                    s = max(s, old)
                    held[slot, h, :o0] = round_e4m3(held[slot, h, :o0] * (old / s))
                    if held is cache.v and s > old and s >= 2.0 ** 120:
                        held[slot, h, o1:] = 0.0
                elif held is cache.v:
                    held[slot, h, o1:] = 0.0
                scale[slot, h] = s
                held[slot, h, o0:o1] = np.where(fine[:, None], round_e4m3(np.where(fine[:, None], x, 0) / s), mark)


def attention(q, cache, block_row, total, window=0, scale=None):
    """q [n, Hq, d], the last n rows of a sequence of `total` tokens; (o, spread) with spread the
    sum of p |v|, which the tests' tolerances go by."""
    n, Hq, d = q.shape
    P, Hk = cache.k.shape[:2]
    scale = d ** -0.5 if scale is None else scale
    q = np.asarray(q, np.float64)
    o, spread = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    nb = min(len(block_row), -(-total // BLOCK) if total > 0 else 0)
    if nb == 0:
        return o, spread
    there = np.array([0 <= block_row[b] < P for b in range(nb)])
    slots = np.where(there, np.asarray(block_row[:nb]), 0)
    j = np.arange(nb * BLOCK)
    p = total - n + np.arange(n)
    seen = (j <= p[:, None]) & np.repeat(there, BLOCK)
    if window:
        seen &= j > p[:, None] - window
    some = seen.any(1)
    for h in range(Hk):
        k, v = (np.where(there[:, None, None], x[slots, h] * s[slots, h][:, None, None], 0.0).reshape(-1, d)
                for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        for g in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
            with np.errstate(invalid="ignore"):
                x = np.where(seen, np.where(seen, q[:, g] @ np.nan_to_num(k).T, 0) * scale, -np.inf)
                x = np.where(seen & np.isnan(k).any(1), np.nan, x)
                x = x - np.where(some, np.nan_to_num(np.nanmax(np.where(some[:, None], x, 0), 1)), 0)[:, None]
                w = np.exp(x)
                w = w / np.where(some, w.sum(1), 1)[:, None]
            o[:, g], spread[:, g] = w @ v, w @ np.abs(v)
    return o, spread
