"""Plain float64 restatement of the 4-bit key/value cache's operators (numpy, no GPU).

Rounding: blocks of 32 channels; the scale is the smallest power of two 2^k with
amax <= 6 * 2^k, k in [-23, 13] (2^0 for a zero block); codes are e2m1, nearest with ties
to the even code, saturating. A block with a non-finite value is scale byte 255: NaN.
"""

from __future__ import annotations

import numpy as np

PAGE, BLOCK = 256, 32
K_MIN, K_MAX = -23, 13
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def norm_rotate(x, gamma, eps, pos, rope_dims, base):
    """x [T, H, D] at positions pos [T] -> normed (gamma None: not) and rotated, float64."""
    x = np.asarray(x, dtype=np.float64)
    if gamma is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(gamma, dtype=np.float64)
    y = x.copy()
    r = rope_dims
    if r:
        theta = float(base) ** (-2.0 * np.arange(r // 2) / r)
        ang = np.asarray(pos, dtype=np.float64)[:, None, None] * theta
        a, b = x[..., x.shape[-1] - r::2], x[..., x.shape[-1] - r + 1::2]
        y[..., x.shape[-1] - r::2] = a * np.cos(ang) - b * np.sin(ang)
        y[..., x.shape[-1] - r + 1::2] = a * np.sin(ang) + b * np.cos(ang)
    return y


def scale_bytes(amax):
    """Scale byte of blocks with these largest magnitudes."""
    amax = np.asarray(amax, dtype=np.float64)
    out = np.full(amax.shape, 127, dtype=np.int64)
    for i, a in np.ndenumerate(amax):
        if not np.isfinite(a):
            out[i] = 255
        elif a > 0:
            k = K_MIN
            while k < K_MAX and a > 6.0 * 2.0 ** k:
                k += 1
            out[i] = k + 127
    return out


def codes_of(x, sbytes):
    """Codes (0..15, one per value) of x [..., dim] under the scale bytes [..., dim/32]."""
    x = np.asarray(x, dtype=np.float64)
    sb = np.repeat(np.asarray(sbytes), BLOCK, axis=-1)
    a = np.abs(np.where(sb == 255, 0, x)) / np.exp2(np.where(sb == 255, 0, sb - 127).astype(np.float64))
    mid = (GRID[1:] + GRID[:-1]) / 2
    mag = np.zeros(a.shape, dtype=np.int64)
    for i, m in enumerate(mid):  # between codes i and i + 1; a tie goes to the even one
        mag += (a > m) | ((a == m) & ((i + 1) % 2 == 0))
    return np.where(sb == 255, 0, mag + 8 * np.signbit(x))


def decode(codes, sbytes):
    """Values of codes [..., dim] (one per value) and scale bytes [..., dim/32]."""
    codes = np.asarray(codes)
    sb = np.repeat(np.asarray(sbytes).astype(np.int64), BLOCK, axis=-1)
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return np.where(sb == 255, np.nan, v * np.exp2((sb - 127).astype(np.float64)))


def unpack(packed):
    packed = np.asarray(packed).astype(np.int64)
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)


def round4(x):
    """x [..., dim] -> the values that its 4-bit form stands for."""
    x = np.asarray(x, dtype=np.float64)
    sb = scale_bytes(amax_of(x))
    return decode(codes_of(x, sb), sb)


def amax_of(x):
    b = np.abs(np.asarray(x, dtype=np.float64)).reshape(*x.shape[:-1], -1, BLOCK)
    return np.where(np.isfinite(b).all(-1), b.max(-1), np.inf)


def attention(q, k, v, start, scale):
    """New tokens q [n, Hq, D] at positions start.. over k, v [start + n, Hk, D]; returns out
    [n, Hq, D], lse [n, Hq], sum_j p_j |v_j| [n, Hq, D], max_j scale * sum_d |q_d k_jd| [n, Hq]."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, top = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        for i in range(n):
            m = min(start + i + 1, k.shape[0])
            if m == 0:
                continue
            s = scale * (kh[:m] @ q[i, h])
            mx = s.max()
            p = np.exp(s - mx)
            lse[i, h] = mx + np.log(p.sum())
            p /= p.sum()
            out[i, h], mag[i, h] = p @ vh[:m], p @ np.abs(vh[:m])
            top[i, h] = scale * (np.abs(kh[:m]) @ np.abs(q[i, h])).max()
    return out, lse, mag, top
