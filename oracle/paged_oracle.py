"""float64 definitions of the rotation by position and of the paged-cache operators (test
infrastructure, numpy only)."""
from __future__ import annotations

import math

import numpy as np

from oracle.cache_oracle import attend

E4M3_TOP = 448.0


def e4m3_values() -> np.ndarray:
    """What the 256 codes of e4m3 stand for: sign, 4 exponent bits (bias 7), 3 mantissa bits; no
    infinities, the two codes with all other bits set are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if c & 127 == 127 else -x if c & 128 else x
    return out


def frequencies(rot_dim, theta, scaling="plain", factor=1.0, low=1.0, high=1.0, context=1.0):
    """(radians per position of each pair, factor of the rotated part)."""
    w = np.array([theta ** (-2.0 * j / rot_dim) for j in range(rot_dim // 2)])
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "bands":
        wave = 2 * math.pi / w
        m = (context / wave - low) / (high - low)
        return np.where(wave < context / high, w, np.where(wave > context / low, w / factor,
                                                           (1 - m) * w / factor + m * w)), 1.0
    if scaling == "ramp":
        at = [rot_dim * math.log(context / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high, low)]
        a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot_dim - 1)
        m = np.clip((np.arange(rot_dim // 2) - a) / max(b - a, 0.001), 0.0, 1.0)
        return m * w / factor + (1 - m) * w, 0.1 * math.log(factor) + 1.0
    return w, 1.0


def rotate(x, pos, layout, w, gain=1.0):
    """x [n, heads, 128] turned by pos [n]; returns (y, |a| + |b| of each element's pair, 0 where
    nothing turns)."""
    x = np.asarray(x, dtype=np.float64)
    n = len(w)
    i = np.arange(n) if layout == "halves" else 2 * np.arange(n)
    j = i + (n if layout == "halves" else 1)
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * w
    c, s = np.cos(ang) * gain, np.sin(ang) * gain
    y, size = x.copy(), np.zeros_like(x)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return y, size


def gather(pool, pages, n):
    """Positions 0 .. n - 1 of one sequence: pool [page, slot, head, 128] -> [n, head, 128]."""
    ps = pool.shape[1]
    at = np.arange(n)
    return pool[np.asarray(pages)[at // ps], at % ps]


def decode(q, k, v):
    """One sequence: q [n_kv, 4, 128], k, v [L, n_kv, 128].  (h, sum a |v|, largest sum |q_i k_i|)."""
    L, n = k.shape[:2]
    h, mean, mag = np.zeros(q.shape), np.zeros(q.shape), 0.0
    for g in range(n if L else 0):
        _, hg, mg, big = attend(q[None, g], k[:, g], v[:, g], np.ones((1, L), dtype=bool))
        h[g], mean[g], mag = hg[0], mg[0], max(mag, big)
    return h, mean, mag
