"""float64 definitions of the cache operators (test infrastructure, numpy only): attention of
drafted trees over caches of per-sequence length, the accumulated key weights of a decode step,
the commit of an accepted path and eviction by weight."""
from __future__ import annotations

import math

import numpy as np

from oracle.gqa_oracle import f64, linear, rope

HPG = 4  # query heads per kv head


def tree_visibility(parents) -> np.ndarray:
    """bool [T, T] of a tree given by each token's parent (-1: the prefix): a token sees itself
    and its ancestors."""
    T = len(parents)
    vis = np.zeros((T, T), dtype=bool)
    for t, p in enumerate(parents):
        if p >= 0:
            vis[t] = vis[p]
        vis[t, t] = True
    return vis


def mask_words(vis) -> np.ndarray:
    """int32 words [B, T, ceil(T/32)] of visibility bits [B, T, T]."""
    B, T, _ = vis.shape
    W = (T + 31) // 32
    out = np.zeros((B, T, W), dtype=np.uint32)
    for j in range(T):
        out[:, :, j // 32] |= vis[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def attend(q, k, v, visible):
    """One kv head of one sequence: q [T, 4, 128], k, v [L, 128], visible [T, L] (bool).
    Returns (a [T, 4, L], h [T, 4, 128], |v| mean [T, 4, 128], largest sum |q_i k_i|); keys
    nobody sees may hold anything."""
    seen = visible.any(0)
    k = np.where(seen[:, None], f64(k), 0.0)
    v = np.where(seen[:, None], f64(v), 0.0)
    e = np.einsum("thd,ld->thl", f64(q), k) / math.sqrt(q.shape[-1])
    e = np.where(visible[:, None, :], e, -np.inf)
    top = e.max(-1, keepdims=True, initial=-np.inf)
    p = np.exp(e - np.where(np.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdims=True)
    a = p / np.where(total == 0, 1.0, total)
    mag = float((np.abs(f64(q)).reshape(-1, q.shape[-1]) @ np.abs(k).T).max(initial=0.0))
    return a, a @ v, a @ np.abs(v), mag


def cache_attention(q, cache_k, cache_v, lens, vis=None, n_new=0):
    """q [B, T, n_kv, 4, 128]; row t of sequence b sees positions < lens[b] and lens[b] + j for
    vis[b][t, j] (all n_new of them where vis is None).  Returns (h [B, T, n_kv, 4, 128],
    mean |v| of the same shape, key weights [B, n_kv, S] summed over rows and heads, largest
    sum |q_i k_i|)."""
    B, T, n = q.shape[:3]
    S = cache_k.shape[1]
    h = np.zeros(q.shape)
    av = np.zeros(q.shape)
    w = np.zeros((B, n, S))
    mag = 0.0
    for b in range(B):
        L = int(lens[b])
        end = L + n_new
        visible = np.ones((T, end), dtype=bool)
        if vis is not None:
            visible[:, L:] = vis[b][:, :n_new]
        for g in range(n):
            a, h[b, :, g], av[b, :, g], m = attend(q[b, :, g], cache_k[b, :end, g], cache_v[b, :end, g], visible)
            w[b, g, :end] = a.sum((0, 1))
            mag = max(mag, m)
    return h, av, w, mag


def block_ragged(x, wq, wk, wv, wo, R, cache_k, cache_v, lens, vis=None):
    """The block for T new positions of each sequence behind its own length: x [B, T, 4096], R
    [B, T, 64, 2].  Returns (delta [B, T, 4096], caches with the new positions, key weights)."""
    x = f64(x)
    B, T, _ = x.shape
    n = cache_k.shape[2]
    q = linear(x, wq).reshape(B, T, n * HPG, 128)
    k = linear(x, wk).reshape(B, T, n, 128)
    v = linear(x, wv).reshape(B, T, n, 128)
    ck, cv = f64(cache_k).copy(), f64(cache_v).copy()
    qr = np.empty_like(q)
    for b in range(B):
        qr[b] = rope(q[b:b + 1], R[b])[0]
        ck[b, lens[b]:lens[b] + T] = rope(k[b:b + 1], R[b])[0]
        cv[b, lens[b]:lens[b] + T] = v[b]
    h, _, w, _ = cache_attention(qr.reshape(B, T, n, HPG, 128), ck, cv, lens, vis, T)
    return linear(h.reshape(B, T, n * HPG * 128), wo), ck, cv, w


def commit(cache, lens, paths):
    """Copy of `cache` [B, S, ...] with positions lens[b] + paths[b][i] moved to lens[b] + i."""
    out = cache.copy()
    for b, path in enumerate(paths):
        at = [int(lens[b]) + j for j in path]
        out[b, lens[b]:lens[b] + len(path)] = cache[b, at]
    return out


def evict_positions(weights, length, budget, n_first, n_recent):
    """Ascending positions one kv head keeps: weights [S]."""
    if length <= budget:
        return list(range(length))
    middle = range(n_first, length - n_recent)
    heaviest = sorted(middle, key=lambda s: (math.isnan(weights[s]), -weights[s] if weights[s] == weights[s] else 0, s))
    keep = heaviest[:budget - n_first - n_recent]
    return sorted(list(range(n_first)) + keep + list(range(length - n_recent, length)))
