"""The operators around a bounded paged KV cache, as plain definitions in fp64.

Test infrastructure only (see the package docstring): the product never imports this.

* ``norm_rope``: per-head RMS norm and rotation by position of [T, H, D] heads.
* ``lse_and_weights``: every query row's log-sum-exp over its causal keys, and the weight every
  cached key received from a sequence's rows, summed over the rows and the q heads of a KV head.
* ``evict``: which of a head's cache entries stay (protected first, then heavier, ties to the
  lower index) and where they go (the k-th stray into the k-th hole).
"""
from __future__ import annotations

import math

import numpy as np

from .paged_attention import gather, row_positions

__all__ = ["norm_rope", "lse_and_weights", "evict"]


def norm_rope(x, weight, eps, inv_freq, axes, positions, interleaved):
    """x [T, H, D] float64; weight [D] or None; positions [n_axes, T]; returns (y, mag), mag
    [T, H, D] being the sum of magnitudes that went into each element (for error bounds)."""
    T, H, D = x.shape
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * weight
    out, mag = y.copy(), np.abs(y)
    n = len(inv_freq)
    for i in range(n):
        a = positions[axes[i]].astype(np.float64) * inv_freq[i]
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        out[..., u] = y[..., u] * c - y[..., v] * s
        out[..., v] = y[..., u] * s + y[..., v] * c
        mag[..., u] = mag[..., v] = np.abs(y[..., u]) + np.abs(y[..., v])
    return out, mag


def lse_and_weights(q, k_pool, block_table, cu_seqlens_q, ctx_lens, lse=None):
    """q [T, Hq, D], k_pool [nb, bs, Hkv, D] as floats. Returns (lse [T, Hq], per sequence the
    weights [Hkv, ctx]). With lse given, the weights are taken against it."""
    T, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    g = Hq // Hkv
    seq_of, pos_of = row_positions(cu_seqlens_q, ctx_lens)
    out = np.empty((T, Hq))
    weights = [np.zeros((Hkv, int(c))) for c in ctx_lens]
    keys = [gather(k_pool, block_table[s], int(c)) for s, c in enumerate(ctx_lens)]
    for t in range(T):
        s, n = int(seq_of[t]), int(pos_of[t]) + 1
        for h in range(Hq):
            x = keys[s][h // g, :n] @ q[t, h] / math.sqrt(D)
            m = x.max()
            out[t, h] = m + math.log(np.exp(x - m).sum())
            ref = out[t, h] if lse is None else lse[t, h]
            weights[s][h // g, :n] += np.exp(x - ref)
    return out, weights


def evict(weights, positions, n_tokens, budget, recent, sink):
    """One head: weights and token positions of its ctx entries. Returns source [min(ctx, budget)]:
    the entry that ends up at each index (itself where it stays)."""
    ctx = len(weights)
    length = min(ctx, budget)

    def order(j):
        w = weights[j]
        if positions[j] < sink or positions[j] >= n_tokens - recent:
            return (0, 0, 0.0, j)
        return (1, 0 if math.isnan(w) else 1, 0.0 if math.isnan(w) else -w, j)

    keep = set(sorted(range(ctx), key=order)[:length])
    source = list(range(length))
    strays = [j for j in range(length, ctx) if j in keep]
    for hole, stray in zip([j for j in range(length) if j not in keep], strays):
        source[hole] = stray
    return np.array(source, np.int64)
