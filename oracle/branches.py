"""Float64 definitions of the operators that decode several branches of one prompt.

Plain numpy on the host, one row, branch or beam at a time. Inputs are float
arrays (widened by the caller), outputs float64 or integers; nothing is shared
with the GPU path.
"""
from __future__ import annotations

import numpy as np


def rotate(x, pos, inv_freq, rot, interleaved, factor=1.0):
    """x [..., d]: its first `rot` elements rotated by pos * inv_freq."""
    y = np.array(x, dtype=np.float64)
    if rot == 0:
        return y
    ang = float(pos) * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang) * factor, np.sin(ang) * factor
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    xa, xb = np.array(y[..., a]), np.array(y[..., b])
    y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
    return y


def norm_rope(x, gain, eps, pos, inv_freq, rot, interleaved, factor=1.0):
    """One row's heads x [heads, d]: RMS norm (gain None: none), then rotate."""
    x = np.asarray(x, dtype=np.float64)
    if gain is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(gain, dtype=np.float64)
    return rotate(x, pos, inv_freq, rot, interleaved, factor)


def attend(q, k, v, scale):
    """q [group, d] over k, v [n, d]: (outputs, log of the softmax denominator, sum of p |v|)."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    if k.shape[0] == 0:
        z = np.zeros_like(q)
        return z, np.full(q.shape[0], -np.inf), z
    s = q @ k.T * scale
    m = np.max(s, axis=1, keepdims=True)
    p = np.exp(s - m)
    l = np.sum(p, axis=1, keepdims=True)
    return p @ v / l, (m + np.log(l))[:, 0], p @ np.abs(v) / l


def beam_select(logits, scores, n_out):
    """(scores, parents, tokens) [n_out] of the best continuations; lowest flat index among equals."""
    x = np.array(logits, dtype=np.float64)
    x[np.isnan(x)] = -np.inf
    cand = []
    for b in range(x.shape[0]):
        m = np.max(x[b])
        if not np.isfinite(m) or not np.isfinite(scores[b]):
            continue
        key = float(scores[b]) + ((x[b] - m) - np.log(np.sum(np.exp(x[b] - m))))  # (m first: it may be the lowest float)
        v = np.flatnonzero(x[b] > -np.inf)
        v = v[np.argsort(-key[v], kind="stable")][:n_out]
        cand += [(-key[t], b, int(t)) for t in v]
    cand.sort()
    cand = cand[:n_out] + [(np.inf, -1, -1)] * (n_out - min(n_out, len(cand)))
    return (np.array([-c[0] for c in cand]), np.array([c[1] for c in cand], dtype=np.int64),
            np.array([c[2] for c in cand], dtype=np.int64))


def beam_reorder(pools, old_table, old_len, parents, spare, page):
    """pools: list of [layers][pages][n_kv][page][d], copied; returns (pools, new_table, new_len)."""
    pools = [np.array(p) for p in pools]
    table, length = np.full_like(old_table, -1), np.full_like(old_len, -1)
    for i, p in enumerate(parents):
        if p < 0 or old_len[p] < 0:
            continue
        full, rest = divmod(int(old_len[p]), page)
        table[i, :full], table[i, full], length[i] = old_table[p, :full], spare[i], old_len[p]
        if rest:
            for pool in pools:
                pool[:, spare[i], :, :rest] = pool[:, old_table[p, full], :, :rest]
    return pools, table, length
