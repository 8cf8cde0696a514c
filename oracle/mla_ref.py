"""Latent attention in plain float64 numpy: what enters the paged cache, the
absorbed attention over it and the expanded attention of ragged prompts, from
the definitions (softmax(q k) v, RMSNorm, plane rotations).  Row by row, with
no tiles and no running maxima.

Each attention returns, beside the output and the log-sum-exp, the sums of
magnitudes that bound what roundings can do: ``mag`` = sum_j w_j |v_j| of an
output, ``smag`` = max_j scale * sum_k |q_k| |k_jk| of a row's scores.
"""

from __future__ import annotations

import numpy as np


def rmsnorm(x: np.ndarray, gamma: np.ndarray, eps: float) -> np.ndarray:
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * gamma


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [..., R] turned pair by pair; cos, sin broadcast to [..., R / 2]."""
    R = x.shape[-1]
    out = np.empty_like(x)
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        out[..., a] = x[..., a] * cos[..., i] - x[..., b] * sin[..., i]
        out[..., b] = x[..., b] * cos[..., i] + x[..., a] * sin[..., i]
    return out


def store_rows(kv, gamma, eps, cos_sin, positions, L, interleaved):
    """The cache rows [T, L + R] of the new tokens."""
    R = kv.shape[1] - L
    cs = cos_sin[positions]
    key = rotate(kv[:, L:], cs[:, : R // 2], cs[:, R // 2:], interleaved)
    return np.concatenate((rmsnorm(kv[:, :L], gamma, eps), key), axis=1)


def store_queries(q, cos_sin, positions, interleaved):
    R = q.shape[-1]
    cs = cos_sin[positions][:, None]
    return rotate(q, cs[..., : R // 2], cs[..., R // 2:], interleaved)


def attend(q, k, v, scale):
    """One query [D] over keys [n, D] and values [n, E]: (out, lse, mag, smag)."""
    if k.shape[0] == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    s = scale * (k @ q)
    m = s.max()
    w = np.exp(s - m)
    total = w.sum()
    w = w / total
    smag = abs(scale) * (np.abs(k) @ np.abs(q)).max()
    return w @ v, m + np.log(total), w @ np.abs(v), smag


def decode(q_lat, q_rope, cache, table, lens, q_len, scale):
    """q_lat [H, T, L], q_rope [T, H, R], cache [pages, page, L + R], table
    [S, W], lens [S] -> out [H, T, L], lse [T, H], mag, smag."""
    H, T, L = q_lat.shape
    page = cache.shape[1]
    out, mag = np.zeros((H, T, L)), np.zeros((H, T, L))
    lse, smag = np.full((T, H), -np.inf), np.zeros((T, H))
    for s, n in enumerate(lens):
        rows = np.array([cache[table[s, j // page], j % page] for j in range(int(n))]).reshape(-1, cache.shape[2])
        for i in range(q_len):
            t, see = s * q_len + i, max(0, int(n) - q_len + 1 + i)
            for h in range(H):
                q = np.concatenate((q_lat[h, t], q_rope[t, h]))
                out[h, t], lse[t, h], mag[h, t], smag[t, h] = attend(q, rows[:see], rows[:see, :L], scale)
    return out, lse, mag, smag


def prefill(q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, scale, causal):
    """[T, H, *] tensors -> out [Tq, H, dv], lse [Tq, H], mag, smag."""
    Tq, H, _ = q_nope.shape
    dv = v.shape[2]
    out, mag = np.zeros((Tq, H, dv)), np.zeros((Tq, H, dv))
    lse, smag = np.full((Tq, H), -np.inf), np.zeros((Tq, H))
    for s in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        for h in range(H):
            k = np.concatenate((k_nope[k0:k1, h], k_rope[k0:k1]), axis=1)
            for i in range(q1 - q0):
                see = max(0, min(k1 - k0, i + 1 + (k1 - k0) - (q1 - q0))) if causal else k1 - k0
                q = np.concatenate((q_nope[q0 + i, h], q_rope[q0 + i, h]))
                t = q0 + i
                out[t, h], lse[t, h], mag[t, h], smag[t, h] = attend(q, k[:see], v[k0:k0 + see, h], scale)
    return out, lse, mag, smag
