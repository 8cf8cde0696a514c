"""Mixture of experts in plain float64 numpy: the router's choice, each routed
token times its expert's MXFP4 weights, and the experts' gated network, from
the definitions.  Token by token and slot by slot, with no sorting by expert.

Beside a product each function returns the sums of magnitudes that bound what
fp32 sums and roundings can do to it.
"""

from __future__ import annotations

import numpy as np

from oracle import mxfp4_ref as ref


def route(logits, bias, top_k, softmax, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """logits [T, E] float64 -> (weights [T, top_k], ids [T, top_k])."""
    T, E = logits.shape
    weights, ids = np.zeros((T, top_k)), np.full((T, top_k), -1, dtype=np.int32)
    for t in range(T):
        x = np.where(np.isnan(logits[t]), -np.inf, logits[t])
        on = x > -np.inf
        s = np.zeros(E)
        if softmax:
            if on.any():
                m = x.max()
                s[on] = np.where(x[on] == m, 1.0, np.exp(np.minimum(x[on], 1e300) - min(m, 1e300)))
                s /= s.sum()
        else:
            s[on] = 1 / (1 + np.exp(-x[on]))
        c = x if bias is None else s + bias
        c = np.where(on & ~np.isnan(c), c, -np.inf)
        if n_group > 1:
            v = s if bias is None and group_top == 2 else c
            v = np.where(c > -np.inf, v, -np.inf).reshape(n_group, -1)
            value = []
            for g in range(n_group):
                best = sorted((a for a in v[g] if a > -np.inf), reverse=True)[:group_top]
                value.append(sum(best) if best else -np.inf)
            kept = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
            for g in range(n_group):
                if g not in kept:
                    c[g * (E // n_group):(g + 1) * (E // n_group)] = -np.inf
        chosen = sorted((i for i in range(E) if c[i] > -np.inf), key=lambda i: (-c[i], i))[:top_k]
        w = s[chosen]
        if renormalize and len(chosen):
            if softmax:      # the scores' ratios from the logits: they do not vanish together
                xs = x[chosen]
                w = np.where(xs == xs.max(), 1.0, np.exp(np.minimum(xs, 1e300) - min(xs.max(), 1e300)))
            elif w.sum() == 0:
                w = np.exp(x[chosen] - x[chosen].max())
            w = w / w.sum()
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = scale * w
    return weights, ids


def product(x, codes, scales, K, bias=None):
    """Rows of MXFP4 (values) times one expert's weights: (y, magnitudes)."""
    w = ref.dequantize_mxfp4(codes, scales, K)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    return y, mag


def quantized(x, K):
    """The values that the MXFP4 quantization of x stands for."""
    codes, scales = ref.quantize_mxfp4(x)
    return ref.dequantize_mxfp4(codes, scales, K)


def act(kind, gate, up, alpha=1.702, limit=7.0):
    with np.errstate(over="ignore"):
        if kind == "silu":
            return gate / (1 + np.exp(-gate)) * up
        if kind == "gelu":
            return 0.5 * gate * (1 + np.tanh(np.sqrt(2 / np.pi) * (gate + 0.044715 * gate ** 3))) * up
        gate, up = np.minimum(gate, limit), np.clip(up, -limit, limit)
        return gate / (1 + np.exp(-alpha * gate)) * (up + 1)


def linear(x, ids, codes, scales, K, bias=None):
    """x [T, K] float64, ids [T, k], codes [E, N, K / 2] -> (y, mag) [T, k, N]."""
    T, k = ids.shape
    q = quantized(x, K)
    y = np.zeros((T, k, codes.shape[1]))
    mag = np.zeros_like(y)
    for e in np.unique(ids[(ids >= 0) & (ids < codes.shape[0])]):
        t, j = np.nonzero(ids == e)
        y[t, j], mag[t, j] = product(q[t], codes[e], scales[e], K, None if bias is None else bias[e])
    return y, mag
