"""Inputs, calls and tolerances of the mixture-of-experts tests.

Tolerances, from the roundings that the kernels make (bf16 half step 2^-8
relative, fp32 2^-24):
- a router's weight: the exponential's argument is rounded in fp32 (|x - m| up
  to 40 in the tests: 40 * 2^-24), the exponential is good to 2 ulp, the sums
  of up to E terms and the divisions add a few more: together below 2^-17.
- moe_linear: helpers.check_close, as for the GEMM.
- moe_ffn: the fp32 sums of the first product (n_acc additions of its sum of
  magnitudes, as for the GEMM) and the activation (fast exponential and
  division, 2^-17 relative with arguments up to 40) move h by at most d.
  Where that can change a block's scale or an element's code, the largest
  change counts, times the second product's weights.  Then the second
  product's fp32 sums, the rounding of each slot's result to bf16, the fp32
  sum over slots and the result's rounding.
"""

from __future__ import annotations

import numpy as np
import torch

from helpers import dev_bf16, dev_u8, empty_u8, host_bits, pack_weights
from mxfp4_quantized_gemm_gb300 import synth
from oracle import moe_ref
from oracle import mxfp4_ref as ref

HALF = float(torch.finfo(torch.bfloat16).eps) / 2      # 2^-8
U32 = 2.0 ** -24
WEIGHT_TOL = 2.0 ** -17


def n_acc(K: int) -> int:
    return -(-K // 64) + 4


def routing(T: int, E: int, k: int, seed: int, empty: float = 0.0, skew: float = 0.0):
    """ids int32 [T, k] (a share `empty` of the slots -1) and weights fp32."""
    g = np.random.default_rng(seed)
    p = np.exp(-skew * np.arange(E))
    ids = np.array([g.choice(E, size=k, replace=False, p=p / p.sum()) for _ in range(T)], dtype=np.int32)
    ids[g.random((T, k)) < empty] = -1
    return ids, g.random((T, k), dtype=np.float32) + np.float32(0.1)


class Experts:
    """E random matrices [N, K] in codes and scales, packed on the device."""

    def __init__(self, capi, E: int, N: int, K: int, seed: int, bias: bool):
        at = -round(np.log2(2.9 * np.sqrt(K)))
        self.E, self.N, self.K = E, N, K
        self.codes = synth.weight_codes(N, K, seed, batch=E)
        self.scales = synth.weight_scales(N, K, at - 1, at + 1, seed, batch=E)
        self.bias = np.stack([synth.bias(N, seed=seed + e, sigma=0.3) for e in range(E)]) if bias else None
        self.packed = pack_weights(capi, self.codes, self.scales, K) if capi else None
        self.bias_dev = dev_bf16(self.bias) if capi and bias else None

    def bias64(self, e: int):
        return None if self.bias is None else ref.bf16_bits_to_f64(self.bias[e])


def dev_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def dev_f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def run_route(capi, logits, bias, top_k, score, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0,
              stream=None):
    T, E = logits.shape
    w = torch.full((T, top_k), float("nan"), device="cuda")
    ids = torch.full((T, top_k), -7, dtype=torch.int32, device="cuda")
    capi.mxfp4_moe_route(logits, capi.DTYPE_BF16 if logits.dtype == torch.bfloat16 else capi.DTYPE_F32, logits.stride(0),
                         bias, T, E, top_k, capi.MOE_SOFTMAX if score == "softmax" else capi.MOE_SIGMOID, n_group,
                         topk_group, group_top, renormalize, scale, w, ids, stream)
    return w, ids


def workspace(n: int) -> torch.Tensor:
    """A workspace as a caller may leave it: 0xFF everywhere (NaN scales, -1 counts)."""
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")


def run_linear(capi, x, ids, w: Experts, out=None, ws=None, stream=None):
    T, k = ids.shape
    if out is None:
        out = torch.full((T * k, w.N), float("nan"), dtype=torch.bfloat16, device="cuda")
    n = capi.mxfp4_moe_linear_workspace_bytes(T, k, w.E, w.N, w.K)
    ws = workspace(n) if ws is None else ws
    capi.mxfp4_moe_linear(x, x.stride(0), ids, w.packed, w.bias_dev, out, out.stride(0), T, k, w.E, w.N, w.K, ws, n,
                          stream)
    return out


def run_ffn(capi, x, ids, weights, up: Experts, down: Experts, act: str, residual=None, out=None, ws=None, stream=None):
    T, k = ids.shape
    kind = {"silu": capi.MOE_SILU, "gelu": capi.MOE_GELU_TANH, "swiglu": capi.MOE_SWIGLU_CLAMP}[act]
    if out is None:
        out = torch.full((T, down.N), float("nan"), dtype=torch.bfloat16, device="cuda")
    n = capi.mxfp4_moe_ffn_workspace_bytes(T, k, up.E, up.K, down.K, down.N)
    ws = workspace(n) if ws is None else ws
    capi.mxfp4_moe_ffn(x, x.stride(0), ids, weights, up.packed, up.bias_dev, down.packed, down.bias_dev, residual,
                       0 if residual is None else residual.stride(0), out, out.stride(0), T, k, up.E, up.K, down.K,
                       down.N, kind, 1.702, 7.0, ws, n, stream)
    return out


def _moves(h, d):
    """How far the quantized values of blocks h [rows, n] can move where h is off by at most d."""
    rows, n = h.shape
    pad = -n % 32
    hb = np.pad(h, ((0, 0), (0, pad))).reshape(rows, -1, 32)
    db = np.pad(d, ((0, 0), (0, pad))).reshape(rows, -1, 32)

    def at(v, e):
        a = np.minimum(np.abs(np.ldexp(v, -e)), 6.0)
        q = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
        return np.copysign(np.ldexp(np.rint(a / q) * q, e), v)

    most = np.abs(hb).max(2, keepdims=True)
    lo, hi = (np.abs(hb) - db).max(2, keepdims=True), (np.abs(hb) + db).max(2, keepdims=True)

    def exponent(m):
        return np.maximum(np.frexp(np.maximum(m, 1e-300))[1] - 1, -125) - 2

    here = at(hb, exponent(most))
    far = np.zeros_like(hb)
    for e in (exponent(lo), exponent(hi)):
        for v in (hb - db, hb + db):
            far = np.maximum(far, np.abs(at(v, e) - here))
    return here.reshape(rows, -1)[:, :n], far.reshape(rows, -1)[:, :n]


def want_ffn(x_bits, ids, weights, up: Experts, down: Experts, act: str, residual_bits=None):
    """(exact value, tolerance) of moe_ffn's output."""
    T, k = ids.shape
    q = moe_ref.quantized(ref.bf16_bits_to_f64(x_bits), up.K)
    out, tol = np.zeros((T, down.N)), np.zeros((T, down.N))
    if residual_bits is not None:
        out = ref.bf16_bits_to_f64(residual_bits)
    mags = np.abs(out)
    for e in np.unique(ids[(ids >= 0) & (ids < up.E)]):
        t, j = np.nonzero(ids == e)
        z, mag = moe_ref.product(q[t], up.codes[e], up.scales[e], up.K, up.bias64(e))
        dz = n_acc(up.K) * U32 * mag
        gate, upv = z[:, 0::2], z[:, 1::2]
        dg, du = dz[:, 0::2], dz[:, 1::2]
        h = moe_ref.act(act, gate, upv)
        outer = np.abs(np.clip(upv, -7, 7) + 1) if act == "swiglu" else np.abs(upv)
        d = 1.2 * outer * dg + np.abs(gate) * du + 2.0 ** -17 * np.abs(h)    # |act'| < 1.2, |act(g)| <= |g|
        hq, far = _moves(h, d)
        y, ymag = moe_ref.product(hq, down.codes[e], down.scales[e], down.K, down.bias64(e))
        w2 = np.abs(ref.dequantize_mxfp4(down.codes[e], down.scales[e], down.K))
        ty = far @ w2.T + n_acc(down.K) * U32 * ymag
        ty = ty + HALF * (np.abs(y) + ty)
        w = weights[t, j].astype(np.float64)[:, None]
        np.add.at(out, t, w * y)
        np.add.at(tol, t, np.abs(w) * ty)
        np.add.at(mags, t, np.abs(w * y))
    tol = tol + (k + 1) * U32 * mags
    return out, tol + HALF * (np.abs(out) + tol)


def check_ffn(out, want, what: str):
    exact, tol = want
    got = ref.bf16_bits_to_f64(host_bits(out))
    assert np.isfinite(got).all(), f"{what}: {int((~np.isfinite(got)).sum())} outputs are not finite"
    err = np.abs(got - exact)
    bad = err > tol + 1e-30
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outputs off, worst {np.max(err / (tol + 1e-30)):.2f} " \
        f"tolerances, first at {tuple(np.argwhere(bad)[0])}"
    norm = np.linalg.norm(exact)
    assert np.linalg.norm(got - exact) <= 2 * HALF * norm + 1e-30, f"{what}: the tensor is off by more than 2^-7"
