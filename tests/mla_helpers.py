"""Inputs, calls and tolerances of the latent-attention tests.

Tolerances, from the roundings that the kernels make (bf16 half step 2^-8
relative, fp32 2^-24):
- an attention output: its own rounding, 2^-8 |out|, and the softmax weights'
  rounding, 2^-8 sum_j w_j |v_j|; the scores' fp32 sums, the exponentials and
  the fp32 sums of the output add relative weight errors far below 2^-9 at the
  tests' sizes, for which another 2^-9 of the same sum is left.  Over a whole
  tensor the roundings are independent, each at most 2^-8 / sqrt(3) of its
  value in the mean square: together below 2^-8 of the tensor's norm.
- a log-sum-exp: (terms of a score + terms of the sum) 2^-24 times the
  scores' sums of magnitudes (plus 1 for the sum of weights).
"""

from __future__ import annotations

import numpy as np
import torch

BF = torch.bfloat16
HALF = float(torch.finfo(BF).eps) / 2      # 2^-8
U32 = 2.0 ** -24


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def rnd(seed: int, *shape, scale: float = 1.0, device="cuda") -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(BF).to(device)


def check_attention(out, lse, want, keys: int, dims: int, what: str) -> None:
    w_out, w_lse, mag, smag = want
    got, got_lse = f64(out), f64(lse)
    assert np.isfinite(got).all(), f"{what}: {int((~np.isfinite(got)).sum())} outputs are not finite"
    err = np.abs(got - w_out)
    tol = HALF * np.abs(w_out) + (HALF + HALF / 2) * mag + 1e-30
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outputs off, worst {np.max(err / tol):.2f} tolerances, " \
        f"first at {tuple(np.argwhere(bad)[0])}"
    norm = np.linalg.norm(w_out)
    assert np.linalg.norm(got - w_out) <= HALF * norm + 1e-30, f"{what}: relative error of the tensor above 2^-8"
    empty = np.isneginf(w_lse)
    assert np.array_equal(np.isneginf(got_lse), empty), f"{what}: empty rows"
    ltol = (dims + keys) * U32 * (smag + 1) + 4 * U32 * np.abs(np.where(empty, 0, w_lse))
    bad = np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, w_lse)) > ltol
    assert not bad.any(), f"{what}: {int(bad.sum())} log-sums off"


def paged(seed: int, lens, page: int, L: int = 512, R: int = 64, extra: int = 1, fill: float = 1.0, width=None):
    """A cache in shuffled pages whose unused rows hold NaN, and its table
    (unused entries -1)."""
    need = [-(-int(n) // page) for n in lens]
    pages = sum(need) + extra
    cache = rnd(seed, pages, page, L + R, scale=fill, device="cpu")
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 1))
    table = torch.full((len(lens), max(1, max(need)) if width is None else width), -1, dtype=torch.int32)
    used = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for s, n in enumerate(lens):
        for i in range(need[s]):
            p = int(order[at])
            table[s, i] = p
            used[p, : min(page, int(n) - i * page)] = True
            at += 1
    cache[~used] = float("nan")
    return cache.cuda(), table.cuda()


def run_decode(capi, q_lat, q_rope, cache, table, lens, q_len: int, scale: float, out=None, lse=None, stream=None):
    """q_lat [H, T, L] and q_rope [T, H, R] views, through the C ABI."""
    H, T, L = q_lat.shape
    S, R = lens.shape[0], q_rope.shape[2]
    if out is None:
        out = torch.full((H, T, L), float("nan"), dtype=BF, device="cuda")
    if lse is None:
        lse = torch.full((T, H), float("nan"), dtype=torch.float32, device="cuda")
    n = capi.mxfp4_mla_decode_workspace_bytes(S, q_len, H, L, table.shape[1] * cache.shape[1])
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    capi.mxfp4_mla_decode(q_lat, q_lat.stride(1), q_lat.stride(0), q_rope, q_rope.stride(0), q_rope.stride(1), cache,
                          cache.stride(0), cache.shape[1], cache.shape[0], table, table.stride(0), table.shape[1], lens,
                          out, out.stride(1), out.stride(0), lse, S, q_len, H, L, R, scale, ws, n, stream)
    return out, lse


def run_prefill(capi, q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, scale: float, causal: bool, out=None, lse=None,
                stream=None):
    Tq, H, dn = q_nope.shape
    Tk, dv = v.shape[0], v.shape[2]
    if out is None:
        out = torch.full((Tq, H, dv), float("nan"), dtype=BF, device="cuda")
    if lse is None:
        lse = torch.full((Tq, H), float("nan"), dtype=torch.float32, device="cuda")
    capi.mxfp4_mla_prefill(q_nope, q_nope.stride(0), q_nope.stride(1), q_rope, q_rope.stride(0), q_rope.stride(1),
                           k_nope, k_nope.stride(0), k_nope.stride(1), k_rope, k_rope.stride(0), v, v.stride(0),
                           v.stride(1), cu_q, cu_k, cu_q.shape[0] - 1, out, out.stride(0), out.stride(1), lse, Tq, Tk,
                           H, dn, k_rope.shape[1], dv, scale, causal, stream)
    return out, lse
