"""The latent-attention oracle for calls of many rows: the same definitions and
results as ``oracle.mla_ref`` (which goes row by row), in float64 tensors, all
heads of a sequence at a time, on the device of the inputs."""

from __future__ import annotations

import numpy as np
import torch


def attend(q, k, v, see, scale):
    """q [H, m, D], k [H or 1, n, D], v [H or 1, n, E], see [m] visible keys of
    each row -> out [H, m, E], lse [H, m], mag [H, m, E], smag [H, m]."""
    H, m, _ = q.shape
    n = k.shape[1]
    if n == 0 or m == 0:
        z = q.new_zeros(H, m, v.shape[2])
        return z, q.new_full((H, m), -float("inf")), z.clone(), q.new_zeros(H, m)
    hidden = torch.arange(n, device=q.device) >= see[:, None]
    s = (scale * (q @ k.transpose(1, 2))).masked_fill_(hidden, -float("inf"))
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    w = w / torch.where(total > 0, total, torch.ones_like(total))
    smag = (abs(scale) * (q.abs() @ k.abs().transpose(1, 2))).masked_fill_(hidden, 0.0).amax(-1)
    return w @ v, lse, w @ v.abs(), smag


def decode(q_lat, q_rope, cache, table, lens, q_len, scale):
    """As oracle.mla_ref.decode, of tensors; numpy results."""
    H, T, L = q_lat.shape
    page, width = cache.shape[1], cache.shape[2]
    flat, dev = cache.reshape(-1, width), q_lat.device
    q = torch.cat((q_lat, q_rope.transpose(0, 1)), 2).double()
    out, lse = torch.zeros(H, T, L, dtype=torch.float64, device=dev), torch.zeros(T, H, dtype=torch.float64, device=dev)
    mag, smag = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        j = torch.arange(int(n), device=dev)
        rows = flat[table[b].long()[j // page] * page + j % page].double()[None]
        t = slice(b * q_len, (b + 1) * q_len)
        see = (int(n) - q_len + 1 + torch.arange(q_len, device=dev)).clamp(min=0)
        out[:, t], a, mag[:, t], c = attend(q[:, t], rows, rows[..., :L], see, scale)
        lse[t], smag[t] = a.T, c.T
    return tuple(x.cpu().numpy() for x in (out, lse, mag, smag))


def prefill(q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, scale, causal):
    """As oracle.mla_ref.prefill, of tensors; numpy results."""
    Tq, H, _ = q_nope.shape
    dev = q_nope.device
    out = torch.zeros(Tq, H, v.shape[2], dtype=torch.float64, device=dev)
    lse = torch.zeros(Tq, H, dtype=torch.float64, device=dev)
    mag, smag = torch.zeros_like(out), torch.zeros_like(lse)
    for s in range(len(cu_q) - 1):
        q0, q1, k0, k1 = (int(x) for x in (cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]))
        n = k1 - k0
        see = torch.full((q1 - q0,), n, device=dev)
        if causal:
            see = (torch.arange(q1 - q0, device=dev) + 1 + n - (q1 - q0)).clamp(0, n)
        q = torch.cat((q_nope[q0:q1], q_rope[q0:q1]), 2).double().transpose(0, 1)
        kr = k_rope[k0:k1, None].expand(n, H, k_rope.shape[1])
        k = torch.cat((k_nope[k0:k1], kr), 2).double().transpose(0, 1)
        o, a, g, c = attend(q, k, v[k0:k1].double().transpose(0, 1), see, scale)
        out[q0:q1], lse[q0:q1], mag[q0:q1], smag[q0:q1] = o.transpose(0, 1), a.T, g.transpose(0, 1), c.T
    return tuple(x.cpu().numpy() for x in (out, lse, mag, smag))


# ------------------------------------------------- how the kernels share work
def decode_units(lens, row_groups: int, over: int, tile: int = 64) -> list[int]:
    """Work units of each row group in order: `over` for going over to it and
    its tiles, or one for an empty sequence."""
    return [1 if n == 0 else over + -(-int(n) // tile) for n in lens for _ in range(row_groups)]


def cut_places(units: list[int], blocks: int, over: int) -> set[int]:
    """Where blocks begin inside a group that holds anything, in units from the
    group's first: 0 .. over, and -1 for further in."""
    ends = np.cumsum(units)
    total = int(ends[-1])
    q, r = divmod(total, blocks)
    at = set()
    for b in range(1, blocks):
        u = b * q + min(b, r)
        g = int(np.searchsorted(ends, u, side="right"))
        off = u - (int(ends[g]) - units[g])
        if units[g] > 1:
            at.add(off if off <= over else -1)
    return at
