"""One MLA layer with MXFP4 weights: a prompt, then tokens one by one.

    python examples/latent_attention.py [--heads 64] [--prompt 1000] [--steps 4]

The prompt goes through the expanded form (K and V of every head from the
latents, then ``mla_prefill``), each later token through the absorbed form (the
K-up product, ``mla_decode`` over the paged latent cache, the V-up product).
Both read the cache rows that ``mla_store`` wrote.  The last prompt token is
computed both ways, which must agree to bf16 roundings.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mxfp4_quantized_gemm_gb300 import ops  # noqa: E402,F401  (registers torch.ops.mxfp4.*)

L, R, DN, DV, PAGE, EPS = 512, 64, 192, 256, 64, 1e-6
mx = torch.ops.mxfp4


def fp4_codes(*shape: int, gen: torch.Generator) -> torch.Tensor:
    """Random E2M1 values as one 4-bit code per byte."""
    return torch.randint(0, 16, shape, generator=gen, device="cuda", dtype=torch.uint8)


def pack(values: torch.Tensor, exponent: int) -> torch.Tensor:
    """[.., N, K] E2M1 values, one per byte, all scaled by 2^exponent -> packed weights."""
    codes = values[..., 0::2] | (values[..., 1::2] << 4)
    K = values.shape[-1]
    scales = torch.full((*values.shape[:-1], -(-K // 32)), 127 + exponent, dtype=torch.uint8, device="cuda")
    return mx.pack_weights(codes.contiguous(), scales, K)


class LatentAttention:
    """Query and latent projections, the latent cache, and both forms of the
    attention; weights are random."""

    def __init__(self, hidden: int, heads: int, pages: int, most_positions: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.scale = heads, (DN + R) ** -0.5
        self.w_q = pack(fp4_codes(heads * (DN + R), hidden, gen=gen), -7)
        self.w_kv = pack(fp4_codes(L + R, hidden, gen=gen), -7)
        # the expanding matrix of each head: DN rows give its keys, DV rows its
        # values.  One scale throughout, so that its transpose (the absorbed
        # K-up) is the same matrix.
        up = fp4_codes(heads, DN + DV, L, gen=gen)
        self.w_expand = pack(up, -6)
        self.w_k_up = pack(up[:, :DN].transpose(1, 2).contiguous(), -6)
        self.w_v_up = pack(up[:, DN:].contiguous(), -6)
        self.gamma = torch.ones(L, dtype=torch.bfloat16, device="cuda")
        freq = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        angles = torch.arange(most_positions, device="cuda", dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat((angles.cos(), angles.sin()), 1).float()
        self.cache = torch.zeros(pages, PAGE, L + R, dtype=torch.bfloat16, device="cuda")

    def _project(self, x, positions, slots):
        """Queries of the new tokens (the rotated part apart), their rows in the cache."""
        q = mx.linear(x, self.w_q, None, self.H * (DN + R)).view(-1, self.H, DN + R)
        kv = mx.linear(x, self.w_kv, None, L + R)
        q_rope = mx.mla_store(kv, self.gamma, EPS, q[..., DN:], self.cos_sin, positions, slots, self.cache, True)
        return q[..., :DN], q_rope

    def prefill(self, x, positions, slots, cu):
        """New prompts x [T, hidden], sequence s in rows cu[s] .. cu[s + 1]: [T, H, DV]."""
        q_nope, q_rope = self._project(x, positions, slots)
        rows = self.cache.view(-1, L + R)[slots]
        latents = rows[:, :L].expand(self.H, -1, -1)
        kv = mx.a16wfp4_bmm(latents, self.w_expand, DN + DV, True)                    # [T, H, DN + DV]
        return mx.mla_prefill(q_nope, q_rope, kv[..., :DN], rows[:, L:], kv[..., DN:], cu, cu, self.scale, True)[0]

    def decode(self, x, positions, slots, page_table, seq_lens):
        """The newest tokens x [S, hidden] of S sequences (seq_lens with them): [S, H, DV]."""
        q_nope, q_rope = self._project(x, positions, slots)
        q_lat = mx.a16wfp4_bmm(q_nope.transpose(0, 1), self.w_k_up, L, False)         # [H, S, L]
        o, _ = mx.mla_decode(q_lat, q_rope, self.cache, page_table, seq_lens, self.scale)
        return mx.a16wfp4_bmm(o, self.w_v_up, DV, True)                               # [S, H, DV]


def run(heads: int = 64, prompt: int = 1000, steps: int = 4, hidden: int = 1024) -> float:
    """Largest difference of the two forms for the last prompt token, relative to its largest value."""
    total = prompt + steps
    need = -(-total // PAGE)
    layer = LatentAttention(hidden, heads, need + 3, total)
    table = (torch.randperm(need + 3, device="cuda")[:need]).to(torch.int32)[None]
    at = torch.arange(total, device="cuda")
    slots = table[0, at // PAGE].long() * PAGE + at % PAGE
    x = torch.randn(total, hidden, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, prompt], dtype=torch.int32, device="cuda")
    expanded = layer.prefill(x[:prompt], at[:prompt], slots[:prompt], cu)
    last = prompt - 1

    def step(t: int):
        return layer.decode(x[t:t + 1], at[t:t + 1], slots[t:t + 1], table,
                            torch.tensor([t + 1], dtype=torch.int32, device="cuda"))

    absorbed = step(last)
    for t in range(prompt, total):
        out = step(t)
        assert out.isfinite().all()
    diff = (absorbed[0].float() - expanded[last].float()).abs().max() / expanded[last].float().abs().max()
    return float(diff)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    print(f"{a.prompt} prompt tokens, {a.steps} decoded, {a.heads} heads: absorbed against expanded form of the last "
          f"prompt token, relative difference {run(a.heads, a.prompt, a.steps):.4f}")
