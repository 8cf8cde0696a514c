"""One mixture-of-experts layer with MXFP4 weights.

    python examples/mixture_of_experts.py [--tokens 64] [--experts 32]

A router (``moe_route``) picks experts for each token by sigmoid scores with a
bias for balance; their gated networks (``moe_ffn``) are summed onto the shared
expert, a dense gated network, which is the same call with one expert.  The
layer is computed a second time from the experts' two products (``moe_linear``)
with the activation in between.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mxfp4_quantized_gemm_gb300 import ops  # noqa: E402,F401  (registers torch.ops.mxfp4.*)

mx = torch.ops.mxfp4


class MixtureOfExperts:
    """Router, experts and shared expert; weights are random."""

    def __init__(self, hidden: int, inner: int, experts: int, top_k: int, seed: int = 0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.K, self.I, self.E, self.top_k = hidden, inner, experts, top_k
        self.gate = torch.randn(hidden, experts, device="cuda", generator=self.gen) * hidden ** -0.5
        self.balance = torch.randn(experts, device="cuda", generator=self.gen) * 0.05
        self.gate_up, self.down = self._weights(experts, 2 * inner, hidden, mx.pack_gate_up), self._weights(
            experts, hidden, inner, mx.pack_weights)
        self.shared_gate_up, self.shared_down = self._weights(1, 2 * inner, hidden, mx.pack_gate_up), self._weights(
            1, hidden, inner, mx.pack_weights)

    def _weights(self, n: int, rows: int, K: int, pack) -> torch.Tensor:
        codes = torch.randint(0, 256, (n, rows, K // 2), generator=self.gen, device="cuda", dtype=torch.uint8)
        exponent = round(torch.log2(torch.tensor(2.9 * K ** 0.5)).item())    # products of unit rows near 1
        return pack(codes, torch.full((n, rows, -(-K // 32)), 127 - exponent, dtype=torch.uint8, device="cuda"), K)

    def route(self, x):
        return mx.moe_route(x.float() @ self.gate, self.balance, self.top_k, "sigmoid", 4, 2, 2, True, 2.5)

    def forward(self, x):
        """x [tokens, hidden] -> x + shared(x) + the sum of the experts' weighted results."""
        weights, ids = self.route(x)
        one, zero = torch.ones_like(weights[:, :1]), torch.zeros_like(ids[:, :1])
        y = mx.moe_ffn(x, zero, one, self.shared_gate_up, None, self.shared_down, None, x, 1, self.I, self.K, "silu", 1.0,
                       0.0)
        return mx.moe_ffn(x, ids, weights, self.gate_up, None, self.down, None, y, self.E, self.I, self.K, "silu", 1.0, 0.0)

    def in_steps(self, x):
        """The experts' sum alone, product by product."""
        weights, ids = self.route(x)
        z = mx.moe_linear(x, ids, self.gate_up, None, self.E, 2 * self.I)
        h = torch.nn.functional.silu(z[..., 0::2].float()) * z[..., 1::2].float()
        h = h.to(torch.bfloat16).view(-1, self.I)
        y = mx.moe_linear(h, ids.view(-1, 1), self.down, None, self.E, self.K).view(*ids.shape, self.K)
        return (y.float() * weights[..., None]).sum(1)

    def experts(self, x):
        weights, ids = self.route(x)
        return mx.moe_ffn(x, ids, weights, self.gate_up, None, self.down, None, None, self.E, self.I, self.K, "silu", 1.0,
                          0.0)


def run(tokens: int = 64, hidden: int = 1024, inner: int = 512, experts: int = 32, top_k: int = 4) -> float:
    """Difference of the fused experts and the ones put together, relative to the result (2-norms)."""
    layer = MixtureOfExperts(hidden, inner, experts, top_k)
    x = torch.randn(tokens, hidden, device="cuda", generator=layer.gen).to(torch.bfloat16)
    out = layer.forward(x)
    assert out.shape == x.shape and out.isfinite().all()
    want = layer.in_steps(x)
    return float((layer.experts(x).float() - want).norm() / want.norm())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=32)
    a = ap.parse_args()
    print(f"{a.tokens} tokens, {a.experts} experts: fused against stepwise experts, relative difference "
          f"{run(a.tokens, experts=a.experts):.4f}")
