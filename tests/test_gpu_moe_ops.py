"""The mixture-of-experts operators of torch.ops.mxfp4 on the GPU: equal to the
C-ABI calls, views that need a copy, empty batches, opcheck, tracing, and the
layer of the example."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from helpers import dev_bf16, dev_u8
from moe_helpers import Experts, dev_f32, dev_i32, routing, run_ffn, run_linear, run_route
from mxfp4_quantized_gemm_gb300 import ops  # noqa: F401
from mxfp4_quantized_gemm_gb300 import synth

pytestmark = pytest.mark.gpu
mx = torch.ops.mxfp4
BF = torch.bfloat16


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


@pytest.fixture(scope="module")
def layer(capi):
    T, E, k, K, I, N = 42, 6, 3, 256, 96, 264
    up, down = Experts(capi, E, 2 * I, K, 1, True), Experts(capi, E, N, I, 2, True)
    ids, w = routing(T, E, k, 3, 0.1)
    return dict(up=up, down=down, x=dev_bf16(synth.activations(T, K, 4)), ids=dev_i32(ids), w=dev_f32(w),
                r=dev_bf16(synth.residual(T, N, 5)))


def ffn_args(L, **change):
    up, down = L["up"], L["down"]
    a = dict(x=L["x"], ids=L["ids"], weights=L["w"], w_gate_up=up.packed, bias_gate_up=up.bias_dev, w_down=down.packed,
             bias_down=down.bias_dev, residual=L["r"], E=up.E, I=down.K, N=down.N, act="silu", alpha=1.702, limit=7.0)
    return dict(a, **change)


def test_route_is_the_c_call(capi):
    x, b = torch.randn(30, 64, device="cuda"), torch.randn(64, device="cuda") * 0.1
    w, ids = mx.moe_route(x, b, 6, "sigmoid", 8, 4, 2, True, 2.5)
    w2, i2 = run_route(capi, x, b, 6, "sigmoid", 8, 4, 2, True, 2.5)
    assert torch.equal(w, w2) and torch.equal(ids, i2)
    # leading dimensions, rows with a stride, a transposed view, bf16
    w3, i3 = mx.moe_route(x.view(2, 15, 64), b, 6, "sigmoid", 8, 4, 2, True, 2.5)
    assert w3.shape == (2, 15, 6) and torch.equal(w3.view(30, 6), w) and torch.equal(i3.view(30, 6), ids)
    wide = torch.randn(30, 80, device="cuda")
    wide[:, 8:72] = x
    assert torch.equal(mx.moe_route(wide[:, 8:72], b, 6, "sigmoid", 8, 4, 2, True, 2.5)[1], ids)
    assert torch.equal(mx.moe_route(x.t().contiguous().t(), b, 6, "sigmoid", 8, 4, 2, True, 2.5)[1], ids)
    assert torch.equal(mx.moe_route(x[:1].expand(4, 64), b, 6, "sigmoid", 8, 4, 2, True, 2.5)[1], ids[:1].expand(4, 6))
    wb, ib = mx.moe_route(x.to(BF), None, 6, "softmax", 1, 1, 1, False, 1.0)
    w4, i4 = run_route(capi, x.to(BF), None, 6, "softmax", renormalize=False)
    assert torch.equal(wb, w4) and torch.equal(ib, i4)


def test_linear_and_ffn_are_the_c_calls(capi, layer):
    L, up = layer, layer["up"]
    T, k = L["ids"].shape
    y = mx.moe_linear(L["x"], L["ids"], up.packed, up.bias_dev, up.E, up.N)
    assert y.shape == (T, k, up.N) and torch.equal(y.view(T * k, -1), run_linear(capi, L["x"], L["ids"], up))
    out = mx.moe_ffn(**ffn_args(L))
    assert torch.equal(out, run_ffn(capi, L["x"], L["ids"], L["w"], up, L["down"], "silu", L["r"]))
    # leading dimensions; rows with a stride; a view that is copied; an odd offset of the weights
    lead = {n: L[n].view(2, T // 2, -1) for n in ("x", "ids", "w", "r")}
    got = mx.moe_ffn(**ffn_args(L, x=lead["x"], ids=lead["ids"], weights=lead["w"], residual=lead["r"]))
    assert got.shape == (2, T // 2, L["down"].N) and torch.equal(got.view(T, -1), out)
    wide = torch.zeros(T, 300, dtype=BF, device="cuda")
    wide[:, 7:263] = L["x"]
    assert torch.equal(mx.moe_ffn(**ffn_args(L, x=wide[:, 7:263])), out)
    assert torch.equal(mx.moe_ffn(**ffn_args(L, x=L["x"].t().contiguous().t(), ids=L["ids"].t().contiguous().t())), out)
    odd = torch.empty(up.packed.numel() + 1, dtype=torch.uint8, device="cuda")[1:].copy_(up.packed)
    assert torch.equal(mx.moe_ffn(**ffn_args(L, w_gate_up=odd)), out)


def test_pack_gate_up_interleaves(capi, layer):
    up = layer["up"]
    first = [torch.cat((v[:, 0::2], v[:, 1::2]), 1) for v in (dev_u8(up.codes), dev_u8(up.scales))]
    assert torch.equal(mx.pack_gate_up(*first, up.K), up.packed)
    one = [v[0] for v in first]
    assert torch.equal(mx.pack_gate_up(*one, up.K), up.packed[: up.packed.numel() // up.E])


def test_empty_batches(capi, layer):
    L, up = layer, layer["up"]
    w, ids = mx.moe_route(torch.randn(0, 64, device="cuda"), None, 4, "softmax", 1, 1, 1, True, 1.0)
    assert w.shape == ids.shape == (0, 4)
    assert mx.moe_linear(L["x"][:0], L["ids"][:0], up.packed, None, up.E, up.N).shape == (0, 3, up.N)
    assert mx.moe_ffn(**ffn_args(L, x=L["x"][:0], ids=L["ids"][:0], weights=L["w"][:0],
                                 residual=L["r"][:0])).shape == (0, L["down"].N)


def test_opcheck(capi, layer):
    L, up = layer, layer["up"]
    checks = ("test_schema", "test_faketensor")
    x = torch.randn(9, 32, device="cuda")
    torch.library.opcheck(mx.moe_route.default, (x, None, 4, "softmax", 4, 2, 1, True, 1.0), test_utils=checks)
    torch.library.opcheck(mx.moe_linear.default, (L["x"], L["ids"], up.packed, up.bias_dev, up.E, up.N), test_utils=checks)
    torch.library.opcheck(mx.moe_ffn.default, tuple(ffn_args(L).values()), test_utils=checks)
    torch.library.opcheck(mx.pack_gate_up.default, (dev_u8(up.codes), dev_u8(up.scales), up.K), test_utils=checks)


def test_compiled_layer_is_the_eager_one(capi, layer):
    L = layer
    gate = torch.randn(256, 6, device="cuda", dtype=BF)

    def block(x, r):
        w, ids = mx.moe_route(x @ gate, None, 3, "softmax", 1, 1, 1, True, 1.0)
        return torch.relu(mx.moe_ffn(**ffn_args(L, x=x, ids=ids, weights=w, residual=r)))

    want = block(L["x"], L["r"])
    assert torch.equal(torch.compile(block, backend="aot_eager", fullgraph=True)(L["x"], L["r"]), want)


def test_host_tensor_is_refused(capi, layer):
    with pytest.raises(RuntimeError, match="not a CUDA device"):
        mx.moe_ffn(**ffn_args(layer, ids=layer["ids"].cpu()))


def test_example_layer(capi):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixture_of_experts.py")
    spec = importlib.util.spec_from_file_location("mixture_of_experts_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # the fused network and the one put together from moe_linear differ where
    # the latter rounds gate, up and h to bf16 (2^-8 each) before h is rounded
    # to 4 bits: at most one step (2^-1 of a value in [4, 6]) of the few values
    # that lie that near a border (3 * 2^-8 / 2^-2 of them), summed over I
    # independent terms, beside the outputs' own roundings
    assert m.run(tokens=50, hidden=256, inner=128, experts=8) < np.sqrt(3 * 2.0 ** -6) * 0.5
    assert capi.mxfp4_get_device_error() == capi.OK
