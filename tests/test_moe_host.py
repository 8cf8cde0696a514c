"""Mixture of experts on the host: the oracle's pins, the refusals of the entry
points, the operators on meta tensors (no compute call is made)."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import moe_ref
from oracle import mxfp4_ref as ref


# ----------------------------------------------------------------- oracle
def test_route_closed_forms():
    x = np.log(np.array([[1.0, 5.0, 2.0, 8.0]]))
    w, ids = moe_ref.route(x, None, 2, True, renormalize=False)
    assert ids.tolist() == [[3, 1]] and np.allclose(w, [[8 / 16, 5 / 16]])
    w, ids = moe_ref.route(x, None, 2, True, renormalize=True, scale=2.5)
    assert np.allclose(w, [[2.5 * 8 / 13, 2.5 * 5 / 13]])
    w, ids = moe_ref.route(x, None, 4, False, renormalize=False)        # sigmoid(log a) = a / (1 + a)
    assert np.allclose(w, [[8 / 9, 5 / 6, 2 / 3, 1 / 2]]) and ids.tolist() == [[3, 1, 2, 0]]


def test_route_by_rationals():
    # scores a / (1 + a) plus a bias, groups of two by the sum of their best two:
    # the choice of exact fractions
    a = [Fraction(n, d) for n, d in ((3, 1), (1, 2), (4, 1), (1, 9), (2, 3), (5, 2), (7, 1), (1, 1))]
    b = [Fraction(n, 100) for n in (3, -40, -20, 55, 10, 0, -60, 21)]
    c = [v / (1 + v) + w for v, w in zip(a, b)]
    groups = sorted(range(4), key=lambda g: (-(c[2 * g] + c[2 * g + 1]), g))[:2]
    order = sorted((i for i in range(8) if i // 2 in groups), key=lambda i: (-c[i], i))[:3]
    x = np.log(np.array([[float(v) for v in a]]))
    w, ids = moe_ref.route(x, np.array([float(v) for v in b]), 3, False, 4, 2, 2)
    s = [a[i] / (1 + a[i]) for i in order]
    assert ids.tolist() == [order] and np.allclose(w[0], [float(v / sum(s)) for v in s], atol=1e-14)


def test_route_ties_masks_and_nothing_left():
    x = np.zeros((4, 6))
    x[1, :4] = -np.inf
    x[2] = -np.inf
    x[3, 2] = np.nan
    w, ids = moe_ref.route(x, None, 3, True)
    assert ids.tolist() == [[0, 1, 2], [4, 5, -1], [-1, -1, -1], [0, 1, 3]]
    assert np.allclose(w, [[1 / 3] * 3, [0.5, 0.5, 0], [0, 0, 0], [1 / 3] * 3])
    x[0, 3] = np.inf
    w, ids = moe_ref.route(x[:1], None, 2, True)
    assert ids[0, 0] == 3 and w[0].tolist() == [1, 0]


def test_linear_is_the_dense_product_of_each_expert():
    g = np.random.default_rng(0)
    codes = g.integers(0, 256, (3, 10, 16), dtype=np.uint8)
    scales = g.integers(120, 130, (3, 10, 1), dtype=np.uint8)
    x = g.standard_normal((4, 32))
    ids = np.array([[0, 2], [1, 1], [-1, 0], [2, 5]])
    y, mag = moe_ref.linear(x, ids, codes, scales, 32)
    xc, xs = ref.quantize_mxfp4(x)
    for t in range(4):
        for j in range(2):
            e = ids[t, j]
            if 0 <= e < 3:
                want, m = ref.mxfp4_gemm_f64(xc[t:t + 1], xs[t:t + 1], codes[e], scales[e], 32)
                assert np.allclose(y[t, j], want[0]) and np.allclose(mag[t, j], m[0])
            else:
                assert (y[t, j] == 0).all()


def test_activations():
    g, u = np.array([0.0, 1.0, -30.0, 9.0]), np.array([2.0, 3.0, 1.0, -20.0])
    assert np.allclose(moe_ref.act("silu", g, u), [0, 3 / (1 + np.exp(-1)), -30 * np.exp(-30), -180 / (1 + np.exp(-9))])
    assert np.allclose(moe_ref.act("swiglu", g, u)[[0, 3]], [0, 7 / (1 + np.exp(-1.702 * 7)) * -6])
    # the tanh form follows x Phi(x) to 1e-3
    phi = 0.8413447460685429
    assert abs(moe_ref.act("gelu", np.array([1.0]), np.array([1.0]))[0] - phi) < 1e-3


def test_epilogue_warps_leave_together():
    # a hardware barrier does not end without a warp that has left its role: the
    # warps that share it leave by what they all see, not by a wait that one of them
    # gave up, and no other role has such a barrier
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "mxfp4_quantized_gemm_gb300", "csrc", "moe_gemm.cu")) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    start = source.index("if (warp < kFirstEpiWarp)")
    epilogue = source.index("setmaxnreg.inc", start)
    end = source.index("__syncthreads", epilogue)
    assert "epi_barrier" not in source[start:epilogue] and "__syncthreads" not in source[start:end]
    role = source[epilogue:end]
    assert "epi_barrier();" in role and "next_of_all()" in role
    assert "next_segment()" not in role and not re.search(r"\b(break|return)\b", role)
    wait = source[source.index("auto next_of_all"):start]
    assert "mbar_wait(" not in wait and "clock64" not in wait and "no_more" in wait


# --------------------------------------------------------------- refusals
A = 1 << 20   # an aligned address that no refused call reads
ROUTE = dict(logits=A, dtype=0, ld=64, bias=A, T=4, E=64, top_k=8, score=1, n_group=8, topk_group=4, group_top=2,
             renormalize=True, scale=1.0, weights=A, ids=A)
LINEAR = dict(x=A, ldx=256, ids=A, w_packed=A, bias=A, out=A, ldo=512, T=4, top_k=2, E=8, N=512, K=256, workspace=A,
              workspace_bytes=1 << 40)
FFN = dict(x=A, ldx=256, ids=A, weights=A, w_gate_up=A, bias_gate_up=A, w_down=A, bias_down=A, residual=A, ldr=512,
           out=A, ldo=512, T=4, top_k=2, E=8, K=256, I=128, N=512, act=0, alpha=1.0, limit=7.0, workspace=A,
           workspace_bytes=1 << 40)
CALLS = {"mxfp4_moe_route": ROUTE, "mxfp4_moe_linear": LINEAR, "mxfp4_moe_ffn": FFN}


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import build
    build.build()
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


def status(capi, fn, base, **change):
    a = dict(base, **change)
    try:
        getattr(capi, fn)(*a.values(), stream=0)
    except capi.Mxfp4Error as e:
        return e.status
    return capi.OK


@pytest.mark.parametrize("fn", CALLS)
def test_refusals_common(capi, fn):
    base = CALLS[fn]
    may_be_null = ("bias", "bias_gate_up", "bias_down", "residual")
    for k in [k for k, v in base.items() if v == A and k != "workspace"]:
        if k not in may_be_null:
            assert status(capi, fn, base, **{k: None}) == capi.ERR_INVALID_ARG, k
        assert status(capi, fn, base, **{k: A + 1}) == capi.ERR_MISALIGNED, k
    for k in [k for k in base if k in ("T", "E", "top_k", "N", "K", "I", "n_group", "topk_group")]:
        assert status(capi, fn, base, **{k: 0}) == capi.ERR_INVALID_ARG, k
        assert status(capi, fn, base, **{k: -2}) == capi.ERR_INVALID_ARG, k
    for k in [k for k in base if k.startswith("ld")]:
        assert status(capi, fn, base, **{k: base[k] - 1}) == capi.ERR_UNSUPPORTED_SHAPE, k
    assert status(capi, fn, base, E=1025 if fn != "mxfp4_moe_route" else 1032) == capi.ERR_UNSUPPORTED_SHAPE
    assert status(capi, fn, base, top_k=33) == capi.ERR_UNSUPPORTED_SHAPE
    if "workspace" in base:
        assert status(capi, fn, base, K=255) == capi.ERR_UNSUPPORTED_SHAPE
        assert status(capi, fn, base, T=1 << 28) == capi.ERR_UNSUPPORTED_SHAPE
        assert status(capi, fn, base, T=1 << 27, K=1024, ldx=1024) == capi.ERR_UNSUPPORTED_SHAPE   # row tiles x k-tiles
        assert status(capi, fn, base, workspace=None) == capi.ERR_WORKSPACE
        assert status(capi, fn, base, workspace_bytes=1000) == capi.ERR_WORKSPACE
        assert status(capi, fn, base, workspace=A + 8) == capi.ERR_MISALIGNED
        for k in ("w_packed", "w_gate_up", "w_down"):
            if k in base:
                assert status(capi, fn, base, **{k: A + 8}) == capi.ERR_MISALIGNED


def test_refusals_of_each(capi):
    bad, shape = capi.ERR_INVALID_ARG, capi.ERR_UNSUPPORTED_SHAPE
    for change, want in ((dict(dtype=2), bad), (dict(score=2), bad), (dict(group_top=0), bad), (dict(group_top=3), bad),
                         (dict(n_group=7), shape), (dict(n_group=64), shape), (dict(topk_group=9), shape),
                         (dict(topk_group=1, top_k=9), shape), (dict(n_group=1, topk_group=2), shape)):
        assert status(capi, "mxfp4_moe_route", ROUTE, **change) == want, change
    assert status(capi, "mxfp4_moe_route", ROUTE, dtype=1, logits=A + 2) == capi.ERR_MISALIGNED
    assert status(capi, "mxfp4_moe_ffn", FFN, act=3) == bad
    assert status(capi, "mxfp4_moe_ffn", FFN, act=-1) == bad
    assert status(capi, "mxfp4_moe_ffn", FFN, I=127) == shape


def test_ffn_refuses_clamps_without_a_meaning(capi):
    nan, inf = float("nan"), float("inf")
    clamp = dict(FFN, act=2, workspace_bytes=0)         # (what is accepted goes as far as the workspace)
    for change in (dict(limit=-1.0), dict(limit=nan), dict(limit=-inf), dict(alpha=nan), dict(alpha=inf)):
        assert status(capi, "mxfp4_moe_ffn", clamp, **change) == capi.ERR_INVALID_ARG, change
        for act in (0, 1):                              # they ignore both
            assert status(capi, "mxfp4_moe_ffn", dict(clamp, act=act), **change) == capi.ERR_WORKSPACE, change
    for change in (dict(), dict(limit=0.0), dict(limit=inf), dict(alpha=0.0), dict(alpha=-3e38)):
        assert status(capi, "mxfp4_moe_ffn", clamp, **change) == capi.ERR_WORKSPACE, change
    from mxfp4_quantized_gemm_gb300 import ops
    ffn = dict(x=meta(7, 256), ids=meta(7, 2, dtype=torch.int32), weights=meta(7, 2, dtype=torch.float32),
               w_gate_up=meta(ops._packed_weight_bytes(8, 192, 256), dtype=torch.uint8), bias_gate_up=None,
               w_down=meta(ops._packed_weight_bytes(8, 300, 96), dtype=torch.uint8), bias_down=None, residual=None, E=8,
               I=96, N=300, act="swiglu_clamp", alpha=1.702, limit=inf)
    assert torch.ops.mxfp4.moe_ffn(**ffn).shape == (7, 300)
    for change in (dict(limit=-1.0), dict(limit=nan), dict(alpha=inf)):
        with pytest.raises(RuntimeError, match="mxfp4::moe_ffn"):
            torch.ops.mxfp4.moe_ffn(**dict(ffn, **change))


def test_workspace_queries(capi):
    lin, ffn = capi.mxfp4_moe_linear_workspace_bytes, capi.mxfp4_moe_ffn_workspace_bytes
    assert lin(0, 8, 64, 512, 256) == 0 and lin(4, 8, 64, 512, 255) == 0 and lin(4, 33, 64, 512, 256) == 0
    assert ffn(4, 8, 64, 256, 0, 512) == 0 and ffn(4, 8, 64, 256, 127, 512) == 0 and ffn(4, 8, 2000, 256, 128, 512) == 0
    assert 0 < lin(4, 8, 64, 512, 256) < ffn(4, 8, 64, 256, 128, 512)
    # the tokens' blocks: one row tile of 17408 bytes per k-tile and expert at least
    assert lin(1000, 8, 64, 512, 512) - lin(1000, 8, 64, 512, 256) == (8000 // 128 + 64) * 17408


# -------------------------------------------------- operators without a GPU
def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_operators_trace_and_refuse_on_meta_tensors():
    from mxfp4_quantized_gemm_gb300 import ops
    mx, i32, f32, u8 = torch.ops.mxfp4, torch.int32, torch.float32, torch.uint8

    def packed(E, N, K):
        return meta(ops._packed_weight_bytes(E, N, K), dtype=u8)

    route = dict(logits=meta(2, 5, 64), bias=meta(64, dtype=f32), top_k=6, score="sigmoid", n_group=8, topk_group=4,
                 group_top=2, renormalize=True, scale=2.5)
    w, ids = mx.moe_route(**route)
    assert w.shape == ids.shape == (2, 5, 6) and w.dtype == f32 and ids.dtype == i32
    linear = dict(x=meta(2, 5, 256), ids=meta(2, 5, 6, dtype=i32), w_packed=packed(8, 300, 256), bias=meta(8, 300), E=8,
                  N=300)
    assert mx.moe_linear(**linear).shape == (2, 5, 6, 300)
    ffn = dict(x=meta(7, 256), ids=meta(7, 2, dtype=i32), weights=meta(7, 2, dtype=f32), w_gate_up=packed(8, 192, 256),
               bias_gate_up=meta(8, 192), w_down=packed(8, 300, 96), bias_down=None, residual=meta(7, 300), E=8, I=96,
               N=300, act="silu", alpha=1.0, limit=7.0)
    assert mx.moe_ffn(**ffn).shape == (7, 300)
    assert mx.pack_gate_up(meta(3, 600, 128, dtype=u8), meta(3, 600, 8, dtype=u8), 256).numel() == 3 * 3 * 34816

    def refuses(op, base, **change):
        with pytest.raises(RuntimeError, match="mxfp4::moe|mxfp4::pack"):
            op(**dict(base, **change))

    for change in (dict(logits=meta(2, 64, dtype=torch.float16)), dict(bias=meta(64)), dict(bias=meta(63, dtype=f32)),
                   dict(top_k=33), dict(top_k=0), dict(score="relu"), dict(n_group=7), dict(topk_group=0),
                   dict(group_top=3), dict(top_k=17, topk_group=2), dict(logits=meta(2, 1032))):
        refuses(mx.moe_route, route, **change)
    for change in (dict(x=meta(2, 5, 256, dtype=f32)), dict(ids=meta(2, 5, 6, dtype=torch.int64)),
                   dict(ids=meta(10, 6, dtype=i32)), dict(w_packed=packed(7, 300, 256)), dict(bias=meta(7, 300)),
                   dict(ids=meta(2, 5, 33, dtype=i32)), dict(E=0)):
        refuses(mx.moe_linear, linear, **change)
    for change in (dict(weights=meta(7, 3, dtype=f32)), dict(weights=meta(7, 2)), dict(act="relu"), dict(I=95),
                   dict(residual=meta(7, 256)), dict(w_gate_up=packed(7, 192, 256)), dict(w_down=packed(4, 300, 96)),
                   dict(bias_gate_up=meta(8, 96)), dict(bias_down=meta(300))):
        refuses(mx.moe_ffn, ffn, **change)
    refuses(mx.pack_gate_up, dict(codes=meta(3, 601, 128, dtype=u8), scales=meta(3, 601, 8, dtype=u8), K=256))
