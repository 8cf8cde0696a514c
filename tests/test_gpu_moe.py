"""Mixture of experts on the GPU against the plain 64-bit oracle: the router's
choice and weights, the experts' products and the gated network, at sizes and
routings where they can go wrong."""

import numpy as np
import pytest
import torch

from helpers import check_close, dev_bf16, host_bits
from moe_helpers import (Experts, WEIGHT_TOL, check_ffn, dev_f32, dev_i32, n_acc, routing, run_ffn, run_linear,
                         run_route, want_ffn)
from mxfp4_quantized_gemm_gb300 import synth
from oracle import moe_ref
from oracle import mxfp4_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


def ok(capi):
    torch.cuda.synchronize()
    assert capi.mxfp4_get_device_error() == capi.OK


# ------------------------------------------------------------------- route
def check_route(capi, logits, bias, top_k, score, **kw):
    dev = logits.cuda()
    w, ids = run_route(capi, dev, None if bias is None else bias.cuda(), top_k, score, **kw)
    ok(capi)
    want_w, want = moe_ref.route(logits.double().numpy(), None if bias is None else bias.double().numpy(), top_k,
                                 score == "softmax", **kw)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want), f"rows {np.unique(np.nonzero(got != want)[0])[:8]}"
    got_w = w.double().cpu().numpy()
    assert (np.abs(got_w - want_w) <= WEIGHT_TOL * np.abs(want_w) + 1e-37).all(), np.abs(got_w - want_w).max()
    return got


def logits_of(T, E, seed, bf16=False, scale=1.5):
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * scale
    return x.to(BF) if bf16 else x


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,keep,top", [
    (1, 1, 1, 1, 1, 1), (3, 5, 5, 1, 1, 1), (33, 33, 4, 1, 1, 1), (70, 64, 8, 1, 1, 1), (129, 128, 8, 8, 3, 1),
    (50, 160, 6, 8, 3, 2), (97, 256, 8, 8, 4, 2), (31, 255, 32, 1, 1, 1), (20, 513, 7, 1, 1, 1),
    (9, 1024, 32, 32, 32, 2), (17, 96, 3, 32, 5, 2), (40, 60, 16, 4, 2, 2)])
@pytest.mark.parametrize("bias,bf16,renorm", [(False, True, True), (True, False, False), (True, True, True)])
def test_route(capi, score, T, E, k, groups, keep, top, bias, bf16, renorm):
    x = logits_of(T, E, T + E, bf16)
    b = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.1 if bias else None
    check_route(capi, x, b, k, score, n_group=groups, topk_group=keep, group_top=top, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(96, 8), (96, 12), (72, 8), (160, 8), (160, 4), (192, 8), (192, 12), (384, 8),
                                      (384, 4), (300, 3), (384, 1), (160, 1)])
@pytest.mark.parametrize("bias,bf16,top", [(False, True, 1), (False, False, 1), (True, True, 2), (False, True, 2)])
def test_route_groups_that_are_whole_lanes_or_not(capi, score, E, groups, bias, bf16, top):
    x = logits_of(60, E, E + groups, bf16)
    x[40:] = torch.round(x[40:])                     # ties of experts and of groups
    x[:, 5::7] = -float("inf")
    b = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.1 if bias else None
    keep = max(1, groups // 3)
    check_route(capi, x, b, min(8, E // groups * keep), score, n_group=groups, topk_group=keep, group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_ties_go_to_the_lower_index(capi, score, bias):
    x = torch.zeros(40, 64)
    x[10:] = torch.randint(0, 3, (30, 64), generator=torch.Generator().manual_seed(1)).float()
    b = torch.zeros(64) if bias else None
    got = check_route(capi, x, b, 8, score)
    assert (got[:10] == np.arange(8)).all()
    check_route(capi, x, b, 8, score, n_group=8, topk_group=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_decides_near_values_in_64_bits(capi, score, groups):
    # a bias that all but cancels the scores' differences: neighbours differ by
    # less than an fp32 step
    T, E = 64, 128
    row = logits_of(1, E, 5)
    x = row.repeat(T, 1)
    s = torch.softmax(row.double(), 1)[0] if score == "softmax" else torch.sigmoid(row.double())[0]
    b = (0.9 - s).float()
    c = s + b.double()
    assert c.max() - c.min() < 2 ** -23 and len(torch.unique(c)) > E // 2
    x[T // 2:, ::2] += logits_of(T // 2, E // 2, 6, scale=0.3)
    check_route(capi, x, b, 8, score, n_group=groups, topk_group=max(1, groups // 2), group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masks_infinities_and_nan(capi, score, bias, groups):
    x = logits_of(12, 40, 9)
    x[0] = -np.inf                          # nothing left
    x[1, 3:] = -np.inf                      # fewer than top_k
    x[2] = float("nan")
    x[3, ::2] = float("nan")
    x[4, 7] = np.inf
    x[5, [2, 30]] = np.inf                  # two share the weight
    x[6] = torch.finfo(torch.float32).min
    x[7, 20:] = torch.finfo(torch.float32).min
    x[8] = 200.0                            # saturated scores
    x[9] = -200.0
    x[9, 4] = -199.0
    x[10] = -torch.arange(40.0) * 40        # scores from 1 down to nothing
    b = torch.linspace(-0.3, 0.3, 40) if bias else None
    if bias:
        b[0], b[5] = -np.inf, float("nan")
    got = check_route(capi, x, b, 6, score, n_group=groups, topk_group=max(1, groups // 2), group_top=2)
    assert (got[0] == -1).all() and (got[2] == -1).all() and (got[1, 3:] == -1).all()


def test_route_strided_rows_and_the_last_row_alone(capi):
    wide = logits_of(21, 80, 11).cuda()
    a = run_route(capi, wide[:, 8:72], None, 4, "softmax")
    b = run_route(capi, wide[:, 8:72].contiguous(), None, 4, "softmax")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    w, ids = run_route(capi, wide[20:, 8:72], None, 4, "softmax")
    assert torch.equal(ids[0], a[1][20]) and torch.equal(w[0], a[0][20])
    ok(capi)


# ------------------------------------------------------------------ linear
def check_linear(capi, T, k, E, N, K, seed=0, bias=True, empty=0.0, skew=0.0, ids=None, x=None, **kw):
    w = Experts(capi, E, N, K, seed, bias)
    x = synth.activations(T, K, seed) if x is None else x
    if ids is None:
        ids = routing(T, E, k, seed, empty, skew)[0]
    out = run_linear(capi, dev_bf16(x), dev_i32(ids), w, **kw)
    ok(capi)
    acc, mag = moe_ref.linear(ref.bf16_bits_to_f64(x), ids, w.codes, w.scales, K,
                              None if w.bias is None else ref.bf16_bits_to_f64(w.bias))
    got = host_bits(out)[:, :N].reshape(T, k, N)
    check_close(got, acc, mag, n_acc(K), what=f"moe_linear T={T} k={k} E={E} N={N} K={K}", K=K)
    assert (got[ids < 0] == 0).all()
    return out


@pytest.mark.parametrize("T,k,E,N,K", [
    (1, 1, 1, 64, 64), (1, 8, 16, 300, 512), (5, 2, 3, 257, 34), (16, 4, 8, 512, 1024), (130, 1, 2, 256, 256),
    (64, 3, 5, 1001, 1510), (300, 2, 4, 130, 770), (700, 2, 3, 768, 2048)])
@pytest.mark.parametrize("bias", [False, True])
def test_linear(capi, T, k, E, N, K, bias):
    check_linear(capi, T, k, E, N, K, seed=T + N, bias=bias)


@pytest.mark.parametrize("counts", [[128], [129], [127, 0, 1], [0, 0, 256], [16, 17, 15, 1], [0, 640, 3]])
def test_linear_rows_at_the_tiles_edges(capi, counts):
    ids = np.concatenate([np.full(n, e) for e, n in enumerate(counts)]).astype(np.int32)
    ids = np.random.default_rng(3).permutation(ids)[:, None]
    check_linear(capi, len(ids), 1, len(counts), 520, 600, ids=ids)


def test_linear_empty_slots_and_edge_rows(capi):
    x = synth.with_edge_rows(synth.activations(90, 512, 4), seed=4)
    check_linear(capi, 90, 4, 7, 260, 512, empty=0.4, x=x)
    check_linear(capi, 6, 2, 3, 100, 64, ids=np.full((6, 2), -1, dtype=np.int32))


def test_linear_more_tiles_than_blocks(capi):
    # whole rounds of tiles, then cut ones
    check_linear(capi, 260, 4, 12, 4100, 300, skew=0.2)


def test_linear_the_same_expert_twice_and_ids_out_of_range(capi):
    w = Experts(capi, 4, 200, 128, 2, True)
    x = dev_bf16(synth.activations(3, 128, 2))
    ids = np.array([[1, 1, 3], [0, 4, 1 << 20], [-5, 2, -(1 << 31)]], dtype=np.int32)
    out = run_linear(capi, x, dev_i32(ids), w)
    torch.cuda.synchronize()
    assert capi.mxfp4_get_device_error() == capi.ERR_INDEX
    assert capi.mxfp4_get_device_error() == capi.OK
    out = host_bits(out).reshape(3, 3, 200)
    assert np.array_equal(out[0, 0], out[0, 1]) and (out[1, 1:] == 0).all() and (out[2, 0] == 0).all()
    good = np.where((ids >= 0) & (ids < 4), ids, -1)
    acc, mag = moe_ref.linear(ref.bf16_bits_to_f64(synth.activations(3, 128, 2)), good, w.codes, w.scales, 128,
                              ref.bf16_bits_to_f64(w.bias))
    check_close(out, acc, mag, n_acc(128), what="ids out of range", K=128)


def test_linear_a_row_that_is_not_finite_stays_alone(capi):
    x = synth.activations(40, 256, 8)
    x[7, 3], x[9, 40] = 0x7F80, 0x7FC1
    w = Experts(capi, 3, 64, 256, 8, False)
    ids = routing(40, 3, 2, 8)[0]
    got = ref.bf16_bits_to_f64(host_bits(run_linear(capi, dev_bf16(x), dev_i32(ids), w))).reshape(40, 2, 64)
    ok(capi)
    bad = np.zeros(40, dtype=bool)
    bad[[7, 9]] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def test_linear_strides_and_what_lies_between(capi):
    T, k, E, N, K = 19, 3, 4, 130, 200
    w = Experts(capi, E, N, K, 6, True)
    x = synth.activations(T, K, 6)
    ids = routing(T, E, k, 6, 0.2)[0]
    plain = run_linear(capi, dev_bf16(x), dev_i32(ids), w)
    for ldx, ldo, at in ((K + 8, N + 6, 0), (K + 3, N + 1, 1), (K, N + 8, 8)):
        xw = torch.zeros(T * ldx + 8, dtype=BF, device="cuda")[at:at + T * ldx].view(T, ldx)
        xw[:, :K] = dev_bf16(x)
        out = torch.full((T * k * ldo + 8,), 7.0, dtype=BF, device="cuda")[at:at + T * k * ldo].view(T * k, ldo)
        run_linear(capi, xw, dev_i32(ids), w, out=out)
        assert torch.equal(out[:, :N], plain) and (out[:, N:] == 7).all()
    ok(capi)


# --------------------------------------------------------------------- ffn
def check_network(capi, T, k, E, K, I, N, act="silu", seed=0, bias=True, res=True, empty=0.0, skew=0.0, ids=None):
    up, down = Experts(capi, E, 2 * I, K, seed, bias), Experts(capi, E, N, I, seed + 100, bias)
    x = synth.activations(T, K, seed)
    drawn, weights = routing(T, E, k, seed, empty, skew)
    ids = drawn if ids is None else ids
    weights[ids < 0] = np.nan                          # an empty slot's weight is not used
    r = synth.residual(T, N, seed, sigma=1.0) if res else None
    out = run_ffn(capi, dev_bf16(x), dev_i32(ids), dev_f32(weights), up, down, act, dev_bf16(r) if res else None)
    ok(capi)
    check_ffn(out, want_ffn(x, ids, weights, up, down, act, r), f"moe_ffn T={T} k={k} E={E} K={K} I={I} N={N} {act}")
    return out


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("T,k,E,K,I,N,bias,res", [
    (1, 1, 1, 64, 32, 64, False, False), (1, 8, 16, 512, 256, 512, False, True), (7, 2, 3, 98, 66, 101, True, True),
    (33, 4, 9, 1000, 362, 1000, True, False), (200, 2, 3, 640, 130, 264, True, True), (140, 1, 1, 256, 640, 300, False, True)])
def test_ffn(capi, act, T, k, E, K, I, N, bias, res):
    check_network(capi, T, k, E, K, I, N, act, seed=T + K, bias=bias, res=res)


@pytest.mark.parametrize("I", [2, 30, 64, 126, 128, 130, 254, 256, 258, 384, 386])
def test_ffn_widths_around_the_tiles(capi, I):
    check_network(capi, 20, 2, 3, 128, I, 72, seed=I)


def test_ffn_empty_slots_and_tokens_without_experts(capi):
    ids = routing(50, 6, 3, 5, 0.5)[0]
    ids[40:] = -1                                      # padding of a captured batch
    check_network(capi, 50, 3, 6, 256, 128, 256, ids=ids, seed=5)
    out = check_network(capi, 4, 2, 3, 64, 32, 40, ids=np.full((4, 2), -1, dtype=np.int32), res=False)
    assert (out == 0).all()


def test_ffn_many_tokens_of_one_expert(capi):
    check_network(capi, 900, 2, 5, 320, 192, 328, skew=1.0, seed=12)
