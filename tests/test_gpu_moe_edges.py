"""Mixture of experts on the GPU at inputs that lie on a border: experts that
fp32 cannot tell apart beside equal ones, scores that vanish, groups whose
values cancel, gates whose square is infinite, rows that are not finite, clamps
at their limits."""

import numpy as np
import pytest
import torch

from helpers import dev_bf16, host_bits, pack_weights
from moe_helpers import Experts, dev_f32, dev_i32, routing, run_ffn, run_route
from mxfp4_quantized_gemm_gb300 import synth
from oracle import moe_ref
from oracle import mxfp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


def check_choice(capi, logits, bias, top_k, score, **kw):
    """The kernel's ids are those of the 64-bit oracle."""
    _, ids = run_route(capi, logits.cuda(), None if bias is None else bias.cuda(), top_k, score, **kw)
    torch.cuda.synchronize()
    assert capi.mxfp4_get_device_error() == capi.OK
    _, want = moe_ref.route(logits.double().numpy(), None if bias is None else bias.double().numpy(), top_k,
                            score == "softmax", **kw)
    got = ids.cpu().numpy()
    rows = np.unique(np.nonzero(got != want)[0])
    assert not len(rows), f"{len(rows)} rows, first {rows[0]}: {got[rows[0]]} for {want[rows[0]]}"


# numbers of experts for each number of logits a lane
SIZES = [33, 64, 96, 128, 160, 192, 256, 384, 512, 1024]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", SIZES)
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
@pytest.mark.parametrize("base,ulps", [(1.0, 1), (2.0 ** -20, 1), (-3.0, 2)])
def test_route_finds_a_higher_expert_behind_equal_ones(capi, score, E, bias, base, ulps):
    # all logits equal but for 0 to 12 that are a step of fp32 higher or two (the
    # scores of 2^-20 and its neighbour differ by 2^-45: more than pairs of fp32 tell)
    g = np.random.default_rng(E)
    x = np.full((40, E), base, dtype=np.float32)
    up = np.float32(base)
    for _ in range(ulps):
        up = np.nextafter(up, np.float32(100.0))
    higher = np.nextafter(up, np.float32(100.0))
    for t in range(1, 40):
        at = g.permutation(E)[:t % 13]
        x[t, at] = np.where(g.random(len(at)) < 0.3, higher, up)
    x[1, :], x[1, E - 1] = base, up                    # the last expert alone
    b = None if bias is None else torch.full((E,), bias)
    for k in (1, 8):
        check_choice(capi, torch.from_numpy(x), b, k, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", SIZES)
def test_route_finds_a_higher_bias_behind_equal_ones(capi, score, E):
    x, b = torch.ones(8, E), torch.zeros(E)
    b[E - 2] = 1e-7 if score == "sigmoid" else 1e-9
    x[4:, ::3] = -2.0
    for k in (1, 5):
        check_choice(capi, x, b, k, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(16, 4), (40, 4), (64, 8), (96, 32), (160, 8), (256, 8), (300, 3), (1024, 8)])
@pytest.mark.parametrize("bias", [None, 0.0])
def test_route_groups_whose_scores_vanish(capi, score, E, groups, bias):
    # scores down to 1e-200: nothing in fp32, and still in order
    gen = torch.Generator().manual_seed(E)
    x = 60.0 * torch.randn(60, E, generator=gen)
    if score == "sigmoid":
        x = -90.0 - x.abs()
    x[0] = -(400.0 / E) * torch.arange(E - 1, -1, -1.0)    # rising, the last group highest
    x[1] = -(400.0 / E) * torch.randperm(E, generator=gen)
    x[2] = -100.0                                       # all alike
    x[3] = torch.round(x[3] / 40) * 40                  # few values
    b = None if bias is None else torch.full((E,), bias)
    for keep in (2, groups - 1):
        k = min(32, E // groups * keep)
        check_choice(capi, x, b, k, score, n_group=groups, topk_group=keep, group_top=2)
        check_choice(capi, x, b, k, score, n_group=groups, topk_group=keep, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 32), (96, 32), (128, 32), (320, 32), (512, 32), (1024, 32)])
@pytest.mark.parametrize("large", [2.0 ** 14, 2.0 ** 18, 2.0 ** 40])
def test_route_groups_whose_best_two_cancel(capi, score, E, groups, large):
    # half of the groups: a bias of +large and one of -large, so that the sum is that of
    # two scores with an error that the other groups' sums do not have
    size = E // groups
    g = np.random.default_rng(E)
    x = torch.from_numpy(g.standard_normal((300, E)).astype(np.float32) * 3)
    b = np.full(E, -np.inf, dtype=np.float32)
    for n in range(groups):
        b[n * size:n * size + 2] = (large, -large) if n % 2 else (0.0, 0.0)
    if score == "softmax":
        b[~np.isfinite(b)] = -4 * large                  # these count for the sum, no further
    for keep in (1, 7, 16, 31):
        check_choice(capi, x, torch.from_numpy(b), min(32, 2 * keep), score, n_group=groups, topk_group=keep,
                     group_top=2)


@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (384, 8), (1024, 8)])
@pytest.mark.parametrize("at", [2.0 ** 17, -2.0 ** 19, 2.0 ** 21])
def test_route_groups_of_large_logits(capi, E, groups, at):
    # what a key drops of such a logit is not small beside 1
    x = at + 4.0 * torch.randn(100, E, generator=torch.Generator().manual_seed(E))
    for keep in (1, 3):
        check_choice(capi, x, None, 8, "softmax", n_group=groups, topk_group=keep, group_top=2)


@pytest.mark.parametrize("E", [256, 1024])
def test_route_softmax_scores_whose_sum_is_off(capi, E):
    # biases that cancel the scores to 2^-25 of them: what is left is as small as the
    # error of the sum of E exponentials, which is common to all scores
    for v in np.linspace(5.5, 9.0, 500).astype(np.float32):
        x = np.full((1, E), -v, dtype=np.float32)
        x[0, 5] = 0.0
        s = np.exp(x[0].astype(np.float64))
        b = (-s / s.sum()).astype(np.float32)
        check_choice(capi, torch.from_numpy(x), torch.from_numpy(b), 1, "softmax")


# ------------------------------------------------------------- large gates
def powers_network(capi, K=64, I=64, N=40):
    """Gates x[0], ups 1.5 x[32], results 32 h_0 + ...: every code is one power of two or 1.5."""
    up, down = Experts(capi, 1, 2 * I, K, 0, False), Experts(capi, 1, N, I, 0, False)
    up.codes[:], down.codes[:] = 0, 0x22                # (two codes a byte; 1.0 is 2, 1.5 is 3)
    up.codes[0, 0::2, 0] = 0x02
    up.codes[0, 1::2, 16] = 0x03
    for w in (up, down):
        w.scales[:] = 127
        w.packed = pack_weights(capi, w.codes, w.scales, w.K)
    return up, down


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("T", [14, 70, 300])
def test_ffn_gates_whose_square_is_infinite(capi, act, T):
    up, down = powers_network(capi)
    e = np.resize([3, 60, 63, 64, 66, 90, 110], T)
    sign = np.where(np.arange(T) % 14 < 7, 1.0, -1.0)
    x = np.zeros((T, 64), dtype=np.float32)
    x[:, 0], x[:, 32] = sign * 2.0 ** e, 1.0
    bits = synth.f32_to_bf16_bits(x)
    ids, w = np.zeros((T, 1), dtype=np.int32), np.ones((T, 1), dtype=np.float32)
    got = ref.bf16_bits_to_f64(host_bits(run_ffn(capi, dev_bf16(bits), dev_i32(ids), dev_f32(w), up, down, act)))
    torch.cuda.synchronize()
    assert capi.mxfp4_get_device_error() == capi.OK
    # h is one value in all columns, far from the borders of its rounding
    h = moe_ref.act(act, x[:, :1].astype(np.float64), np.full((T, 1), 1.5))
    q = moe_ref.quantized(np.repeat(h, 64, axis=1), 64)
    want = np.repeat(q.sum(1, keepdims=True), 40, axis=1)
    assert np.isfinite(got).all()
    far = np.abs(x[:, 0]) > 8                          # (at -8 the oracle's 1 + tanh has no digits left)
    assert np.array_equal(got[far], want[far])
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 1e-12)[~far & (x[:, 0] > 0)].all()


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("T", [20, 200])
def test_ffn_rows_that_are_not_finite_stay_alone(capi, act, T):
    up, down = Experts(capi, 3, 2 * 70, 192, 1, True), Experts(capi, 3, 100, 70, 2, True)
    ids, w = routing(T, 3, 2, 5)
    x = synth.activations(T, 192, 3)
    want = host_bits(run_ffn(capi, dev_bf16(x), dev_i32(ids), dev_f32(w), up, down, act))
    bad = x.copy()
    rows = [0, 7, T - 1]
    bad[0, 3], bad[7, 100], bad[T - 1, 191] = 0x7F80, 0x7FC1, 0xFF80
    got = host_bits(run_ffn(capi, dev_bf16(bad), dev_i32(ids), dev_f32(w), up, down, act))
    torch.cuda.synchronize()
    assert capi.mxfp4_get_device_error() == capi.OK
    assert np.isnan(ref.bf16_bits_to_f64(got[rows])).all()
    keep = np.setdiff1d(np.arange(T), rows)
    assert np.array_equal(got[keep], want[keep])


@pytest.mark.parametrize("alpha,limit", [(1.702, 0.0), (1.702, 0.5), (1.0, float("inf")), (0.0, 7.0), (3e38, 7.0)])
def test_ffn_clamps_give_the_same_bits_for_few_and_many_rows(capi, alpha, limit):
    # I = 70 ends inside a block of 32: what pads it has to be nothing
    up, down = Experts(capi, 1, 2 * 70, 192, 1, True), Experts(capi, 1, 100, 70, 2, True)
    x = dev_bf16(synth.activations(200, 192, 3))

    def run(T):
        ids, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
        out = torch.empty(T, 100, dtype=torch.bfloat16, device="cuda")
        n = capi.mxfp4_moe_ffn_workspace_bytes(T, 1, 1, 192, 70, 100)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        capi.mxfp4_moe_ffn(x, 192, ids, w, up.packed, up.bias_dev, down.packed, down.bias_dev, None, 0, out, 100, T, 1, 1,
                           192, 70, 100, capi.MOE_SWIGLU_CLAMP, alpha, limit, ws, n)
        torch.cuda.synchronize()
        return out

    many, few = run(200), run(20)
    assert many.isfinite().all() and torch.equal(many[:20], few)
    assert capi.mxfp4_get_device_error() == capi.OK
