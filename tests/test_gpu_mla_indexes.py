"""What the latent-attention kernels do with prompt offsets and lengths on the
device that are out of range: the header's promise, case by case."""

import pytest
import torch

from mla_helpers import paged, rnd, run_decode, run_prefill

pytestmark = pytest.mark.gpu

L, R, H = 128, 64, 2


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# 40 query rows and 90 keys; the third sequence is a good one in every case
GOOD = ([0, 10, 20, 40], [0, 30, 60, 90])


@pytest.mark.parametrize("cu_q,cu_k", [
    ([1, 10, 20, 40], GOOD[1]),              # a row before the first sequence
    ([-1, 10, 20, 40], GOOD[1]),
    ([0, 21, 20, 40], GOOD[1]),              # descending
    ([0, 10, 20, 39], GOOD[1]),              # a row behind the last
    ([0, 10, 20, 41], GOOD[1]),              # past the tensor
    (GOOD[0], [-1, 30, 60, 90]),
    (GOOD[0], [0, 61, 60, 90]),
    (GOOD[0], [0, 30, 60, 91]),
    (GOOD[0], [0, 2 ** 31 - 1, 60, 90]),
    ([0, -2 ** 31, 20, 40], GOOD[1])])
@pytest.mark.parametrize("many", [False, True])
def test_prompt_offsets_out_of_range_are_reported(capi, cu_q, cu_k, many):
    if many:                                 # more sequences than a warp has lanes, the bad one in front
        cu_q, cu_k = cu_q + [cu_q[-1]] * 40, cu_k + [cu_k[-1]] * 40
    q, kv, kr = rnd(1, 40, H, 64 + R), rnd(2, 90, H, 128), rnd(3, 90, R)
    args = (q[..., :64], q[..., 64:], kv[..., :64], kr, kv[..., 64:])
    guard = torch.full((3, 40, H, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    good, good_lse = run_prefill(capi, *args, i32(*GOOD[0]), i32(*GOOD[1]), 0.09, True)
    assert capi.mxfp4_get_device_error() == capi.OK
    bad, bad_lse = run_prefill(capi, *args, i32(*cu_q), i32(*cu_k), 0.09, True, out=guard[1])
    assert capi.mxfp4_get_device_error() == capi.ERR_INDEX
    assert capi.mxfp4_get_device_error() == capi.OK
    assert (guard[0] == 5).all() and (guard[2] == 5).all()
    if cu_q[:3] == [0, 10, 20] and cu_k[1:3] == [30, 60]:
        assert torch.equal(bad[10:20], good[10:20]) and torch.equal(bad_lse[10:20], good_lse[10:20])


def test_keys_left_over_and_empty_sequences_are_no_error(capi):
    q, kv, kr = rnd(4, 40, H, 64 + R), rnd(5, 90, H, 128), rnd(6, 90, R)
    args = (q[..., :64], q[..., 64:], kv[..., :64], kr, kv[..., 64:])
    a = run_prefill(capi, *args, i32(0, 0, 20, 20, 40), i32(7, 7, 40, 45, 80), 0.09, True)
    b = run_prefill(capi, *args[:2], *(t[7:80] for t in args[2:]), i32(0, 20, 40), i32(0, 33, 73), 0.09, True)
    assert capi.mxfp4_get_device_error() == capi.OK
    # (the second sequence's keys begin at 45 in one and at 40 in the other)
    assert torch.equal(a[0][:20], b[0][:20]) and torch.isfinite(a[0].float()).all() and torch.isfinite(a[1]).all()


def test_lengths_out_of_range_are_cut_without_an_error(capi):
    page, S = 16, 5
    q_lat, q_rope = rnd(7, H, S, L), rnd(8, S, H, R)
    cache, table = paged(9, [64] * S, page, L, R)
    a = run_decode(capi, q_lat, q_rope, cache, table, i32(64, 65, -1, 2 ** 31 - 1, -2 ** 31), 1, 0.07)
    b = run_decode(capi, q_lat, q_rope, cache, table, i32(64, 64, 0, 64, 0), 1, 0.07)
    assert capi.mxfp4_get_device_error() == capi.OK
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (a[0][:, 2] == 0).all() and torch.isneginf(a[1][4]).all()


def test_a_negative_page_is_reported(capi):
    lens, page = [40, 200], 64
    q_lat, q_rope = rnd(10, H, 2, L), rnd(11, 2, H, R)
    cache, table = paged(12, lens, page, L, R)
    good = run_decode(capi, q_lat, q_rope, cache, table, i32(*lens), 1, 0.05)
    assert capi.mxfp4_get_device_error() == capi.OK     # (its unused entries are -1)
    table[0, 0] = -1
    bad = run_decode(capi, q_lat, q_rope, cache, table, i32(*lens), 1, 0.05)
    assert capi.mxfp4_get_device_error() == capi.ERR_INDEX
    assert torch.equal(good[0][:, 1], bad[0][:, 1]) and torch.equal(good[1][1], bad[1][1])
