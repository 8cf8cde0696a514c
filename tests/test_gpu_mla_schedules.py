"""The plans by which the latent-attention kernels share their work, in the
sizes at which each is taken: prefill's lists of query tiles dealt by their keys
(up to 32 sequences and 64 rounds), decode's cuts where going over to another row
group counts as three tiles (24 units a block and more).  Small widths keep the
64-bit values cheap; each test asserts that its sizes reach the plan."""

import numpy as np
import pytest
import torch

import mla_wide
from mla_helpers import check_attention, paged, rnd, run_decode, run_prefill

pytestmark = pytest.mark.gpu

R = 64


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


@pytest.fixture(autouse=True)
def no_device_error(capi):
    yield
    assert capi.mxfp4_get_device_error() == capi.OK


def sms() -> int:
    return torch.cuda.get_device_properties(0).multi_processor_count


# ----------------------------------------------------------------- prefill
def prefill_rounds(new, H) -> tuple[bool, int, int]:
    """(pairs, query tiles of all heads, blocks or pairs at most)."""
    pairs = sum(new) > 128 * len(new)
    tiles = sum(-(-n // (256 if pairs else 128)) for n in new)
    return pairs, tiles * H, sms() // 2 if pairs else sms()


def prefill_case(capi, new, old, H, dn, dv, causal, seed):
    total = [max(0, a + b) for a, b in zip(new, old)]
    cu_q, cu_k = (np.concatenate(([0], np.cumsum(x))) for x in (new, total))
    Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
    q, kv, kr = rnd(seed, Tq, H, dn + R), rnd(seed + 1, Tk, H, dn + dv), rnd(seed + 2, Tk, R)
    args = (q[..., :dn], q[..., dn:], kv[..., :dn], kr, kv[..., dn:])
    cq, ck = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k))
    scale = (dn + R) ** -0.5
    out, lse = run_prefill(capi, *args, cq, ck, scale, causal)
    want = mla_wide.prefill(*args, cu_q, cu_k, scale, causal)
    check_attention(out, lse, want, max(total), dn + R, f"new {new} old {old} H {H} causal {causal}")
    again, lse2 = run_prefill(capi, *args, cq, ck, scale, causal)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


PAIRS = ([700, 300, 257, 256, 1, 130, 900, 0, 513, 4], [0, 200, -300, 64, 700, 129, -150, 90, -513, 0])
SINGLE = ([200, 1, 128, 129, 60, 300, 7, 0, 256, 90, 33, 140, 2, 127, 64, 255, 5, 100, 31, 77],
          [0, 400, -128, 64, 300, -200, 0, 50, 129, -90, 128, 1, 256, 0, -64, -10, 200, 64, 128, 500])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("what,H", [("pairs", 11), ("pairs", 41), ("single", 12), ("single", 25)])
def test_prefill_tiles_dealt_over_a_few_rounds(capi, what, H, causal):
    # some prompts without a key, some of whose first queries see none
    new, old = PAIRS if what == "pairs" else SINGLE
    pairs, tiles, blocks = prefill_rounds(new, H)
    assert pairs == (what == "pairs") and len(new) <= 32 and 2 * blocks < tiles <= 32 * blocks
    prefill_case(capi, new, old, H, 64, 64, causal, seed=H)


@pytest.mark.parametrize("S", [1, 31, 32])
def test_prefill_tiles_dealt_up_to_every_lane(capi, S):
    g = np.random.default_rng(S)
    new = [int(v) for v in g.integers(100, 600, S)]
    old = [int(v) for v in g.integers(-300, 300, S)]
    H = 9 if S > 1 else 170
    pairs, tiles, blocks = prefill_rounds(new, H)
    assert pairs and 2 * blocks < tiles <= 32 * blocks
    prefill_case(capi, new, old, H, 8, 72, True, seed=S)


@pytest.mark.parametrize("what,new,old,causal", [
    ("pairs", [300, 5], [40, 0], True), ("pairs", [300, 5], [-260, 33], False),
    ("single", [100, 130, 1], [30, -100, -1], True), ("single", [100, 130, 1], [-60, 0, 40], False)])
def test_prefill_more_rounds_than_lanes(capi, what, new, old, causal):
    tiles = prefill_rounds(new, 1)[1]
    H = -(-35 * (sms() // 2 if what == "pairs" else sms()) // tiles)
    pairs, tiles, blocks = prefill_rounds(new, H)
    assert pairs == (what == "pairs") and 32 * blocks < tiles <= 40 * blocks
    prefill_case(capi, new, old, H, 64, 64, causal, seed=H)


@pytest.mark.parametrize("more", [0, 1])
def test_prefill_at_the_longest_list_and_just_above(capi, more):
    # 4 tiles a head: 64 rounds of single blocks exactly, or the plan without a list
    H = 16 * sms() + more
    pairs, tiles, blocks = prefill_rounds([90, 130, 1], H)
    assert not pairs and tiles == 64 * blocks + 4 * more
    prefill_case(capi, [90, 130, 1], [20, -60, 3], H, 8, 8, True, seed=more)


def test_prefill_pairs_above_the_longest_list(capi):
    H = 22 * sms() // 2
    pairs, tiles, blocks = prefill_rounds([300, 5], H)
    assert pairs and tiles > 64 * blocks
    prefill_case(capi, [300, 5], [-100, 20], H, 64, 64, True, seed=3)


# ------------------------------------------------------------------ decode
def decode_case(capi, lens, H, q_len, seed, lat=128, page=64):
    scale = (lat + R) ** -0.5
    S = len(lens)
    T = S * q_len
    q_lat, q_rope = rnd(seed, H, T, lat), rnd(seed + 1, T, H, R)
    cache, table = paged(seed + 2, lens, page, lat, R)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = run_decode(capi, q_lat, q_rope, cache, table, ln, q_len, scale)      # (its workspace holds NaN before)
    want = mla_wide.decode(q_lat, q_rope, cache, table, lens, q_len, scale)
    check_attention(out, lse, want, max(lens), lat + R, f"S {S} H {H} q_len {q_len}")
    again, lse2 = run_decode(capi, q_lat, q_rope, cache, table, ln, q_len, scale)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


def row_groups(H: int, q_len: int) -> int:
    assert H >= 64                       # a token's heads in groups of 64
    return -(-H // 64) * q_len


@pytest.mark.parametrize("S,H,q_len", [(2, 64, 1), (31, 64, 1), (40, 64, 1), (63, 128, 3), (64, 128, 3), (65, 128, 3),
                                       (33, 64, 5), (150, 100, 2), (400, 64, 2)])
def test_decode_long_stretches(capi, S, H, q_len):
    # ragged lengths, empty sequences and single positions among them, to 30
    # units a block, whose cuts fall on each unit of going over
    g = np.random.default_rng(S)
    RT, blocks = row_groups(H, q_len), sms()
    part = g.uniform(0.4, 1.6, S)
    lens = [int(v) for v in part / part.sum() * 30 * blocks * 64 / RT]
    if S > 30:
        for i in range(0, S, 11):
            lens[i] = (0, 1, 64, 65)[i // 11 % 4]
    units = sum(mla_wide.decode_units(lens, RT, 1))
    assert units >= 24 * blocks, units / blocks
    if RT * S > 300:
        assert {0, 1, 2, 3} <= mla_wide.cut_places(mla_wide.decode_units(lens, RT, 3), blocks, 3)
    decode_case(capi, lens, H, q_len, seed=S)


@pytest.mark.parametrize("S,H,q_len", [(50, 64, 2), (64, 64, 1), (90, 64, 2)])
def test_decode_just_below_and_at_long_stretches(capi, S, H, q_len):
    # the last sequence grown tile by tile through the border of 24 units a block
    RT, blocks = row_groups(H, q_len), sms()
    goal = 24 * blocks // RT                              # units of all sequences, one row group each
    g = np.random.default_rng(S)
    lens = [int(v) for v in g.uniform(0.5, 1.4, S) * (goal / S - 1) * 64]
    lens[3] = lens[S // 2] = 0
    rest = goal - sum(mla_wide.decode_units(lens[:-1], 1, 1)) - 1
    assert rest > 4
    for step in (-1, 0, 1, 2, 3):
        lens[-1] = (rest + step) * 64 - 7
        units = sum(mla_wide.decode_units(lens, RT, 1))
        assert (units >= 24 * blocks) == (step >= (0 if goal * RT == 24 * blocks else 1)), (step, units)
        decode_case(capi, lens, H, q_len, seed=S + step)


def test_decode_full_width_long_stretches(capi):
    # the widest latent, pages of 16 (many copies a tile) and of 64
    g = np.random.default_rng(7)
    lens = [int(v) for v in g.uniform(2200, 7600, 50)]
    lens[10] = 0
    for page in (16, 64):
        assert sum(mla_wide.decode_units(lens, 1, 1)) >= 24 * sms()
        decode_case(capi, lens, 64, 1, seed=page, lat=512, page=page)
