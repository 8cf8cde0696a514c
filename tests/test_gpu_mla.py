"""Latent attention on the GPU against the float64 oracle: the cache store,
the absorbed decode over pages and the expanded prefill."""

import numpy as np
import pytest
import torch

from oracle import mla_ref as ref
from mla_helpers import BF, HALF, U32, check_attention, f64, paged, rnd, run_decode, run_prefill

pytestmark = pytest.mark.gpu

L, R = 512, 64


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


@pytest.fixture(autouse=True)
def no_device_error(capi):
    yield
    assert capi.mxfp4_get_device_error() == capi.OK


# ------------------------------------------------------------------- store
def table_of_angles(n: int) -> torch.Tensor:
    freq = 10000.0 ** (-np.arange(0, R, 2) / R)
    ang = np.arange(n)[:, None] * freq
    return torch.from_numpy(np.concatenate((np.cos(ang), np.sin(ang)), 1)).float().cuda()


def run_store(capi, kv, gamma, eps, q, q_out, cos_sin, positions, slots, cache, lat, interleaved, stream=None):
    T, H = q.shape[:2]
    capi.mxfp4_mla_store(kv, kv.stride(0), gamma, eps, q if H else None, q.stride(0), q.stride(1),
                         q_out if H else None, q_out.stride(0), q_out.stride(1), H, cos_sin, cos_sin.shape[0],
                         positions, slots, cache, cache.stride(0), cache.shape[1], cache.shape[0], T, lat, R,
                         interleaved, stream)


def check_store(kv, gamma, eps, q, q_out, cos_sin, positions, slots, before, cache, lat, interleaved):
    cs, pos = f64(cos_sin), positions.cpu().numpy()
    rows = ref.store_rows(f64(kv), f64(gamma), eps, cs, pos, lat, interleaved)
    want = f64(before).reshape(-1, lat + R).copy()
    tol = np.zeros_like(want)
    bound = np.concatenate((np.abs(rows[:, :lat]) * (HALF + 2.0 ** -15),
                            np.abs(rows[:, lat:]) * HALF + 8 * U32 * np.abs(f64(kv)[:, lat:]).max() + 0 * rows[:, lat:]),
                           1)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s], tol[s] = rows[t], bound[t]
    got = f64(cache).reshape(-1, lat + R)
    assert (np.abs(got - want) <= tol).all()
    if q.shape[1]:
        wq = ref.store_queries(f64(q), cs, pos, interleaved)
        assert (np.abs(f64(q_out) - wq) <= np.abs(wq) * HALF + 8 * U32 * np.abs(f64(q)).max()).all()


@pytest.mark.parametrize("T,H,page,lat,interleaved", [
    (1, 64, 64, 512, True), (1, 1, 8, 512, False), (5, 3, 16, 128, True), (33, 16, 64, 384, False),
    (200, 64, 128, 512, True), (257, 80, 24, 256, False), (64, 0, 64, 512, True)])
def test_store(capi, T, H, page, lat, interleaved):
    pages = -(-T // page) + 2
    kv = rnd(1, T, lat + R + 24, scale=3)[:, :lat + R]              # rows of a wider tensor
    gamma, q = rnd(2, lat), rnd(3, T, max(H, 1), 192 + R)[:, :H, 192:]
    q_out = torch.full((T, max(H, 1), R), 7.0, dtype=BF, device="cuda")[:, :H]
    cs = table_of_angles(5000)
    g = torch.Generator().manual_seed(4)
    positions = torch.randint(0, 5000, (T,), generator=g).cuda()
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[T - T // 3:] = -1
    slots = slots.cuda()
    backing = rnd(5, pages, page * (lat + R) + 64)                  # pages further apart than they are long
    cache = backing[:, : page * (lat + R)].view(pages, page, lat + R)
    before = cache.clone()
    run_store(capi, kv, gamma, 1e-5, q, q_out, cs, positions, slots, cache, lat, interleaved)
    check_store(kv, gamma, 1e-5, q, q_out, cs, positions, slots, before, cache, lat, interleaved)
    assert torch.equal(backing[:, page * (lat + R):], rnd(5, pages, page * (lat + R) + 64)[:, page * (lat + R):])


def test_store_rotates_queries_in_place_and_handles_special_rows(capi):
    T, H, page = 6, 4, 8
    kv = rnd(11, T, L + R)
    kv[0] = 0                                                       # eps alone under the root
    kv[1, 5] = float("inf")
    kv[2, 7] = float("nan")
    q = rnd(12, T, H, R)
    q0, cs = q.clone(), table_of_angles(64)
    pos, slots = torch.arange(T).cuda() * 7, torch.arange(T).cuda() + 3
    cache = torch.zeros(2, page, L + R, dtype=BF, device="cuda")
    gamma = rnd(13, L)
    run_store(capi, kv, gamma, 1e-6, q, q, cs, pos, slots, cache, L, True)
    wq = ref.store_queries(f64(q0), f64(cs), pos.cpu().numpy(), True)
    assert (np.abs(f64(q) - wq) <= np.abs(wq) * HALF + 8 * U32 * np.abs(f64(q0)).max()).all()
    flat = f64(cache).reshape(-1, L + R)
    assert (flat[3, :L] == 0).all() and np.isnan(flat[5, :L]).all()
    assert np.isnan(flat[4, 5]) and (np.delete(flat[4, :L], 5) == 0).all()      # inf / inf, and x / inf
    want = ref.store_rows(f64(kv)[3:], f64(gamma), 1e-6, f64(cs), pos.cpu().numpy()[3:], L, True)
    assert np.abs(flat[6:9] - want).max() <= np.abs(want).max() * (HALF + 2.0 ** -15)


# ------------------------------------------------------------------ decode
def decode_case(capi, lens, H, q_len, page, lat=512, scale=None, seed=0, q_scale=1.0, fill=1.0, width=None):
    scale = (lat + R) ** -0.5 if scale is None else scale
    S = len(lens)
    T = S * q_len
    q_lat, q_rope = rnd(seed + 21, H, T, lat, scale=q_scale), rnd(seed + 22, T, H, R, scale=q_scale)
    cache, table = paged(seed + 23, lens, page, lat, R, fill=fill, width=width)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = run_decode(capi, q_lat, q_rope, cache, table, ln, q_len, scale)
    want = ref.decode(f64(q_lat), f64(q_rope), f64(cache), table.cpu().numpy(), lens, q_len, scale)
    check_attention(out, lse, want, max(lens), lat + R, f"lens {lens} H {H} q_len {q_len} page {page}")


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 127, 128, 129, 255, 257, 640, 1500])
def test_decode_one_sequence(capi, n):
    decode_case(capi, [n], 16, 1, 64, seed=n)


@pytest.mark.parametrize("H,q_len", [(1, 1), (8, 1), (16, 1), (17, 1), (32, 1), (33, 1), (40, 2), (64, 1), (64, 2),
                                     (65, 1), (100, 1), (128, 1), (8, 4), (16, 3), (3, 7), (8, 9)])
def test_decode_head_layouts(capi, H, q_len):
    decode_case(capi, [200, 7, 385], H, q_len, 32, seed=H)


@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 128, 192, 256])
def test_decode_page_sizes(capi, page):
    decode_case(capi, [page, page - 1, page + 1, 3 * page + 5, 300], 8, 1, page, seed=page)


@pytest.mark.parametrize("lat", [128, 256, 384, 512])
def test_decode_latent_widths(capi, lat):
    decode_case(capi, [150, 290], 24, 2, 16, lat=lat, seed=lat)


def test_decode_empty_and_short_sequences(capi):
    # lengths of zero, below q_len (some tokens see nothing), and equal to it
    decode_case(capi, [0, 1, 2, 3, 4, 0, 130, 0], 8, 4, 16)
    decode_case(capi, [0, 0], 64, 1, 64, width=4)
    decode_case(capi, [0], 5, 1, 8, width=1)


def test_decode_many_sequences(capi):
    # more sequences than threads of a block
    g = np.random.default_rng(3)
    decode_case(capi, [int(v) for v in g.integers(0, 40, 300)], 4, 1, 8)


def test_decode_long_ragged_sequences(capi):
    # blocks that go from one sequence into the next, and sequences over many blocks
    decode_case(capi, [5000, 1, 2900, 64, 65, 3777, 0, 1234, 700], 64, 1, 64)
    decode_case(capi, [2100, 63, 1500, 1], 48, 2, 128, seed=9)


@pytest.mark.parametrize("lat", [128, 256, 512])
def test_decode_many_short_sequences(capi, lat):
    # several sequences to a block, so that the next one's queries and
    # positions are asked for while the last one's are in use
    g = np.random.default_rng(lat)
    decode_case(capi, [int(v) for v in g.integers(0, 200, 700)], 16, 1, 64, lat=lat, seed=lat)


@pytest.mark.parametrize("S", [31, 32, 33, 50, 63, 64, 65])
def test_decode_sequences_per_lane(capi, S):
    # lengths of one, two and more sequences to a lane, empty ones among them
    g = np.random.default_rng(S)
    decode_case(capi, [int(v) * int(v % 7 > 0) for v in g.integers(0, 400, S)], 64, 1, 64, lat=128, seed=S)


def test_decode_lengths_written_just_before(capi):
    # each call's lengths differ from the last call's and are written on the
    # device right before it, with another of the library's kernels between
    H, page, lat = 16, 64, 128
    full = [640] * 5
    q_lat, q_rope = rnd(131, H, 5, lat), rnd(132, 5, H, R)
    cache, table = paged(133, full, page, lat, R)
    lens = [[640, 3, 0, 129, 64], [1, 640, 500, 0, 65], [640] * 5, [0, 0, 63, 1, 0], [333, 222, 111, 55, 27]] * 3
    on_device = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ln = torch.zeros(5, dtype=torch.int32, device="cuda")
    got = []
    for i in range(len(lens)):
        ln.copy_(on_device[i])
        got.append(run_decode(capi, q_lat, q_rope, cache, table, ln, 1, 0.07))
        run_decode(capi, q_lat, q_rope, cache, table, ln, 1, 0.07)
    for n, (out, lse) in zip(lens, got):
        want = ref.decode(f64(q_lat), f64(q_rope), f64(cache), table.cpu().numpy(), n, 1, 0.07)
        check_attention(out, lse, want, max(n), lat + R, f"lens {n}")


@pytest.mark.parametrize("S", [4, 40])
def test_decode_lengths_written_by_the_kernel_ahead(capi, S):
    # the store kernel lets the next kernel start before it writes; here what it
    # writes (a rotated query: 1.0 pairs are a length beyond the table, -1.0
    # pairs a negative one) is the lengths, others in each call
    H, page, lat, cap = 8, 64, 128, 256
    q_lat, q_rope = rnd(141, H, S, lat), rnd(142, S, H, R)
    cache, table = paged(143, [cap] * S, page, lat, R)
    kv, gamma = rnd(144, 1, lat + R), rnd(145, lat)
    cos_sin = torch.cat((torch.ones(1, R // 2), torch.zeros(1, R // 2)), 1).cuda()
    pos, no_slot = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.full((1,), -1, dtype=torch.int64, device="cuda")
    g = np.random.default_rng(S)
    masks = [g.integers(0, 2, 2 * R // 2) for _ in range(12)]
    qs = [torch.from_numpy(np.where(np.repeat(m, 2), 1.0, -1.0)).to(BF).reshape(1, 2, R).cuda() for m in masks]
    q_out = torch.zeros(1, 2, R, dtype=BF, device="cuda")
    lens = q_out.view(torch.int32).reshape(-1)[:S]
    ws = torch.empty(capi.mxfp4_mla_decode_workspace_bytes(S, 1, H, lat, cap), dtype=torch.uint8, device="cuda")
    got = [(torch.empty(H, S, lat, dtype=BF, device="cuda"), torch.empty(S, H, device="cuda")) for _ in qs]

    def calls():
        for q, (out, lse) in zip(qs, got):
            run_store(capi, kv, gamma, 1e-6, q, q_out, cos_sin, pos, no_slot, cache, lat, True)
            capi.mxfp4_mla_decode(q_lat, q_lat.stride(1), q_lat.stride(0), q_rope, q_rope.stride(0), q_rope.stride(1),
                                  cache, cache.stride(0), page, cache.shape[0], table, table.stride(0), table.shape[1],
                                  lens, out, out.stride(1), out.stride(0), lse, S, 1, H, lat, R, 0.07, ws, ws.numel(),
                                  None)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()              # (one call right behind the other)
    with torch.cuda.graph(graph):
        calls()
    for out, lse in got:
        out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for m, (out, lse) in zip(masks, got):
        n = [cap * int(v) for v in m[:S]]
        want = ref.decode(f64(q_lat), f64(q_rope), f64(cache), table.cpu().numpy(), n, 1, 0.07)
        check_attention(out, lse, want, cap, lat + R, f"lens {n}")


def test_decode_many_row_groups(capi):
    # 24 row groups a sequence: dozens of tiles for every block, cut in the middle
    decode_case(capi, [1000, 0, 900, 64, 1, 1111, 777, 1024], 192, 8, 64, lat=128, seed=4)


def test_decode_rising_and_peaked_scores(capi):
    # scores that keep passing the running maximum, far outside the slack, and
    # weights of one position alone
    lens, H, page = [700], 16, 64
    q_lat, q_rope = rnd(31, H, 1, L), rnd(32, 1, H, R)
    cache, table = paged(33, lens, page)
    ramp = torch.linspace(0.05, 6.0, 704, device="cuda")
    for i, p in enumerate(table[0].tolist()):
        rows = cache[p].float() * ramp[i * page:(i + 1) * page, None]
        cache[p] = rows.to(BF)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for scale in (0.05, 1.0, -0.3):
        out, lse = run_decode(capi, q_lat, q_rope, cache, table, ln, 1, scale)
        want = ref.decode(f64(q_lat), f64(q_rope), f64(cache), table.cpu().numpy(), lens, 1, scale)
        check_attention(out, lse, want, 700, L + R, f"scale {scale}")


def test_decode_strided_views_and_untouched_gaps(capi):
    S, H, q_len, page = 3, 20, 2, 16
    T, lens = S * q_len, [90, 33, 200]
    big_q = rnd(41, T, H, L + R + 32)
    q_lat, q_rope = big_q[..., :L].transpose(0, 1), big_q[..., L:L + R]
    base, table = paged(42, lens, page)
    pages = base.shape[0]
    backing = torch.full((pages, 2 * page * (L + R) + 8), float("nan"), dtype=BF, device="cuda")
    cache = backing[:, 8: 8 + page * (L + R)].view(pages, page, L + R)
    cache.copy_(base)
    wide = torch.full((S, table.shape[1] + 3), -5, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table
    buf = torch.full((T, H, L + 8), 9.0, dtype=BF, device="cuda")
    out, lse = run_decode(capi, q_lat, q_rope, cache, wide[:, : table.shape[1]],
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), q_len, 0.05,
                          out=buf[..., :L].transpose(0, 1))
    want = ref.decode(f64(q_lat), f64(q_rope), f64(base), table.cpu().numpy(), lens, q_len, 0.05)
    check_attention(out, lse, want, 200, L + R, "strided")
    assert (buf[..., L:] == 9).all()


def test_decode_is_deterministic_and_captures(capi):
    lens, H = [3000, 10, 1111], 64
    q_lat, q_rope = rnd(51, H, 3, L), rnd(52, 3, H, R)
    cache, table = paged(53, lens, 64)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = run_decode(capi, q_lat, q_rope, cache, table, ln, 1, 0.06)
    b = run_decode(capi, q_lat, q_rope, cache, table, ln, 1, 0.06)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # captured, then replayed with other lengths and queries in the same buffers
    n = capi.mxfp4_mla_decode_workspace_bytes(3, 1, H, L, table.shape[1] * 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])

    def call():
        capi.mxfp4_mla_decode(q_lat, q_lat.stride(1), q_lat.stride(0), q_rope, q_rope.stride(0), q_rope.stride(1),
                              cache, cache.stride(0), 64, cache.shape[0], table, table.stride(0), table.shape[1], ln,
                              out, out.stride(1), out.stride(0), lse, 3, 1, H, L, R, 0.06, ws, n)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    ln.copy_(torch.tensor([2000, 0, 700], dtype=torch.int32))
    q_lat.copy_(rnd(54, H, 3, L))
    graph.replay()
    torch.cuda.synchronize()
    c = run_decode(capi, q_lat, q_rope, cache, table, ln, 1, 0.06)
    assert torch.equal(out, c[0]) and torch.equal(lse, c[1])


def test_decode_on_a_side_stream(capi):
    lens, H = [900, 1000], 32
    q_lat, q_rope = rnd(61, H, 2, L), rnd(62, 2, H, R)
    cache, table = paged(63, lens, 32)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = run_decode(capi, q_lat, q_rope, cache, table, ln, 1, 0.06)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = run_decode(capi, q_lat, q_rope, cache, table, ln, 1, 0.06, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_cache_past_32_bits(capi):
    # pages whose element offsets pass 2^31 and byte offsets 2^32
    page, H = 64, 16
    pages = 2 ** 32 // (page * (L + R)) + 3
    cache = torch.zeros(pages, page, L + R, dtype=BF, device="cuda")
    small, table = paged(71, [300], page, extra=0)
    where = torch.tensor([pages - 1, 1, pages - 3, pages // 2, pages - 2])
    for i in range(5):
        cache[where[i]] = small[int(table[0, i])]
    far = where.to(torch.int32)[None].cuda()
    q_lat, q_rope = rnd(72, H, 1, L), rnd(73, 1, H, R)
    ln = torch.tensor([300], dtype=torch.int32, device="cuda")
    a = run_decode(capi, q_lat, q_rope, small, table, ln, 1, 0.05)
    b = run_decode(capi, q_lat, q_rope, cache, far, ln, 1, 0.05)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ----------------------------------------------------------------- prefill
def prefill_case(capi, new, old, H, dn, dv, causal, seed=0, scale=None, kv_scale=1.0):
    scale = (dn + R) ** -0.5 if scale is None else scale
    total = [a + b for a, b in zip(new, old)]
    cu_q = np.concatenate(([0], np.cumsum(new)))
    cu_k = np.concatenate(([0], np.cumsum(total)))
    Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
    q, kv, kr = rnd(seed + 81, Tq, H, dn + R), rnd(seed + 82, Tk, H, dn + dv, scale=kv_scale), rnd(seed + 83, Tk, R)
    args = (q[..., :dn], q[..., dn:], kv[..., :dn], kr, kv[..., dn:])
    cq, ck = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k))
    out, lse = run_prefill(capi, *args, cq, ck, scale, causal)
    want = ref.prefill(*(f64(t) for t in args), cu_q, cu_k, scale, causal)
    check_attention(out, lse, want, max(total), dn + R, f"new {new} old {old} H {H} dn {dn} dv {dv} causal {causal}")


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 200, 257, 400])
def test_prefill_one_prompt(capi, n):
    prefill_case(capi, [n], [0], 2, 192, 256, True, seed=n)


@pytest.mark.parametrize("dn,dv", [(8, 8), (64, 64), (72, 40), (120, 136), (128, 128), (128, 200), (192, 128),
                                   (192, 256), (64, 256), (184, 248)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_widths(capi, dn, dv, causal):
    prefill_case(capi, [70, 140], [0, 33], 2, dn, dv, causal, seed=dn + dv)


@pytest.mark.parametrize("dn,dv", [(64, 64), (8, 8), (72, 40), (128, 136), (192, 128), (120, 256), (184, 200)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_widths_in_pairs(capi, dn, dv, causal):
    # prompts above 128 tokens on average take pairs of blocks
    prefill_case(capi, [300, 150], [0, 45], 2, dn, dv, causal, seed=dn + dv)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_ragged_with_context(capi, causal):
    prefill_case(capi, [5, 130, 1, 64, 1], [300, 0, 129, 64, 0], 3, 192, 256, causal)


def test_prefill_empty_rows_and_sequences(capi):
    # no new tokens; no keys; fewer keys than queries (the first see nothing)
    prefill_case(capi, [0, 3, 0, 140, 20], [7, -3, 0, -100, -15], 2, 192, 256, True)
    prefill_case(capi, [0, 3, 0, 40], [7, -3, 0, -10], 2, 64, 64, False)


def test_prefill_many_prompts(capi):
    g = np.random.default_rng(5)
    prefill_case(capi, [int(v) for v in g.integers(0, 5, 500)], [int(v) for v in g.integers(0, 4, 500)], 1, 64, 64, True)


@pytest.mark.parametrize("most", [400, 200])
def test_prefill_many_tiles_per_block(capi, most):
    # several query tiles for every block (pairs of blocks above 128 tokens a
    # prompt, single blocks below), some of them without a key
    g = np.random.default_rng(most)
    new = [int(v) for v in g.integers(1, most, 40)] + [most]
    old = [int(v) for v in g.integers(-60, 200, 41)]
    old = [max(b, -a) for a, b in zip(new, old)]
    prefill_case(capi, new, old, 9, 64, 64, True)


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_scores_scaled_by_zero_and_below(capi, scale):
    decode_case(capi, [300, 5, 0], 8, 2, 16, scale=scale)
    prefill_case(capi, [70, 200], [0, 30], 2, 64, 72, True, scale=scale)


def test_prefill_rising_and_peaked_scores(capi):
    n, H = 520, 2
    q, kv, kr = rnd(91, n, H, 256), rnd(92, n, H, 448), rnd(93, n, R)
    kv = (kv.float() * torch.linspace(0.05, 8.0, n, device="cuda")[:, None, None]).to(BF)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    args = (q[..., :192], q[..., 192:], kv[..., :192], kr, kv[..., 192:])
    for scale in (0.06, 0.8, -0.2):
        out, lse = run_prefill(capi, *args, cu, cu, scale, True)
        want = ref.prefill(*(f64(t) for t in args), [0, n], [0, n], scale, True)
        check_attention(out, lse, want, n, 256, f"scale {scale}")


@pytest.mark.parametrize("shift", [-64.0, 64.0])
def test_scores_far_from_zero(capi, shift):
    # every score is about -+270 (beyond what 2^x holds), from one value of the
    # rotated key: the sums are those of the rest
    lens, H, page = [700, 40, 64], 8, 16
    q_lat, q_rope = rnd(101, H, 3, L), rnd(102, 3, H, R)
    cache, table = paged(103, lens, page)
    q_rope[..., 0], cache[..., L] = 100.0, torch.where(cache[..., L].isnan(), cache[..., L], shift)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = 1 / 24
    out, lse = run_decode(capi, q_lat, q_rope, cache, table, ln, 1, scale)
    want = ref.decode(f64(q_lat), f64(q_rope), f64(cache), table.cpu().numpy(), lens, 1, scale)
    check_attention(out, lse, want, 700, L + R, f"decode, shift {shift}")
    n = 300
    q, kv, kr = rnd(104, n, H, 192 + R), rnd(105, n, H, 192 + 256), rnd(106, n, R)
    q[..., 192], kr[:, 0] = 100.0, shift
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    args = (q[..., :192], q[..., 192:], kv[..., :192], kr, kv[..., 192:])
    out, lse = run_prefill(capi, *args, cu, cu, scale, True)
    want = ref.prefill(*(f64(t) for t in args), [0, n], [0, n], scale, True)
    check_attention(out, lse, want, n, 256, f"prefill, shift {shift}")


def test_prefill_ignores_what_lies_past_a_sequence(capi):
    # the rows after each sequence's keys are another's, or NaN
    H, n = 2, 150
    q, kv, kr = rnd(101, n, H, 256), rnd(102, n + 90, H, 448), rnd(103, n + 90, R)
    kv[n:] = float("nan")
    kr[n:] = float("nan")
    kv[n + 40:] = float("inf")
    cu_q = torch.tensor([0, n, n], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, n, n + 90], dtype=torch.int32, device="cuda")
    args = (q[..., :192], q[..., 192:], kv[..., :192], kr, kv[..., 192:])
    for causal in (True, False):
        out, lse = run_prefill(capi, *args, cu_q, cu_k, 0.0625, causal)
        alone = tuple(t[:n] for t in args)
        want = ref.prefill(*(f64(t) for t in alone), [0, n], [0, n], 0.0625, causal)
        check_attention(out, lse, want, n, 256, "past the end")


def test_prefill_strides_determinism_and_capture(capi):
    n, H, dn, dv = 300, 4, 128, 128
    q, kr = rnd(111, n, H + 1, dn + R + 8), rnd(112, n, R + 16)
    k, v = rnd(113, H, n, dn), rnd(114, n, H, dv + 24)
    buf = torch.full((H, n, dv + 8), 3.0, dtype=BF, device="cuda")
    cu = torch.tensor([0, 170, n], dtype=torch.int32, device="cuda")
    args = (q[:, :H, :dn], q[:, 1:, dn:dn + R], k.transpose(0, 1), kr[:, 8:8 + R], v[..., 16:16 + dv])
    out = buf[..., :dv].transpose(0, 1)
    _, lse = run_prefill(capi, *args, cu, cu, 0.07, True, out=out)
    want = ref.prefill(*(f64(t) for t in args), [0, 170, n], [0, 170, n], 0.07, True)
    check_attention(out, lse, want, n, dn + R, "strided")
    assert (buf[..., dv:] == 3).all()
    again, lse2 = run_prefill(capi, *args, cu, cu, 0.07, True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    graph = torch.cuda.CUDAGraph()
    out3, lse3 = torch.empty_like(again), torch.empty_like(lse)
    with torch.cuda.graph(graph):
        run_prefill(capi, *args, cu, cu, 0.07, True, out=out3, lse=lse3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out3, again) and torch.equal(lse3, lse)


def test_decode_agrees_with_prefill_over_the_same_latents(capi):
    # the absorbed and the expanded form of one attention: with K-up and V-up
    # matrices that pick latent values, both are exact in bf16
    n, H = 300, 4
    lat, kr = rnd(121, n, L), rnd(122, n, R)
    qn, qr = rnd(123, 1, H, 192), rnd(124, 1, H, R)
    kv = torch.empty(n, H, 448, dtype=BF, device="cuda")
    q_lat = torch.zeros(H, 1, L, dtype=BF, device="cuda")
    for h in range(H):
        kv[:, h, :192] = lat[:, 60 * h: 60 * h + 192]
        kv[:, h, 192:] = lat[:, 80 * h: 80 * h + 256]
        q_lat[h, 0, 60 * h: 60 * h + 192] = qn[0, h]
    one, all_ = (torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (1, n))
    o, lse = run_prefill(capi, qn, qr, kv[..., :192], kr, kv[..., 192:], one, all_, 0.0625, True)
    cache, table = paged(125, [n], 64)
    for i, p in enumerate(table[0].tolist()):
        rows = torch.cat((lat, kr), 1)[64 * i: 64 * i + 64]
        cache[p, : rows.shape[0]] = rows
    ol, lse2 = run_decode(capi, q_lat, qr, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), 1, 0.0625)
    for h in range(H):
        a, b = f64(o[0, h]), f64(ol[h, 0, 80 * h: 80 * h + 256])
        assert np.abs(a - b).max() <= 4 * HALF * np.abs(f64(lat)).max()
        assert np.linalg.norm(a - b) <= 2 * HALF * np.linalg.norm(a)
    assert np.abs(f64(lse) - f64(lse2)).max() <= 2 * (576 + n) * U32 * 40


# ------------------------------------------------------ indexes out of range
def test_indexes_out_of_range_are_reported_and_touch_nothing(capi):
    T, H, page = 4, 2, 8
    kv, q, gamma = rnd(131, T, L + R), rnd(132, T, H, R), rnd(133, L)
    cache = torch.zeros(2, page, L + R, dtype=BF, device="cuda")
    q_out = torch.zeros(T, H, R, dtype=BF, device="cuda")
    cs = table_of_angles(16)
    pos = torch.tensor([3, 16, -1, 5], device="cuda")
    slots = torch.tensor([0, 1, 2, 16], device="cuda")
    run_store(capi, kv, gamma, 1e-6, q, q_out, cs, pos, slots, cache, L, True)
    assert capi.mxfp4_get_device_error() == capi.ERR_INDEX
    assert capi.mxfp4_get_device_error() == capi.OK
    assert (cache.view(-1, L + R)[1:] == 0).all() and (cache.view(-1, L + R)[0] != 0).any()
    assert (q_out[1:3] == 0).all() and (q_out[0] != 0).any() and (q_out[3] != 0).any()
    # a page outside the cache, and a length above the table's capacity: the
    # other sequence is as it should be
    lens = [40, 200]
    q_lat, q_rope = rnd(134, H, 2, L), rnd(135, 2, H, R)
    cache, table = paged(136, lens, 64)
    good = run_decode(capi, q_lat, q_rope, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1, 0.05)
    table[0, 0] = cache.shape[0] + 7
    bad = run_decode(capi, q_lat, q_rope, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1, 0.05)
    assert capi.mxfp4_get_device_error() == capi.ERR_INDEX
    assert torch.equal(good[0][:, 1], bad[0][:, 1]) and torch.equal(good[1][1], bad[1][1])
