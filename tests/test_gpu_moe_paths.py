"""Mixture of experts on the GPU where the kernels go other ways: few and many
pairs, tiles cut between blocks, k-steps whose scales do not stay, the largest
numbers of experts and slots, unaligned ids, captured graphs, streams and shared
workspaces, the same bits run after run."""

import numpy as np
import pytest
import torch

from helpers import check_close, dev_bf16, host_bits
from moe_helpers import (Experts, check_ffn, dev_f32, dev_i32, n_acc, routing, run_ffn, run_linear, run_route, want_ffn,
                         workspace)
from mxfp4_quantized_gemm_gb300 import synth
from oracle import moe_ref
from oracle import mxfp4_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


def check_rows(capi, T, k, E, N, K, ids, rows, seed=0, bias=True):
    """moe_linear of all T tokens, the tokens `rows` against the oracle."""
    w = Experts(capi, E, N, K, seed, bias)
    x = synth.activations(T, K, seed)
    out = run_linear(capi, dev_bf16(x), dev_i32(ids), w)
    torch.cuda.synchronize()
    assert capi.mxfp4_get_device_error() == capi.OK
    acc, mag = moe_ref.linear(ref.bf16_bits_to_f64(x[rows]), ids[rows], w.codes, w.scales, K,
                              ref.bf16_bits_to_f64(w.bias) if bias else None)
    got = host_bits(out).reshape(T, k, N)
    check_close(got[rows], acc, mag, n_acc(K), what=f"moe_linear T={T} k={k} E={E} N={N} K={K}", K=K)
    assert (got[ids < 0] == 0).all() and np.isfinite(ref.bf16_bits_to_f64(got)).all()


@pytest.mark.parametrize("T,k", [(32, 8), (255, 1), (257, 1), (86, 3), (33, 8), (1000, 1)])
def test_pairs_around_the_one_kernel_plan(capi, T, k):
    ids = routing(T, 12, k, T, 0.1)[0]
    check_rows(capi, T, k, 12, 96, 160, ids, np.arange(T), seed=T)


@pytest.mark.parametrize("T,k", [(51, 5), (28, 9), (23, 11), (15, 17), (14, 18), (13, 19), (12, 21), (11, 23)])
def test_few_pairs_whose_slots_fill_no_power_of_two(capi, T, k):
    # the lanes that count past a token's last slot reach behind the last id here
    ids = routing(T, 24, k, T, 0.1)[0]
    check_rows(capi, T, k, 24, 40, 64, ids, np.arange(T), seed=k)


def test_most_experts_and_slots(capi):
    ids = routing(40, 1024, 32, 1)[0]
    check_rows(capi, 40, 32, 1024, 40, 64, ids, np.arange(40), bias=False)
    ids = routing(5, 1024, 32, 2)[0]
    check_rows(capi, 5, 32, 1024, 40, 64, ids, np.arange(5), bias=True)


def test_many_pairs_and_ids_that_are_not_aligned(capi):
    T, k, E, N, K = 30000, 5, 7, 64, 64
    g = np.random.default_rng(5)
    ids = g.integers(-1, E, (T, k)).astype(np.int32)
    w = Experts(capi, E, N, K, 5, False)
    x = synth.activations(T, K, 5)
    room = torch.empty(T * k + 1, dtype=torch.int32, device="cuda")
    room[1:] = dev_i32(ids).flatten()
    a = run_linear(capi, dev_bf16(x), dev_i32(ids), w)
    b = run_linear(capi, dev_bf16(x), room[1:].view(T, k), w)
    assert torch.equal(a, b)
    rows = np.concatenate((np.arange(40), np.arange(T - 40, T), g.integers(0, T, 100)))
    acc, mag = moe_ref.linear(ref.bf16_bits_to_f64(x[rows]), ids[rows], w.codes, w.scales, K)
    check_close(host_bits(a).reshape(T, k, N)[rows], acc, mag, n_acc(K), what="30000 x 5", K=K)


@pytest.mark.parametrize("N", [1, 2, 3, 7, 31, 63, 127, 129, 191, 255, 257, 385, 1001])
def test_rows_of_odd_widths(capi, N):
    # rows that start at odd columns and end inside a word, many and few of them
    check_rows(capi, 140, 1, 1, N, 192, np.zeros((140, 1), dtype=np.int32), np.arange(0, 140, 3), seed=N)
    check_rows(capi, 60, 2, 3, N, 64, routing(60, 3, 2, N, 0.1)[0], np.arange(60), seed=N, bias=False)


def test_rows_of_odd_widths_and_strides(capi):
    # what lies between and behind the rows stays
    w = Experts(capi, 2, 301, 256, 3, True)
    x, ids = dev_bf16(synth.activations(150, 256, 3)), dev_i32(routing(150, 2, 1, 3)[0])
    want = run_linear(capi, x, ids, w)
    for ldo, at in ((301, 1), (302, 0), (303, 5), (304, 0), (305, 8), (320, 3)):
        room = torch.full((150 * ldo + 16,), 7.0, dtype=BF, device="cuda")
        run_linear(capi, x, ids, w, out=room[at:at + 150 * ldo].view(150, ldo))
        got = room[at:at + 150 * ldo].view(150, ldo)
        assert torch.equal(got[:, :301], want) and (got[:, 301:] == 7).all()
        assert (room[:at] == 7).all() and (room[at + 150 * ldo:] == 7).all()


@pytest.mark.parametrize("T", [3, 40, 200])
def test_cut_tiles(capi, T):
    # one or two tiles of 56 k-steps: cut for several blocks
    ids = np.zeros((T, 1), dtype=np.int32)
    check_rows(capi, T, 1, 1, 300, 14336, ids, np.arange(T), seed=T)


@pytest.mark.parametrize("T", [40, 200])
def test_cut_tiles_of_many_rows(capi, T):
    # 112 k-steps: worth a cut with any number of rows
    ids = np.zeros((T, 1), dtype=np.int32)
    check_rows(capi, T, 1, 1, 300, 28672, ids, np.arange(0, T, 3), seed=T)


@pytest.mark.parametrize("at", [16, 48])
def test_cut_tiles_with_a_workspace_aligned_to_16_bytes(capi, at):
    # the parts of cut tiles are read and written 32 bytes at a time
    T, K = 40, 28672
    w = Experts(capi, 1, 300, K, 8, True)
    x, ids = dev_bf16(synth.activations(T, K, 8)), torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    n = capi.mxfp4_moe_linear_workspace_bytes(T, 1, 1, 300, K)
    room = workspace(n + 128)
    got = run_linear(capi, x, ids, w, ws=room[at:at + n])
    assert torch.equal(got, run_linear(capi, x, ids, w))
    assert (room[at + n:] == 0xFF).all() and (room[:at] == 0xFF).all()
    up, down = Experts(capi, 1, 2 * 130, K, 4, True), Experts(capi, 1, 72, 130, 5, True)
    weights = torch.ones(T, 1, device="cuda")
    n = capi.mxfp4_moe_ffn_workspace_bytes(T, 1, 1, K, 130, 72)
    room = workspace(n + 128)
    got = run_ffn(capi, x, ids, weights, up, down, "silu", ws=room[at:at + n])
    assert torch.equal(got, run_ffn(capi, x, ids, weights, up, down, "silu"))
    assert (room[at + n:] == 0xFF).all() and (room[:at] == 0xFF).all()


def test_cut_tiles_after_whole_rounds(capi):
    T = 5120
    ids = np.zeros((T, 1), dtype=np.int32)
    rows = np.unique(np.concatenate(([0, 127, 128, T - 1], np.random.default_rng(1).integers(0, T, 40))))
    check_rows(capi, T, 1, 1, 1010, 14336, ids, rows, seed=3)


@pytest.mark.parametrize("K", [6144, 6146, 8192])
def test_scales_that_stay_and_that_do_not(capi, K):
    ids = routing(150, 2, 1, K)[0]
    check_rows(capi, 150, 1, 2, 1100, K, ids, np.arange(0, 150, 3), seed=K)


def test_gated_cut_tiles_of_many_rows(capi):
    T, K = 150, 28672
    up, down = Experts(capi, 1, 2 * 130, K, 4, True), Experts(capi, 1, 72, 130, 5, True)
    x = synth.activations(T, K, 4)
    ids, w = np.zeros((T, 1), dtype=np.int32), np.ones((T, 1), dtype=np.float32)
    out = run_ffn(capi, dev_bf16(x), dev_i32(ids), dev_f32(w), up, down, "silu")
    check_ffn(out, want_ffn(x, ids, w, up, down, "silu"), "gated, cut, 150 rows of 28672")


@pytest.mark.parametrize("K", [130, 256, 512, 700, 6144, 6400, 6600])
@pytest.mark.parametrize("T", [5, 60, 70])
def test_halves_of_few_rows(capi, T, K):
    # few tiles: halves on a block each, finished row by row up to 32 rows; scales
    # that stay (up to K = 6144) and that do not
    ids = (np.arange(T) % 3 == 0).astype(np.int32)[:, None]
    check_rows(capi, T, 1, 2, 300, K, ids, np.arange(T), seed=K + T)


@pytest.mark.parametrize("K,I", [(700, 130), (6400, 520)])
def test_gated_halves_of_few_rows(capi, K, I):
    T = 40
    up, down = Experts(capi, 2, 2 * I, K, 4, True), Experts(capi, 2, 300, I, 5, True)
    x = synth.activations(T, K, 4)
    ids, w = routing(T, 2, 1, K)
    out = run_ffn(capi, dev_bf16(x), dev_i32(ids), dev_f32(w), up, down, "silu")
    check_ffn(out, want_ffn(x, ids, w, up, down, "silu"), f"gated halves, K={K}")


@pytest.mark.parametrize("T", [2, 150])
def test_gated_cut_tiles(capi, T):
    up, down = Experts(capi, 1, 2 * 130, 14336, 4, True), Experts(capi, 1, 72, 130, 5, True)
    x = synth.activations(T, 14336, 4)
    ids, w = np.zeros((T, 1), dtype=np.int32), np.ones((T, 1), dtype=np.float32)
    out = run_ffn(capi, dev_bf16(x), dev_i32(ids), dev_f32(w), up, down, "silu")
    check_ffn(out, want_ffn(x, ids, w, up, down, "silu"), f"gated, cut, T={T}")


def ffn_case(capi, T, k, E, K, I, N, seed):
    up, down = Experts(capi, E, 2 * I, K, seed, True), Experts(capi, E, N, I, seed + 1, True)
    ids, w = routing(T, E, k, seed, 0.1)
    return up, down, dev_bf16(synth.activations(T, K, seed)), dev_i32(ids), dev_f32(w), dev_bf16(
        synth.residual(T, N, seed, sigma=1.0))


def ws_bytes(capi, ids, up, down):
    return capi.mxfp4_moe_ffn_workspace_bytes(ids.shape[0], ids.shape[1], up.E, up.K, down.K, down.N)


@pytest.mark.parametrize("T", [9, 400])
def test_the_same_bits_again_and_behind_other_calls(capi, T):
    up, down, x, ids, w, r = ffn_case(capi, T, 4, 10, 512, 256, 384, 7)
    ws = workspace(ws_bytes(capi, ids, up, down))
    first = run_ffn(capi, x, ids, w, up, down, "silu", r, ws=ws)
    other = ids.flip(0).contiguous()
    for _ in range(5):
        run_ffn(capi, x, other, w, up, down, "silu", r, ws=ws)      # leaves another plan in the workspace
        run_linear(capi, x, ids, up)
        assert torch.equal(run_ffn(capi, x, ids, w, up, down, "silu", r, ws=ws), first)
    assert capi.mxfp4_get_device_error() == capi.OK


def test_residual_in_place_and_other_strides(capi):
    up, down, x, ids, w, r = ffn_case(capi, 60, 3, 5, 256, 128, 264, 9)
    want = run_ffn(capi, x, ids, w, up, down, "gelu", r)
    out = r.clone()
    run_ffn(capi, x, ids, w, up, down, "gelu", out, out=out)
    assert torch.equal(out, want)
    for ldr, ldo, at in ((272, 280, 0), (265, 267, 1)):
        rw = torch.zeros(60 * ldr + 8, dtype=BF, device="cuda")[at:at + 60 * ldr].view(60, ldr)
        rw[:, :264] = r
        ow = torch.full((60 * ldo + 8,), 5.0, dtype=BF, device="cuda")[at:at + 60 * ldo].view(60, ldo)
        run_ffn(capi, x, ids, w, up, down, "gelu", rw, out=ow)
        assert torch.equal(ow[:, :264], want) and (ow[:, 264:] == 5).all()
    # without a residual: the same sum with zeros
    none = run_ffn(capi, x, ids, w, up, down, "gelu")
    zero = run_ffn(capi, x, ids, w, up, down, "gelu", torch.zeros_like(r))
    assert torch.equal(none, zero)


@pytest.mark.parametrize("T", [12, 300])
def test_captured_and_replayed_with_new_values(capi, T):
    # router and network in one graph; two graphs share a workspace
    up, down, x, _, _, r = ffn_case(capi, T, 4, 16, 320, 192, 320, 11)
    logits, x1, out1, out2 = torch.randn(T, 16, device="cuda"), x.clone(), r.clone(), r.clone()
    w, ids = torch.empty(T, 4, device="cuda"), torch.empty(T, 4, dtype=torch.int32, device="cuda")
    n = ws_bytes(capi, ids, up, down)
    ws = workspace(n)

    def step(out):
        capi.mxfp4_moe_route(logits, capi.DTYPE_F32, 16, None, T, 16, 4, capi.MOE_SOFTMAX, 1, 1, 1, True, 1.0, w, ids)
        run_ffn(capi, x1, ids, w, up, down, "silu", r, out=out, ws=ws)

    graphs = []
    for out in (out1, out2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(out)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step(out)
        torch.cuda.current_stream().wait_stream(s)
        graphs.append(g)
    for seed in range(4):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        logits.copy_(torch.randn(T, 16, device="cuda", generator=gen))
        logits[seed] = -float("inf")
        x1.copy_(torch.randn(T, 320, device="cuda", generator=gen))
        for g, out in zip(graphs, (out1, out2)):
            out.zero_()
            g.replay()
        eager = r.clone()
        step(eager)
        torch.cuda.synchronize()
        assert torch.equal(out1, eager) and torch.equal(out2, eager) and torch.equal(out1[seed], r[seed])
    assert capi.mxfp4_get_device_error() == capi.OK


@pytest.mark.parametrize("T", [6, 200])
def test_weights_and_ids_written_by_the_kernels_before(capi, T):
    # copies straight before the calls, in one graph: no ordering call is needed
    up, down, x, ids, w, r = ffn_case(capi, T, 4, 6, 512, 320, 384, 31)
    up2, down2, x2, ids2, w2, _ = ffn_case(capi, T, 4, 6, 512, 320, 384, 41)
    want = run_ffn(capi, x2, ids2, w2, up2, down2, "silu", r)
    want_rows = run_linear(capi, x2, ids2, up2)
    out, rows = torch.zeros_like(want), torch.zeros_like(want_rows)
    ws, ws2 = workspace(ws_bytes(capi, ids, up, down)), workspace(ws_bytes(capi, ids, up, down))
    sources = [(x, x2), (ids, ids2), (w, w2), (up.bias_dev, up2.bias_dev), (down.bias_dev, down2.bias_dev),
               (down.packed, down2.packed), (up.packed, up2.packed)]
    first = [a.clone() for a, _ in sources]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for a, b in sources:
                a.copy_(b)
            run_ffn(capi, x, ids, w, up, down, "silu", r, out=out, ws=ws)
            run_linear(capi, x, ids, up, out=rows, ws=ws2)
            for (a, _), b in zip(sources, first):
                a.copy_(b)
    torch.cuda.synchronize()
    for _ in range(5):
        out.zero_()
        rows.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(rows, want_rows)


def test_two_streams_with_a_workspace_each(capi):
    cases = [ffn_case(capi, 50, 3, 6, 256, 128, 256, 20), ffn_case(capi, 333, 2, 4, 384, 256, 200, 21)]
    want = [run_ffn(capi, *c[2:5], c[0], c[1], "silu", c[5]) for c in cases]
    outs = [torch.empty_like(v) for v in want]
    wss = [workspace(ws_bytes(capi, c[3], c[0], c[1])) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, out, ws in zip(cases, streams, outs, wss):
            run_ffn(capi, *c[2:5], c[0], c[1], "silu", c[5], out=out, ws=ws, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_two_host_threads_whose_first_calls_are_theirs(capi):
    # one captures its first call and replays it, the other calls beside it
    import threading
    cases = [ffn_case(capi, 50, 3, 6, 256, 128, 256, 20), ffn_case(capi, 333, 2, 4, 384, 256, 200, 21)]
    want = [run_ffn(capi, *c[2:5], c[0], c[1], "silu", c[5]) for c in cases]
    outs = [torch.zeros_like(v) for v in want]
    wss = [workspace(ws_bytes(capi, c[3], c[0], c[1])) for c in cases]
    torch.cuda.synchronize()
    errors = []

    def call(i, stream=None):
        c = cases[i]
        run_ffn(capi, *c[2:5], c[0], c[1], "silu", c[5], out=outs[i], ws=wss[i], stream=stream)

    def captured():
        try:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, capture_error_mode="thread_local"):
                call(0)
            for _ in range(10):
                graph.replay()
            torch.cuda.synchronize()
        except Exception as e:      # noqa: BLE001 (told to the main thread)
            errors.append(e)

    def eager():
        try:
            s = torch.cuda.Stream()
            for _ in range(10):
                call(1, s)
            s.synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=f) for f in (captured, eager)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_one_expert_is_the_dense_layer(capi):
    # moe_linear of one expert against mxfp4_gemm: both within 2 ulp of the same
    # exact value; here on values whose sums are exact in fp32, so the same bits
    N, K, T = 300, 512, 70
    w = Experts(capi, 1, N, K, 3, False)
    w.scales[:] = 127
    from helpers import gemm_workspace, pack_weights
    w.packed = pack_weights(capi, w.codes, w.scales, K)
    x = synth.f32_to_bf16_bits(np.random.default_rng(0).integers(-4, 5, (T, K)).astype(np.float32))
    a = run_linear(capi, dev_bf16(x), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), w)
    out = torch.empty(T, N, dtype=BF, device="cuda")
    n = capi.mxfp4_gemm_workspace_bytes(T, N, K)
    capi.mxfp4_gemm(dev_bf16(x), K, None, None, 0, w.packed, None, out, N, T, N, K, gemm_workspace(capi, n), n)
    assert torch.equal(a, out)


def test_route_of_a_last_token_beyond_the_block(capi):
    x = torch.randn(4097, 72, device="cuda")
    w, ids = run_route(capi, x, None, 5, "sigmoid")
    w1, i1 = run_route(capi, x[4096:], None, 5, "sigmoid")
    assert torch.equal(w[4096:], w1) and torch.equal(ids[4096:], i1)
