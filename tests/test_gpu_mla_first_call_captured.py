"""A host thread whose first call of the library is made while a stream is
captured: the tensor-map kernels need the thread's device context for their
maps, and must find it without a call that the capture forbids."""

import threading

import pytest
import torch

from mla_helpers import BF, paged, rnd, run_prefill

pytestmark = pytest.mark.gpu
R = 64


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


def in_new_thread(call):
    """call() captured as a new thread's first call, and replayed."""
    errors = []

    def work():
        try:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            graph.replay()
            torch.cuda.synchronize()
        except Exception as e:      # noqa: BLE001 (told to the main thread)
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not errors, errors


def test_prefill(capi):
    n, H = 300, 2
    q, kv, kr = rnd(1, n, H, 64 + R), rnd(2, n, H, 128), rnd(3, n, R)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    args = (q[..., :64], q[..., 64:], kv[..., :64], kr, kv[..., 64:], cu, cu, 0.09, True)
    want = run_prefill(capi, *args)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    in_new_thread(lambda: run_prefill(capi, *args, out=out, lse=lse))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_decode(capi):
    H, S, L, page = 4, 2, 128, 16
    q_lat, q_rope = rnd(4, H, S, L), rnd(5, S, H, R)
    cache, table = paged(6, [300, 40], page, L, R)
    lens = torch.tensor([300, 40], dtype=torch.int32, device="cuda")
    n = capi.mxfp4_mla_decode_workspace_bytes(S, 1, H, L, table.shape[1] * page)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(out, lse):
        capi.mxfp4_mla_decode(q_lat, q_lat.stride(1), q_lat.stride(0), q_rope, q_rope.stride(0), q_rope.stride(1),
                              cache, cache.stride(0), page, cache.shape[0], table, table.stride(0), table.shape[1], lens,
                              out, out.stride(1), out.stride(0), lse, S, 1, H, L, R, 0.07, ws, n)

    a, b = ((torch.zeros(H, S, L, dtype=BF, device="cuda"), torch.zeros(S, H, device="cuda")) for _ in range(2))
    call(*a)
    in_new_thread(lambda: call(*b))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[0].abs().sum() > 0


def test_bmm(capi):
    B, M, N, K = 2, 40, 64, 128
    g = torch.Generator().manual_seed(7)
    codes = torch.randint(0, 256, (B, N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scales = torch.full((B, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    packed = torch.empty(capi.mxfp4_packed_weight_bytes(B, N, K), dtype=torch.uint8, device="cuda")
    capi.mxfp4_pack_weights(codes, scales, B, N, K, packed)
    x = rnd(8, B, M, K)
    a, b = (torch.zeros(B, M, N, dtype=BF, device="cuda") for _ in range(2))
    capi.a16wfp4_bmm(x, packed, a, B, M, N, K, capi.OUT_BMN)
    in_new_thread(lambda: capi.a16wfp4_bmm(x, packed, b, B, M, N, K, capi.OUT_BMN))
    assert torch.equal(a, b) and a.abs().sum() > 0
