"""The latent-attention operators of torch.ops.mxfp4 on the GPU: equal to the
C-ABI calls, views that need a copy, empty batches, opcheck, and the layer of
the example."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from mxfp4_quantized_gemm_gb300 import ops  # noqa: F401
from mla_helpers import BF, paged, rnd, run_decode, run_prefill

pytestmark = pytest.mark.gpu
mx = torch.ops.mxfp4
L, R = 512, 64


@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


def decode_args(H=16, lens=(130, 7)):
    S = len(lens)
    cache, table = paged(3, list(lens), 16)
    return (rnd(1, H, S, L), rnd(2, S, H, R), cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.06)


def prefill_args(H=2, new=(40, 90), dn=64, dv=64):
    T = sum(new)
    q, kv, kr = rnd(4, T, H, dn + R), rnd(5, T, H, dn + dv), rnd(6, T, R)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32, device="cuda")
    return q[..., :dn], q[..., dn:], kv[..., :dn], kr, kv[..., dn:], cu, cu, 0.09, True


def store_args(T=9, H=4, page=8, pages=4):
    g = torch.Generator().manual_seed(7)
    return dict(kv=rnd(8, T, L + R), gamma=rnd(9, L), eps=1e-6, q_rope=rnd(10, T, H, 192 + R)[..., 192:],
                cos_sin=torch.randn(50, R, generator=g).cuda(), positions=torch.arange(T).cuda(),
                slots=torch.randperm(page * pages, generator=g)[:T].cuda(),
                cache=torch.zeros(pages, page, L + R, dtype=BF, device="cuda"), interleaved=True)


def test_decode_is_the_c_call(capi):
    ql, qr, cache, table, lens, scale = decode_args()
    out, lse = mx.mla_decode(ql, qr, cache, table, lens, scale)
    o2, l2 = run_decode(capi, ql, qr, cache, table, lens, 1, scale)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    # head-last queries: read in place; an odd offset: copied
    o3, _ = mx.mla_decode(ql.transpose(0, 1).contiguous().transpose(0, 1), qr, cache, table, lens, scale)
    odd = torch.empty(ql.numel() + 1, dtype=BF, device="cuda")[1:].view(ql.shape).copy_(ql)
    o4, _ = mx.mla_decode(odd, qr, cache, table.t().contiguous().t(), lens, scale)
    assert torch.equal(o3, out) and torch.equal(o4, out)


def test_prefill_is_the_c_call(capi):
    a = prefill_args()
    out, lse = mx.mla_prefill(*a)
    o2, l2 = run_prefill(capi, *a)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    # a value tensor whose innermost dimension is not contiguous is copied
    b = list(a)
    b[4] = a[4].transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(mx.mla_prefill(*b)[0], out)


def test_store_rotates_and_updates_the_cache(capi):
    a, b = store_args(), store_args()
    q = mx.mla_store(**a)
    q2 = torch.empty_like(q)
    kv, qr, cache = b["kv"], b["q_rope"], b["cache"]
    capi.mxfp4_mla_store(kv, kv.stride(0), b["gamma"], 1e-6, qr, qr.stride(0), qr.stride(1), q2, q2.stride(0),
                         q2.stride(1), 4, b["cos_sin"], 50, b["positions"], b["slots"], cache, cache.stride(0), 8, 4, 9,
                         L, R, True)
    assert torch.equal(q, q2) and torch.equal(a["cache"], cache) and cache.abs().sum() > 0


def test_empty_batches(capi):
    a = store_args()
    for k in ("kv", "q_rope", "positions", "slots"):
        a[k] = a[k][:0]
    assert mx.mla_store(**a).shape == (0, 4, R) and (a["cache"] == 0).all()
    b = store_args()
    b["q_rope"] = b["q_rope"][:, :0]
    assert mx.mla_store(**b).shape == (9, 0, R) and (b["cache"] != 0).any()
    ql, qr, cache, table, lens, scale = decode_args()
    out, lse = mx.mla_decode(ql[:, :0], qr[:0], cache, table, lens, scale)
    assert out.shape == (16, 0, L) and lse.shape == (0, 16)
    qn, q_r, kn, kr, v, cu, _, s, c = prefill_args()
    zero = torch.zeros_like(cu)
    out, lse = mx.mla_prefill(qn[:0], q_r[:0], kn, kr, v, zero, cu, s, c)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out, lse = mx.mla_prefill(qn, q_r, kn[:0], kr[:0], v[:0], cu, zero, s, c)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_opcheck(capi):
    for op, args in ((mx.mla_decode, decode_args()), (mx.mla_prefill, prefill_args()),
                     (mx.mla_store, tuple(store_args().values()))):
        torch.library.opcheck(op.default, args, test_utils=("test_schema", "test_faketensor"))


def test_host_tensor_is_refused(capi):
    ql, qr, cache, table, lens, scale = decode_args()
    with pytest.raises(RuntimeError, match="not a CUDA device"):
        mx.mla_decode(ql, qr, cache, table.cpu(), lens, scale)


def test_example_layer(capi):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_attention.py")
    spec = importlib.util.spec_from_file_location("latent_attention_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # each form rounds its intermediate products (K and V, or the absorbed query
    # and the latent sum) and its weights to bf16: a few of its half steps, 2^-8
    assert m.run(heads=8, prompt=150, steps=2, hidden=256) < 8 * 2.0 ** -8
    assert capi.mxfp4_get_device_error() == capi.OK
