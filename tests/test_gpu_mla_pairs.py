"""Prefill in pairs of blocks: what one block of a pair hands to the other
(queries, keys, values, values cleared behind a sequence's end, softmax
weights) must be there when the products that read it are issued.  Whatever
came too early would show as NaN or as other bits in some call."""

import numpy as np
import pytest
import torch

from oracle import mla_ref as ref
from mla_helpers import check_attention, f64, rnd, run_prefill

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


@pytest.mark.parametrize("dn,dv", [(64, 64), (192, 256)])
@pytest.mark.parametrize("causal", [True, False])
def test_pairs_repeat_their_bits_beside_keys_of_nan(capi, dn, dv, causal):
    # every prompt's keys end inside a tile and are followed by the keys of a
    # sequence without queries, which hold NaN; some tiles of 128 and 256 keys
    # exactly have nothing to clear between them
    new = [300, 0, 131, 0, 257, 0, 256, 0, 500, 0, 390, 0]
    old = [0, 150, 45, 130, 0, 140, 128, 129, 7, 133, 250, 128]
    H = 24
    total = [a + b for a, b in zip(new, old)]
    cu_q, cu_k = (np.concatenate(([0], np.cumsum(x))) for x in (new, total))
    Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
    q, kv, kr = rnd(1, Tq, H, dn + R), rnd(2, Tk, H, dn + dv), rnd(3, Tk, R)
    for s in range(1, len(new), 2):
        kv[cu_k[s]:cu_k[s + 1]] = float("nan")
        kr[cu_k[s]:cu_k[s + 1]] = float("nan")
    args = (q[..., :dn], q[..., dn:], kv[..., :dn], kr, kv[..., dn:])
    cq, ck = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k))
    scale = (dn + R) ** -0.5
    out, lse = run_prefill(capi, *args, cq, ck, scale, causal)
    some = [0, 11, H - 1]                       # (the oracle's share; the rest by equality of calls and finiteness)
    want = ref.prefill(*(f64(t[:, some] if t.dim() == 3 else t) for t in args), cu_q, cu_k, scale, causal)
    check_attention(out[:, some], lse[:, some], want, max(total), dn + R, f"dn {dn} dv {dv} causal {causal}")
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    noise = torch.rand(1 << 20, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            noise.sort()                        # other code in the instruction caches
        again, lse2 = run_prefill(capi, *args, cq, ck, scale, causal)
        assert torch.equal(again, out) and torch.equal(lse2, lse), f"call {i}"


def test_pairs_rescale_after_tiles_that_need_none(capi):
    # scores that pass the running maximum by far in some key tiles and not at
    # all in those between, one to five of them
    n, H, dn, dv = 2300, 8, 64, 64
    q, kv, kr = rnd(11, n, H, dn + R), rnd(12, n, H, dn + dv), rnd(13, n, R)
    rise = [0, 1, 3, 4, 7, 12, 13, 17]
    for k, t in enumerate(rise):
        kv[128 * t: 128 * (t + 1), :, :dn] *= 2.0 ** k
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    args = (q[..., :dn], q[..., dn:], kv[..., :dn], kr, kv[..., dn:])
    scale = 0.02
    out, lse = run_prefill(capi, *args, cu, cu, scale, True)
    some = [0, H - 1]
    want = ref.prefill(*(f64(t[:, some] if t.dim() == 3 else t) for t in args), [0, n], [0, n], scale, True)
    check_attention(out[:, some], lse[:, some], want, n, dn + R, "rising in steps")
    for i in range(20):
        again, lse2 = run_prefill(capi, *args, cu, cu, scale, True)
        assert torch.equal(again, out) and torch.equal(lse2, lse), f"call {i}"
