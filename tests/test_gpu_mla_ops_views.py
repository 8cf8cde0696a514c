"""The latent-attention operators on views that the kernels cannot read in
place: they are copied, not refused."""

import pytest
import torch

from mxfp4_quantized_gemm_gb300 import ops  # noqa: F401
from mla_helpers import BF, paged, rnd

pytestmark = pytest.mark.gpu
mx = torch.ops.mxfp4
L, R = 128, 64


def test_decode_takes_any_page_table():
    H, S, page, n = 4, 3, 16, 48
    cache, table = paged(1, [n], page, L, R)
    q_lat, q_rope = rnd(2, H, S, L), rnd(3, S, H, R)
    lens = torch.tensor([40, 7, 33], dtype=torch.int32, device="cuda")
    shared = table.expand(S, -1)                          # one prefix for all sequences
    want = mx.mla_decode(q_lat, q_rope, cache, shared.contiguous(), lens, 0.07)
    flat = torch.cat((table[0], table[0], table[0]))
    overlapping = torch.as_strided(flat, (S, 2), (1, 1))  # rows that share entries
    for t in (shared, shared.contiguous().t().contiguous().t()):
        got = mx.mla_decode(q_lat, q_rope, cache, t, lens, 0.07)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    short = lens.clamp(max=32)
    a = mx.mla_decode(q_lat, q_rope, cache, overlapping, short, 0.07)
    b = mx.mla_decode(q_lat, q_rope, cache, overlapping.clone(), short, 0.07)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = table[:, :1].expand(S, 1)                       # a single page for all
    a = mx.mla_decode(q_lat, q_rope, cache, one, lens.clamp(max=page), 0.07)
    b = mx.mla_decode(q_lat, q_rope, cache, one.contiguous(), lens.clamp(max=page), 0.07)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("off", [1, 4])
def test_store_takes_any_gamma_and_rotation_table(off):
    T, H, page, pages = 5, 2, 8, 2
    kv, gamma, q = rnd(4, T, L + R), rnd(5, L), rnd(6, T, H, R)
    cs = torch.randn(50, R, generator=torch.Generator().manual_seed(7)).cuda()
    pos, slots = torch.arange(T).cuda() * 9, torch.arange(T).cuda() + 4

    def call(g, c):
        cache = torch.zeros(pages, page, L + R, dtype=BF, device="cuda")
        return mx.mla_store(kv, g, 1e-6, q, c, pos, slots, cache, True), cache

    want = call(gamma, cs)
    g = torch.empty(L + off, dtype=BF, device="cuda")[off:].copy_(gamma)
    c = torch.empty(50 * R + off, device="cuda")[off:].view(50, R).copy_(cs)
    if off == 1:
        assert g.data_ptr() % 16 and c.data_ptr() % 16
    for args in ((g, cs), (gamma, c), (g.view(1, L), c), (torch.stack((gamma, gamma), 1)[:, 0], cs)):
        got = call(*args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
