"""The many-row form of the latent-attention oracle is the row-by-row one."""

import numpy as np
import torch

import mla_wide
from oracle import mla_ref as ref


def same(a, b):
    for x, y in zip(a, b):
        assert np.array_equal(np.isneginf(x), np.isneginf(y))
        assert np.allclose(np.where(np.isneginf(x), 0, x), np.where(np.isneginf(y), 0, y), rtol=1e-12, atol=1e-13)


def test_decode():
    g = np.random.default_rng(0)
    H, L, R, page, q_len, lens = 3, 6, 2, 4, 2, [11, 0, 1, 8]
    cache, table = g.normal(size=(9, page, L + R)), np.array([[2, 0, 3], [1, 1, 1], [4, 0, 0], [5, 8, 0]])
    ql, qr = g.normal(size=(H, len(lens) * q_len, L)), g.normal(size=(len(lens) * q_len, H, R))
    want = ref.decode(ql, qr, cache, table, lens, q_len, 0.4)
    got = mla_wide.decode(*(torch.from_numpy(x) for x in (ql, qr, cache, table)), lens, q_len, 0.4)
    same(got, want)


def test_prefill():
    g = np.random.default_rng(1)
    H, dn, R, dv = 2, 5, 3, 4
    cu_q, cu_k = [0, 4, 4, 9, 10, 12], [0, 6, 8, 11, 11, 13]
    args = (g.normal(size=(12, H, dn)), g.normal(size=(12, H, R)), g.normal(size=(13, H, dn)), g.normal(size=(13, R)),
            g.normal(size=(13, H, dv)))
    for causal, scale in ((True, 0.3), (False, -0.2)):
        want = ref.prefill(*args, cu_q, cu_k, scale, causal)
        same(mla_wide.prefill(*(torch.from_numpy(x) for x in args), cu_q, cu_k, scale, causal), want)


def test_cuts():
    units = mla_wide.decode_units([0, 64, 65], 2, 3)
    assert units == [1, 1, 4, 4, 5, 5]
    # 20 units over 6 blocks begin at 0, 4, 8, 11, 14, 17
    # (2, 2, 1, 4 and 2 into the groups that begin at 2, 6, 10, 10 and 15)
    assert mla_wide.cut_places(units, 6, 3) == {2, 1, -1}
    assert mla_wide.cut_places([10, 10], 4, 3) == {-1, 0}
