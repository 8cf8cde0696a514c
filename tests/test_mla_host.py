"""Latent attention on the host: the oracle's pins, and the refusals of the
entry points (no compute call is made)."""

import itertools
from fractions import Fraction

import numpy as np
import pytest

from oracle import mla_ref as ref

L, R = 512, 64


# ----------------------------------------------------------------- oracle
def test_attend_closed_forms():
    v = np.array([[1.0, 2.0], [3.0, 6.0], [5.0, 4.0]])
    out, lse, _, _ = ref.attend(np.zeros(4), np.ones((3, 4)), v, 1.0)       # equal scores: the mean
    assert np.allclose(out, [3, 4], atol=1e-15) and np.isclose(lse, np.log(3))
    k = np.eye(3)
    out, lse, mag, smag = ref.attend(np.array([0.0, np.log(2.0), np.log(5.0)]), k, -v, 1.0)
    assert np.allclose(out, -(v[0] + 2 * v[1] + 5 * v[2]) / 8) and np.isclose(lse, np.log(8))
    assert np.allclose(mag, -out) and np.isclose(smag, np.log(5.0))
    out, lse, _, _ = ref.attend(np.ones(4), np.zeros((0, 4)), np.zeros((0, 2)), 1.0)
    assert (out == 0).all() and np.isneginf(lse)


def test_attend_against_rationals():
    # scores log2 w: weights are exact rationals
    w = [Fraction(1), Fraction(3), Fraction(4)]
    v = [Fraction(7), Fraction(-2), Fraction(1, 2)]
    want = sum(a * b for a, b in zip(w, v)) / sum(w)
    out, lse, _, _ = ref.attend(np.array([1.0]), np.array([[np.log(float(a))] for a in w]),
                                np.array([[float(b)] for b in v]), 1.0)
    assert abs(out[0] - float(want)) < 1e-14 and abs(lse - np.log(8.0)) < 1e-14


def test_rotation_is_a_rotation_and_pairs_differ():
    x = np.arange(1.0, 9.0)
    ang = np.array([0.3, 1.1, -2.0, 0.0])
    for inter in (True, False):
        y = ref.rotate(x, np.cos(ang), np.sin(ang), inter)
        assert np.isclose(np.linalg.norm(x), np.linalg.norm(y))
        assert np.allclose(ref.rotate(y, np.cos(-ang), np.sin(-ang), inter), x)
    quarter = np.full(4, np.pi / 2)
    assert np.allclose(ref.rotate(x, np.cos(quarter), np.sin(quarter), True), [-2, 1, -4, 3, -6, 5, -8, 7])
    assert np.allclose(ref.rotate(x, np.cos(quarter), np.sin(quarter), False), [-5, -6, -7, -8, 1, 2, 3, 4])


def test_decode_is_prefill_of_the_newest_tokens():
    # one head: the absorbed form is the expanded one with K and V the latents
    g = np.random.default_rng(0)
    n, q_len, lat = 11, 3, 6
    cache, table = g.normal(size=(4, 4, lat + 2)), np.array([[2, 0, 3]])
    rows = np.array([cache[table[0, j // 4], j % 4] for j in range(n)])
    ql, qr = g.normal(size=(1, q_len, lat)), g.normal(size=(q_len, 1, 2))
    a = ref.decode(ql, qr, cache, table, [n], q_len, 0.4)
    b = ref.prefill(ql.transpose(1, 0, 2), qr, rows[:, None, :lat], rows[:, lat:], rows[:, None, :lat], [0, q_len],
                    [0, n], 0.4, True)
    assert np.allclose(a[0].transpose(1, 0, 2), b[0]) and np.allclose(a[1], b[1])


# --------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def capi():
    from mxfp4_quantized_gemm_gb300 import build
    build.build()
    from mxfp4_quantized_gemm_gb300 import capi as c
    return c


A = 0x10000       # an aligned, never dereferenced address

STORE = dict(kv=A, ld_kv=576, gamma=A, eps=1e-6, q=A, q_tok=64 * 64, q_head=64, q_out=A, qo_tok=64 * 64, qo_head=64,
             H=64, cos_sin=A, max_pos=100, positions=A, slots=A, cache=A, page_stride=64 * 576, page_size=64,
             num_pages=10, T=4, L=512, R=64, interleaved=True, stream=0)
DECODE = dict(q_lat=A, ql_tok=512, ql_head=4 * 512, q_rope=A, qr_tok=64 * 64, qr_head=64, cache=A, page_stride=64 * 576,
              page_size=64, num_pages=10, page_table=A, table_stride=8, max_pages=8, seq_lens=A, out=A, o_tok=512,
              o_head=4 * 512, lse=A, S=4, q_len=1, H=64, L=512, R=64, scale=0.06, workspace=A, workspace_bytes=1 << 40,
              stream=0)
PREFILL = dict(q_nope=A, qn_tok=64 * 256, qn_head=256, q_rope=A, qr_tok=64 * 256, qr_head=256, k_nope=A,
               kn_tok=64 * 448, kn_head=448, k_rope=A, kr_tok=64, v=A, v_tok=64 * 448, v_head=448, cu_q=A, cu_k=A, S=2,
               out=A, o_tok=64 * 256, o_head=256, lse=A, Tq=100, Tk=100, H=64, dn=192, R=64, dv=256, scale=0.06,
               causal=True, stream=0)


def status(capi, fn, base, **change):
    with pytest.raises(capi.Mxfp4Error) as e:
        getattr(capi, fn)(**{**base, **change})
    return e.value.status


@pytest.mark.parametrize("fn,base", [("mxfp4_mla_store", STORE), ("mxfp4_mla_decode", DECODE),
                                     ("mxfp4_mla_prefill", PREFILL)])
def test_refusals_common(capi, fn, base):
    import torch
    if not torch.cuda.is_available():
        assert status(capi, fn, base) in (capi.ERR_NO_DEVICE, capi.ERR_CUDA)     # arguments fine: only the device is missing
    pointers = [k for k, v in base.items() if v == A and k not in ("lse", "workspace")]
    for k in pointers:
        assert status(capi, fn, base, **{k: None}) == capi.ERR_INVALID_ARG, k
    for k in [k for k in pointers if k not in ("positions", "slots", "page_table", "seq_lens", "cu_q", "cu_k")]:
        assert status(capi, fn, base, **{k: A + 2}) == capi.ERR_MISALIGNED, k
    for k in [k for k in pointers if k in ("positions", "slots", "page_table", "seq_lens", "cu_q", "cu_k")]:
        assert status(capi, fn, base, **{k: A + 2}) == capi.ERR_MISALIGNED, k
    for k in [k for k in base if k in ("T", "S", "L", "R", "q_len", "max_pages", "page_size", "num_pages", "Tq", "Tk",
                                       "dn", "dv", "max_pos")]:
        assert status(capi, fn, base, **{k: 0}) == capi.ERR_INVALID_ARG, k
        assert status(capi, fn, base, **{k: -3}) == capi.ERR_INVALID_ARG, k
    strides = [k for k in base if k.endswith(("_tok", "_head"))]
    for k, bad in itertools.product(strides, (0, -64)):
        if k == "kr_tok" and bad == 0:
            pass
        assert status(capi, fn, base, **{k: bad}) == capi.ERR_UNSUPPORTED_SHAPE, (k, bad)
    for k in strides:
        assert status(capi, fn, base, **{k: base[k] + 4}) == capi.ERR_MISALIGNED, k
        assert status(capi, fn, base, **{k: 1 << 40}) == capi.ERR_UNSUPPORTED_SHAPE, k
    assert status(capi, fn, base, R=32) == capi.ERR_UNSUPPORTED_SHAPE


def test_refusals_of_each(capi):
    bad = capi.ERR_UNSUPPORTED_SHAPE
    for k in ("mxfp4_mla_store", "mxfp4_mla_decode"):
        base = STORE if k == "mxfp4_mla_store" else DECODE
        for change in (dict(L=64), dict(L=640), dict(L=500), dict(page_size=12, page_stride=64 * 576),
                       dict(page_stride=64 * 576 - 8)):
            assert status(capi, k, base, **change) == bad, change
        assert status(capi, k, base, page_stride=64 * 576 + 4) == capi.ERR_MISALIGNED
    assert status(capi, "mxfp4_mla_store", STORE, ld_kv=568) == bad
    assert status(capi, "mxfp4_mla_store", STORE, ld_kv=580) == capi.ERR_MISALIGNED
    assert status(capi, "mxfp4_mla_store", STORE, H=-1) == capi.ERR_INVALID_ARG
    assert status(capi, "mxfp4_mla_store", STORE, eps=-1.0) == capi.ERR_INVALID_ARG
    assert status(capi, "mxfp4_mla_store", STORE, eps=float("nan")) == capi.ERR_INVALID_ARG
    assert status(capi, "mxfp4_mla_decode", DECODE, H=0) == capi.ERR_INVALID_ARG
    assert status(capi, "mxfp4_mla_decode", DECODE, table_stride=7) == bad
    assert status(capi, "mxfp4_mla_decode", DECODE, workspace=None) == capi.ERR_WORKSPACE
    assert status(capi, "mxfp4_mla_decode", DECODE, workspace_bytes=100) == capi.ERR_WORKSPACE
    assert status(capi, "mxfp4_mla_decode", DECODE, workspace=A + 8) == capi.ERR_MISALIGNED
    assert status(capi, "mxfp4_mla_decode", DECODE, S=1 << 20, q_len=1 << 12) == bad
    assert status(capi, "mxfp4_mla_decode", DECODE, lse=A + 2) == capi.ERR_MISALIGNED
    for change in (dict(dn=196), dict(dn=200), dict(dv=260), dict(dv=264), dict(H=70000)):
        assert status(capi, "mxfp4_mla_prefill", PREFILL, **change) == bad, change
    assert status(capi, "mxfp4_mla_prefill", PREFILL, H=0) == capi.ERR_INVALID_ARG


def test_workspace_query(capi):
    q = capi.mxfp4_mla_decode_workspace_bytes
    assert q(4, 1, 64, 512, 64) == 0 and q(0, 1, 64, 512, 4096) == 0 and q(4, 1, 64, 0, 4096) == 0
    assert q(4, 1, 64, 512, 65) > 0
    part = 64 * (512 + 2) * 4
    assert q(1, 1, 64, 512, 128) == 2 * 2 * part                  # two tiles: two blocks, two parts each
    assert q(1000, 4, 128, 512, 10 ** 6) <= 256 * 2 * part        # bounded by the grid
    assert q(1, 1, 8, 512, 10 ** 6) < q(1, 1, 64, 512, 10 ** 6)   # fewer rows, smaller parts


def test_error_status_has_a_name(capi):
    assert capi.mxfp4_status_string(capi.ERR_INDEX) == "MXFP4_ERR_INDEX"


# -------------------------------------------------- operators without a GPU
def test_operators_trace_and_refuse_on_meta_tensors():
    import torch

    from mxfp4_quantized_gemm_gb300 import ops  # noqa: F401
    mx, bf = torch.ops.mxfp4, torch.bfloat16

    def meta(*shape, dtype=bf):
        return torch.empty(*shape, dtype=dtype, device="meta")

    cache = meta(10, 64, 576)
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    q = mx.mla_store(meta(5, 576), meta(512), 1e-6, meta(5, 8, 64), meta(100, 64, dtype=f32), meta(5, dtype=i64),
                     meta(5, dtype=i64), cache, False)
    assert q.shape == (5, 8, 64)
    out, lse = mx.mla_decode(meta(8, 6, 512), meta(6, 8, 64), cache, meta(3, 4, dtype=i32), meta(3, dtype=i32), 0.1)
    assert out.shape == (8, 6, 512) and lse.shape == (6, 8) and lse.dtype == f32
    cu = meta(3, dtype=i32)
    out, lse = mx.mla_prefill(meta(7, 8, 128), meta(7, 8, 64), meta(9, 8, 128), meta(9, 64), meta(9, 8, 256), cu, cu,
                              0.1, True)
    assert out.shape == (7, 8, 256) and lse.shape == (7, 8)

    def store(**change):
        a = dict(kv=meta(5, 576), gamma=meta(512), eps=1e-6, q_rope=meta(5, 8, 64), cos_sin=meta(100, 64, dtype=f32),
                 positions=meta(5, dtype=i64), slots=meta(5, dtype=i64), cache=cache, interleaved=True)
        a.update(change)
        with pytest.raises(RuntimeError, match="mla_store"):
            mx.mla_store(**a)

    store(kv=meta(5, 512))
    store(kv=meta(5, 576, dtype=f32))
    store(gamma=meta(500))
    store(q_rope=meta(5, 8, 32))
    store(q_rope=meta(4, 8, 64))
    store(cos_sin=meta(100, 64))
    store(positions=meta(5, dtype=i32))
    store(slots=meta(6, dtype=i64))
    store(cache=meta(10, 60, 576), kv=meta(5, 576))
    store(cache=meta(10, 64, 564), kv=meta(5, 564))
    store(cache=meta(10, 576, 64).transpose(1, 2))

    def decode(**change):
        a = dict(q_lat=meta(8, 6, 512), q_rope=meta(6, 8, 64), cache=cache, page_table=meta(3, 4, dtype=i32),
                 seq_lens=meta(3, dtype=i32), scale=0.1)
        a.update(change)
        with pytest.raises(RuntimeError, match="mla_decode"):
            mx.mla_decode(**a)

    decode(q_lat=meta(8, 6, 256))
    decode(q_rope=meta(8, 6, 64))
    decode(page_table=meta(3, 4, dtype=i64))
    decode(page_table=meta(2, 4, dtype=i32))
    decode(seq_lens=meta(4, dtype=i32), page_table=meta(4, 4, dtype=i32))
    decode(cache=meta(10, 64, 576, dtype=f32))

    def prefill(**change):
        a = dict(q_nope=meta(7, 8, 128), q_rope=meta(7, 8, 64), k_nope=meta(9, 8, 128), k_rope=meta(9, 64),
                 v=meta(9, 8, 256), cu_q=cu, cu_k=cu, scale=0.1, causal=True)
        a.update(change)
        with pytest.raises(RuntimeError, match="mla_prefill"):
            mx.mla_prefill(**a)

    prefill(q_nope=meta(7, 8, 200), k_nope=meta(9, 8, 200))
    prefill(v=meta(9, 8, 264))
    prefill(v=meta(9, 8, 100))
    prefill(v=meta(9, 4, 256))
    prefill(k_rope=meta(9, 8, 64))
    prefill(q_rope=meta(9, 8, 64))
    prefill(cu_q=meta(4, dtype=i32))
    prefill(cu_k=meta(3, dtype=i64))
