"""The 8-bit operators' C ABI without a GPU: struct layouts, argument checks that come
before any CUDA call, and the 64-bit restatements' own pins."""
import ctypes

import numpy as np
import pytest

import moe_decode_step_gb300 as M
from moe_decode_step_gb300 import _binding as b

import _fp8 as ref
import _serving as s

P, I64, I32, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


@pytest.fixture(scope="module", autouse=True)
def built():
    from moe_decode_step_gb300 import build
    build.build()


def _struct(name, *fields):
    return type(name, (ctypes.Structure,), {"_fields_": list(fields)})


Norm = _struct("Norm", ("x", P), ("x_stride", I64), ("residual", P), ("residual_stride", I64),
               ("gamma", P), ("out", P), ("out_stride", I64), ("codes", P), ("codes_stride", I64),
               ("scales", P), ("scales_stride", I64), ("n_rows", I64), ("d", I32), ("dtype", I32),
               ("gamma_dtype", I32), ("eps", F))
Product = _struct("Product", ("x", P), ("x_stride", I64), ("x_scales", P), ("x_scales_stride", I64),
                  ("w", P), ("w_stride", I64), ("w_expert_stride", I64), ("w_scales", P),
                  ("w_scales_stride", I64), ("w_scales_expert_stride", I64), ("offsets", P),
                  ("rows", P), ("out", P), ("out_stride", I64), ("out_scales", P),
                  ("out_scales_stride", I64),
                  *((n, I32) for n in ("n_rows", "x_rows", "n", "k", "n_experts", "w_format",
                                       "activation", "out_dtype")))
Combine = _struct("Combine", ("y", P), ("y_stride", I64), ("w", P), ("slots", P), ("residual", P),
                  ("residual_stride", I64), ("out", P), ("out_stride", I64),
                  *((n, I32) for n in ("n_tokens", "top_k", "y_rows", "d", "dtype")))

BAD, NO, OK = 1, 2, 0


def test_packed_formats_have_the_structs_layout():
    for fmt, st in ((b.RMS_NORM, Norm), (b.FP8_PRODUCT, Product), (b.COMBINE, Combine)):
        assert fmt.size == ctypes.sizeof(st)
        values = list(range(1, len(st._fields_) + 1))
        got = st.from_buffer_copy(fmt.pack(*values))
        assert [getattr(got, n) for n, _ in st._fields_] == values


def _norm(**kw):
    good = dict(x=4096, x_stride=64, residual=8192, residual_stride=64, gamma=4096, out=4096,
                out_stride=64, codes=4096, codes_stride=64, scales=77, scales_stride=1, n_rows=2,
                d=64, dtype=0, gamma_dtype=2, eps=1e-6)
    return M.lib().moe_rms_norm(None, ctypes.byref(Norm(**{**good, **kw})))


def test_norm_checks():
    assert M.lib().moe_rms_norm(None, None) == BAD
    for kw in (dict(x=None), dict(gamma=None), dict(out=None, codes=None, scales=None),
               dict(codes=None), dict(scales=None), dict(n_rows=-1), dict(d=0), dict(dtype=3),
               dict(dtype=-1), dict(gamma_dtype=3), dict(eps=-1.0), dict(eps=float("nan")),
               dict(residual_stride=56), dict(out_stride=0), dict(codes_stride=56),
               dict(scales_stride=0)):
        assert _norm(**kw) == BAD, kw
    for kw in (dict(d=60), dict(d=16392, x_stride=16392, residual_stride=16392, out_stride=16392,
                                codes_stride=16392, scales_stride=129), dict(x=8), dict(residual=8),
               dict(gamma=8), dict(out=4104), dict(codes=4100), dict(x_stride=65),
               dict(residual_stride=68), dict(out_stride=65), dict(codes_stride=65)):
        assert _norm(**kw) == NO, kw
    assert _norm(n_rows=0, x=None) == OK


def test_quantize_and_pack_checks():
    def q(x=4096, dtype=0, xs=64, rows=2, d=64, codes=4096, cs=64, scales=77, ss=1):
        return M.lib().moe_fp8_quantize(None, x, dtype, xs, rows, d, codes, cs, scales, ss)
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(rows=-1), dict(d=0),
               dict(dtype=3), dict(cs=8), dict(ss=0)):
        assert q(**kw) == BAD, kw
    for kw in (dict(d=12, cs=64), dict(x=8), dict(codes=4), dict(xs=4), dict(cs=68)):
        assert q(**kw) == NO, kw
    assert q(rows=0, x=None) == OK

    def p(w=4096, dtype=0, mats=1, n=3, k=5, codes=1, scales=1):
        return M.lib().moe_fp8_pack(None, w, dtype, mats, n, k, codes, scales)
    for kw in (dict(w=None), dict(codes=None), dict(scales=None), dict(mats=-1), dict(n=0),
               dict(k=0), dict(dtype=3)):
        assert p(**kw) == BAD, kw
    for kw in (dict(w=3), dict(w=4098, dtype=2), dict(n=2 ** 31), dict(mats=2 ** 31 - 1, n=129)):
        assert p(**kw) == NO, kw
    assert p(mats=0, w=None) == OK


def _product(**kw):
    good = dict(x=4096, x_stride=256, x_scales=1, x_scales_stride=2, w=4096, w_stride=256,
                w_expert_stride=65536, w_scales=1, w_scales_stride=2, w_scales_expert_stride=4,
                offsets=64, rows=64, out=4096, out_stride=256, out_scales=1, out_scales_stride=1,
                n_rows=8, x_rows=5, n=256, k=256, n_experts=3, w_format=0, activation=0, out_dtype=0)
    return M.lib().moe_fp8_product(None, ctypes.byref(Product(**{**good, **kw})))


def test_product_checks():
    assert M.lib().moe_fp8_product(None, None) == BAD
    for kw in (dict(x=None), dict(x_scales=None), dict(w=None), dict(w_scales=None), dict(out=None),
               dict(offsets=None), dict(rows=None), dict(n_rows=-1), dict(x_rows=-1),
               dict(x_rows=0), dict(n=0), dict(k=0), dict(n_experts=0), dict(w_format=2),
               dict(activation=2), dict(out_dtype=4), dict(out_dtype=3),
               dict(activation=1, out_dtype=3, out_scales=None), dict(activation=1, n=255),
               dict(x_stride=240), dict(w_stride=240), dict(out_stride=255),
               dict(activation=1, out_dtype=3, out_scales_stride=0)):
        assert _product(**kw) == BAD, kw
    for kw in (dict(k=248), dict(k=8), dict(x=4104), dict(x_stride=264), dict(w=4104),
               dict(w_stride=264), dict(w_expert_stride=65528), dict(n_experts=1025),
               dict(out=4097), dict(out_dtype=2, out=4098),
               dict(w_format=1, k=192), dict(w_format=1, w=4112), dict(w_format=1, w_stride=144),
               dict(n_rows=2 ** 31 - 100), dict(x_stride=2 ** 32)):
        assert _product(**kw) == NO, kw
    assert _product(n_rows=0, x=None, out=None) == OK


def test_dispatch_and_combine_checks():
    def d(idx=64, tokens=2, k=3, experts=4, offsets=64, rows=64, slots=64):
        return M.lib().moe_dispatch(None, idx, tokens, k, experts, offsets, rows, slots)
    for kw in (dict(idx=None), dict(offsets=None), dict(rows=None), dict(slots=None),
               dict(tokens=-1), dict(k=0), dict(experts=0)):
        assert d(**kw) == BAD, kw
    for kw in (dict(experts=1025), dict(tokens=2 ** 24, k=2)):
        assert d(**kw) == NO, kw

    def c(**kw):
        good = dict(y=4096, y_stride=64, w=64, slots=64, residual=4096, residual_stride=64,
                    out=4096, out_stride=64, n_tokens=2, top_k=3, y_rows=6, d=64, dtype=0)
        return M.lib().moe_combine(None, ctypes.byref(Combine(**{**good, **kw})))
    assert M.lib().moe_combine(None, None) == BAD
    for kw in (dict(y=None), dict(w=None), dict(slots=None), dict(out=None), dict(n_tokens=-1),
               dict(top_k=0), dict(y_rows=-1), dict(d=0), dict(dtype=3), dict(out_stride=32)):
        assert c(**kw) == BAD, kw
    for kw in (dict(d=60), dict(top_k=33), dict(y=8), dict(residual=8), dict(out=8),
               dict(y_stride=60), dict(residual_stride=60), dict(out_stride=68)):
        assert c(**kw) == NO, kw
    assert c(n_tokens=0, y=None) == OK


# ---------------------------------------------------------------------------
# The restatements
# ---------------------------------------------------------------------------
def test_exponent_is_the_smallest_that_holds():
    rng = np.random.default_rng(0)
    amax = np.concatenate([2.0 ** rng.uniform(-140, 127, 400), 448.0 * 2.0 ** np.arange(-126, 120),
                           np.nextafter(448.0 * 2.0 ** np.arange(-126, 119), np.inf), [0.0]])
    e = ref.block_exp(amax)
    assert ((e >= -126) & (e <= 120)).all()
    assert (amax <= 448.0 * 2.0 ** e).all()
    assert ((e == -126) | (amax > 448.0 * 2.0 ** (e - 1.0))).all()


def test_values_survive_their_8_bit_form():
    """A value is off by at most half a step of its block's scale."""
    rng = np.random.default_rng(1)
    y = rng.standard_normal((7, 300)) * np.exp(3 * rng.standard_normal((7, 1)))
    codes, scales = ref.quantize(y)
    got = ref.row_values(codes, scales)
    unit = 2.0 ** (np.repeat(scales.astype(int), 128, 1)[:, :300] - 127.0)
    assert (np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * unit)).all()
    w = rng.standard_normal((130, 140))
    codes, scales = ref.pack(w)
    assert scales.shape == (2, 2)
    assert np.abs(ref.weight_values(codes, scales, False) - w).max() <= 2.0 ** -4 * np.abs(w).max()


def test_mxfp4_values_are_the_packers():
    import torch
    rng = np.random.default_rng(2)
    v = rng.standard_normal((5, 64)).astype(np.float32)
    q, sc = M.mxfp4_pack(torch.from_numpy(v))
    got = ref.weight_values(q.numpy(), sc.numpy(), True)
    table = set(ref.E2M1.tolist())
    unit = 2.0 ** (np.repeat(sc.numpy().astype(int), 32, 1) - 127.0)
    assert set((got / unit).ravel().tolist()) <= table
    # nearest: half the widest step beside it, values above 5 become 6
    assert (np.abs(got - v) <= np.where(np.abs(v) / unit > 5, np.abs(np.abs(v) - 6 * unit),
                                        unit * 1.0) + 1e-12).all()


def test_dispatch_restatement():
    off, rows, slots = ref.dispatch(np.array([[2, 0], [0, -1], [2, 1]]), 4)
    assert off.tolist() == [0, 2, 3, 5, 5]
    assert rows.tolist() == [0, 1, 2, 0, 2, -1]
    assert slots.tolist() == [[3, 0], [1, -1], [4, 2]]


def test_e4m3_rounding_of_the_restatement():
    assert s.e4m3_round(np.array([0.0, 448.0, 1e9, np.inf])).tolist() == [0, 126, 126, 126]
