"""GPU tests of the 8-bit products, norms and expert operators against 64-bit
restatements (_fp8.py, which derives the bounds)."""
import numpy as np
import pytest
import torch

import moe_decode_step_gb300 as M

import _fp8 as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _codes(a):
    return _dev(a).view(torch.float8_e4m3fn)


def _scales(a):
    return _dev(a).view(torch.float8_e8m0fnu)


# ---------------------------------------------------------------------------
# Norm, quantisation, packing
# ---------------------------------------------------------------------------
def _rows(rng, rows, d, dtype):
    v = rng.standard_normal((rows, d)) * np.exp(rng.standard_normal((rows, 1)))
    return _dev(v, torch.float32).to(dtype)


@pytest.mark.parametrize("rows,d", [(1, 7168), (3, 8), (5, 72), (9, 128), (2, 1016), (17, 1024),
                                    (4, 1032), (6, 4096), (3, 4104), (2, 8192), (3, 8200),
                                    (2, 16384), (700, 256)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(rows, d, dtype, residual):
    rng = np.random.default_rng(rows * 31 + d)
    x, r = _rows(rng, rows, d, dtype), _rows(rng, rows, d, dtype) if residual else None
    gamma = _dev(1 + 0.2 * rng.standard_normal(d), torch.float32).to(
        dtype if d % 16 else torch.float32)
    z = _np(x) + (_np(r) if residual else 0.0)
    size = np.abs(_np(x)) + (np.abs(_np(r)) if residual else 0.0)
    scale = 1.0 / np.sqrt((z * z).mean(axis=1, keepdims=True) + 1e-5)
    y = z * scale * _np(gamma)
    tol = 64 * 2.0 ** -24 * np.abs(y) + 2.0 ** -24 * size * scale * np.abs(_np(gamma))
    got = M.rms_norm(x, gamma, residual=r, eps=1e-5, quantize=True)
    if residual:
        ref.check_values(r, z, 2.0 ** -24 * size, dtype, "residual")
    ref.check_values(got.out, y, tol, dtype, "out")
    ref.check_codes(got.codes, got.scales, y, tol, "codes")


def test_rms_norm_strides_and_outputs():
    rng = np.random.default_rng(1)
    big = _rows(rng, 6, 3 * 264, torch.bfloat16)
    x = big.view(6, 3, 264)[:, 1]
    gamma = _dev(np.ones(264), torch.bfloat16)
    plain = M.rms_norm(x.contiguous(), gamma)
    assert plain.codes is None and plain.scales is None
    out = torch.full((6, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    r = M.rms_norm(x, gamma, out=out[:, :264])
    assert torch.equal(r.out, plain.out) and (out[:, 264:] == 7).all()
    only = M.rms_norm(x, gamma, out=False, quantize=True)
    both = M.rms_norm(x, gamma, quantize=True)
    assert only.out is None and torch.equal(only.codes.view(torch.uint8),
                                            both.codes.view(torch.uint8))
    # in place, and x as its own residual
    y = x.contiguous()
    assert torch.equal(M.rms_norm(y, gamma, out=y).out, plain.out)
    z = x.contiguous()
    twice = M.rms_norm(z, gamma, residual=z)
    assert torch.equal(z, 2 * x)
    assert torch.equal(twice.out, M.rms_norm(2 * x, gamma).out)
    assert M.rms_norm(x[:0], gamma, quantize=True).codes.shape == (0, 264)


def test_quantize_extremes():
    """All-zero blocks, the largest and smallest values, infinities and NaN: a block's
    scale is its finite values', infinities become 448, NaN stays in its place."""
    big = np.zeros((8, 256))
    big[1, 3] = 3.4e38
    big[2, :] = 2.0 ** -149
    big[3, 0], big[3, 1], big[3, 2] = np.inf, -np.inf, 5.0
    big[4, 7], big[4, 8] = np.nan, 3.0
    big[5, 200] = 448.0 * 2.0 ** 5
    big[6, 200] = 448.0 * 2.0 ** 5 * (1 + 2.0 ** -20)
    big[7] = np.nan
    x = _dev(big, torch.float32)
    q = M.fp8_quantize(x)
    codes, scales = ref.quantize(_np(x))
    got, gs = q.codes.view(torch.uint8).cpu().numpy(), q.scales.view(torch.uint8).cpu().numpy()
    assert np.array_equal(gs, scales)
    nan = np.isnan(big)
    assert np.array_equal((got & 127) == 127, nan)
    assert np.array_equal(got[~nan], codes[~nan])


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_is_exact(dtype):
    """No arithmetic comes before the rounding, so codes and scales are the restatement's."""
    rng = np.random.default_rng(5)
    for rows, d in ((1, 8), (33, 520), (4, 7168), (2, 16384)):
        x = _rows(rng, rows, d, dtype)
        q = M.fp8_quantize(x)
        codes, scales = ref.quantize(_np(x))
        assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy() & 127, codes & 127)
        assert np.array_equal(q.scales.view(torch.uint8).cpu().numpy(), scales)
        nz = (codes & 127) != 0
        assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy()[nz], codes[nz])


@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (129, 127), (3, 300, 77), (2, 2, 64, 256)])
@pytest.mark.parametrize("dtype", TYPES)
def test_pack(shape, dtype):
    rng = np.random.default_rng(7)
    w = _dev(rng.standard_normal(shape), torch.float32).to(dtype)
    q = M.fp8_pack(w)
    n, k = shape[-2:]
    assert q.codes.shape == w.shape
    assert q.scales.shape == shape[:-2] + (ref.blocks(n), ref.blocks(k))
    for got, gs, v in zip(q.codes.view(torch.uint8).cpu().numpy().reshape(-1, n, k),
                          q.scales.view(torch.uint8).cpu().numpy().reshape(
                              -1, ref.blocks(n), ref.blocks(k)), _np(w).reshape(-1, n, k)):
        codes, scales = ref.pack(v)
        assert np.array_equal(got, codes) and np.array_equal(gs, scales)


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------
def _check_product(got, p, tol, swiglu, quantize, dtype, what):
    if swiglu:
        p, tol = ref.swiglu(p, tol)
    if quantize:
        ref.check_codes(got.codes, got.scales, p, tol, what)
    else:
        ref.check_values(got, p, tol, dtype, what)


LINEAR = [  # rows, n, k
    (1, 256, 128), (1, 1, 128), (128, 256, 512), (129, 257, 640), (300, 1000, 1152), (5, 7168, 256),
    (64, 520, 2048), (1000, 130, 128), (17, 384, 7168), (2500, 640, 384), (40, 40000, 128)]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,n,k", LINEAR)
def test_linear(rows, n, k, mx):
    rng = np.random.default_rng(rows + n + k)
    dtype = TYPES[(rows + n) % 3]
    x, xs = ref.random_x(rng, rows, k)
    w, ws = ref.random_w(rng, n, k, mx)
    p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, mx))
    got = M.fp8_linear(_codes(x), _scales(xs), _dev(w) if mx else _codes(w), _scales(ws),
                       out_dtype=dtype)
    assert got.dtype == dtype
    _check_product(got, p, tol, False, False, dtype, (rows, n, k))


@pytest.mark.parametrize("k", [16, 48, 112, 144, 1008])
def test_linear_short_and_odd_k(k):
    rng = np.random.default_rng(k)
    x, xs = ref.random_x(rng, 37, k)
    w, ws = ref.random_w(rng, 200, k, False)
    p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, False))
    got = M.fp8_linear(_codes(x), _scales(xs), _codes(w), _scales(ws), out_dtype=torch.float32)
    _check_product(got, p, tol, False, False, torch.float32, k)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("rows,f,k", [(1, 128, 128), (130, 256, 512), (33, 200, 256), (7, 1, 128),
                                      (64, 1408, 1024), (260, 129, 384), (5, 256, 2048),
                                      (200, 144, 2304)])
def test_swiglu(rows, f, k, quantize, mx):
    rng = np.random.default_rng(rows + f + k)
    x, xs = ref.random_x(rng, rows, k)
    w, ws = ref.random_w(rng, 2 * f, k, mx)
    p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, mx))
    got = M.fp8_linear(_codes(x), _scales(xs), _dev(w) if mx else _codes(w), _scales(ws),
                       activation="swiglu", quantize=quantize, out_dtype=torch.float16)
    _check_product(got, p, tol, True, quantize, torch.float16, (rows, f, k))


def test_linear_strides_and_given_out():
    rng = np.random.default_rng(3)
    x, xs = ref.random_x(rng, 50, 256)
    w, ws = ref.random_w(rng, 300, 256, False)
    plain = M.fp8_linear(_codes(x), _scales(xs), _codes(w), _scales(ws))
    wide = torch.zeros(50, 400, dtype=torch.uint8, device=DEV)
    wide[:, 16:272] = _dev(x)
    sc = torch.zeros(50, 9, dtype=torch.uint8, device=DEV)
    sc[:, 3:5] = _dev(xs)
    ww = torch.zeros(300, 512, dtype=torch.uint8, device=DEV)
    ww[:, 256:] = _dev(w)
    out = torch.full((50, 333), 5.0, dtype=torch.bfloat16, device=DEV)
    got = M.fp8_linear(wide[:, 16:272], sc[:, 3:5], ww[:, 256:], _dev(ws), out=out[:, 7:307])
    assert got.data_ptr() == out[:, 7:].data_ptr() and torch.equal(got, plain)
    assert (out[:, :7] == 5).all() and (out[:, 307:] == 5).all()
    assert M.fp8_linear(_codes(x)[:0], _scales(xs)[:0], _codes(w), _scales(ws)).shape == (0, 300)


def test_linear_nan_and_infinity_stay_in_their_rows():
    rng = np.random.default_rng(4)
    x, xs = ref.random_x(rng, 140, 256)
    w, ws = ref.random_w(rng, 256, 256, False)
    clean = M.fp8_linear(_codes(x), _scales(xs), _codes(w), _scales(ws))
    x[5, 100] = 0x7F
    xs[130, 1] = 255
    got = M.fp8_linear(_codes(x), _scales(xs), _codes(w), _scales(ws))
    bad = torch.zeros(140, dtype=torch.bool, device=DEV)
    bad[5] = bad[130] = True
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], clean[~bad])


# ---------------------------------------------------------------------------
# By expert
# ---------------------------------------------------------------------------
def _experts(rng, counts, n, k, mx):
    e = len(counts)
    w, ws = zip(*(ref.random_w(rng, n, k, mx) for _ in range(e)))
    return np.stack(w), np.stack(ws)


COUNTS = [[3], [0, 5, 0, 0, 130, 1, 128, 0], [0, 0, 0], [1] * 20, [300, 0, 2, 257], [64, 65, 63, 4]]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("mode", ["plain", "swiglu", "quantize"])
@pytest.mark.parametrize("counts", COUNTS)
def test_experts(counts, mode, gather, mx):
    rng = np.random.default_rng(sum(counts) + len(counts))
    n, k = (272, 384) if mode == "plain" else (2 * 200, 256)
    w, ws = _experts(rng, counts, n, k, mx)
    total, tail = sum(counts), 3
    x_rows = 41 if gather else total + tail
    x, xs = ref.random_x(rng, x_rows, k)
    rows = rng.integers(0, x_rows, total + tail)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    kw = dict(activation=None if mode == "plain" else "swiglu", quantize=mode == "quantize")
    if not kw["quantize"]:
        kw["out"] = torch.full((total + tail, n // (1 if mode == "plain" else 2)), 9.0,
                               dtype=torch.bfloat16, device=DEV)
    got = M.expert_linear(_codes(x), _scales(xs), _dev(w) if mx else _codes(w), _scales(ws),
                          _dev(offsets, torch.int32),
                          rows=_dev(rows, torch.int32) if gather else None, **kw)
    xv = ref.row_values(x, xs)[rows if gather else slice(None)]
    if not kw["quantize"]:
        assert (got[total:] == 9).all()
    for e, c in enumerate(counts):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        p, tol = ref.product(xv[a:b], ref.weight_values(w[e], ws[e], mx))
        part = (M.Quantized(got.codes[a:b], got.scales[a:b]) if kw["quantize"] else got[a:b])
        _check_product(part, p, tol, mode != "plain", kw["quantize"], torch.bfloat16, (e, c))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("mode", ["plain", "swiglu", "quantize"])
def test_few_rows_of_experts_split_k(mode, mx):
    """Fewer tiles than the device has room for: K is split; some clusters have no tile."""
    rng = np.random.default_rng(11)
    counts, k, n = [0, 2, 0, 1, 0, 0], 2048, 272
    w, ws = _experts(rng, counts, n, k, mx)
    x, xs = ref.random_x(rng, 4, k)
    rows = np.array([3, 1, 3])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    kw = dict(activation=None if mode == "plain" else "swiglu", quantize=mode == "quantize",
              out_dtype=torch.float16)
    got = M.expert_linear(_codes(x), _scales(xs), _dev(w) if mx else _codes(w), _scales(ws),
                          _dev(offsets, torch.int32), rows=_dev(rows, torch.int32), **kw)
    xv = ref.row_values(x, xs)[rows]
    for e, (a, b) in ((1, (0, 2)), (3, (2, 3))):
        p, tol = ref.product(xv[a:b], ref.weight_values(w[e], ws[e], mx))
        part = M.Quantized(got.codes[a:b], got.scales[a:b]) if kw["quantize"] else got[a:b]
        _check_product(part, p, tol, mode != "plain", kw["quantize"], torch.float16, e)


@pytest.mark.parametrize("k", [16, 144, 528])
def test_rows_by_index_with_odd_k(k):
    rng = np.random.default_rng(k)
    counts = [70, 0, 9]
    w, ws = _experts(rng, counts, 130, k, False)
    x, xs = ref.random_x(rng, 30, k)
    rows = rng.integers(0, 30, 79)
    got = M.expert_linear(_codes(x), _scales(xs), _codes(w), _scales(ws),
                          _dev(np.array([0, 70, 70, 79]), torch.int32), rows=_dev(rows, torch.int32))
    xv = ref.row_values(x, xs)[rows]
    for e, (a, b) in ((0, (0, 70)), (2, (70, 79))):
        p, tol = ref.product(xv[a:b], ref.weight_values(w[e], ws[e], False))
        _check_product(got[a:b], p, tol, False, False, torch.bfloat16, e)


@pytest.mark.parametrize("shift", [1, 4, 8])
def test_scales_of_any_alignment(shift):
    rng = np.random.default_rng(shift)
    x, xs = ref.random_x(rng, 40, 1024)
    w, ws = ref.random_w(rng, 300, 1024, True)
    p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, True))
    wide = torch.zeros(300, 48, dtype=torch.uint8, device=DEV)
    wide[:, shift:shift + 32] = _dev(ws)
    xw = torch.zeros(40, 24, dtype=torch.uint8, device=DEV)
    xw[:, shift:shift + 8] = _dev(xs)
    got = M.fp8_linear(_codes(x), xw[:, shift:shift + 8], _dev(w), wide[:, shift:shift + 32],
                       out_dtype=torch.float32)
    _check_product(got, p, tol, False, False, torch.float32, shift)


def test_rows_and_results_past_4_gib():
    """Codes and results whose places pass 32 bits."""
    rng = np.random.default_rng(9)
    x, xs = ref.random_x(rng, 40, 8192)
    big = torch.zeros(560000, 8192, dtype=torch.uint8, device=DEV)      # 4.6 GB
    sc = torch.full((560000, 64), 127, dtype=torch.uint8, device=DEV)
    big[-40:], sc[-40:] = _dev(x), _dev(xs)
    w, ws = ref.random_w(rng, 256, 8192, False)
    p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, False))
    rows = torch.arange(560000 - 40, 560000, device=DEV, dtype=torch.int32)
    offsets = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    got = M.expert_linear(big, sc, _codes(w)[None], _scales(ws)[None], offsets, rows=rows)
    _check_product(got, p, tol, False, False, torch.bfloat16, "rows")
    one = M.fp8_linear(big, sc, _codes(w)[:64], _scales(ws)[:1])
    _check_product(one[-40:], p[:, :64], tol[:, :64], False, False, torch.bfloat16, "all rows")
    del big, sc, one
    x, xs = ref.random_x(rng, 70000, 128)
    w, ws = ref.random_w(rng, 16384, 128, False)
    got = M.fp8_linear(_codes(x), _scales(xs), _codes(w), _scales(ws), out_dtype=torch.float32)
    assert got.numel() * 4 > 2 ** 32
    p, tol = ref.product(ref.row_values(x[-9:], xs[-9:]), ref.weight_values(w, ws, False))
    _check_product(got[-9:], p, tol, False, False, torch.float32, "results")


def test_refusals():
    rng = np.random.default_rng(1)
    x, xs = ref.random_x(rng, 4, 256)
    w, ws = ref.random_w(rng, 64, 256, False)
    x, xs, w, ws = _codes(x), _scales(xs), _codes(w), _scales(ws)
    bad = [lambda: M.fp8_linear(x.float(), xs, w, ws), lambda: M.fp8_linear(x, xs[:3], w, ws),
           lambda: M.fp8_linear(x, xs, w[None], ws), lambda: M.fp8_linear(x, xs, w[:, :128], ws),
           lambda: M.fp8_linear(x, xs, w, ws[:, :1]), lambda: M.fp8_linear(x, xs, w.T, ws),
           lambda: M.fp8_linear(x, xs, w, ws, activation="relu"),
           lambda: M.fp8_linear(x, xs, w[:63], ws, activation="swiglu"),
           lambda: M.fp8_linear(x, xs, w, ws, quantize=True),
           lambda: M.fp8_linear(x, xs, w, ws, out_dtype=torch.int32),
           lambda: M.fp8_linear(x, xs, w, ws, out=torch.empty(4, 63, device=DEV)),
           lambda: M.fp8_linear(x, xs, w, ws, activation="swiglu", quantize=True,
                                out=torch.empty(4, 32, device=DEV)),
           lambda: M.fp8_linear(x.cpu(), xs, w, ws), lambda: M.fp8_linear(x, xs.cpu(), w, ws),
           lambda: M.expert_linear(x, xs, w, ws, torch.zeros(2, dtype=torch.int32, device=DEV)),
           lambda: M.expert_linear(x, xs, w[None], ws[None], torch.zeros(3, dtype=torch.int32,
                                                                         device=DEV)),
           lambda: M.expert_linear(x, xs, w[None], ws[None], torch.zeros(2, device=DEV)),
           lambda: M.fp8_quantize(x), lambda: M.fp8_quantize(torch.zeros(8, device=DEV)),
           lambda: M.fp8_pack(torch.zeros(8, 8, device=DEV).T[:, :4]),
           lambda: M.rms_norm(torch.zeros(2, 8, device=DEV), torch.ones(9, device=DEV)),
           lambda: M.rms_norm(torch.zeros(2, 8, device=DEV), torch.ones(8, device=DEV), out=False),
           lambda: M.rms_norm(torch.zeros(2, 8, device=DEV), torch.ones(8, device=DEV),
                              residual=torch.zeros(1, 8, device=DEV).expand(2, 8)),
           lambda: M.rms_norm(torch.zeros(2, 8, device=DEV), torch.ones(8, device=DEV),
                              residual=torch.zeros(2, 8, device=DEV).half()),
           lambda: M.moe_dispatch(torch.zeros(4, device=DEV), 3),
           lambda: M.moe_dispatch(torch.zeros(4, 2, dtype=torch.int32, device=DEV), 0),
           lambda: M.moe_combine(torch.zeros(4, 8, device=DEV), torch.zeros(2, 2, device=DEV),
                                 torch.zeros(2, 3, dtype=torch.int32, device=DEV))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(str(i))
    for f in (lambda: M.rms_norm(torch.zeros(2, 12, device=DEV), torch.ones(12, device=DEV)),
              lambda: M.fp8_quantize(torch.zeros(2, 16392, device=DEV)),
              lambda: M.moe_dispatch(torch.zeros(4, 2, dtype=torch.int32, device=DEV), 1025),
              lambda: M.fp8_linear(x[:, :248].contiguous(), xs, w[:, :248].contiguous(), ws)):
        with pytest.raises(M.MoEError):
            f()


def test_combine_broadcast_residual():
    rng = np.random.default_rng(2)
    y = _rows(rng, 6, 64, torch.bfloat16)
    r = _rows(rng, 1, 64, torch.bfloat16)
    slots = torch.arange(6, dtype=torch.int32, device=DEV).view(3, 2)
    w = torch.rand(3, 2, device=DEV)
    assert torch.equal(M.moe_combine(y, w, slots, residual=r.expand(3, 64)),
                       M.moe_combine(y, w, slots, residual=r.repeat(3, 1)))


def test_experts_values_out_of_range_are_bounded():
    """Offsets outside the rows or below earlier ones, sources outside x."""
    rng = np.random.default_rng(8)
    w, ws = _experts(rng, [0] * 4, 256, 128, False)
    x, xs = ref.random_x(rng, 10, 128)
    out = torch.full((20, 256), 3.0, dtype=torch.float32, device=DEV)
    rows = np.arange(20) - 5
    got = M.expert_linear(_codes(x), _scales(xs), _codes(w), _scales(ws),
                          _dev(np.array([-4, 6, 2, 9, 1000]), torch.int32),
                          rows=_dev(rows, torch.int32), out=out)
    xv = ref.row_values(x, xs)[np.clip(rows, 0, 9)]
    for e, (a, b) in enumerate(((0, 6), (6, 6), (6, 9), (9, 20))):
        if a < b:
            p, tol = ref.product(xv[a:b], ref.weight_values(w[e], ws[e], False))
            _check_product(got[a:b], p, tol, False, False, torch.float32, e)


@pytest.mark.parametrize("experts", [511, 512, 513, 1023, 1024])
def test_many_experts(experts):
    """Few rows spread over many experts, most of which have none."""
    rng = np.random.default_rng(experts)
    counts = np.zeros(experts, int)
    counts[rng.choice(experts, 9, replace=False)] = rng.integers(1, 40, 9)
    counts[-1] = 2
    total = counts.sum()
    w, ws = ref.random_w(rng, 128, 128, False)
    x, xs = ref.random_x(rng, total, 128)
    sign = rng.integers(0, 2, experts) * 128        # experts differ in their weights' signs
    we = torch.from_numpy(w)[None] ^ torch.from_numpy(sign.astype(np.uint8))[:, None, None]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    got = M.expert_linear(_codes(x), _scales(xs), we.to(DEV).view(torch.float8_e4m3fn),
                          _scales(ws)[None].expand(experts, -1, -1), _dev(offsets, torch.int32))
    p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, False))
    flip = np.repeat(np.where(sign, -1.0, 1.0), counts)[:, None]
    _check_product(got, p * flip, tol, False, False, torch.bfloat16, experts)


# ---------------------------------------------------------------------------
# Dispatch and combine
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,k,experts", [(1, 1, 1), (1, 16, 896), (64, 16, 896), (33, 4, 60),
                                              (700, 8, 256), (3000, 8, 8), (4097, 2, 1024),
                                              (20000, 8, 128), (33000, 2, 3), (1025, 4, 1024),
                                              (70000, 4, 100), (300000, 2, 17)])
@pytest.mark.parametrize("holes", [False, True])
def test_dispatch(tokens, k, experts, holes):
    rng = np.random.default_rng(tokens + k)
    idx = np.minimum(rng.integers(0, experts, (tokens, k)), rng.integers(0, experts, (tokens, k)))
    if holes:
        idx[rng.random((tokens, k)) < 0.2] = -1
        idx[rng.random((tokens, k)) < 0.05] = experts
    got = M.moe_dispatch(_dev(idx, torch.int32), experts)
    for g, want in zip(got, ref.dispatch(idx, experts)):
        assert np.array_equal(g.cpu().numpy(), want)


def test_dispatch_of_nothing():
    got = M.moe_dispatch(torch.empty(0, 4, dtype=torch.int32, device=DEV), 5)
    assert got.offsets.tolist() == [0] * 6 and got.rows.shape == (0,)
    none = M.moe_dispatch(torch.full((3, 2), -1, dtype=torch.int32, device=DEV), 5)
    assert none.offsets.tolist() == [0] * 6
    assert (none.rows == -1).all() and (none.slots == -1).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,k,d", [(1, 1, 8), (5, 3, 264), (64, 16, 1024), (3, 32, 7168),
                                        (200, 9, 2056)])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(tokens, k, d, residual, dtype):
    rng = np.random.default_rng(tokens + k + d)
    n = tokens * k
    y = _rows(rng, n, d, dtype)
    slots = rng.permutation(n).reshape(tokens, k)
    slots[rng.random(slots.shape) < 0.1] = -1
    slots[0, 0] = n      # outside too
    w = rng.random((tokens, k)).astype(np.float32)
    r = _rows(rng, tokens, d, dtype) if residual else None
    got = M.moe_combine(y, _dev(w), _dev(slots, torch.int32), residual=r)
    ok = (slots >= 0) & (slots < n)
    terms = np.where(ok, w, 0.0)[..., None] * _np(y)[np.where(ok, slots, 0)]
    base = _np(r) if residual else np.zeros((tokens, d))
    tol = (k + 1) * 2.0 ** -24 * (np.abs(terms).sum(axis=1) + np.abs(base))
    ref.check_values(got, terms.sum(axis=1) + base, tol, dtype)
    if residual:
        again = M.moe_combine(y, _dev(w), _dev(slots, torch.int32), residual=r, out=r)
        assert again.data_ptr() == r.data_ptr() and torch.equal(again, got)
