"""8-bit products, norms and the experts of any number of rows: the norm with
the residual's addition, 8-bit activations and weights, products dense or by
expert, the sorting of tokens by expert and the weighted sum of their results.

Argument marshalling only, as in serving.py: every call checks its tensors, then
makes one call of the C ABI (include/moe_decode.h states the formulas and the
rules).  All of it is asynchronous on `stream` (default: the current stream);
tensors made here are allocated on that stream.

8-bit activations are E4M3 codes (float8_e4m3fn or uint8) [rows, d] with E8M0
scales (float8_e8m0fnu or uint8) [rows, ceil(d / 128)]; 8-bit weights codes [n, k]
with scales [ceil(n / 128), ceil(k / 128)]; MXFP4 weights the layer's canonical
layout, uint8 [n, k / 2] with scales [n, k / 32].
"""
from typing import NamedTuple, Optional

import torch

from ._binding import COMBINE, DTYPE_E4M3, FP8_PRODUCT, RMS_NORM, check, lib
from .serving import _CODES, _DTYPE, _SCALES, _raw_stream, _vector, _want
from .serving import _empty as _empty_on

try:   # a private entry, which a torch may lack
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    def _empty_strided_cuda(shape, strides, dtype):
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")

# what the ABI's 32-bit arguments hold: ctypes cuts larger ones without a word (below it
# the library checks its limits)
_INT_MAX = 2 ** 31 - 1
_ACTIVATION = {None: 0, "swiglu": 1}


class Quantized(NamedTuple):
    codes: torch.Tensor     # float8_e4m3fn
    scales: torch.Tensor    # float8_e8m0fnu


class RMSNormed(NamedTuple):
    out: Optional[torch.Tensor]      # 16- or 32-bit, as x
    codes: Optional[torch.Tensor]    # float8_e4m3fn
    scales: Optional[torch.Tensor]   # float8_e8m0fnu


class MoEDispatch(NamedTuple):
    """What moe_dispatch writes: the choices sorted by expert."""
    offsets: torch.Tensor   # int32 [n_experts + 1]: first entry of each expert
    rows: torch.Tensor      # int32 [tokens * top_k]: token of each entry
    slots: torch.Tensor     # int32 [tokens, top_k]: entry of each choice


def _empty(stream, dtype, shape, strides):
    """A new tensor on the current device whose memory belongs to the stream the call
    runs on (what torch.empty_strided does, at a third of its time: behind a launch
    three of its calls cost the host 7 us, these 1.6)."""
    if stream is None:
        return _empty_strided_cuda(shape, strides, dtype)
    with torch.cuda.stream(stream):
        return _empty_strided_cuda(shape, strides, dtype)


def _rows(stream, dtype, rows, d):
    return _empty(stream, dtype, (rows, d), (max(d, 1), 1))


def _stream(stream, device):
    """cudaStream_t of the call (see _raw_stream, which has the checks)."""
    if stream is None and device.index == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(device.index)
    return _raw_stream(stream, device)


def _blocks(n):
    return (n + 127) // 128


def _matrix(t, name, dtypes, device=None):
    """Rows with a contiguous last dimension, on `device` (None: any CUDA device):
    how many, how long, and their stride (of one row its length rounded up to 16)."""
    if t.dtype in dtypes and t.is_cuda and t.dim() == 2 and (device is None or t.device == device):
        rows, d = t.shape
        s0, s1 = t.stride()
        if s1 == 1 or d <= 1:
            return rows, d, s0 if rows > 1 else (d + 15) // 16 * 16
    _want(False, name, f"{' or '.join(map(str, dtypes))} [rows, columns] with a contiguous last "
          f"dimension on {device or 'a CUDA device'}", t)


def _alike(t, name, dtype, rows, d, device, written=True):
    """The row stride of a matrix [rows, d]; of one that is written, rows apart."""
    r, c, stride = _matrix(t, name, (dtype,), device)
    if r != rows or c != d or (written and stride < d):
        _want(False, name, f"[{rows}, {d}]{', rows apart' if written else ''}", t)
    return stride


def _new_codes(stream, rows, d):
    b = (d + 127) // 128
    return (_empty(stream, torch.float8_e4m3fn, (rows, d), (max(d, 1), 1)),
            _empty(stream, torch.float8_e8m0fnu, (rows, b), (max(b, 1), 1)))


def rms_norm(x, gamma, residual=None, eps=1e-6, out=True, quantize=False, stream=None):
    """Norm of rows with the residual's addition (moe_rms_norm): x bfloat16,
    float16 or float32 [rows, d], residual the same (updated in place) or None,
    gamma [d].  Returns an RMSNormed: out in x's type (out=True, or a tensor to
    write; None where out=False), and with quantize the 8-bit form of the same
    unrounded values."""
    dev, dtype = x.device, x.dtype
    rows, d, xs = _matrix(x, "x", _DTYPE)
    rs = os = 0
    if residual is not None:
        rs = _alike(residual, "residual", dtype, rows, d, dev)
    _vector(gamma, d, gamma.dtype if gamma.dtype in _DTYPE else torch.float32, "gamma", dev)
    raw = _stream(stream, dev)
    if out is True:
        out, os = _rows(stream, dtype, rows, d), d
    elif out is False or out is None:
        out = None
        _want(quantize, "out", "an output: out or quantize", out)
    else:
        os = _alike(out, "out", dtype, rows, d, dev)
    codes = scales = None
    if quantize:
        codes, scales = _new_codes(stream, rows, d)
    args = RMS_NORM.pack(
        x.data_ptr(), xs, residual.data_ptr() if residual is not None else 0, rs,
        gamma.data_ptr(), out.data_ptr() if out is not None else 0, os,
        codes.data_ptr() if quantize else 0, d,
        scales.data_ptr() if quantize else 0, _blocks(d), rows, d, _DTYPE[dtype],
        _DTYPE[gamma.dtype], eps)
    check(lib().moe_rms_norm(raw, args), "moe_rms_norm")
    return RMSNormed(out, codes, scales)


def fp8_quantize(x, stream=None):
    """The 8-bit form of activations x bfloat16, float16 or float32 [rows, d]
    (moe_fp8_quantize): Quantized(codes, scales)."""
    rows, d, xs = _matrix(x, "x", _DTYPE)
    if d > _INT_MAX:
        _want(False, "x", "rows of at most 16384 columns", x)
    raw = _stream(stream, x.device)
    codes, scales = _new_codes(stream, rows, d)
    check(lib().moe_fp8_quantize(raw, x.data_ptr(), _DTYPE[x.dtype], xs, rows, d, codes.data_ptr(),
                                 d, scales.data_ptr(), _blocks(d)), "moe_fp8_quantize")
    return Quantized(codes, scales)


def fp8_pack(w, stream=None):
    """The 8-bit form of weights w bfloat16, float16 or float32 [..., n, k],
    contiguous (moe_fp8_pack): Quantized(codes [..., n, k], scales [...,
    ceil(n / 128), ceil(k / 128)])."""
    if w.dim() < 2 or w.dtype not in _DTYPE or not w.is_cuda or not w.is_contiguous():
        _want(False, "w", "bfloat16, float16 or float32 [..., n, k] contiguous on a CUDA device", w)
    n, k = w.shape[-2:]
    raw = _stream(stream, w.device)
    codes = _empty_on(stream, torch.float8_e4m3fn, w.device, *w.shape)
    scales = _empty_on(stream, torch.float8_e8m0fnu, w.device, *w.shape[:-2], _blocks(n),
                       _blocks(k))
    check(lib().moe_fp8_pack(raw, w.data_ptr(), _DTYPE[w.dtype], w.numel() // max(n * k, 1), n, k,
                             codes.data_ptr(), scales.data_ptr()), "moe_fp8_pack")
    return Quantized(codes, scales)


def _product(what, x, x_scales, w, w_scales, experts, offsets, rows, activation, quantize,
             out_dtype, out, stream):
    """fp8_linear (experts 0) and expert_linear."""
    dev = x.device
    x_rows, k, xs = _matrix(x, "x", _CODES)
    kb = (k + 127) // 128
    sr, sc, ss = _matrix(x_scales, "x_scales", _SCALES, dev)
    if sr != x_rows or sc != kb:
        _want(False, "x_scales", f"E8M0 scales {(x_rows, kb)}", x_scales)
    shape = w.shape
    n, width = shape[-2:]
    mx = w.dtype == torch.uint8 and 2 * width == k
    if ((not mx and (w.dtype not in _CODES or width != k)) or w.device != dev
            or (width > 1 and w.stride(-1) != 1)):
        _want(False, "w", f"E4M3 codes [..., n, {k}] or MXFP4 bytes [..., n, {k // 2}], rows "
              f"contiguous on {dev}", w)
    want = (n, k // 32) if mx else ((n + 127) // 128, kb)
    if (w_scales.shape != (shape[:-2] + want) or w_scales.dtype not in _SCALES
            or w_scales.device != dev or (want[1] > 1 and w_scales.stride(-1) != 1)):
        _want(False, "w_scales", f"E8M0 scales {want} for each matrix, rows contiguous on {dev}",
              w_scales)
    _want(activation in _ACTIVATION, "activation", "None or 'swiglu'", activation)
    cols = n
    if activation:
        _want(n % 2 == 0, "w", "gates and ups: an even number of rows", w)
        cols = n // 2
    else:
        _want(not quantize, "quantize", "an activation", activation)
    n_rows = x_rows
    at_offsets = at_rows = w_expert = ws_expert = 0
    if experts:
        _vector(offsets, experts + 1, torch.int32, "offsets", dev)
        at_offsets = offsets.data_ptr()
        if rows is not None:
            _vector(rows, None, torch.int32, "rows", dev)
            n_rows, at_rows = rows.shape[0], rows.data_ptr()
        if experts > 1:
            w_expert, ws_expert = w.stride(0), w_scales.stride(0)
    raw = _stream(stream, dev)
    scales, at_scales, os = None, 0, cols
    if quantize:
        _want(out is None, "out", "None with quantize", out)
        out, scales = _new_codes(stream, n_rows, cols)
        kind, at_scales = DTYPE_E4M3, scales.data_ptr()
    elif out is None:
        if out_dtype not in _DTYPE:
            _want(False, "out_dtype", "bfloat16, float16 or float32", out_dtype)
        out, kind = _rows(stream, out_dtype, n_rows, cols), _DTYPE[out_dtype]
    else:
        os = _alike(out, "out", out.dtype if out.dtype in _DTYPE else torch.bfloat16, n_rows, cols,
                    dev)
        kind = _DTYPE[out.dtype]
    args = FP8_PRODUCT.pack(
        x.data_ptr(), xs, x_scales.data_ptr(), ss, w.data_ptr(),
        w.stride(-2) if n > 1 else (width + 31) // 32 * 32, w_expert, w_scales.data_ptr(),
        w_scales.stride(-2), ws_expert, at_offsets, at_rows, out.data_ptr(), os, at_scales,
        _blocks(cols), n_rows, x_rows, n, k, experts or 1, mx, _ACTIVATION[activation], kind)
    check(lib().moe_fp8_product(raw, args), what)
    return Quantized(out, scales) if quantize else out


def fp8_linear(x, x_scales, w, w_scales, activation=None, quantize=False,
               out_dtype=torch.bfloat16, out=None, stream=None):
    """x W^T of 8-bit activations x [rows, k] with 8-bit weights w [n, k] or MXFP4
    weights w uint8 [n, k / 2] (moe_fp8_product).  activation 'swiglu' takes w as
    n / 2 gate rows and n / 2 up rows and returns silu(gate) * up.  Returns out
    [rows, n or n / 2] in out_dtype (or the given out), or with quantize (and an
    activation) its 8-bit form, Quantized(codes, scales)."""
    if w.dim() != 2:
        _want(False, "w", "a matrix", w)
    return _product("fp8_linear", x, x_scales, w, w_scales, 0, None, None, activation, quantize,
                    out_dtype, out, stream)


def expert_linear(x, x_scales, w, w_scales, offsets, rows=None, activation=None, quantize=False,
                  out_dtype=torch.bfloat16, out=None, stream=None):
    """fp8_linear by expert: w [experts, n, k or k / 2]; output rows offsets[e] ..
    offsets[e + 1) (int32 [experts + 1], a dispatch's) go through matrix e, output
    row i reading row rows[i] of x (int32, a dispatch's rows; None: row i).  Rows
    of no expert are left as they are."""
    if w.dim() != 3 or w.shape[0] < 1:
        _want(False, "w", "a matrix for each expert", w)
    return _product("expert_linear", x, x_scales, w, w_scales, w.shape[0], offsets, rows,
                    activation, quantize, out_dtype, out, stream)


def moe_dispatch(idx, n_experts, stream=None):
    """Tokens by expert (moe_dispatch) from moe_route's idx, int32 [tokens, top_k]
    contiguous: a MoEDispatch.  Choices outside [0, n_experts) are left out."""
    if idx.dim() != 2 or idx.dtype != torch.int32 or not idx.is_cuda or not idx.is_contiguous():
        _want(False, "idx", "torch.int32 [tokens, top_k] contiguous on a CUDA device", idx)
    tokens, k = idx.shape
    dev = idx.device
    n_experts = int(n_experts)
    _want(1 <= n_experts <= _INT_MAX, "n_experts", "1 to 1024", n_experts)
    if tokens > _INT_MAX or k > _INT_MAX:
        _want(False, "idx", "at most 2^24 choices", idx)
    raw = _stream(stream, dev)
    offsets = _empty(stream, torch.int32, (n_experts + 1,), (1,))
    rows = _empty(stream, torch.int32, (tokens * k,), (1,))
    slots = _rows(stream, torch.int32, tokens, k)
    check(lib().moe_dispatch(raw, idx.data_ptr(), tokens, k, n_experts, offsets.data_ptr(),
                             rows.data_ptr(), slots.data_ptr()), "moe_dispatch")
    return MoEDispatch(offsets, rows, slots)


def moe_combine(y, w, slots, residual=None, out=None, stream=None):
    """Weighted sums of the experts' rows (moe_combine): y bfloat16, float16 or
    float32 [entries, d], w float32 and slots int32 [tokens, top_k] (moe_route's
    weights, a dispatch's slots), residual [tokens, d] in y's type or None.
    Returns out [tokens, d]; out may be residual."""
    dev = y.device
    y_rows, d, ys = _matrix(y, "y", _DTYPE)
    if (slots.dim() != 2 or slots.dtype != torch.int32 or slots.device != dev
            or not slots.is_contiguous()):
        _want(False, "slots", f"torch.int32 [tokens, top_k] contiguous on {dev}", slots)
    tokens, k = slots.shape
    if (w.dtype != torch.float32 or w.shape != slots.shape or w.device != dev
            or not w.is_contiguous()):
        _want(False, "w", f"torch.float32 {(tokens, k)} contiguous on {dev}", w)
    rs = 0
    if residual is not None:
        rs = _alike(residual, "residual", y.dtype, tokens, d, dev, written=False)
    raw = _stream(stream, dev)
    if out is None:
        out, os = _rows(stream, y.dtype, tokens, d), d
    else:
        os = _alike(out, "out", y.dtype, tokens, d, dev)
    args = COMBINE.pack(y.data_ptr(), ys, w.data_ptr(), slots.data_ptr(),
                        residual.data_ptr() if residual is not None else 0, rs, out.data_ptr(), os,
                        tokens, k, y_rows, d, _DTYPE[y.dtype])
    check(lib().moe_combine(raw, args), "moe_combine")
    return out
