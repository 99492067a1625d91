"""GPU tests of the 8-bit products, norms and expert operators at the edges of what
their documentation allows, against 64-bit restatements (_fp8.py, which derives the
bounds)."""
import numpy as np
import pytest
import torch

import moe_decode_step_gb300 as M

import _fp8 as ref
from test_gpu_fp8 import _codes, _dev, _scales

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _u8(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("k", [128, 512])
def test_scales_of_batches_in_a_row(k, mx):
    """64 tokens at a time share the barrier that their largest results cross the CTAs
    by: tiles of 240 tokens and several tiles a pair, 64 tokens a million times larger
    or smaller than those before and after, so that a largest result taken from other
    tokens shows in the scale; the same bits again and again."""
    rng = np.random.default_rng(k)
    rows, f = 2400, 2048
    x, xs = ref.random_x(rng, rows, k)
    xs = (xs.astype(int) + np.where(np.arange(rows) % 240 // 64 % 2, 20, 0)[:, None]).astype(
        np.uint8)
    w, ws = ref.random_w(rng, 2 * f, k, mx)
    args = (_codes(x), _scales(xs), _dev(w) if mx else _codes(w), _scales(ws))
    got = M.fp8_linear(*args, activation="swiglu", quantize=True)
    # (the restatement of all 2,400 x 4,096 takes seconds; every eighth row has rows of
    # each 64)
    some = np.arange(0, rows, 8)
    p, tol = ref.swiglu(*ref.product(ref.row_values(x, xs)[some], ref.weight_values(w, ws, mx)))
    ref.check_codes(got.codes[::8], got.scales[::8], p, tol, k)
    for _ in range(50):
        again = M.fp8_linear(*args, activation="swiglu", quantize=True)
        assert torch.equal(_u8(again.codes), _u8(got.codes))
        assert torch.equal(_u8(again.scales), _u8(got.scales))


def _product(mode, k, mx, rows, seed, index):
    """A call of two tiles: what it returns, as a list of tensors of values."""
    rng = np.random.default_rng(seed)
    n = 512                                    # two tiles of 256, or of 128 gates and ups
    x, xs = ref.random_x(rng, rows, k)
    w, ws = ref.random_w(rng, n, k, mx)
    x, xs, w, ws = _codes(x), _scales(xs), _dev(w) if mx else _codes(w), _scales(ws)
    kw = dict(activation=None if mode == "plain" else "swiglu", quantize=mode == "quantize")

    def run():
        if index:
            got = M.expert_linear(x, xs, w[None], ws[None],
                                  torch.tensor([0, rows], dtype=torch.int32, device=DEV),
                                  rows=torch.arange(rows, dtype=torch.int32, device=DEV), **kw)
        else:
            got = M.fp8_linear(x, xs, w, ws, **kw)
        if mode != "quantize":
            return got.float()
        return got.codes.float() * got.scales.float().repeat_interleave(128, 1)
    return run


@pytest.mark.parametrize("mode", ["plain", "swiglu", "quantize"])
@pytest.mark.parametrize("k,mx,index", [(256, False, False), (256, True, True),
                                        (2048, False, True), (2048, True, False)])
def test_a_wait_that_runs_out_leaves_nan(k, mx, index, mode):
    """A pair of CTAs that gets no weights: its tile is NaN in both CTAs' columns, and
    (K = 2,048 is split over four pairs) whichever pair of the cluster it is; the other
    tile and the calls after it are right."""
    run = _product(mode, k, mx, 16, k, index)
    clean = run()
    cols = 256 if mode == "plain" else 128
    assert clean.isfinite().all()
    for fault in (1,) if k == 256 else (1, 2, 4):
        assert M.lib().moe_debug_set_product_fault(fault, 20_000_000) == 0
        try:
            got = run()
            torch.cuda.synchronize()
        finally:
            assert M.lib().moe_debug_set_product_fault(0, 0) == 0
        assert got[:, :cols].isnan().all(), fault
        assert torch.equal(got[:, cols:], clean[:, cols:]), fault
        assert torch.equal(run(), clean)


def test_without_torchs_private_allocator_entry(monkeypatch):
    """What a torch without it falls back to gives the same tensors."""
    import importlib
    import torch._C._dynamo.guards as guards
    from moe_decode_step_gb300 import fp8
    x = torch.randn(5, 264, device=DEV).to(torch.bfloat16)
    gamma = torch.ones(264, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = M.rms_norm(x, gamma, quantize=True)
    fast = fp8._empty_strided_cuda
    monkeypatch.delattr(guards, "_empty_strided_cuda")
    try:
        importlib.reload(fp8)
        assert fp8._empty_strided_cuda is not fast
        for stream in (None, s):
            got = fp8.rms_norm(x, gamma, quantize=True, stream=stream)
            torch.cuda.synchronize()
            assert all(a.stride() == b.stride() and torch.equal(_u8(a), _u8(b))
                       for a, b in zip(got, want))
    finally:
        monkeypatch.undo()
        importlib.reload(fp8)
    assert fp8._empty_strided_cuda is fast


@pytest.mark.parametrize("d", [8, 264, 1032, 4104, 16384])
@pytest.mark.parametrize("dtype,eps", [(torch.float32, 0.0), (torch.float32, 1e-6),
                                       (torch.bfloat16, 0.0), (torch.bfloat16, 1e-36)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_values_whose_squares_leave_fp32(d, dtype, eps, residual):
    """Rows whose squares are infinite, zero or denormal in 32 bits, beside ordinary
    ones; magnitudes that differ within a row.  Held to the same bounds."""
    rng = np.random.default_rng(d)
    size = 2.0 ** np.array([0.0, 62, 64, 66, 100, 125, -45, -52, -60, -70, -100, -120, 60, -50])
    v = rng.standard_normal((len(size), d)) * size[:, None]
    # (a few far smaller ones beside the large)
    v[3, ::5] *= 2.0 ** -70
    v[5, ::3] *= 2.0 ** -90
    v = np.clip(v, -2.0 ** 126, 2.0 ** 126)
    x = _dev(v, torch.float32).to(dtype)
    r = _dev(v[:, ::-1] * 0.5, torch.float32).to(dtype) if residual else None
    gamma = _dev(1 + 0.2 * rng.standard_normal(d), torch.float32)
    z = x.double().cpu().numpy() + (r.double().cpu().numpy() if residual else 0.0)
    mag = np.abs(x.double().cpu().numpy()) + (np.abs(r.double().cpu().numpy()) if residual else 0)
    scale = 1.0 / np.sqrt((z * z).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    g = gamma.double().cpu().numpy()
    y = z * scale * g
    # (denormal values and sums of the inputs' type: half of fp32's smallest step)
    tol = (64 * 2.0 ** -24 * np.abs(y) + (2.0 ** -24 * mag + 2.0 ** -150) * scale * np.abs(g)
           + 2.0 ** -149)
    got = M.rms_norm(x, gamma, residual=r, eps=eps, quantize=True)
    ref.check_values(got.out, y, tol, dtype, "out")
    ref.check_codes(got.codes, got.scales, y, tol, "codes")


def test_norm_of_zeros_infinities_and_nan():
    """As the formula has them: 0 / sqrt(0 + eps), 0 / 0 without eps, infinity / infinity,
    finite values over infinity; rows beside them are as they are alone."""
    x = torch.randn(6, 2056, device=DEV)
    x[1] = 0
    x[2, 7], x[3, 2000] = float("inf"), float("nan")
    gamma = torch.ones(2056, device=DEV)
    for eps in (0.0, 1e-6):
        out = M.rms_norm(x, gamma, eps=eps).out
        assert (out[1].isnan() if eps == 0 else out[1] == 0).all()
        assert out[2, 7].isnan() and (out[2, :7] == 0).all() and (out[2, 8:] == 0).all()
        assert out[3].isnan().all()
        for i in (0, 4, 5):
            assert torch.equal(out[i], M.rms_norm(x[i:i + 1], gamma, eps=eps).out[0])


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,f,k", [(1, 128, 128), (33, 200, 256), (260, 129, 384),
                                      (5, 256, 2048), (300, 144, 512)])
def test_swiglu_in_32_bits(rows, f, k, mx):
    rng = np.random.default_rng(rows + f + k)
    x, xs = ref.random_x(rng, rows, k)
    w, ws = ref.random_w(rng, 2 * f, k, mx)
    p, tol = ref.swiglu(*ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, mx)))
    got = M.fp8_linear(_codes(x), _scales(xs), _dev(w) if mx else _codes(w), _scales(ws),
                       activation="swiglu", out_dtype=torch.float32)
    ref.check_values(got, p, tol, torch.float32, (rows, f, k))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_swiglu_over_the_range_of_gates(dtype):
    """Gates of -224 to 224, each a product of one term: silu to its bound, and 0 where the
    documentation has it 0 (below -87.3, where silu is less than 1.1e-36)."""
    rng = np.random.default_rng(6)
    k = f = 128
    x = np.zeros((k, k), np.uint8)
    np.fill_diagonal(x, 0x38)                                   # 1.0
    w = rng.integers(0, 256, (2 * f, k), np.uint8)
    w[(w & 127) == 127] = 0
    xs, ws = np.full((k, 1), 127, np.uint8), np.array([[126], [110]], np.uint8)
    p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, False))
    low = np.where(p[:, :f] < -87.3, 1.1e-36 * np.abs(p[:, f:]), 0.0)
    assert (p[:, :f] < -88).sum() > 500 and (p[:, :f] > 88).sum() > 500
    want, tol = ref.swiglu(p, tol)
    got = M.fp8_linear(_codes(x), _scales(xs), _codes(w), _scales(ws), activation="swiglu",
                       out_dtype=dtype)
    ref.check_values(got, want, tol + low, dtype)


@pytest.mark.parametrize("mode", ["plain", "swiglu", "quantize"])
def test_more_token_tiles_than_a_pass(mode):
    """Sixteen tiles of tokens share a pass over the weights: 40 tiles of one matrix and 21,
    1 and 17 of experts, every row compared."""
    rng = np.random.default_rng(12)
    kw = dict(activation=None if mode == "plain" else "swiglu", quantize=mode == "quantize")
    k, n = 128, 300

    def check(got, x, xs, w, ws, what):
        p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, False))
        if mode != "plain":
            p, tol = ref.swiglu(p, tol)
        if mode == "quantize":
            ref.check_codes(got.codes, got.scales, p, tol, what)
        else:
            ref.check_values(got, p, tol, torch.bfloat16, what)

    x, xs = ref.random_x(rng, 9500, k)
    w, ws = ref.random_w(rng, n, k, False)
    check(M.fp8_linear(_codes(x), _scales(xs), _codes(w), _scales(ws), **kw), x, xs, w, ws, "dense")
    counts = [5000, 0, 17, 4000]
    w, ws = (np.stack(t) for t in zip(*(ref.random_w(rng, n, k, False) for _ in counts)))
    off = np.concatenate([[0], np.cumsum(counts)])
    rows = rng.integers(0, 9500, off[-1])
    for src in (None, rows):
        got = M.expert_linear(_codes(x[:off[-1]] if src is None else x),
                              _scales(xs[:off[-1]] if src is None else xs), _codes(w), _scales(ws),
                              _dev(off, torch.int32),
                              rows=None if src is None else _dev(src, torch.int32), **kw)
        at = np.arange(off[-1]) if src is None else src
        for e, (a, b) in enumerate(zip(off, off[1:])):
            if a < b:
                part = M.Quantized(*(t[a:b] for t in got)) if mode == "quantize" else got[a:b]
                check(part, x[at[a:b]], xs[at[a:b]], w[e], ws[e], (e, src is None))


@pytest.mark.parametrize("rows", [3, 70, 500])
def test_rows_by_index_of_one_matrix(rows):
    """The C call without offsets and with rows, which Python has no name for."""
    from moe_decode_step_gb300._binding import FP8_PRODUCT
    rng = np.random.default_rng(rows)
    k, n = 384, 200
    x, xs = ref.random_x(rng, 41, k)
    w, ws = ref.random_w(rng, n, k, False)
    src = rng.integers(0, 41, rows)
    t = [_dev(x), _dev(xs), _dev(w), _dev(ws), _dev(src, torch.int32)]
    out = torch.empty(rows, n, dtype=torch.float32, device=DEV)
    args = FP8_PRODUCT.pack(t[0].data_ptr(), k, t[1].data_ptr(), 3, t[2].data_ptr(), k, 0,
                            t[3].data_ptr(), 3, 0, 0, t[4].data_ptr(), out.data_ptr(), n, 0, 1,
                            rows, 41, n, k, 1, 0, 0, 2)
    assert M.lib().moe_fp8_product(torch.cuda.current_stream().cuda_stream, args) == M.MOE_OK
    p, tol = ref.product(ref.row_values(x, xs)[src], ref.weight_values(w, ws, False))
    ref.check_values(out, p, tol, torch.float32, rows)


@pytest.mark.parametrize("tiles", [9, 15, 16, 19, 20, 36, 37, 38, 39])
@pytest.mark.parametrize("mx", [False, True])
def test_tiles_beside_the_splits_of_k(tiles, mx):
    """Numbers of tiles around those up to which K is split over a cluster of two and of
    four pairs: what fits beside one another is fewer than the SMs would make."""
    rng = np.random.default_rng(tiles)
    rows, n, k = 5, 256 * tiles, 1024
    x, xs = ref.random_x(rng, rows, k)
    w, ws = ref.random_w(rng, n, k, mx)
    p, tol = ref.product(ref.row_values(x, xs), ref.weight_values(w, ws, mx))
    got = M.fp8_linear(_codes(x), _scales(xs), _dev(w) if mx else _codes(w), _scales(ws),
                       out_dtype=torch.float32)
    ref.check_values(got, p, tol, torch.float32, tiles)


def test_first_call_of_a_process_is_captured():
    """What the host asks the device once (how many clusters fit) a capture allows."""
    code = """
import torch, moe_decode_step_gb300 as M
x = torch.randint(0, 120, (5, 2048), dtype=torch.uint8, device="cuda")
w = torch.randint(0, 120, (4096, 2048), dtype=torch.uint8, device="cuda")
xs = torch.full((5, 16), 120, dtype=torch.uint8, device="cuda")
ws = torch.full((32, 16), 120, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = M.fp8_linear(x, xs, w, ws)
g.replay()
torch.cuda.synchronize()
assert torch.equal(out, M.fp8_linear(x, xs, w, ws))
"""
    import os
    import subprocess
    import sys
    subprocess.run([sys.executable, "-c", code], check=True,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
