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
