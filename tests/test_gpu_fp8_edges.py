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
