"""Refusals of the 8-bit operators without a GPU that lie past the packed structs: the
test hook, sizes that do not fit the ABI's integers, the package without torch's
private allocator entry."""
import os
import subprocess
import sys

import pytest
import torch

import moe_decode_step_gb300 as M
from moe_decode_step_gb300 import fp8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from moe_decode_step_gb300 import build
    build.build()


def test_product_fault_hook():
    assert M.lib().moe_debug_set_product_fault(-1, 0) == M.MOE_ERR_INVALID_ARG
    assert M.lib().moe_debug_set_product_fault(0, 0) == M.MOE_OK


class _Shaped:
    """What the checks look at of a contiguous tensor on a device, of any size."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return True


@pytest.mark.parametrize("call", [
    lambda: M.fp8_quantize(_Shaped(torch.bfloat16, 1, 2 ** 32 + 8)),
    lambda: M.fp8_quantize(_Shaped(torch.float32, 2, 2 ** 31)),
    lambda: M.moe_dispatch(_Shaped(torch.int32, 2 ** 32, 1), 8),
    lambda: M.moe_dispatch(_Shaped(torch.int32, 2 ** 31, 2), 8),
    lambda: M.moe_dispatch(_Shaped(torch.int32, 1, 2 ** 32 + 1), 8),
    lambda: M.moe_dispatch(_Shaped(torch.int32, 4, 2), 2 ** 32 + 3)])
def test_sizes_past_32_bits_are_refused(call, monkeypatch):
    """They must not reach the library cut to 32 bits."""
    monkeypatch.setattr(fp8, "_stream", lambda *a: None)
    monkeypatch.setattr(fp8, "_empty", lambda *a: pytest.fail("went past the checks"))
    with pytest.raises(ValueError):
        call()


def test_import_without_torchs_private_allocator_entry():
    """The package, MoELayer included, does not hang on it."""
    code = ("import torch, torch._C._dynamo.guards as g; del g._empty_strided_cuda; "
            "import moe_decode_step_gb300 as M; M.MoELayer; "
            "assert 'moe_decode_step_gb300' in M.fp8._empty_strided_cuda.__module__")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
