"""Sizes of the serving operators that do not fit the ABI's 32-bit integers are refused
before the library sees them cut; without a GPU."""
import pytest
import torch

import moe_decode_step_gb300 as M
from moe_decode_step_gb300 import serving


class _Shaped:
    """What the checks look at of a contiguous tensor on a device, of any size."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return (*self.shape[1:], 1)[i]

    def is_contiguous(self):
        return True


def _i32(*shape):
    return _Shaped(torch.int32, *shape)


def _plan(n_slots=8, block_size=16, width=4, free=64, rows=2):
    return M.kv_plan(_i32(rows), _i32(rows), _i32(rows, width), _i32(free), _i32(1), block_size,
                     n_slots)


def _release(block_size=16, width=4, free=64, rows=2):
    return M.kv_release(_Shaped(torch.bool, rows), _i32(rows), _i32(rows, width), _i32(free),
                        _i32(1), block_size)


def _append(n):
    cache = object.__new__(M.KVCache)
    cache.n_kv_heads, cache.head_dim, cache.device = 2, 64, _Shaped.device
    new = _Shaped(torch.bfloat16, n, 2, 64)
    return cache.append(new, new, _i32(n))


@pytest.mark.parametrize("call", [
    lambda: _plan(n_slots=2 ** 32 + 8), lambda: _plan(block_size=2 ** 32 + 16),
    lambda: _plan(width=2 ** 31), lambda: _plan(free=2 ** 32), lambda: _plan(rows=2 ** 32 + 2),
    lambda: _release(block_size=2 ** 32 + 16), lambda: _release(width=2 ** 31),
    lambda: _release(free=2 ** 32), lambda: _release(rows=2 ** 32 + 2),
    lambda: _append(2 ** 32 + 1)])
def test_sizes_past_32_bits_are_refused(call, monkeypatch):
    def past(*args):
        pytest.fail("went past the checks")
    for name in ("_raw_stream", "_empty", "lib"):
        monkeypatch.setattr(serving, name, past)
    with pytest.raises(ValueError):
        call()
