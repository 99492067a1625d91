"""Refusals of the 8-bit operators without a GPU that lie past the packed structs: the
test hook, sizes that do not fit the ABI's integers, the package without torch's
private allocator entry."""
import pytest

import moe_decode_step_gb300 as M


@pytest.fixture(scope="module", autouse=True)
def built():
    from moe_decode_step_gb300 import build
    build.build()


def test_product_fault_hook():
    assert M.lib().moe_debug_set_product_fault(-1, 0) == M.MOE_ERR_INVALID_ARG
    assert M.lib().moe_debug_set_product_fault(0, 0) == M.MOE_OK
