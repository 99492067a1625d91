"""Argument checks of the serving operators' C ABI that come before any CUDA
call (no GPU): the forms that test_serving_abi.py does not have."""
import pytest

import moe_decode_step_gb300 as M


@pytest.fixture(scope="module", autouse=True)
def built():
    from moe_decode_step_gb300 import build
    build.build()


def test_release_past_checks():
    bad = M.MOE_ERR_INVALID_ARG
    good = [64, 64, 2, 64, 64, 4, 4, 64, 4, 64, 16, 64]
    call = lambda a: M.lib().moe_kv_release_past(None, *a)   # noqa: E731
    for i, v in ((3, None), (4, None), (7, None), (9, None), (11, None), (2, 0), (5, 3), (6, 0),
                 (8, -1), (10, 8)):
        args = list(good)
        args[i] = v
        assert call(args) == bad, (i, v)
    assert call([None, None] + good[2:]) == bad
    assert call(good[:2] + [16385] + good[3:]) == M.MOE_ERR_UNSUPPORTED
