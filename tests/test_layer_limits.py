"""The largest sizes that the token operators take, on the CPU: what is past
them is refused, whatever else the arguments say.
"""
import ctypes

import pytest

import fp8_fine_grained_quantize_amd as fb

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = ctypes.c_void_p(0x100000)  # never dereferenced


def _dispatch(T, K, C):
    return fb.lib().fp8blk_moe_dispatch(FAKE, T, C, C, K, FAKE, FAKE, C, None)


def _dispatch_fp8(T, K, C):
    return fb.lib().fp8blk_moe_dispatch_fp8(FAKE, T, C, C, FAKE, K, FAKE, FAKE, FAKE, C, FAKE, None)


def _combine(T, K, C, flags=0):
    return fb.lib().fp8blk_moe_combine(FAKE, T, K, C, C, FAKE, FAKE, FAKE, C, flags, None)


def _combine_backward(T, K, C, flags=0):
    return fb.lib().fp8blk_moe_combine_backward(FAKE, C, FAKE, C, T, K, C, FAKE, FAKE, FAKE, C, FAKE, flags, None)


@pytest.mark.parametrize("call", [_dispatch, _dispatch_fp8, _combine, _combine_backward])
@pytest.mark.parametrize("C", [2 ** 41, 2 ** 43, 2 ** 44, 2 ** 44 + 2 ** 20, 2 ** 45, 2 ** 58, 2 ** 62])
def test_rows_that_no_memory_holds(call, C):
    assert call(1, 1, C) == UNSUPPORTED


def test_tokens_past_the_lanes_of_a_launch():
    """64 lanes at least for a token's row, 256 for codes."""
    assert _dispatch(2 ** 26, 1, 64) == _combine(2 ** 26, 1, 64) == _combine_backward(2 ** 26, 1, 64) == UNSUPPORTED
    assert _dispatch_fp8(2 ** 24, 1, 64) == UNSUPPORTED
    assert _combine(2 ** 20, 1, 2 ** 14, 1) == UNSUPPORTED   # FP32 rows: 4 channels a lane
    assert _combine_backward(2 ** 23, 4, 8192) == UNSUPPORTED and _combine_backward(2 ** 24, 3, 8192) == UNSUPPORTED
