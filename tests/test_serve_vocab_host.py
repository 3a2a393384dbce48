"""Refusals of tt_vocab_strings (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import exact_byte_level_amd as tt


@pytest.mark.parametrize("sizes, code", [((-1, 10), tt.TT_EINVAL), ((10, -1), tt.TT_EINVAL), ((256, 256), tt.TT_ENOTLOADED)])
def test_vocab_strings_refuses(sizes, code):
    call = ctypes.CDLL(tt.LIB_PATH).tt_vocab_strings
    call.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64]
    strings, offsets = np.full(300, 7, np.uint8), np.full(300, 7, np.int32)
    assert call(strings.ctypes.data, offsets.ctypes.data, *sizes) == code
    assert (strings == 7).all() and (offsets == 7).all()
