"""CPU: argument checks of shapes without BF16 windows (fake pointers, nothing runs)."""
import ctypes

import pytest

from bit_kv_cache_evict_gb300 import build as B
from bit_kv_cache_evict_gb300 import oscar as O

F = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return O.lib()


def call(lib, bits, sink, recent, kv, batch=0, room=1 << 40):
    n = ctypes.c_size_t(room)
    sh = O.make_shape(4, 1, sink=sink, recent=recent)
    if bits == 4:
        return lib.oscar_decode_attn_int4(ctypes.byref(sh), batch, F, kv, F, F, F, 4, 1, F, F, ctypes.c_float(1.0), F, 0, F, ctypes.byref(n),
                                          None, None)
    return lib.oscar_decode_attn(ctypes.byref(sh), batch, F, kv, F, F, F, 4, 1, F, F, ctypes.c_float(1.0), F, F, ctypes.byref(n), None, None)


@pytest.mark.parametrize("bits", [2, 4])
def test_the_window_rows_may_be_null_only_without_windows(lib, bits):
    assert call(lib, bits, 64, 256, None, batch=1) == O.OSCAR_ERR_INVALID_ARG
    assert call(lib, bits, 1, 0, None, batch=1) == O.OSCAR_ERR_INVALID_ARG
    assert call(lib, bits, 0, 0, None, room=0) == O.OSCAR_ERR_WORKSPACE
    assert call(lib, bits, 0, 0, None) == O.OSCAR_OK


@pytest.mark.parametrize("bits", [2, 4])
def test_windows_whose_sum_passes_32_bits_are_refused(lib, bits):
    big = (1 << 31) - 1
    for sink, recent in ((big, big), (big, 1), (321, 0), (0, 321), (161, 160)):
        assert call(lib, bits, sink, recent, F) == O.OSCAR_ERR_UNSUPPORTED
