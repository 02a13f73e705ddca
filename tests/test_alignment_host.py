"""CPU: index arrays at odd addresses are refused before any launch (fake pointers, nothing runs)."""
import ctypes

import pytest

from bit_kv_cache_evict_gb300 import build as B
from bit_kv_cache_evict_gb300 import oscar as O

P = ctypes.c_void_p
F, M = P(4096), P(4098)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return O.lib()


def evict(lib, bits, row=F, seq=F, pos=F, table=F):
    call = lib.oscar_evict_quantize_int4 if bits == 4 else lib.oscar_evict_quantize
    return call(ctypes.byref(O.make_shape(4, 1)), 1, F, 1, row, seq, pos, None, F, F, F, table, 1, 1, 1, None, None)


def decode(lib, bits, bl=F, table=F, hl=F):
    n, sh = ctypes.c_size_t(1 << 40), O.make_shape(4, 1)
    if bits == 4:
        return lib.oscar_decode_attn_int4(ctypes.byref(sh), 1, F, F, bl, F, table, 4, 1, hl, F, ctypes.c_float(1.0), F, 0, F, ctypes.byref(n),
                                          None, None)
    return lib.oscar_decode_attn(ctypes.byref(sh), 1, F, F, bl, F, table, 4, 1, hl, F, ctypes.c_float(1.0), F, F, ctypes.byref(n), None, None)


@pytest.mark.parametrize("bits", [2, 4])
def test_misaligned_index_arrays_are_refused(lib, bits):
    for name in ("row", "seq", "pos", "table"):
        assert evict(lib, bits, **{name: M}) == O.OSCAR_ERR_INVALID_ARG, name
    for name in ("bl", "table", "hl"):
        assert decode(lib, bits, **{name: M}) == O.OSCAR_ERR_INVALID_ARG, name
