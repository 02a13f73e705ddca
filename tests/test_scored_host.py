"""CPU: sizes and refusals of the decode that accumulates attention weight, of the
choice of tokens and of the decode of shared pages (fake pointers, nothing runs), and
the test scenes' unpacking against the oracle's."""
import ctypes

import numpy as np
import pytest

from bit_kv_cache_evict_gb300 import build as B
from bit_kv_cache_evict_gb300 import oscar as O
from history_scene import Scene, unpack
from oracle import int4 as I

P = ctypes.c_void_p
OK, BAD, UNSUP, WS = O.OSCAR_OK, O.OSCAR_ERR_INVALID_ARG, O.OSCAR_ERR_UNSUPPORTED, O.OSCAR_ERR_WORKSPACE
F, M = P(4096), P(4098)  # a fake device pointer, and a misaligned one


@pytest.fixture(scope="module")
def lib():
    B.build()
    return O.lib()


def sh(hq=32, hk=8, **k):
    return O.make_shape(hq, hk, **k)


def weights(lib, s=None, bits=4, B=4, q=F, kv=F, bl=F, pool=F, table=F, max_pages=10, num_pages=1, hl=F, U=F, scale=1.0, out=F,
            kind=O.OSCAR_OUT_F32, w=F, stride=640, sw=None, decay=1.0, ws=F, room=1 << 40, status=None):
    n = ctypes.c_size_t(room)
    return lib.oscar_decode_attn_weights(ctypes.byref(s or sh()), bits, B, q, kv, bl, pool, table, max_pages, num_pages, hl, U, scale, out, kind,
                                         w, stride, sw, decay, ws, ctypes.byref(n), status, None)


def test_weights_refusals(lib):
    need = O.oscar_decode_workspace_bytes_weights(sh(), 4, 4, 10)
    assert need >= O.oscar_decode_workspace_bytes_int4(sh(), 4, 10) + 4 * 32 * 640 * 4
    assert weights(lib, room=need - 1) == WS
    assert weights(lib, B=0, q=None, kv=None, bl=None, table=None, hl=None, U=None, out=None, w=None) == OK
    for name in ("q", "kv", "bl", "pool", "table", "hl", "U", "out", "w"):
        assert weights(lib, **{name: None}) == BAD, name
    for name in ("q", "kv", "pool", "U", "out", "ws", "status", "w", "sw", "bl", "hl", "table"):
        assert weights(lib, **{name: M}) == BAD, name
    assert weights(lib, stride=639) == BAD                  # a score for every position of the table
    for decay in (-0.1, 1.1, float("nan"), float("inf")):
        assert weights(lib, decay=decay) == BAD
    assert weights(lib, kind=2) == BAD and weights(lib, scale=float("nan")) == BAD
    assert weights(lib, max_pages=0) == BAD and weights(lib, max_pages=1 << 26) == BAD and weights(lib, num_pages=-1) == BAD
    for bits in (0, 1, 3, 8):
        assert weights(lib, bits=bits) == UNSUP
    assert weights(lib, s=sh(hq=24)) == UNSUP


def shared(lib, s=None, bits=4, B=4, q=F, kv=F, bl=F, pool=F, table=F, max_pages=10, num_pages=1, hl=F, group=F, n_groups=2, pages=F, least=0, U=F,
           scale=1.0, out=F, kind=O.OSCAR_OUT_F32, ws=F, room=1 << 40, status=None):
    n = ctypes.c_size_t(room)
    return lib.oscar_decode_attn_shared(ctypes.byref(s or sh()), bits, B, q, kv, bl, pool, table, max_pages, num_pages, hl, group, n_groups, pages, least,
                                        U, scale, out, kind, ws, ctypes.byref(n), status, None)


def test_shared_refusals(lib):
    need = O.oscar_decode_workspace_bytes_shared(sh(), 2, 4, 10, 2)
    assert need > O.oscar_decode_workspace_bytes(sh(), 4, 10)
    assert shared(lib, bits=2, room=need - 1) == WS
    assert shared(lib, B=0, q=None, kv=None, bl=None, table=None, hl=None, U=None, out=None, group=None, pages=None) == OK
    for name in ("q", "kv", "bl", "pool", "table", "hl", "U", "out", "group", "pages"):
        assert shared(lib, **{name: None}) == BAD, name
    for name in ("q", "kv", "pool", "U", "out", "ws", "status", "group", "pages", "bl", "hl", "table"):
        assert shared(lib, **{name: M}) == BAD, name
    assert shared(lib, least=-1) == BAD
    assert shared(lib, n_groups=-1) == BAD and shared(lib, n_groups=8193) == BAD
    assert shared(lib, kind=2) == BAD and shared(lib, scale=float("nan")) == BAD and shared(lib, max_pages=0) == BAD
    for bits in (0, 1, 3, 8):
        assert shared(lib, bits=bits) == UNSUP


def select(lib, batch=2, w=F, stride=100, hl=F, budget=F, protect=0, keep=F, kstride=50, n=F, kw=None, kwstride=0, status=None):
    return lib.oscar_history_select(batch, w, stride, hl, budget, protect, keep, kstride, n, kw, kwstride, status, None)


def test_select_refusals(lib):
    assert select(lib, batch=0, w=None, hl=None, budget=None, keep=None, n=None) == OK
    for name in ("w", "hl", "budget", "keep", "n"):
        assert select(lib, **{name: None}) == BAD, name
    for name in ("w", "hl", "budget", "keep", "n", "kw", "status"):
        assert select(lib, **{name: M}) == BAD, name
    for name in ("batch", "stride", "protect", "kstride", "kwstride"):
        assert select(lib, **{name: -1}) == BAD, name
    assert select(lib, stride=(1 << 31) - 1) == BAD and select(lib, batch=1 << 29) == BAD
    assert select(lib, kw=F, kwstride=50) == BAD            # over the scores themselves
    assert select(lib, kw=P(4096 + 796), kwstride=50) == BAD and select(lib, kw=P(4096 - 396), kwstride=50) == BAD


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("g", [32, 64, 128])
def test_the_scenes_values_are_the_oracles(bits, g):
    c = Scene(1, bits, [130, 70], 4, 2, g, groups=[0, 0], shared=1)
    assert c.table[0, 0] == c.table[1, 0]
    vals = unpack(c.pool, c.hk, bits, g)
    for b in range(2):
        pos = np.arange(int(c.hist[b]))
        for h in range(2):
            for w in (0, 1):
                assert np.array_equal(vals[c.table[b, pos // 64], h, w, pos % 64], I.values(c.pool, c.table, b, pos, h, w, 2, bits, g))
    want = c.want()
    q, kv = (np.asarray(x, np.float64) for x in (I_f64(c.q), I_f64(c.kv)))
    ref, mag = I.decode(q, kv, c.len, c.pool, c.table, c.hist, c.U, 1 / np.sqrt(128), g, bits=bits)
    assert np.abs(want[0] - ref).max() < 1e-12 and np.allclose(want[3], mag)
    assert np.allclose(want[1].sum(1) + want[2].sum(1), 4)


def I_f64(bits):
    from history_scene import f64
    return f64(bits)
