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


class Fake:
    """What the binding looks at of a contiguous CUDA tensor."""

    is_cuda = True

    def __init__(self, *shape, dtype=None):
        import torch
        self.shape, self.dtype = shape, dtype or torch.int32

    def numel(self):
        return int(np.prod(self.shape))

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096


def test_the_binding_refuses_wrong_tensors(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # (no GPU here)
    O._torch_names()
    monkeypatch.setattr(O, "_raw_stream", lambda d: 0)
    monkeypatch.setattr(O, "_current_device", lambda: 0)
    f32, bf16, u8 = torch.float32, torch.bfloat16, torch.uint8
    B_, hq, hk, pages = 2, 8, 2, 3
    good = dict(q=Fake(B_, hq, 128, dtype=bf16), kv=Fake(B_, 320, hk, 2, 128, dtype=bf16), len=Fake(B_), pool=Fake(9 * hk * 10240, dtype=u8),
                table=Fake(B_, pages), hist=Fake(B_), U=Fake(hk, 2, 128, 128, dtype=f32), out=Fake(B_, hq, 128, dtype=f32),
                ws=Fake(1 << 40, dtype=u8), w=Fake(B_, 64 * pages, dtype=f32), sw=Fake(B_, 320, dtype=f32), group=Fake(B_), gp=Fake(1))

    def weights(**k):
        a = good | k
        O.oscar_decode_attn_weights(sh(hq, hk), 4, a["q"], a["kv"], a["len"], a["pool"], a["table"], pages, 9, a["hist"], a["U"], 0.1, a["out"], a["w"],
                                    a["ws"], slot_weight=a["sw"])

    def shared(**k):
        a = good | k
        O.oscar_decode_attn_shared(sh(hq, hk), 4, a["q"], a["kv"], a["len"], a["pool"], a["table"], pages, 9, a["hist"], a["group"], a["gp"], a["U"],
                                   0.1, a["out"], a["ws"])

    bad = (dict(q=Fake(B_, hq, 128, dtype=f32)), dict(kv=Fake(5, dtype=bf16)), dict(len=Fake(1)), dict(pool=Fake(9 * hk * 10240 - 1, dtype=u8)),
           dict(table=Fake(B_, pages - 1)), dict(hist=Fake(1)), dict(U=Fake(1, dtype=f32)), dict(out=Fake(B_, hq, 127, dtype=f32)),
           dict(out=Fake(B_, hq, 128, dtype=torch.float16)))
    for k in bad:
        with pytest.raises((TypeError, ValueError)):
            weights(**k)
        with pytest.raises((TypeError, ValueError)):
            shared(**k)
    for k in (dict(w=Fake(1, 64 * pages, dtype=f32)), dict(w=Fake(B_ * 64 * pages, dtype=f32)), dict(w=Fake(B_, 64 * pages)), dict(sw=Fake(B_, 319, dtype=f32))):
        with pytest.raises((TypeError, ValueError)):
            weights(**k)
    with pytest.raises(O.OscarError):                       # the library's own refusal: rows too short for the table
        weights(w=Fake(B_, 64 * pages - 1, dtype=f32))
    for k in (dict(group=Fake(1)), dict(gp=Fake(1, dtype=f32))):
        with pytest.raises((TypeError, ValueError)):
            shared(**k)
    ok = dict(weight=Fake(2, 50, dtype=f32), hist_len=Fake(2), budget=Fake(2), keep=Fake(2, 10), n_keep=Fake(2), kept_weight=Fake(2, 10, dtype=f32))
    for k in (dict(keep=Fake(1, 10)), dict(kept_weight=Fake(1, 10, dtype=f32)), dict(kept_weight=Fake(20, dtype=f32)), dict(hist_len=Fake(1)),
              dict(budget=Fake(2, dtype=f32)), dict(n_keep=Fake(1)), dict(weight=Fake(2, 50))):
        with pytest.raises((TypeError, ValueError)):
            O.oscar_history_select(**(ok | k))
    with pytest.raises(O.OscarError):                       # every Fake lies at one address: kept_weight over weight
        O.oscar_history_select(**ok)


def I_f64(bits):
    from history_scene import f64
    return f64(bits)
