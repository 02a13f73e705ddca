"""CPU tests of the 4-bit history's and the history-moving calls: sizes, and
every refusal before a launch (fake pointers, nothing runs)."""
import ctypes

import numpy as np
import pytest

from bit_kv_cache_evict_gb300 import build as B
from bit_kv_cache_evict_gb300 import oscar as O
from oracle import int4 as I

P = ctypes.c_void_p
OK, BAD, UNSUP, WS = O.OSCAR_OK, O.OSCAR_ERR_INVALID_ARG, O.OSCAR_ERR_UNSUPPORTED, O.OSCAR_ERR_WORKSPACE
F = P(4096)        # a fake device pointer, 16-byte aligned
M = P(4098)        # misaligned


@pytest.fixture(scope="module")
def lib():
    B.build()
    return O.lib()


def sh(hq=32, hk=8, **k):
    return O.make_shape(hq, hk, **k)


def test_block_bytes(lib):
    for g in (32, 64, 128):
        assert O.block_bytes_int4(sh(quant_group=g)) == I.block_bytes(4, g)
        assert O.block_bytes(sh(quant_group=g)) == I.block_bytes(2, g)
    assert O.block_bytes_int4(sh(quant_group=16)) == 0


def evict(lib, s=None, n=3, src=F, rows=3, row=None, seq=F, pos=F, new=None, U=F, clip=F, pool=F, table=F, batch=1,
          max_pages=1, num_pages=1, status=None):
    return lib.oscar_evict_quantize_int4(ctypes.byref(s or sh()), n, src, rows, row, seq, pos, new, U, clip, pool, table,
                                         batch, max_pages, num_pages, status, None)


def test_evict_refusals(lib):
    assert evict(lib, n=0, src=None, seq=None, pos=None, U=None, clip=None, pool=None, table=None) == OK
    for name in ("src", "seq", "pos", "U", "clip", "pool", "table"):
        assert evict(lib, **{name: None}) == BAD, name
    for name in ("src", "new", "U", "pool", "clip", "status"):
        assert evict(lib, **{name: M}) == BAD, name
    assert evict(lib, n=-1) == BAD and evict(lib, batch=-1) == BAD and evict(lib, max_pages=0) == BAD
    assert evict(lib, max_pages=1 << 26) == BAD           # positions would not fit 32 bits
    assert evict(lib, rows=2) == BAD                       # three tokens from two rows
    assert evict(lib, s=sh(quant_group=16)) == UNSUP and evict(lib, s=sh(hq=24)) == UNSUP


def decode(lib, s=None, B=4, q=F, kv=F, bl=F, pool=F, table=F, max_pages=10, num_pages=1, hl=F, U=F, scale=1.0, out=F,
           kind=O.OSCAR_OUT_F32, ws=F, room=1 << 40, status=None):
    n = ctypes.c_size_t(room)
    return lib.oscar_decode_attn_int4(ctypes.byref(s or sh()), B, q, kv, bl, pool, table, max_pages, num_pages, hl, U,
                                      ctypes.c_float(scale), out, kind, ws, ctypes.byref(n), status, None)


def test_decode_refusals(lib):
    need = O.oscar_decode_workspace_bytes_int4(sh(), 4, 10)
    assert need > 0
    assert decode(lib, room=need - 1) == WS
    assert decode(lib, B=0, q=None, kv=None, bl=None, table=None, hl=None, U=None, out=None) == OK
    for name in ("q", "kv", "bl", "pool", "table", "hl", "U", "out"):
        assert decode(lib, **{name: None}) == BAD, name
    for name in ("q", "kv", "pool", "U", "out", "ws", "status"):
        assert decode(lib, **{name: M}) == BAD, name
    assert decode(lib, out=P(4104)) == BAD                 # fp32 rows: 16 bytes
    assert decode(lib, kind=2) == BAD and decode(lib, kind=-1) == BAD
    assert decode(lib, max_pages=0) == BAD and decode(lib, max_pages=1 << 26) == BAD and decode(lib, num_pages=-1) == BAD
    assert decode(lib, scale=float("nan")) == BAD
    assert decode(lib, s=sh(quant_group=48)) == BAD and decode(lib, s=sh(hq=24)) == UNSUP
    assert decode(lib, B=1 << 20, max_pages=1 << 16, ws=None) == BAD       # item counts past 32 bits


def read(lib, s=None, bits=4, n=3, seq=F, pos=F, pool=F, table=F, batch=1, max_pages=1, num_pages=1, out=F,
         kind=O.OSCAR_OUT_BF16, status=None):
    return lib.oscar_history_read(ctypes.byref(s or sh()), bits, n, seq, pos, pool, table, batch, max_pages, num_pages,
                                  out, kind, status, None)


def test_read_refusals(lib):
    assert read(lib, n=0, seq=None, pos=None, pool=None, table=None, out=None) == OK
    for name in ("seq", "pos", "pool", "table", "out"):
        assert read(lib, **{name: None}) == BAD, name
    for name in ("seq", "pos", "pool", "table", "out", "status"):
        assert read(lib, **{name: M}) == BAD, name
    for bits in (0, 1, 3, 8):
        assert read(lib, bits=bits) == UNSUP
    assert read(lib, n=-1) == BAD and read(lib, batch=-1) == BAD and read(lib, max_pages=0) == BAD
    assert read(lib, n=(1 << 31) - 1) == BAD
    assert read(lib, max_pages=1 << 26) == BAD and read(lib, num_pages=-1) == BAD and read(lib, kind=7) == BAD
    assert read(lib, s=sh(head_dim=64)) == UNSUP


def gather(lib, s=None, bits=2, batch=2, pool=F, boost=None, src=F, smax=4, dst=F, dmax=4, keep=F, stride=10, n=F,
           num_pages=8, status=None):
    return lib.oscar_history_gather(ctypes.byref(s or sh()), bits, batch, pool, boost, src, smax, dst, dmax, keep, stride,
                                    n, num_pages, status, None)


def test_gather_refusals(lib):
    assert gather(lib, batch=0, pool=None, src=None, dst=None, keep=None, n=None) == OK
    assert gather(lib, stride=0, keep=None) == OK
    for name in ("pool", "src", "dst", "keep", "n"):
        assert gather(lib, **{name: None}) == BAD, name
    for name in ("pool", "boost", "src", "dst", "keep", "n", "status"):
        assert gather(lib, **{name: M}) == BAD, name
    assert gather(lib, bits=4, boost=F) == BAD             # boost records belong to 2-bit pools
    assert gather(lib, bits=3) == UNSUP
    for name in ("batch", "stride", "num_pages"):
        assert gather(lib, **{name: -1}) == BAD, name
    for name in ("smax", "dmax"):
        assert gather(lib, **{name: 0}) == BAD and gather(lib, **{name: 1 << 26}) == BAD, name
    assert gather(lib, batch=1 << 20, dmax=1 << 12) == BAD  # more pages than a launch counts


def copy(lib, page_bytes=49152, n=2, src=F, dst=F, pools=(4096, 8192), n_pools=None, num_pages=4, status=None):
    arr = (ctypes.c_void_p * max(len(pools), 1))(*pools) if pools is not None else None
    return lib.oscar_pages_copy_device(page_bytes, n, src, dst, arr, len(pools or ()) if n_pools is None else n_pools,
                                       num_pages, status, None)


def test_copy_refusals(lib):
    assert copy(lib, n=0, src=None, dst=None) == OK and copy(lib, pools=()) == OK
    assert copy(lib, src=None) == BAD and copy(lib, dst=None) == BAD and copy(lib, src=M) == BAD and copy(lib, dst=M) == BAD
    assert copy(lib, pools=(4096, 0)) == BAD and copy(lib, pools=(4096, 8200)) == BAD and copy(lib, pools=None, n_pools=1) == BAD
    assert copy(lib, page_bytes=0) == BAD and copy(lib, page_bytes=24) == BAD
    assert copy(lib, n=-1) == BAD and copy(lib, n_pools=-1) == BAD and copy(lib, num_pages=-1) == BAD
    assert copy(lib, pools=tuple([4096] * 129)) == BAD and copy(lib, status=M) == BAD
    assert copy(lib, page_bytes=1 << 30, n=1 << 20) == BAD  # more pieces than a launch counts
    for page_bytes in (1 << 35, (1 << 64) - 16, (1 << 64) - 16384):  # (a sum with them would wrap around)
        assert copy(lib, page_bytes=page_bytes, n=1, pools=(4096,)) == BAD


class Fake:
    """What the binding looks at of a CUDA tensor."""

    def __init__(self, *shape, dtype=None, device=0, contiguous=True, at=4096):
        import torch
        self.shape, self.dtype, self.is_cuda, self._d, self._c, self._at = shape, dtype or torch.int32, True, device, contiguous, at

    def numel(self):
        return int(np.prod(self.shape))

    def is_contiguous(self):
        return self._c

    def get_device(self):
        return self._d

    def data_ptr(self):
        return self._at


def test_binding_refuses_wrong_tensors(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # (no GPU here)
    u8, i = torch.uint8, Fake(2)
    O._torch_names()
    monkeypatch.setattr(O, "_raw_stream", lambda d: 0)
    monkeypatch.setattr(O, "_current_device", lambda: 0)

    def copy(src=i, dst=i, pools=(Fake(256, dtype=u8),), n=4):
        O.oscar_pages_copy_device(64, src, dst, list(pools), n)

    for bad, what in ((dict(src=torch.zeros(2, dtype=torch.int32)), TypeError), (dict(dst=[0, 1]), TypeError),
                      (dict(dst=Fake(2, dtype=torch.int64)), TypeError), (dict(dst=Fake(1)), ValueError),
                      (dict(dst=Fake(2, device=1)), ValueError), (dict(src=Fake(2, contiguous=False)), ValueError),
                      (dict(pools=[Fake(255, dtype=u8)]), ValueError), (dict(pools=[Fake(256)]), TypeError),
                      (dict(pools=[Fake(256, dtype=u8)] * 129), ValueError)):
        with pytest.raises(what):
            copy(**bad)
    with pytest.raises(O.OscarError):                       # the library's own refusal: a pool at an odd address
        copy(pools=[Fake(256, dtype=u8, at=4104)])
    out = Fake(2, 8, 2, 128, dtype=torch.float32)
    pool = Fake(8 * 10240, dtype=u8)
    for bad, what in ((dict(out=Fake(2, 8, 2, 128, dtype=torch.float16)), TypeError), (dict(out=Fake(2, 8, 2, 127, dtype=torch.bfloat16)), ValueError),
                      (dict(pool=Fake(8 * 10240 - 1, dtype=u8)), ValueError), (dict(pos=Fake(1)), ValueError), (dict(table=Fake(0)), ValueError)):
        k = dict(out=out, pool=pool, pos=i, table=Fake(1)) | bad
        with pytest.raises(what):
            O.oscar_history_read(sh(), 4, i, k["pos"], k["pool"], k["table"], 1, 1, 1, k["out"])
    with pytest.raises(ValueError):
        O.oscar_history_gather(sh(), 4, pool, Fake(2, 1), Fake(1, 1), Fake(2, 1), i, 1)
    assert O._out_type(torch.zeros(1)) == O.OSCAR_OUT_F32 and O._out_type(torch.zeros(1, dtype=torch.bfloat16)) == O.OSCAR_OUT_BF16
    for g in (32, 64, 128):
        assert [O._pool_block(sh(quant_group=g), b) for b in (2, 4)] == [O.block_bytes(sh(quant_group=g)), O.block_bytes_int4(sh(quant_group=g))]
    assert O.block_bytes_int4(sh()) == 10240 and O.block_bytes_int4(sh(quant_group=128)) == 8704
