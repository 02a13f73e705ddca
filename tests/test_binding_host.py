"""CPU tests of the binding's first call: the names it keeps are all there once a
thread may rely on them."""
import pytest

from bit_kv_cache_evict_gb300 import oscar as O

torch = pytest.importorskip("torch")

NAMES = ("_F32", "_BF16", "_I32", "_U8", "_raw_stream", "_current_device")


class Watch:
    """torch, noting what the binding has set whenever one of its names is looked up."""

    def __init__(self, of, seen):
        self._of, self._seen = of, seen

    def __getattr__(self, name):
        self._seen.append({n: getattr(O, n) for n in NAMES})
        v = getattr(self._of, name)
        return Watch(v, self._seen) if name in ("_C", "cuda") else v


def test_the_guard_is_set_after_everything_it_stands_for(monkeypatch):
    """A second thread that finds _F32 set goes on to use the others at once."""
    import sys
    for n in NAMES:
        monkeypatch.setattr(O, n, None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # (no GPU here)
    seen = []
    monkeypatch.setitem(sys.modules, "torch", Watch(torch, seen))
    O._torch_names()
    assert len(seen) >= len(NAMES) - 1
    for at in seen:
        assert at["_F32"] is None or all(v is not None for v in at.values()), at
    assert all(getattr(O, n) is not None for n in NAMES)


class Fake:
    """What the binding looks at of a contiguous CUDA tensor."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.int32):
        self.shape, self.dtype = shape, dtype

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096 if self.numel() else 0


def test_an_empty_workspace_is_refused(monkeypatch):
    """Its address is null, which to the library is the question for the size: nothing would run."""
    from bit_kv_cache_evict_gb300 import build as B
    B.build()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # (no GPU here)
    O._torch_names()
    monkeypatch.setattr(O, "_raw_stream", lambda d: 0)
    monkeypatch.setattr(O, "_current_device", lambda: 0)
    sh = O.make_shape(4, 1)

    def call(B, workspace):
        O.oscar_decode_attn_int4(sh, Fake(B, 4, 128, dtype=torch.bfloat16), Fake(B, 320, 1, 2, 128, dtype=torch.bfloat16), Fake(B), Fake(10240, dtype=torch.uint8),
                                 Fake(B, 4), 4, 1, Fake(B), Fake(1, 2, 128, 128, dtype=torch.float32), 1.0, Fake(B, 4, 128, dtype=torch.float32), workspace)

    with pytest.raises(ValueError):
        call(2, Fake(0, dtype=torch.uint8))
    with pytest.raises(O.OscarError):                      # too small: the library's own refusal
        call(2, Fake(16, dtype=torch.uint8))
    call(0, Fake(0, dtype=torch.uint8))                    # an empty batch needs none
