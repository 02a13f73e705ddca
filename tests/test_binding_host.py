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
