"""CPU: the figure of captured DRAM traffic is tied to every source of its kernel."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "bit_kv_cache_evict_gb300", "csrc")


def test_every_library_header_of_the_kernel_is_in_the_hash():
    seen = bench.int2_sources()
    assert "splitk.cuh" in seen and "oscar_common.cuh" in seen
    for name, text in seen.items():
        for f in re.findall(r'#include "([^"]+)"', text):
            f = os.path.basename(f)
            assert f in seen or not os.path.exists(os.path.join(CSRC, f)), (name, f)


def test_a_change_of_a_header_changes_the_hash(monkeypatch):
    old, texts = bench.kernel_source_hash(), dict(bench.int2_sources())
    for name in texts:
        changed = dict(texts, **{name: texts[name] + "\nint one_more;\n"})
        monkeypatch.setattr(bench, "int2_sources", lambda t=changed: t)
        assert bench.kernel_source_hash() != old, name
        monkeypatch.setattr(bench, "int2_sources", lambda t=dict(texts, **{name: texts[name] + "\n// a comment\n"}): t)
        assert bench.kernel_source_hash() == old, name
