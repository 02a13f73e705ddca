"""CPU: the split-K plan of the 4-bit decode, restated, never makes more items than
the workspace that the library asks for has room for."""
import random

import pytest

from bit_kv_cache_evict_gb300 import build as B
from bit_kv_cache_evict_gb300 import oscar as O


def pages_of(hist):
    return [-(-int(h) // 64) for h in hist]


def plan4(hist, hk, blocks):
    """(pages of a long item, pages in short items) for these lengths."""
    pages = pages_of(hist)
    total = sum(pages) * hk
    lo, hi = max(4, -(-max(pages) // 64)), 256

    def items(size):
        return sum(-(-n // size) for n in pages) * hk

    if lo <= hi and items(hi) <= blocks:
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if items(mid) <= blocks else (mid + 1, hi)
        if lo <= 16 or lo * blocks <= total + total // 4:
            return lo, 0
    pps = min(256, max(16, total // (4 * blocks)))
    return pps, 32 if pps > 16 else 0


def items_of(hist, hk, blocks):
    pps, tail = plan4(hist, hk, blocks)
    return sum(-(-(n - min(n, tail)) // pps) + -(-min(n, tail) // 16) for n in pages_of(hist)) * hk


@pytest.fixture(scope="module")
def lib():
    B.build()
    return O.lib()


def test_the_workspace_has_room_for_every_plan(lib):
    rng = random.Random(1)
    for _ in range(4000):
        batch, hk, G = int(2 ** rng.uniform(0, 9)), rng.choice([1, 2, 3, 8, 24]), rng.choice([1, 4, 8])
        wide, kind = int(2 ** rng.uniform(0, 12)), rng.random()
        hist = [64 * wide if kind < 0.3 else rng.randint(0, 64 * wide) if kind < 0.7 else min(64 * wide, int(2 ** rng.uniform(0, 19)))
                for _ in range(batch)]
        stride = -(-G * 130 // 4) * 4                      # floats of a partial: outputs, maximum and sum of G heads
        room = O.oscar_decode_workspace_bytes_int4(O.make_shape(G * hk, hk), batch, wide)
        for blocks in (152 * 2, 152 * 3, 132, 512):
            assert items_of(hist, hk, blocks) * 4 * stride * 4 <= room, (batch, hk, G, wide, blocks)


def test_a_plan_of_known_lengths():
    assert plan4([32449] * 8, 8, 456) == (73, 0)           # 448 items on 456 blocks
    assert plan4([705], 1, 456) == (4, 0)
    assert plan4([0], 1, 456) == (4, 0)
    assert plan4([64 * 40] * 64, 8, 456) == (16, 0)        # sixteen pages at least
    assert plan4([64 * 508] * 64, 8, 456) == (142, 32)
    assert plan4([30000], 1, 456) == (8, 0)                # no longer than the other form's smallest items
    assert plan4([100000], 1, 456) == (16, 0)              # 25 pages would leave six of seven blocks idle


def test_sizes_past_32_bits_are_refused(lib):
    for batch, hk in ((1 << 30, 8), (1 << 20, 1 << 12)):
        with pytest.raises(O.OscarError):
            O.oscar_decode_workspace_bytes_int4(O.make_shape(hk, hk), batch, 1)
