"""CPU: the plan of shared pages, restated, never makes more items, tiles of queries or partials than the workspace that
the library asks for has room for, and no run of more than 256 pages."""
import random

import pytest

from bit_kv_cache_evict_gb300 import build as B
from bit_kv_cache_evict_gb300 import oscar as O


@pytest.fixture(scope="module")
def lib():
    B.build()
    return O.lib()


def up(a, b):
    return -(-a // b)


def plan(count, pages, G, hk, max_pages, rows, blocks):
    """Pages of a run at most, for groups of count[g] members that attend pages[g] pages together."""
    tiles = [up(c * G, rows) for c in count]

    def items(n):
        return sum(t * up(p, n) for t, p in zip(tiles, pages)) * hk

    lo, hi = 4, min(max(4, max_pages), 256)
    if items(hi) <= blocks:
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if items(mid) <= blocks else (mid + 1, hi)
        return lo
    share = sum(t * p for t, p in zip(tiles, pages)) * hk // (4 * blocks)
    return max(16, min(max_pages, 256, share))


def test_the_workspace_has_room_for_every_plan(lib):
    rng = random.Random(1)
    for _ in range(1500):
        G, hk, batch = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 8, 64]), rng.choice([2, 3, 8, 33, 160, 1000, 5000])
        n_groups = rng.randint(1, min(8192, rng.choice([1, 3, 80, batch, 2 * batch])))
        max_pages, bits = rng.choice([1, 3, 16, 17, 255, 256, 257, 400, 2000, 16384]), rng.choice([2, 4])
        count = [0] * n_groups
        for _ in range(batch):
            if rng.random() < 0.9:
                count[rng.randrange(n_groups)] += 1
        both = [(c, rng.choice([max_pages, rng.randint(0, max_pages)])) for c in count if c >= rng.choice([2, 2, 3])]
        count, pages = [c for c, p in both if p], [p for c, p in both if p]
        sh = O.make_shape(G * hk, hk)
        stride = up(G * 130, 4) * 4                        # floats of a partial: outputs, maximum and sum of G heads
        try:
            plain = (O.oscar_decode_workspace_bytes if bits == 2 else O.oscar_decode_workspace_bytes_int4)(sh, batch, max_pages)
            room = O.oscar_decode_workspace_bytes_shared(sh, bits, batch, max_pages, n_groups) - plain
        except O.OscarError:                               # (more partials than the device's indices)
            assert batch * hk * max_pages > 1 << 24
            continue
        for rows in (128, 256):
            for blocks in (152, 132):
                n = plan(count, pages, G, hk, max_pages, rows, blocks)
                splits = [up(p, n) for p in pages]
                assert all(up(p, s) <= 256 for p, s in zip(pages, splits))
                items = sum(up(c * G, rows) * s for c, s in zip(count, splits)) * hk
                parts = sum(c * s for c, s in zip(count, splits)) * hk
                tiles = sum(up(c * G, 128) for c in count) * hk
                # items of 32 bytes, tiles of 64 KB (two parts) and 128 scales, partials; 36 bytes per sequence
                assert items * 32 + tiles * (65536 + 512) + parts * stride * 4 + 36 * batch <= room


def test_plans_of_known_groups():
    assert plan([64], [448], 4, 8, 508, 256, 152) == 24     # 8 KV heads x 19 runs on 152 blocks
    assert plan([2], [3], 4, 1, 3, 256, 152) == 4           # no runs of fewer pages than four where one will do
    assert plan([2] * 80, [16384] * 80, 1, 1, 16384, 256, 152) == 256
    assert plan([2] * 90, [2] * 90, 1, 3, 2, 128, 152) == 16
