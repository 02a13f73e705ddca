"""Compaction in the launch form that gives a thread block four KV heads in turn
(many destination pages), with head counts that do not divide by four: byte copies, so equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gpu_harness as H  # noqa: E402
from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from oracle import int4 as I  # noqa: E402
from test_gpu_history import random_pool  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


@pytest.mark.parametrize("bits,g,hk,boost", [(2, 32, 3, True), (2, 128, 6, False), (4, 32, 6, False), (4, 64, 1, False), (4, 128, 9, False)])
def test_four_heads_in_turn(bits, g, hk, boost):
    rng = np.random.default_rng(bits * g + hk)
    wide = 4 * 912 // (3 * hk) + 1                         # destination pages of a row: mostly unused
    hist, keeps = [300, 64, 200], [np.sort(rng.permutation(300)[:171]), np.zeros(0, int), rng.integers(0, 200, 70)]
    need, fresh = [(h + 63) // 64 for h in hist], [3, 0, 2]
    pages = sum(need) + sum(fresh) + 2
    ids, at = rng.permutation(pages), 0
    src, dst = np.full((3, 5), -1, np.int32), np.full((3, wide), -1, np.int32)
    for t, counts in ((src, need), (dst, fresh)):
        for b, n in enumerate(counts):
            t[b, :n] = ids[at:at + n]
            at += n
    assert 3 * wide * hk >= 4 * 912
    keep = np.full((3, 200), -1, np.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = k
    n_keep = np.array([len(k) for k in keeps], np.int32)
    pool = random_pool(rng, pages, hk, bits, g)
    want = I.gather(pool, src, dst, keep, n_keep, hk, bits, g)
    rec = rng.integers(0, 256, pages * hk * O.BOOST_BLOCK_BYTES).astype(np.uint8)
    wrec = rec.copy().reshape(pages, hk, 64, 16)
    for b, k in enumerate(keeps):
        for i, x in enumerate(k):
            wrec[dst[b, i // 64], :, i % 64] = rec.reshape(pages, hk, 64, 16)[src[b, x // 64], :, x % 64]
    dev, drec, status = H.u8_t(pool), H.u8_t(rec), torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_history_gather(O.make_shape(hk, hk, quant_group=g), bits, dev, H.i32_t(src), H.i32_t(dst), H.i32_t(keep), H.i32_t(n_keep), pages,
                           boost=drec if boost else None, dev_status=status)
    assert int(status) == 0
    assert np.array_equal(dev.cpu().numpy(), want)
    assert np.array_equal(drec.cpu().numpy(), wrec.ravel() if boost else rec)
