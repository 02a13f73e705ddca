"""4-bit eviction with a clip ratio of its own for every (KV head, K|V), and rows of
unlike sizes per head: a ratio or matrix taken from another head or from the
other of K and V shows.  Tolerances are those of test_gpu_int4.compare_pools."""
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
from test_gpu_int4 import compare_pools, f64, kv_bits, rotation  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("n,hk", [(7, 3), (120, 4), (700, 3)])   # one vector per block; more of them; tensor cores
def test_each_head_has_its_own_clip_ratio(n, hk, g):
    rng = np.random.default_rng(n + g)
    pages = (n + 63) // 64
    table, pos = rng.permutation(pages).astype(np.int32)[None], rng.permutation(n).astype(np.int32)
    rows, U = kv_bits(rng, n, hk), rotation(rng, hk)
    clip = (0.45 + 0.6 * rng.permutation(2 * hk).reshape(hk, 2) / (2 * hk)).astype(np.float32)
    clip[hk - 1, 1] = 1.0
    want = np.full(pages * hk * I.block_bytes(4, g), 0x5A, np.uint8)
    dev = H.u8_t(want)
    aux = I.evict(want, f64(rows), U, clip, table, np.zeros(n, int), pos, g)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_evict_quantize_int4(O.make_shape(hk, hk, quant_group=g), H.bf16_t(rows), H.i32_t(np.zeros(n)), H.i32_t(pos), H.f32_t(U), H.f32_t(clip),
                                dev, H.i32_t(table), 1, pages, pages, dev_status=status)
    assert int(status) == 0
    compare_pools(dev.cpu().numpy(), want, table, [(i, 0, int(pos[i])) for i in range(n)], aux, hk, g)
