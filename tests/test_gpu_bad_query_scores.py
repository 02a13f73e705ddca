"""The scores of a sequence with a bad query on the GPU: NaN at every token that it attends, and nothing else."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from history_scene import NSLOT, SCALE, Scene, out_tolerance, weight_tolerance  # noqa: E402

D = 128


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("bad", [0x7F80, 0x7FC0])          # bf16 infinity, NaN
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,hk", [(8, 2), (8, 1)])
def test_scores_of_a_bad_query(bits, bad, dtype, hq, hk):
    B.build()
    c = Scene(80, bits, [700, 64, 130], hq, hk, 64)
    c.len[:] = [NSLOT, 7, 100]
    want = c.want()
    c.q[0, 1, 7] = bad
    c.q[1, 6, 0] = bad
    d = c.device()
    out = torch.full((c.B, hq, D), float("nan"), dtype=dtype, device="cuda")
    w, sw = torch.full((c.B, 64 * c.max_pages), 0.5, device="cuda"), torch.full((c.B, NSLOT), 0.25, device="cuda")
    ws = torch.full((O.oscar_decode_workspace_bytes_weights(c.sh, bits, c.B, c.max_pages),), 0xFF, dtype=torch.uint8, device="cuda")
    O.oscar_decode_attn_weights(c.sh, bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"], d["U"], SCALE,
                                out, w, ws, slot_weight=sw)
    w, sw, out = w.cpu().numpy(), sw.cpu().numpy(), out.float().cpu().numpy()
    for b in (0, 1):
        assert np.isnan(w[b, :c.hist[b]]).all() and (w[b, c.hist[b]:] == 0.5).all()
        assert np.isnan(sw[b, :c.len[b]]).all() and (sw[b, c.len[b]:] == 0.25).all()
    rows = np.zeros((3, hq), bool)
    rows[0, 1] = rows[1, 6] = True
    assert np.isnan(out[rows]).all()
    assert (np.abs(out - want[0]) <= out_tolerance(want[0], want[3], bits, dtype == torch.bfloat16))[~rows].all()
    n, m = c.hist[2], c.len[2]
    assert (np.abs(w[2, :n].astype(np.float64) - 0.5 - want[1][2, :n]) <= weight_tolerance(want[1], want[4], 0.5, hq, bits)[2, :n]).all()
    assert (np.abs(sw[2, :m].astype(np.float64) - 0.25 - want[2][2, :m]) <= weight_tolerance(want[2], want[5], 0.25, hq, bits)[2, :m]).all()
    assert (w[2, n:] == 0.5).all() and (sw[2, m:] == 0.25).all()
