"""The rotated queries do not depend on which sequences share a thread block: a sequence decoded alone, as the second of
a pair and behind a pair gives the same bits, for every number of heads per KV head, and is within the bound of float64."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from history_scene import SCALE, Scene, out_tolerance  # noqa: E402

D = 128


@pytest.mark.parametrize("call", ["plain", "weights", "shared"])
@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (4, 1), (8, 1), (3, 3), (24, 3)])
def test_alone_and_beside_others(call, bits, hq, hk):
    B.build()
    c = Scene(90 + hq, bits, [130, 70, 199], hq, hk, 64)       # (histories of one item each)
    c.len[:] = [300, 5, 64]
    d, want = c.device(), c.want()

    def run(rows):
        n = len(rows)
        t = {k: d[k][rows].contiguous() for k in ("q", "kv", "len", "table", "hist")}
        out = torch.full((n, hq, D), float("nan"), device="cuda")
        args = (c.sh, t["q"], t["kv"], t["len"], d["pool"], t["table"], c.max_pages, c.num_pages, t["hist"])
        if call == "plain":
            size, f = (O.oscar_decode_workspace_bytes, O.oscar_decode_attn) if bits == 2 else (O.oscar_decode_workspace_bytes_int4, O.oscar_decode_attn_int4)
            ws = torch.empty(size(c.sh, n, c.max_pages), dtype=torch.uint8, device="cuda")
            f(*args, d["U"], SCALE, out, ws)
        elif call == "weights":
            ws = torch.empty(O.oscar_decode_workspace_bytes_weights(c.sh, bits, n, c.max_pages), dtype=torch.uint8, device="cuda")
            O.oscar_decode_attn_weights(args[0], bits, *args[1:], d["U"], SCALE, out, torch.zeros(n, 64 * c.max_pages, device="cuda"), ws)
        else:
            ws = torch.empty(O.oscar_decode_workspace_bytes_shared(c.sh, bits, n, c.max_pages, 0), dtype=torch.uint8, device="cuda")
            none = torch.full((n,), -1, dtype=torch.int32, device="cuda")
            O.oscar_decode_attn_shared(args[0], bits, *args[1:], none, none[:0], d["U"], SCALE, out, ws)
        return out

    whole = run([0, 1, 2])
    err = np.abs(whole.cpu().numpy() - want[0])
    assert (err <= (out_tolerance(want[0], want[3], bits, False) if call != "plain" or bits == 4 else 2e-3)).all(), err.max()
    for rows in ([0], [1], [2], [1, 0], [2, 1], [2, 0, 1], [0, 1, 2, 1, 0]):
        assert torch.equal(run(rows), whole[rows]), rows
