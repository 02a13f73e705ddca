"""Histories whose values are small, or have little weight, in 2 bits on the GPU against float64: an fp32 output of the
modes is as exact for them as for others (tests/history_scene.py, with its tolerances)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from bit_kv_cache_evict_gb300 import synth as S  # noqa: E402
from history_scene import SCALE, Scene, out_tolerance  # noqa: E402

D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def scene(bits, hq, hk, g, std, hist=(1, 64, 65, 700, 1153)):
    c = Scene(70, bits, list(hist), hq, hk, g, groups=[-1, 0, 0, 0, -1], shared=1, std=std)
    c.len[:] = 0
    return c


def run(c, call):
    d = c.device()
    out = torch.full((c.B, c.hq, D), float("nan"), device="cuda")
    args = (c.sh, c.bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"])
    if call == "weights":
        ws = torch.empty(O.oscar_decode_workspace_bytes_weights(c.sh, c.bits, c.B, c.max_pages), dtype=torch.uint8, device="cuda")
        O.oscar_decode_attn_weights(*args, d["U"], SCALE, out, torch.zeros(c.B, 64 * c.max_pages, device="cuda"), ws)
    else:
        ws = torch.empty(O.oscar_decode_workspace_bytes_shared(c.sh, c.bits, c.B, c.max_pages, c.n_groups), dtype=torch.uint8, device="cuda")
        O.oscar_decode_attn_shared(*args, d["group"], d["group_pages"], d["U"], SCALE, out, ws, min_members=2)
    return out.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("call", ["weights", "shared"])
@pytest.mark.parametrize("hq,hk,g", [(1, 1, 128), (4, 1, 32), (8, 2, 64), (8, 1, 128), (16, 2, 32)])
@pytest.mark.parametrize("std", [2.0 ** -9, 2.0 ** -13])
def test_small_values(bits, call, hq, hk, g, std):
    """Scales of 2^-9 and 2^-13: products of a weight and a scale that are fp16 subnormals unless a power of two lifts them."""
    c = scene(bits, hq, hk, g, std)
    ref, _, _, mag, _, _ = c.want()
    err = np.abs(run(c, call) - ref)
    assert (err <= out_tolerance(ref, mag, bits, False)).all(), (err / out_tolerance(ref, mag, bits, False)).max()


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("call", ["weights", "shared"])
@pytest.mark.parametrize("hq,hk", [(4, 1), (8, 1)])
def test_scales_that_differ_from_page_to_page(bits, call, hq, hk):
    """Pages whose values grow and shrink by powers of two from 2^-12 to 2^12; a page of zeros."""
    c = scene(bits, hq, hk, 32, 1.0)
    for b in range(c.B):
        for i, page in enumerate(c.table[b][c.table[b] >= 0]):
            if b in (2, 3) and i == 0:
                continue                                   # (the shared one)
            f = 0.0 if i == 3 else 2.0 ** ((5 * i + 7 * b) % 25 - 12)
            for h in range(hk):
                for t in range(64):
                    v = c.pairs(page, h, 1, t).astype(np.float64) * f
                    c.set_pairs(page, h, 1, t, v)
    ref, _, _, mag, _, _ = c.want()
    err = np.abs(run(c, call) - ref)
    assert (err <= out_tolerance(ref, mag, bits, False)).all(), (err / out_tolerance(ref, mag, bits, False)).max()


def one_token_above(bits, hq, hk, hist, gaps, s):
    """Histories whose values are all s times the highest code: every rounding of a weight times a scale goes one way.  The
    logits of all tokens but one are 0; that of token 5 is above them by gaps[b] to 1.9 gaps[b] (by head) in base 2."""
    c = scene(bits, hq, hk, 128, 1.0, hist)
    blk = c.pool.reshape(c.num_pages, hk, -1)
    codes = 2048 if bits == 2 else 4096 + 256
    blk[:, :, codes:codes + (2048 if bits == 2 else 4096)] = 0xFF
    for b in range(c.B):
        for i, page in enumerate(c.table[b][c.table[b] >= 0]):
            for h in range(hk):
                for t in range(64):
                    c.set_pairs(page, h, 0, t, np.float16([[0, 1.0 if 64 * i + t == 5 else 0]]))
                    c.set_pairs(page, h, 1, t, np.float16([[s, 0]]))
    head = np.arange(hq)
    f = np.array(gaps)[:, None] * (1 + 0.9 * head / hq) * np.log(2) / (D * SCALE)
    c.q = S.bf16_bits(f[:, :, None] * np.stack([c.R[h * hk // hq][0] @ np.ones(D) for h in head]))
    return c


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("call", ["weights", "shared"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (8, 1), (16, 2)])
@pytest.mark.parametrize("gaps", [(0.1, 0.2, 0.3, 0.4, 0.45), (13.1, 13.2, 13.3, 13.4, 13.5)])
def test_roundings_that_go_one_way(bits, call, hq, hk, gaps):
    """Flat weights of small values; and values of ordinary size with a long tail of little weight behind one token."""
    c = one_token_above(bits, hq, hk, [65, 64, 130, 700, 4096], gaps, 2.0 ** -14 if gaps[0] < 1 else 1.0)
    ref, _, _, mag, _, _ = c.want()
    err = np.abs(run(c, call) - ref)
    assert (err <= out_tolerance(ref, mag, bits, False)).all(), (err / out_tolerance(ref, mag, bits, False)).max()
