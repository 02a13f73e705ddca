"""The decode that accumulates attention weight on the GPU against float64 (tests/history_scene.py, with its tolerances)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gpu_harness as H  # noqa: E402
from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from history_scene import NSLOT, SCALE, Scene, out_tolerance, weight_tolerance  # noqa: E402

D = 128
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def run(c, dtype=F32, decay=1.0, slots=True, old=None, old_slots=None, status=None, stream=None, ws=None, stride=None):
    d = getattr(c, "d", None) or c.device()
    out = torch.full((c.B, c.hq, D), float("nan"), dtype=dtype, device="cuda")
    stride = stride or 64 * c.max_pages
    w = torch.full((c.B, stride), 0.5, device="cuda") if old is None else old.clone()
    sw = None if not slots else torch.full((c.B, NSLOT), 0.25, device="cuda") if old_slots is None else old_slots.clone()
    if ws is None:
        ws = torch.full((O.oscar_decode_workspace_bytes_weights(c.sh, c.bits, c.B, c.max_pages),), 0xFF, dtype=torch.uint8, device="cuda")
    O.oscar_decode_attn_weights(c.sh, c.bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"], d["U"],
                                SCALE, out, w, ws, slot_weight=sw, decay=decay, dev_status=status, stream=stream)
    return out, w, sw


def check(c, got, want, dtype, decay=1.0, old=0.5, old_slots=0.25):
    out, w, sw = got
    ref, rw, rsw, mag, we, swe = want
    g = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all()
    assert (np.abs(g - ref) <= out_tolerance(ref, mag, c.bits, dtype == BF16)).all()
    inside = np.arange(rw.shape[1]) < c.hist[:, None]
    w = w.cpu().numpy().astype(np.float64)
    err = np.abs(w[:, :rw.shape[1]] - (decay * old + rw))
    assert (err[inside] <= weight_tolerance(rw, we, decay * old, c.hq, c.bits)[inside]).all(), (err[inside].max())
    assert (w[:, :rw.shape[1]][~inside] == old).all() and (w[:, rw.shape[1]:] == old).all()   # left as they were
    if sw is not None:
        inside = np.arange(NSLOT) < c.len[:, None]
        s = sw.cpu().numpy().astype(np.float64)
        err = np.abs(s - (decay * old_slots + rsw))
        assert (err[inside] <= weight_tolerance(rsw, swe, decay * old_slots, c.hq, c.bits)[inside]).all(), err[inside].max()
        assert (s[~inside] == old_slots).all()


SHAPES = [(1, 1, 32), (2, 1, 64), (4, 1, 128), (8, 2, 32), (8, 1, 32), (16, 2, 64), (24, 3, 128), (4, 4, 64)]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hq,hk,g", SHAPES)
def test_output_and_weights_match_float64(bits, dtype, hq, hk, g):
    c = Scene(hq + g, bits, [0, 1, 63, 64, 65, 700, 0, 1153], hq, hk, g, std=2.0).poison()
    c.len[6] = 0                                           # an empty context
    c.len[0] = 17
    c.poison()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(c, dtype, status=status)
    check(c, got, c.want(), dtype)
    assert int(status) == 0
    total = got[1].double().sum(1) - 0.5 * got[1].shape[1] + got[2].double().sum(1) - 0.25 * NSLOT
    full = c.hist + c.len > 0
    assert (np.abs(total.cpu().numpy() - np.where(full, hq, 0)) < 1e-3 * hq).all()   # every head's weights add up to 1


@pytest.mark.parametrize("bits", [2, 4])
def test_decay_and_wider_rows(bits):
    c = Scene(3, bits, [130, 2000], 8, 2, 64)
    want = c.want()
    check(c, run(c, decay=0.75, stride=64 * c.max_pages + 37), want, F32, decay=0.75)
    bad = torch.full((2, 64 * c.max_pages), float("nan"), device="cuda")
    bad_slots = torch.full((2, NSLOT), float("inf"), device="cuda")
    out, w, sw = run(c, decay=0.0, old=bad, old_slots=bad_slots)   # 0 replaces, whatever was there
    inside = torch.arange(w.shape[1], device="cuda") < torch.from_numpy(c.hist).cuda()[:, None]
    assert w[inside].isfinite().all() and w[~inside].isnan().all() and sw.isfinite().all()
    ref = want[1][inside.cpu().numpy()]
    assert (np.abs(w[inside].cpu().numpy() - ref) <= weight_tolerance(want[1], want[4], 0, 8, bits)[inside.cpu().numpy()]).all()
    check(c, run(c, slots=False), want, F32)


@pytest.mark.parametrize("bits", [2, 4])
def test_a_flat_softmax_over_a_long_history(bits):
    """Keys of scale 0: every token has the same weight; the result is far smaller than the values."""
    c = Scene(4, bits, [7000, 5], 4, 1, 32, std=0.02)
    check(c, run(c), c.want(), F32)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("hq,hk", [(4, 1), (8, 1)])
def test_a_bad_page_is_reported_and_has_weight_0(bits, hq, hk):
    c = Scene(5, bits, [700, 300], hq, hk, 32)
    bad = [c.table[0, 3], c.table[1, 4]]
    c.table[0, 3], c.table[1, 4] = -1, c.num_pages
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(c, status=status)
    assert int(status) == O.OSCAR_STATUS_BAD_PAGE
    check(c, got, c.want(), F32)
    assert (got[1][0, 192:256] == 0.5).all() and (got[1][1, 256:300] == 0.5).all() and bad


@pytest.mark.parametrize("bits", [2, 4])
def test_a_nan_logit_makes_its_rows_and_weights_nan(bits):
    c = Scene(6, bits, [200, 90, 300], 8, 2, 32)
    want = c.want()
    v = c.pairs(c.table[0, 1], 1, 0, 5)
    v[0, 0] = np.nan
    c.set_pairs(c.table[0, 1], 1, 0, 5, v)
    out, w, sw = run(c)
    assert out[0, 4:].isnan().all() and out[0, :4].isfinite().all()
    assert w[0, :200].isnan().all() and (w[0, 200:] == 0.5).all() and sw[0].isnan().all()
    ref, rw = want[0], want[1]
    tol = out_tolerance(ref, want[3], bits, False)
    assert (np.abs(out[1:].cpu().numpy() - ref[1:]) <= tol[1:]).all()
    assert (np.abs(w[1:].cpu().numpy() - 0.5 - rw[1:])[:, :90] <= weight_tolerance(rw, want[4], 0.5, 8, bits)[1:, :90]).all()


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("bad", [0x7F80, 0x7FC0])          # bf16 infinity, NaN
def test_a_bad_query_leaves_the_other_heads_of_its_group(bits, bad):
    c = Scene(10, bits, [700, 64], 8, 2, 64)
    want = c.want()
    c.q[0, 1, 7] = bad
    c.q[1, 6, 0] = bad
    out, w, _ = run(c)
    rows = np.zeros((2, 8), bool)
    rows[0, 1] = rows[1, 6] = True
    assert out.isnan().cpu().numpy()[rows].all()
    tol = out_tolerance(want[0], want[3], bits, False)
    assert (np.abs(out.cpu().numpy() - want[0]) <= tol)[~rows].all()


@pytest.mark.parametrize("bits", [2, 4])
def test_same_bits_streams_and_graphs(bits):
    c = Scene(7, bits, [1000, 3, 4200], 32, 8, 32)
    first = run(c)
    again = run(c)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(c)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    # a captured step replayed three times accumulates three steps
    ws = torch.zeros(O.oscar_decode_workspace_bytes_weights(c.sh, bits, c.B, c.max_pages), dtype=torch.uint8, device="cuda")
    w, sw = torch.zeros(c.B, 64 * c.max_pages, device="cuda"), torch.zeros(c.B, NSLOT, device="cuda")
    out = torch.zeros(c.B, c.hq, D, device="cuda")
    d = c.d
    call = lambda: O.oscar_decode_attn_weights(c.sh, bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages,  # noqa: E731
                                               d["hist"], d["U"], SCALE, out, w, ws, slot_weight=sw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    w.zero_(), sw.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    three = w.clone()
    w.zero_(), sw.zero_()
    for _ in range(3):
        call()
    assert torch.equal(three, w) and torch.equal(out, first[0])


def test_layers_accumulate_into_one_array():
    """Two layers' calls with the step's decay at the first: the scores of both."""
    a, b = Scene(8, 4, [500, 70], 8, 2, 32), Scene(9, 4, [500, 70], 4, 1, 64)
    w = torch.full((2, 64 * a.max_pages), 2.0, device="cuda")
    _, w, _ = run(a, decay=0.5, old=w, slots=False)
    _, w, _ = run(b, decay=1.0, old=w, slots=False)
    wa, wb = a.want(), b.want()
    ref = 1.0 + wa[1] + wb[1]
    inside = np.arange(ref.shape[1]) < a.hist[:, None]
    tol = weight_tolerance(wa[1], wa[4], 1.0, 8, 4) + weight_tolerance(wb[1], wb[4], 2.0, 4, 4)
    assert (np.abs(w.cpu().numpy() - ref)[inside] <= tol[inside]).all()


@pytest.mark.parametrize("bits", [2, 4])
def test_the_widest_table(bits):
    """64 * max_pages positions just below 2^31 (the scores and the workspace take 9 GB each)."""
    c = Scene(11, bits, [700], 1, 1, 128)
    want, d, most = c.want(), c.device(), (2**31 - 1) // 64
    c.d = dict(d, table=torch.cat([d["table"], torch.full((1, most - c.max_pages), -1, dtype=torch.int32, device="cuda")], 1))
    c.max_pages = most
    out, w, sw = run(c)
    n = want[1].shape[1]
    assert bool((w[:, n:] == 0.5).all())
    check(c, (out, w[:, :n], sw), want, F32)
