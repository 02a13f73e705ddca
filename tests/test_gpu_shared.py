"""The decode of shared first pages on the GPU against float64 (tests/history_scene.py, with its tolerances)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gpu_harness as H  # noqa: E402
from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from history_scene import SCALE, Scene, out_tolerance  # noqa: E402

D = 128
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def run(c, dtype=F32, status=None, stream=None, ws=None, group=None, group_pages=None, min_members=2):
    d = getattr(c, "d", None) or c.device()
    out = torch.full((c.B, c.hq, D), float("nan"), dtype=dtype, device="cuda")
    gp = d["group_pages"] if group_pages is None else group_pages
    if ws is None:
        ws = torch.full((O.oscar_decode_workspace_bytes_shared(c.sh, c.bits, c.B, c.max_pages, gp.numel()),), 0xFF, dtype=torch.uint8, device="cuda")
    own = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    O.oscar_decode_attn_shared(c.sh, c.bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"],
                               d["group"] if group is None else group, gp, d["U"], SCALE, out, ws, min_members=min_members, dev_status=own, stream=stream)
    if status is None:
        (stream or torch.cuda.current_stream()).synchronize()
        assert int(own) == 0                               # no wait of the kernels ran out either
    return out


def check(c, out, want, dtype, rows=slice(None)):
    ref, mag = want[0][rows], want[3][rows]
    got = out.float().cpu().numpy().astype(np.float64)[rows]
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= out_tolerance(ref, mag, c.bits, dtype == BF16, fp16_shared=dtype == BF16)).all(), err.max()
    # all in all: 2^-8 for the rounding of a bf16 output and as much again for its fp16 products; fp32: 2^-15
    assert np.linalg.norm(err) <= np.linalg.norm(ref) * (2.0 ** -7 if dtype == BF16 else 2.0 ** -15), np.linalg.norm(err) / np.linalg.norm(ref)


BOTH = pytest.mark.parametrize("bits", [2, 4])
TYPES = pytest.mark.parametrize("dtype", [F32, BF16])


@BOTH
@TYPES
@pytest.mark.parametrize("hq,hk,g", [(1, 1, 32), (2, 1, 64), (4, 1, 128), (8, 2, 32), (8, 1, 128), (16, 2, 64), (24, 3, 32), (3, 3, 128)])
def test_groups_match_float64(bits, dtype, hq, hk, g):
    """Two groups, one sequence of its own, one whose history ends inside the prefix, one that is the prefix, an empty one."""
    hist = [64 * 5 + 1, 64 * 5, 700, 10, 64 * 5 + 64, 64 * 4 + 63, 900, 0]
    c = Scene(hq + g, bits, hist, hq, hk, g, groups=[0, 0, 1, -1, 1, 0, 1, -1], shared=5, std=2.0)
    c.len[7] = 0
    c.poison()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(c, run(c, dtype, status=status), c.want(), dtype)
    assert int(status) == 0


@BOTH
@TYPES
@pytest.mark.parametrize("members,hq,hk", [(2, 1, 1), (17, 8, 1), (33, 4, 1), (64, 4, 1), (65, 4, 1), (129, 2, 1), (70, 16, 2)])
def test_rows_that_fill_tiles_or_not(bits, dtype, members, hq, hk):
    rng = np.random.default_rng(members)
    hist = (64 * 3 + rng.integers(0, 130, members)).tolist()
    c = Scene(members, bits, hist, hq, hk, 32, groups=[0] * members, shared=3, std=2.0)
    c.len[:] = rng.integers(0, 50, members)
    check(c, run(c, dtype), c.want(), dtype)


@BOTH
@TYPES
@pytest.mark.parametrize("pages", [1, 2, 3, 4, 5, 9, 63, 150])
def test_prefix_lengths(bits, dtype, pages):
    """From one page to more runs of pages than one merge batch takes; peaked weights."""
    c = Scene(pages, bits, [64 * pages + 30, 64 * pages, 64 * pages + 1], 4, 1, 64, groups=[0, 0, 0], shared=pages, std=4.0)
    check(c, run(c, dtype), c.want(), dtype)


@BOTH
def test_more_whole_groups_than_blocks(bits):
    """90 pairs of sequences, three KV heads: 270 items, some of them on the same block."""
    n = 90
    groups = np.repeat(np.arange(n), 2)
    rng = np.random.default_rng(1)
    groups = groups[rng.permutation(2 * n)]
    for dtype in (F32, BF16):
        c = Scene(11, bits, [64 * 2 + (i % 3) for i in range(2 * n)], 3, 3, 128, groups=groups, shared=2)
        c.len[:] = 8
        check(c, run(c, dtype), c.want(), dtype)


@BOTH
@TYPES
def test_maxima_that_grow_and_fall(bits, dtype):
    """Pages whose keys grow from page to page (each passes the maximum so far), and pages that shrink."""
    pages = 12
    for order in (1, -1):
        c = Scene(12, bits, [64 * pages + 5] * 40, 4, 1, 32, groups=[0] * 40, shared=pages, std=1.0)
        for i in range(pages):
            f = np.float16(1.35 ** (i if order > 0 else pages - i))
            for t in range(64):
                c.set_pairs(c.table[0, i], 0, 0, t, c.pairs(c.table[0, i], 0, 0, t) * f)
        check(c, run(c, dtype), c.want(), dtype)


@BOTH
def test_a_flat_softmax_over_a_long_prefix(bits):
    c = Scene(13, bits, [64 * 100 + 3] * 3, 4, 1, 32, groups=[0] * 3, shared=100, std=0.02)
    check(c, run(c), c.want(), F32)


@BOTH
def test_groups_that_are_none(bits):
    """Groups of one, no group at all, no shared pages, no sequence: the plain decode."""
    c = Scene(14, bits, [300, 64 * 4, 64 * 7 + 9], 8, 2, 32)
    want = c.want()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for group, pages in (([0, 1, 2], [2, 2, 2]), ([-1, -1, -1], [3]), ([0, 0, 0], [0]), ([-5, -1, -2], [])):
        for dtype in (F32, BF16):
            check(c, run(c, dtype, group=i32(group), group_pages=i32(pages)), want, dtype)
    sh = c.sh
    O.oscar_decode_attn_shared(sh, bits, torch.empty(0, 8, D, dtype=BF16, device="cuda"), None, i32([]), None, i32([]), 4, 0, i32([]), i32([]), i32([]),
                               c.d["U"], SCALE, torch.empty(0, 8, D, device="cuda"), torch.empty(4096, dtype=torch.uint8, device="cuda"))


@BOTH
@TYPES
def test_bad_pages_and_groups_are_reported(bits, dtype):
    c = Scene(15, bits, [64 * 6 + 10] * 4, 4, 1, 32, groups=[0] * 4, shared=6)
    for at, bad in ((0, -1), (5, c.num_pages), (2, 1 << 30)):
        c.table[:, at] = bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(c, dtype, status=status)
    assert int(status) == O.OSCAR_STATUS_BAD_PAGE
    check(c, out, c.want(), dtype)
    c = Scene(16, bits, [64 * 6 + 10] * 4, 4, 1, 32, groups=[0] * 4, shared=6)
    c.table[:, :6] = -1                                    # nothing of the prefix can be read
    status.zero_()
    out = run(c, dtype, status=status)
    assert int(status) == O.OSCAR_STATUS_BAD_PAGE
    check(c, out, c.want(), dtype)
    c = Scene(17, bits, [64 * 3 + 10] * 4, 4, 1, 32, groups=[0, 0, 1, 1], shared=3)
    want = c.want()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for group, pages in (([0, 0, 2, 1], [3, 3]), ([0, 0, 1, 1], [3, -1]), ([0, 0, 1, 1], [c.max_pages + 1, 3])):
        status.zero_()
        out = run(c, dtype, status=status, group=i32(group), group_pages=i32(pages))
        assert int(status) == O.OSCAR_STATUS_BAD_POS
        check(c, out, want, dtype)


@BOTH
@TYPES
def test_nan_in_a_shared_page_reaches_the_group_alone(bits, dtype):
    c = Scene(18, bits, [64 * 3 + 10] * 6, 8, 2, 32, groups=[0, 0, 1, 1, 1, -1], shared=3)
    want = c.want()
    v = c.pairs(c.table[0, 1], 1, 0, 9)
    v[0, 0] = np.nan
    c.set_pairs(c.table[0, 1], 1, 0, 9, v)
    out = run(c, dtype)
    assert out[:2, 4:].isnan().all() and out[:2, :4].isfinite().all()
    check(c, out, want, dtype, rows=slice(2, 6))


@BOTH
@TYPES
@pytest.mark.parametrize("bad", [0x7F80, 0x7FC0])          # bf16 infinity, NaN
def test_a_bad_query_is_its_rows_matter_alone(bits, dtype, bad):
    c = Scene(22, bits, [64 * 4 + 10] * 3 + [200], 8, 2, 64, groups=[0, 0, 0, -1], shared=4)
    want = c.want()
    rows = np.zeros((4, 8), bool)
    for b, h in ((0, 1), (2, 7), (3, 0)):
        c.q[b, h, 11] = bad
        rows[b, h] = True
    out = run(c, dtype)
    assert out.isnan().cpu().numpy()[rows].all()
    err = np.abs(out.float().cpu().numpy() - want[0])
    assert (err <= out_tolerance(want[0], want[3], bits, dtype == BF16, dtype == BF16))[~rows].all()


@BOTH
@TYPES
def test_same_bits_streams_and_a_graph_that_follows_the_groups(bits, dtype):
    c = Scene(19, bits, [64 * 9 + 17 * i for i in range(12)], 16, 4, 32, groups=[i % 2 for i in range(12)], shared=9)
    want = c.want()
    first = run(c, dtype)
    check(c, first, want, dtype)
    assert torch.equal(first, run(c, dtype))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(c, dtype)
    side.synchronize()
    assert torch.equal(first, other)
    d = c.d
    ws = torch.zeros(O.oscar_decode_workspace_bytes_shared(c.sh, bits, c.B, c.max_pages, 2), dtype=torch.uint8, device="cuda")
    out = torch.zeros(c.B, c.hq, D, dtype=dtype, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O.oscar_decode_attn_shared(c.sh, bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"], d["group"],
                                   d["group_pages"], d["U"], SCALE, out, ws, min_members=2)
    for group, pages in (([i % 2 for i in range(12)], [9, 9]), ([-1] * 6 + [i % 2 for i in range(6)], [4, 9]), ([-1] * 12, [0, 0])):
        d["group"].copy_(torch.tensor(group, dtype=torch.int32))
        d["group_pages"].copy_(torch.tensor(pages, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(c, out, want, dtype)


@BOTH
def test_wide_tables_and_no_windows(bits):
    c = Scene(20, bits, [64 * 3 + 10] * 3, 4, 1, 32, groups=[0] * 3, shared=3, wide=300)
    c.len[:] = 0
    c.sh = O.make_shape(4, 1, quant_group=32, sink=0, recent=0)
    want = c.want()
    for dtype in (F32, BF16):
        check(c, run(c, dtype), want, dtype)


@BOTH
@TYPES
def test_the_librarys_rule_on_both_sides_of_its_border(bits, dtype):
    """min_members 0 shares where it is faster, by members and pages; a minimum above the members shares nothing.  The
    result is the same to its tolerance on both sides: 70 sequences of 8 KV heads, 3 and 9 of 64, fewer and more pages."""
    for members, hk, pages in ((70, 8, 7), (70, 8, 12), (9, 64, 20), (9, 64, 30), (3, 64, 20)):
        c = Scene(21, bits, [64 * pages + i for i in range(members)], hk, hk, 128, groups=[0] * members, shared=pages)
        c.len[:] = 4
        want = c.want()
        for least in (0, 2, members, members + 1):
            check(c, run(c, dtype, min_members=least), want, dtype)
