"""The 4-bit decode where the listed scenes of test_gpu_int4.py do not come:
items in which a warp takes several pages, and queues with short items behind
the long ones, tables wider than the histories, shapes without BF16 windows; and
its bf16 output, which is the fp32 output rounded once.

Tolerances are test_gpu_int4.check's.  Its share for the value sums, 2^-15 of the
largest value, holds here too: a page's four tensor-core steps from zero lose 2^-19 of
it at most, a warp adds at most 64 pages (256-page items), each rounded: 2^-18, and
the merge at most 256 partials in batches: 2^-16 with the un-rotation's 22 bits.

The scenes alias a few pages many times (a table may name a page more than
once), so that the float64 oracle computes each page's part once.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gpu_harness as H  # noqa: E402
import oracle  # noqa: E402
from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from bit_kv_cache_evict_gb300 import synth as S  # noqa: E402
from oracle import int4 as I  # noqa: E402
from test_int4_plan_host import plan4  # noqa: E402
from test_gpu_int4 import SCALE, Cache, check, f64, rotation  # noqa: E402

D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


class Aliased:
    """`batch` sequences of the given lengths (tokens) over a pool of `pages`
    pages named again and again: table[b, i] = pages in an order of the sequence's own.
    grow: the V scales of page p are 2^(grow * p / pages) times larger."""

    def __init__(self, seed, hist, hq, hk, g, pages=8, grow=0.0, q_std=1.0, order=None):
        self.rng = rng = np.random.default_rng(seed)
        self.hist, self.hq, self.hk, self.g, self.B = np.array(hist, np.int32), hq, hk, g, len(hist)
        self.sh = O.make_shape(hq, hk, quant_group=g)
        self.num_pages = pages
        self.max_pages = int((self.hist.max() + 63) // 64)
        self.U = rotation(rng, hk)
        bb, ng = I.block_bytes(4, g), D // g
        pool = rng.integers(0, 256, (pages, hk, bb)).astype(np.uint8)
        for w, base in ((0, 4096), (1, 8192 + 256 * ng)):
            lo, hi = -2 * rng.uniform(0.8, 1.2, (pages, hk, 64 * ng)), 2 * rng.uniform(0.8, 1.2, (pages, hk, 64 * ng))
            size = 2.0 ** (grow * np.arange(pages) / pages)[:, None, None] if w else 1.0
            sz = (np.stack([(hi - lo) / 15, lo], -1) * np.expand_dims(size, -1)).astype(np.float16)
            pool[:, :, base:base + 256 * ng] = sz.view(np.uint8).reshape(pages, hk, 256 * ng)
        self.pool = pool.ravel()
        i = np.arange(self.max_pages)
        self.table = np.stack([order(b, i, self.max_pages) if order else rng.permutation(pages)[i % pages] for b in range(self.B)]).astype(np.int32)
        self.q = S.bf16_bits(rng.standard_normal((self.B, hq, D)) * q_std)
        self.kv = S.bf16_bits(rng.standard_normal((self.B, S.NSLOT, hk, 2, D)))
        self.len = rng.integers(1, S.NSLOT + 1, self.B).astype(np.int32)

    def decode(self, dtype=torch.float32, wide=0):
        d = dict(q=H.bf16_t(self.q), kv=H.bf16_t(self.kv), len=H.i32_t(self.len), pool=H.u8_t(self.pool), hist=H.i32_t(self.hist), U=H.f32_t(self.U))
        table = np.full((self.B, max(wide, self.max_pages)), -1, np.int32)
        table[:, :self.max_pages] = self.table
        out = torch.full((self.B, self.hq, D), float("nan"), dtype=dtype, device="cuda")
        ws = torch.full((O.oscar_decode_workspace_bytes_int4(self.sh, self.B, table.shape[1]),), 0xFF, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        O.oscar_decode_attn_int4(self.sh, d["q"], d["kv"], d["len"], d["pool"], H.i32_t(table), table.shape[1], self.num_pages, d["hist"], d["U"],
                                 SCALE, out, ws, dev_status=status)
        assert int(status) == 0
        self.plan = ws[:256].view(torch.int32)[8:10].tolist()   # pages of a long item, pages in short ones
        return out

    def want(self):
        """float64 attention: every page's tokens once, weighted by how often whole pages
        occur, and the last page's tokens by themselves."""
        orc = oracle.get()
        G = self.hq // self.hk
        out, mag = np.zeros((self.B, self.hq, D)), np.zeros((self.B, self.hq, 2))
        tab = np.arange(self.num_pages, dtype=np.int32)[None]
        for kv in range(self.hk):
            R = [orc.build_R(self.U[kv, w].astype(np.float64)) for w in (0, 1)]
            ks, vs = (I.values(self.pool, tab, 0, np.arange(64 * self.num_pages), kv, w, self.hk, 4, self.g) for w in (0, 1))
            for b in range(self.B):
                n, m = int(self.hist[b]), int(self.len[b])
                times = np.zeros((self.num_pages, 64))
                np.add.at(times, self.table[b, :n // 64], 1)
                if n % 64:
                    times[self.table[b, n // 64], :n % 64] += 1
                times = times.ravel()
                keys, vals = f64(self.kv[b, :m, kv, 0]), f64(self.kv[b, :m, kv, 1])
                for h in range(kv * G, (kv + 1) * G):
                    q = f64(self.q[b, h])
                    lh, lb = SCALE * (ks @ (q @ R[0])), SCALE * (keys @ q)
                    top = max(lh[times > 0].max(initial=-np.inf), lb.max())
                    ph, pb = times * np.exp(np.where(times > 0, lh, top) - top), np.exp(lb - top)
                    out[b, h] = ((ph @ vs) @ R[1].T + pb @ vals) / (ph.sum() + pb.sum())
                    terms = [(np.abs(ks) @ np.abs(q @ R[0]))[times > 0], np.abs(keys) @ np.abs(q)]
                    mag[b, h] = SCALE * max(t.max(initial=0.0) for t in terms), max(np.abs(vs[times > 0]).max(initial=0.0), np.abs(vals).max())
        return out, mag


def pages_per_warp(hist, hk, blocks):
    """Whether even items of one size for each block give some warp a second page (four warps an item)."""
    return sum((h + 63) // 64 for h in hist) * hk > 4 * blocks


RAGGED = [int(64 * 40 * (i % 16 + 1) / 16) - i for i in range(64)]


@pytest.mark.parametrize("hq,hk,g", [(8, 8, 32), (32, 8, 32), (16, 8, 64), (32, 8, 128), (64, 8, 32), (64, 8, 64), (64, 8, 128)])
def test_several_pages_of_an_item_in_each_warp(hq, hk, g):
    """Maximum and sums over pages, the ring's turns, long and short items: 64 ragged sequences of eight KV heads."""
    c = Aliased(hq + g, RAGGED, hq, hk, g, q_std=3.0)
    assert pages_per_warp(c.hist, hk, 512)
    want, mag = c.want()
    out = c.decode()
    check(out, want, mag)
    check(c.decode(torch.bfloat16), want, mag, dtype=torch.bfloat16)


@pytest.mark.parametrize("hq,hk,g", [(32, 8, 32), (32, 8, 128), (64, 8, 32), (64, 8, 64)])
@pytest.mark.parametrize("back", [False, True])
def test_value_scales_that_grow_inside_an_item(hq, hk, g, back):
    """The V scales grow by 2^13 over every sixteen pages, an item's (or shrink):
    the sums taken so far are rescaled."""
    def order(b, i, n):
        at = i % 16 * 24 // 16
        return 23 - at if back else at

    c = Aliased(7 + g, RAGGED, hq, hk, g, pages=24, grow=14.0, order=order)
    assert pages_per_warp(c.hist, hk, 512)
    want, mag = c.want()
    check(c.decode(), want, mag)
    check(c.decode(torch.bfloat16), want, mag, dtype=torch.bfloat16)


@pytest.mark.parametrize("hist", [[64 * 400, 64 * 200 - 3, 5], [64 * 1500 - 1]])
@pytest.mark.parametrize("hq,hk,g", [(4, 1, 32), (8, 1, 64)])
def test_few_long_sequences(hist, hq, hk, g):
    c = Aliased(11, hist, hq, hk, g, pages=16)
    want, mag = c.want()
    check(c.decode(), want, mag)


def test_equal_lengths_of_one_item_size():
    c = Aliased(12, [64 * 130] * 8, 32, 8, 32, pages=16)
    want, mag = c.want()
    check(c.decode(), want, mag)


@pytest.mark.parametrize("hist,hq,hk", [(RAGGED, 32, 8), ([700, 90, 1, 0], 4, 1), ([64 * 300], 8, 1), ([100000], 4, 1), ([64 * 100] * 8, 64, 8)])
@pytest.mark.parametrize("wide", [512, 4096])
def test_a_wider_table_changes_nothing(hist, hq, hk, wide):
    """Unused entries behind the histories: the plan goes by the lengths.  (Outputs may
    differ by the merge's order: it has as many warps to a row as the table may need.)"""
    c = Aliased(13, hist, hq, hk, 32)
    want, mag = c.want()
    narrow, plan = c.decode(), c.plan
    out = c.decode(wide=wide)
    check(out, want, mag)
    assert c.plan == plan == list(plan4(c.hist, hk, 152 * (2 if hq // hk == 8 else 3)))
    assert (out - narrow).abs().max() <= 4e-6 * narrow.abs().max()


@pytest.mark.parametrize("hq,hk,g", [(1, 1, 32), (4, 1, 32), (16, 8, 64), (64, 8, 128)])
def test_bf16_output_is_the_fp32_output_rounded_once(hq, hk, g):
    c = Cache(14 + hq, [0, 1, 63, 64, 65, 300, 1025], hq, hk, g)
    assert torch.equal(c.decode(dtype=torch.bfloat16), c.decode().bfloat16())
    a = Aliased(15, RAGGED, hq, hk, g)
    assert torch.equal(a.decode(torch.bfloat16), a.decode().bfloat16())


def test_the_same_call_gives_the_same_bits():
    a = Aliased(16, RAGGED, 32, 8, 32)
    first = a.decode()
    for _ in range(5):
        assert torch.equal(a.decode(), first)


# ---------------------------------------------------------------------------
# shapes without BF16 windows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,hk,g", [(4, 1, 32), (16, 2, 128)])
def test_a_shape_without_windows(hq, hk, g, dtype):
    c = Cache(17, [500, 0, 64, 1], hq, hk, g)
    c.sh, c.len = O.make_shape(hq, hk, quant_group=g, sink=0, recent=0), np.zeros(4, np.int32)
    want, mag = c.want()
    c.kv = np.zeros((4, 0, hk, 2, D), np.uint16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.decode(dtype=dtype, status=status)
    assert int(status) == 0 and (out[1] == 0).all()
    check(out, want, mag, dtype=dtype)


def test_the_2bit_decode_of_a_shape_without_windows():
    """History tokens alone: equal to the float64 attention over the values that oscar_history_read gives."""
    from test_gpu_history import random_pool
    rng = np.random.default_rng(18)
    hq, hk, g, n = 4, 1, 32, 300
    sh = O.make_shape(hq, hk, quant_group=g, sink=0, recent=0)
    pool, table, U = random_pool(rng, 6, hk, 2, g), np.arange(5, dtype=np.int32)[None], rotation(rng, hk)
    q = S.bf16_bits(rng.standard_normal((1, hq, D)))
    out = torch.full((1, hq, D), float("nan"), device="cuda")
    ws = torch.zeros(O.oscar_decode_workspace_bytes(sh, 1, 5), dtype=torch.uint8, device="cuda")
    kv = torch.zeros(1, 0, hk, 2, D, dtype=torch.bfloat16, device="cuda")
    O.oscar_decode_attn(sh, H.bf16_t(q), kv, H.i32_t([0]), H.u8_t(pool), H.i32_t(table), 5, 6, H.i32_t([n]), H.f32_t(U), SCALE, out, ws)
    want, mag = I.decode(f64(q), np.zeros((1, 0, hk, 2, D)), [0], pool, table, [n], U, SCALE, g, bits=2)
    check(out, want, mag)
