"""The 4-bit history on the GPU against the float64 oracle (oracle/int4.py):
eviction codes and pairs, decode attention, both output types, edge lengths,
bad indices, streams and captured graphs.

Tolerances, from the kernels' arithmetic:
- eviction: a rotated value is within 128^2 2^-48 sum|x u| (compensated sum)
  + 7 2^-44 |y| of the exact one, below 1e-8 code units for these scenes, so a
  code may differ only where u lies within 1e-8 of a border k + 1/2, and s or z
  only where the value before rounding lies within 1e-8 (relative) of an fp16
  midpoint;
- decode: a base-2 logit is a sum of products with q' to 22 bits, accumulated
  in fp32 with truncation: within A 2^-19, A the largest sum of absolute terms
  of a token (8 accumulations of 2^-23, q' 2^-22, the final fp32 sums 2^-21),
  so each p is off by at most 2 A 2^-19 relative to the sum; the value sums (W
  to 22 bits, fp32 accumulation over at most 2^7 steps per warp here, bf16
  window weights in 17 bits) add 2^-15 of the largest value.
"""
import numpy as np
import pytest

from bit_kv_cache_evict_gb300 import synth as S
from oracle import int4 as I

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gpu_harness as H  # noqa: E402
from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402

D = 128
SCALE = 1 / np.sqrt(D)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def rotation(rng, hk):
    return np.linalg.qr(rng.standard_normal((hk, 2, D, D)))[0].astype(np.float32)


def kv_bits(rng, *shape, outlier=20.0):
    x = rng.standard_normal((*shape, 2, D))
    x[..., [3, 77]] *= outlier
    return S.bf16_bits(x)


def f64(bits):
    return S.bf16_to_f32(bits).astype(np.float64)


class Cache:
    """A 4-bit pool with histories of the given lengths, on host and device."""

    def __init__(self, seed, hist, hq, hk, g, std=1.0, v_std=None, spare=0, extra=0):
        self.rng = rng = np.random.default_rng(seed)
        self.hq, self.hk, self.g, self.B = hq, hk, g, len(hist)
        self.hist = np.array(hist, np.int32)
        self.sh = O.make_shape(hq, hk, quant_group=g)
        need = (self.hist + extra + 63) // 64
        self.max_pages = max(1, int(need.max())) + 1
        self.num_pages = int(need.sum()) + spare + 1
        ids = rng.permutation(self.num_pages - 1)
        self.table = np.full((self.B, self.max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.spare = ids[at:]
        self.U = rotation(rng, hk)
        bb, ng = I.block_bytes(4, g), D // g
        pool = rng.integers(0, 256, (self.num_pages, hk, bb)).astype(np.uint8)
        half = 2.0 * np.array([std, std if v_std is None else v_std])
        for w, base in ((0, 4096), (1, 8192 + 256 * ng)):
            lo = -half[w] * rng.uniform(0.8, 1.2, (self.num_pages, hk, 64 * ng))
            hi = half[w] * rng.uniform(0.8, 1.2, lo.shape)
            sz = np.stack([(hi - lo) / 15, lo], -1).astype(np.float16)
            pool[:, :, base:base + 256 * ng] = sz.view(np.uint8).reshape(self.num_pages, hk, 256 * ng)
        self.pool = pool.ravel()
        self.q = S.bf16_bits(rng.standard_normal((self.B, hq, D)))
        self.kv = S.bf16_bits(rng.standard_normal((self.B, S.NSLOT, hk, 2, D)) * half[None, None, None, :, None] / 2)
        self.len = np.where(self.hist > 0, S.NSLOT, rng.integers(0, S.NSLOT + 1, self.B)).astype(np.int32)

    def poison(self):
        """NaN pairs in every slot behind the histories and in unused pages, NaN in the unused BF16 slots."""
        ng = D // self.g
        pool = self.pool.reshape(self.num_pages, self.hk, -1)
        nan = np.full(2 * ng, 0x7E00, np.uint16).view(np.uint8)
        live = np.zeros((self.num_pages, 64), bool)
        for b in range(self.B):
            for x in range(int(self.hist[b])):
                live[self.table[b, x // 64], x % 64] = True
        for p, t in zip(*np.nonzero(~live)):
            for w in (0, 1):
                pool[p][:, I.pair_bytes(4, self.g, w, t).ravel()] = nan
        for b in range(self.B):
            self.kv[b, self.len[b]:] = 0x7FC0
        return self

    def device(self):
        self.d = {k: H.i32_t(getattr(self, k)) for k in ("table", "hist", "len")}
        self.d.update(pool=H.u8_t(self.pool), U=H.f32_t(self.U), q=H.bf16_t(self.q), kv=H.bf16_t(self.kv))
        return self.d

    def decode(self, dtype=torch.float32, status=None, stream=None, out=None, ws=None, hist=None, table=None):
        d = getattr(self, "d", None) or self.device()
        if out is None:
            out = torch.full((self.B, self.hq, D), float("nan"), dtype=dtype, device="cuda")
        if ws is None:
            ws = torch.full((O.oscar_decode_workspace_bytes_int4(self.sh, self.B, self.max_pages),), 0xFF, dtype=torch.uint8,
                            device="cuda")
        t = d["table"] if table is None else table
        O.oscar_decode_attn_int4(self.sh, d["q"], d["kv"], d["len"], d["pool"], t, t.shape[1], self.num_pages,
                                 d["hist"] if hist is None else hist, d["U"], SCALE, out, ws, dev_status=status, stream=stream)
        return out

    def want(self, hist=None, table=None):
        return I.decode(f64(self.q), f64(np.where(self.kv == 0x7FC0, 0, self.kv)), self.len, self.pool,
                        self.table if table is None else table, self.hist if hist is None else hist, self.U, SCALE, self.g)


def check(out, want, mag, dtype=torch.float32):
    got = out.float().cpu().numpy().astype(np.float64)
    logit = mag[..., :1] / np.log(2)
    tol = mag[..., 1:] * (4 * logit * 2.0 ** -19 + 2.0 ** -15) + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + np.abs(want) * 2.0 ** -8
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), (err.max(), float((err / tol).max()))
    return float(np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300))


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def near_midpoint(v, got):
    """Whether the fp16 value `got` is a rounding of something within 1e-8 (relative) of v."""
    return got in (np.float16(v * (1 - 1e-8)), np.float16(v * (1 + 1e-8)))


def compare_pools(got, want, table, items, aux, hk, g):
    """Codes and pairs of the listed (row, sequence, position), with the exemptions above; every other byte equal."""
    u, sp, zp = aux
    exempt, touched = 0, []
    got, want = got.copy(), want.copy()
    for i, b, x in items:
        for h in range(hk):
            for w in (0, 1):
                cg, pg = I.raw(got, table, b, [x], h, w, hk, 4, g)
                co, po = I.raw(want, table, b, [x], h, w, hk, 4, g)
                same = np.ones(D // g, bool)
                for k in range(D // g):
                    if (pg[0, k].view(np.uint16) != po[0, k].view(np.uint16)).any():
                        assert near_midpoint(sp[i, h, w, k], pg[0, k, 0]) and near_midpoint(zp[i, h, w, k], pg[0, k, 1])
                        same[k] = False
                        exempt += g
                for j in np.nonzero(cg[0] != co[0])[0]:
                    uu = u[i, h, w, j]
                    assert not same[j // g] or abs(uu - np.floor(uu) - 0.5) < 1e-8, (b, x, h, w, j, cg[0, j], co[0, j], uu)
                    exempt += 1
                base = (int(table[b, x // 64]) * hk + h) * I.block_bytes(4, g)
                touched.append(base + I.code_bytes(4, g, w, x % 64)[0])
                touched.append(base + I.pair_bytes(4, g, w, x % 64).ravel())
    if touched:
        at = np.concatenate(touched)
        got[at] = want[at] = 0
    assert np.array_equal(got, want)                      # no stray writes
    assert exempt <= 1e-4 * len(items) * hk * 2 * D
    return exempt


@pytest.mark.parametrize("n,hk,g,clip", [(1, 1, 32, 0.95), (3, 2, 64, 1.0), (70, 4, 32, 0.9), (33, 8, 128, 0.95), (130, 2, 32, 0.5),
                                         (5, 3, 64, 0.95)])
def test_eviction_matches_the_oracle(n, hk, g, clip):
    rng = np.random.default_rng(n * 10 + hk)
    pages = (n + 63) // 64 + 1
    table = rng.permutation(pages + 2)[:pages].astype(np.int32).reshape(1, -1)
    pos = np.sort(rng.permutation(pages * 64)[:n]).astype(np.int32)
    rows, U, cl = kv_bits(rng, n, hk), rotation(rng, hk), np.full((hk, 2), clip, np.float32)
    rows[0, 0, 0] = S.bf16_bits(np.zeros(D))              # a zero vector: s = 0
    if n > 1:
        rows[1] = S.bf16_bits(f64(rows[1]) * 2.0 ** -18)  # subnormal fp16 scales
    pool = rng.integers(0, 256, (pages + 2) * hk * I.block_bytes(4, g)).astype(np.uint8)
    want = pool.copy()
    aux = I.evict(want, f64(rows), U, cl, table, np.zeros(n, int), pos, g)
    dev, status = H.u8_t(pool), torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_evict_quantize_int4(O.make_shape(hk, hk, quant_group=g), H.bf16_t(rows), H.i32_t(np.zeros(n)), H.i32_t(pos), H.f32_t(U),
                                H.f32_t(cl), dev, H.i32_t(table), 1, pages, pages + 2, dev_status=status)
    assert int(status) == 0
    compare_pools(dev.cpu().numpy(), want, table, [(i, 0, int(pos[i])) for i in range(n)], aux, hk, g)


@pytest.mark.parametrize("B_", [2, 40])
def test_eviction_appends_into_the_ring_and_skips_bad_indices(B_):
    rng = np.random.default_rng(5)
    hk, g, n = 8, 32, B_
    table = rng.permutation(n * 2).astype(np.int32).reshape(n, 2)
    kv, new, U = kv_bits(rng, n * 20, hk), kv_bits(rng, n, hk), rotation(rng, hk)
    row, pos, seq = (np.arange(n) * 20 + 7).astype(np.int32), rng.integers(0, 128, n).astype(np.int32), np.arange(n, dtype=np.int32)
    pool = rng.integers(0, 256, n * 2 * hk * I.block_bytes(4, g)).astype(np.uint8)
    bad = pos.copy()
    bad[0] = 128                                           # behind the table's row
    tb = table.copy()
    tb[1] = n * 2                                          # a page id out of range
    cl = np.full((hk, 2), 0.95, np.float32)
    want = pool.copy()
    ok = np.arange(2, n)
    aux = I.evict(want, f64(kv[row[ok]]), U, cl, table, seq[ok], pos[ok], g) if len(ok) else (None,) * 3
    dev, dkv, status = H.u8_t(pool), H.bf16_t(kv), torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_evict_quantize_int4(O.make_shape(32, hk), dkv, H.i32_t(seq), H.i32_t(bad), H.f32_t(U), H.f32_t(cl), dev, H.i32_t(tb),
                                n, 2, n * 2, src_row=H.i32_t(row), new_kv=H.bf16_t(new), dev_status=status)
    assert int(status) == O.OSCAR_STATUS_BAD_POS | O.OSCAR_STATUS_BAD_PAGE
    compare_pools(dev.cpu().numpy(), want, table, [(i, int(b), int(pos[b])) for i, b in enumerate(ok)], aux, hk, g)
    kv[row] = new                                          # the rows were read, so the new tokens are in
    assert np.array_equal(dkv.view(torch.int16).cpu().numpy().view(np.uint16), kv)


def evict_in_calls(rows, U, clip, pos, seq, table, g, per_call, src_row=None, new=None, kv=None):
    """A fresh pool after evicting the tokens `per_call` at a time (None: in one call)."""
    n, hk = len(pos), rows.shape[1]
    pages = int(table.max()) + 1
    pool = torch.full((pages * hk * I.block_bytes(4, g),), 0xA5, dtype=torch.uint8, device="cuda")
    sh, dt = O.make_shape(hk, hk, quant_group=g), H.i32_t(table)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    src = rows if kv is None else kv
    for a in range(0, n, per_call or n):
        s = slice(a, a + (per_call or n))
        part = src[s].contiguous() if src_row is None else src
        O.oscar_evict_quantize_int4(sh, part, seq[s].contiguous(), pos[s].contiguous(), U, clip, pool, dt, table.shape[0], table.shape[1], pages,
                                    src_row=None if src_row is None else src_row[s].contiguous(),
                                    new_kv=None if new is None else new[s].contiguous(), dev_status=status)
    return pool, int(status)


@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("kind", ["outliers", "flat", "scales", "offset", "grid", "wide_U"])
def test_many_tokens_at_once_give_the_same_bytes(kind, g):
    """The kernel for many tokens and the one for few agree in every byte, on
    values that put many decisions next to a border (equal values, grids,
    subnormal scales) as well."""
    hk, n = 4, 1200
    gen = torch.Generator("cuda").manual_seed(g)
    x = torch.randn(n, hk, 2, D, device="cuda", generator=gen)
    U = torch.from_numpy(rotation(np.random.default_rng(g), hk)).cuda()
    clip = torch.tensor([0.95, 1.0, 0.6, 0.99] * (hk // 2), device="cuda").reshape(hk, 2)
    if kind == "outliers":
        x[..., [5, 90]] *= 20
    elif kind == "scales":
        x *= torch.exp2(torch.randint(-40, 14, (n, 1, 1, 1), device="cuda", generator=gen).float())
        x[7], x[8, :, :, 1:] = 0.0, 0.0
    elif kind == "offset":                                 # one direction far larger than the rest: |z| over the range
        x = x * 0.01 + U.sum(-1).unsqueeze(0)
    elif kind == "grid":                                   # R^T of a few levels: ties and equal values
        x = torch.randint(-2, 3, x.shape, device="cuda", generator=gen).float()
        U = torch.eye(D, device="cuda").expand(hk, 2, D, D).contiguous()
    elif kind == "wide_U":
        U = (U * 37.5).contiguous()
    x = x.bfloat16()
    table = np.random.default_rng(1).permutation(21).astype(np.int32).reshape(1, 21)
    pos, seq = H.i32_t(np.arange(n) + 5), H.i32_t(np.zeros(n))
    few, st1 = evict_in_calls(x, U, clip, pos, seq, table, g, 31)
    many, st2 = evict_in_calls(x, U, clip, pos, seq, table, g, None)
    assert st1 == 0 and st2 == 0
    assert torch.equal(few, many), int((few != many).sum())


@pytest.mark.parametrize("n", [96, 97, 111, 112, 333])
def test_many_tokens_scattered_with_append_and_bad_indices(n):
    rng = np.random.default_rng(n)
    hk, g, pages = 24, 32, 12                              # 48 vectors a token: one call of n is bulk, calls of 13 are not
    table = rng.permutation(pages).astype(np.int32).reshape(2, 6)
    at = rng.permutation(2 * 384)[:n]
    seq, pos = (at // 384).astype(np.int32), (at % 384).astype(np.int32)
    row = rng.permutation(2 * n)[:n].astype(np.int32)
    seq[3], pos[5], row[11] = 2, 384, 2 * n                # each skipped; the third one's row is not touched either
    kv, new = kv_bits(rng, 2 * n, hk), kv_bits(rng, n, hk)
    U, clip = H.f32_t(rotation(rng, hk)), torch.full((hk, 2), 0.95, device="cuda")
    pools, states, rows = [], [], []
    for per_call in (13, None):
        dkv = H.bf16_t(kv)
        p, st = evict_in_calls(dkv, U, clip, H.i32_t(pos), H.i32_t(seq), table, g, per_call, src_row=H.i32_t(row), new=H.bf16_t(new), kv=dkv)
        pools.append(p)
        states.append(st)
        rows.append(dkv.view(torch.int16).cpu().numpy().view(np.uint16))
    assert states == [O.OSCAR_STATUS_BAD_POS] * 2
    assert torch.equal(pools[0], pools[1])
    want = kv.copy()
    ok = np.arange(n) != 11
    want[row[ok]] = new[ok]
    assert np.array_equal(rows[0], want) and np.array_equal(rows[1], want)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 300, 1025]


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (4, 1), (8, 1), (16, 2), (8, 8)])
@pytest.mark.parametrize("g", [32, 64, 128])
def test_decode_edge_lengths(hq, hk, g):
    c = Cache(hq * 100 + hk + g, LENGTHS if hk < 8 else LENGTHS[::4], hq, hk, g).poison()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.decode(status=status)
    assert int(status) == 0
    check(out, *c.want())
    bf = c.decode(dtype=torch.bfloat16)
    assert torch.equal(bf, out.bfloat16()) or (bf.float() - out).abs().max() <= (out.abs() * 2.0 ** -8 + 1e-4).max()
    check(bf, *c.want(), dtype=torch.bfloat16)


def test_decode_of_an_empty_context_is_zero():
    c = Cache(3, [0, 70], 4, 1, 32)
    c.len[:] = 0
    out = c.decode()
    assert (out[0] == 0).all()
    check(out, *c.want())


@pytest.mark.parametrize("hq,hk,g", [(4, 1, 32), (8, 1, 128)])
def test_decode_long_histories(hq, hk, g):
    """Several split-K items per sequence; a flat softmax, where the sums are far larger than the result."""
    c = Cache(11, [9000, 4097], hq, hk, g)
    c.q = S.bf16_bits(f64(c.q) * 0.05)
    c.len[:] = 320
    want, mag = c.want()
    rel = check(c.decode(), want, mag)
    assert rel < 2e-5, rel


@pytest.mark.parametrize("std,v_std", [(1.0, 1e-3), (1.0, 2e4), (1.0, 3e4), (1e-3, 1.0), (6.0, 6.0)])
@pytest.mark.filterwarnings("ignore:overflow", "ignore:invalid")
def test_decode_does_not_depend_on_the_values_size(std, v_std):
    c = Cache(13, [700, 64, 3], 4, 1, 32, std=std, v_std=v_std)
    want, mag = c.want()
    if not np.isfinite(want).all():                        # 3e4: zeros beyond fp16's 65504 are stored as infinities
        assert v_std == 3e4 and np.array_equal(np.isfinite(c.decode().cpu().numpy()), np.isfinite(want))
        return
    rel = check(c.decode(), want, mag)
    assert rel < 2e-5, rel                                 # fp16 parts scaled by a power of two: 22 bits at any size


def test_decode_with_one_huge_scale_and_equal_groups():
    c = Cache(17, [500], 4, 1, 32)
    pool = c.pool.reshape(c.num_pages, c.hk, -1)
    for x in range(0, 500, 7):                             # s = 0: every value of the group is z
        at = I.pair_bytes(4, 32, 1, x % 64)[x % 4]
        pool[c.table[0, x // 64], 0, at] = np.array([0.0, 0.5], np.float16).view(np.uint8)
    at = I.pair_bytes(4, 32, 1, 400 % 64)[2]               # the last pages see a much larger scale
    pool[c.table[0, 400 // 64], 0, at] = np.array([900.0, -7000.0], np.float16).view(np.uint8)
    check(c.decode(), *c.want())


def test_bad_pages_and_lengths_are_reported():
    c = Cache(19, [200, 500], 4, 1, 32)
    d = c.device()
    table = c.table.copy()
    table[1, 2] = c.num_pages
    table[1, 3] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.decode(status=status, table=H.i32_t(table))
    assert int(status) == O.OSCAR_STATUS_BAD_PAGE
    want, mag = c.want()
    assert np.abs(out[0].cpu().numpy() - want[0]).max() <= 1e-3   # the other sequence is untouched
    assert torch.isfinite(out).all()
    status.zero_()
    hist = c.hist.copy()
    hist[0], hist[1] = -5, 64 * c.max_pages + 1
    out = c.decode(status=status, hist=H.i32_t(hist))
    assert int(status) & O.OSCAR_STATUS_BAD_POS and torch.isfinite(out).all()
    assert d is c.d


def test_decode_on_another_stream_and_two_calls_at_once():
    a, b = Cache(21, [1000, 3000], 8, 2, 32), Cache(22, [70, 2000, 5], 8, 1, 64)
    for c in (a, b):
        c.device()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        oa = torch.zeros(a.B, a.hq, D, device="cuda")
        ob = torch.zeros(b.B, b.hq, D, dtype=torch.bfloat16, device="cuda")
        wa = torch.zeros(O.oscar_decode_workspace_bytes_int4(a.sh, a.B, a.max_pages), dtype=torch.uint8, device="cuda")
        wb = torch.zeros(O.oscar_decode_workspace_bytes_int4(b.sh, b.B, b.max_pages), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        outs.append((a.decode(stream=s1, out=oa, ws=wa), b.decode(stream=s2, out=ob, ws=wb)))
    torch.cuda.synchronize()
    for oa, ob in outs:
        check(oa, *a.want())
        check(ob, *b.want(), dtype=torch.bfloat16)


def test_step_in_a_graph_replayed_as_the_history_grows():
    """Eviction and decode captured once; each replay reads the lengths and
    rows that the arrays hold then."""
    c = Cache(23, [100, 63], 4, 1, 32, extra=10)
    d = c.device()
    rng = np.random.default_rng(1)
    rows = kv_bits(rng, 4, c.B, 1, outlier=1.0)
    src, pos = H.bf16_t(rows[0]), H.i32_t(c.hist)
    seq, clip = H.i32_t(np.arange(c.B)), torch.full((1, 2), 0.95, device="cuda")
    hist = H.i32_t(c.hist + 1)
    out = torch.zeros(c.B, c.hq, D, device="cuda")
    ws = torch.zeros(O.oscar_decode_workspace_bytes_int4(c.sh, c.B, c.max_pages), dtype=torch.uint8, device="cuda")

    def step():
        O.oscar_evict_quantize_int4(c.sh, src, seq, pos, d["U"], clip, d["pool"], d["table"], c.B, c.max_pages, c.num_pages)
        c.decode(out=out, ws=ws, hist=hist)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    now = c.hist.copy()
    for i in range(4):
        src.copy_(H.bf16_t(rows[i]))
        pos.copy_(H.i32_t(now))
        hist.copy_(H.i32_t(now + 1))
        graph.replay()
        torch.cuda.synchronize()
        I.evict(c.pool, f64(rows[i]), c.U, np.full((1, 2), 0.95, np.float32), c.table, np.arange(c.B), now, 32)
        now = now + 1
        check(out, *c.want(hist=now))


def test_every_output_row_is_written_and_nothing_else():
    c = Cache(25, [130, 0, 64], 8, 2, 32)
    room = torch.full((c.B + 2, c.hq, D), 7.0, device="cuda")
    c.decode(out=room[1:1 + c.B])
    assert (room[0] == 7).all() and (room[-1] == 7).all()
    check(room[1:1 + c.B], *c.want())


def test_zero_queries_average_the_values():
    c = Cache(27, [100, 5], 4, 1, 32)
    c.q[:] = 0
    check(c.decode(), *c.want())
    c = Cache(28, [64 * 3], 8, 1, 64)
    c.q[0, 1:] = 0                                        # one head of a KV group alone is not zero
    check(c.decode(), *c.want())


def test_eviction_then_decode_in_a_chain_without_waits():
    """Eviction, decode, compaction, decode, copies, read: launched one behind
    the other, each reading what the one before wrote."""
    c = Cache(29, [640, 300], 8, 2, 32, spare=16, extra=1)
    d = c.device()
    rows = kv_bits(c.rng, c.B, c.hk, outlier=1.0)
    clip = np.full((c.hk, 2), 0.95, np.float32)
    src, seq, pos, dclip = H.bf16_t(rows), H.i32_t(np.arange(c.B)), H.i32_t(c.hist), H.f32_t(clip)
    hist = H.i32_t(c.hist + 1)
    keeps = [np.arange(0, 641, 3), np.arange(1, 301, 2)]
    keep = np.zeros((2, 256), np.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = k
    n_keep = np.array([len(k) for k in keeps], np.int32)
    fresh = np.full((2, 4), -1, np.int32)
    fresh[0], fresh[1, :3] = c.spare[:4], c.spare[4:7]
    dk, dn, df = H.i32_t(keep), H.i32_t(n_keep), H.i32_t(fresh)
    copies = (H.i32_t(fresh[0]), H.i32_t(c.spare[8:12]))
    moved = H.i32_t(np.stack([c.spare[8:12], fresh[1]]))
    o1, o2, o3 = (torch.zeros(c.B, c.hq, D, device="cuda") for _ in range(3))
    back = torch.zeros(n_keep[0], c.hk, 2, D, device="cuda")
    ws = torch.zeros(O.oscar_decode_workspace_bytes_int4(c.sh, c.B, c.max_pages), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):                                     # (the same again changes nothing)
        O.oscar_evict_quantize_int4(c.sh, src, seq, pos, d["U"], dclip, d["pool"], d["table"], c.B, c.max_pages, c.num_pages)
        c.decode(out=o1, ws=ws, hist=hist)
        O.oscar_history_gather(c.sh, 4, d["pool"], d["table"], df, dk, dn, c.num_pages)
        c.decode(out=o2, ws=ws, hist=dn, table=df)
        O.oscar_pages_copy_device(c.hk * I.block_bytes(4, 32), *copies, [d["pool"]], c.num_pages)
        c.decode(out=o3, ws=ws, hist=dn, table=moved)
        O.oscar_history_read(c.sh, 4, H.i32_t(np.zeros(n_keep[0])), H.i32_t(np.arange(n_keep[0])), d["pool"], moved, 2, 4, c.num_pages, back)
    I.evict(c.pool, f64(rows), c.U, clip, c.table, np.arange(c.B), c.hist, 32)
    check(o1, *c.want(hist=c.hist + 1))
    c.pool = I.gather(c.pool, c.table, fresh, keep, n_keep, c.hk, 4, 32)
    check(o2, *c.want(hist=n_keep, table=fresh))
    assert (o3 - o2).abs().max() <= 1e-5 * o2.abs().max()
    ref = np.stack([np.stack([I.values(c.pool, fresh, 0, np.arange(n_keep[0]), h, w, c.hk, 4, 32) for w in (0, 1)], 1)
                    for h in range(c.hk)], 1)
    assert np.array_equal(back.cpu().numpy(), ref.astype(np.float32))


def test_queries_and_lengths_written_just_before_the_call():
    """No wait between the kernels that write q and the lengths and the call."""
    c = Cache(30, [700, 90, 1], 8, 2, 32)
    d = c.device()
    n, rng = 12, np.random.default_rng(2)
    qs = H.bf16_t(S.bf16_bits(rng.standard_normal((n, c.B, c.hq, D))))
    hists = H.i32_t(np.stack([rng.integers(0, c.hist + 1) for _ in range(n)]))
    q, hist, alone = d["q"], d["hist"], []
    ws = torch.zeros(O.oscar_decode_workspace_bytes_int4(c.sh, c.B, c.max_pages), dtype=torch.uint8, device="cuda")
    for i in range(n):
        q.copy_(qs[i])
        hist.copy_(hists[i])
        torch.cuda.synchronize()
        alone.append(c.decode(ws=ws))
        torch.cuda.synchronize()
    outs = torch.zeros(n, c.B, c.hq, D, device="cuda")
    torch.cuda.synchronize()
    for i in range(n):
        hist.copy_(hists[i])
        q.copy_(qs[i])
        c.decode(out=outs[i], ws=ws)
    assert torch.equal(outs, torch.stack(alone))


def test_two_graphs_share_a_workspace():
    a, b = Cache(31, [1500, 40], 8, 2, 32), Cache(32, [64, 900, 3], 8, 1, 128)
    need = max(O.oscar_decode_workspace_bytes_int4(c.sh, c.B, c.max_pages) for c in (a, b))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(c.B, c.hq, D, device="cuda") for c in (a, b)]
    graphs = []
    for c, o in zip((a, b), outs):
        c.device()
        c.decode(out=o, ws=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.decode(out=o, ws=ws)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
    for c, o in zip((a, b), outs):
        check(o, *c.want())


def test_eviction_and_decode_past_32_bit_offsets():
    """The same pages at the end of a pool of 4.9 GB: equal bytes and outputs."""
    c = Cache(33, [300, 77], 32, 8, 32, extra=300)
    d = c.device()
    page = c.hk * I.block_bytes(4, 32)
    pages, base = 60000, 60000 - c.num_pages
    assert base * page > 1 << 32
    big = torch.zeros(pages, page, dtype=torch.uint8, device="cuda")
    big[base:] = d["pool"].view(-1, page)
    up = H.i32_t(np.where(c.table >= 0, c.table + base, -1))
    clip = torch.full((c.hk, 2), 0.95, device="cuda")
    for n in (1, 260):                                     # one vector per block, tensor cores
        rows = H.bf16_t(kv_bits(c.rng, 2 * n, c.hk))
        seq, pos = H.i32_t(np.repeat([0, 1], n)), H.i32_t(np.concatenate([h + np.arange(n) for h in c.hist]))
        for pool, table, np_ in ((d["pool"], d["table"], c.num_pages), (big.view(-1), up, pages)):
            O.oscar_evict_quantize_int4(c.sh, rows, seq, pos, d["U"], clip, pool, table, c.B, c.max_pages, np_)
    assert torch.equal(big[base:], d["pool"].view(-1, page)) and not big[:base:997].any()
    hist = H.i32_t(c.hist + 260)
    low = c.decode(hist=hist)
    high = torch.zeros_like(low)
    ws = torch.zeros(O.oscar_decode_workspace_bytes_int4(c.sh, c.B, c.max_pages), dtype=torch.uint8, device="cuda")
    O.oscar_decode_attn_int4(c.sh, d["q"], d["kv"], d["len"], big.view(-1), up, c.max_pages, pages, hist, d["U"], SCALE, high, ws)
    assert torch.equal(low, high) and low.isfinite().all()


@pytest.mark.parametrize("hk,n", [(5, 450), (80, 40), (1, 2111)])
def test_many_tokens_with_other_counts_of_kv_heads(hk, n):
    """More (KV head, K|V) pairs than SMs, one, and a count that divides nothing."""
    rng = np.random.default_rng(hk)
    x, U = H.bf16_t(kv_bits(rng, n, hk)), H.f32_t(rotation(rng, hk))
    clip = torch.full((hk, 2), 0.9, device="cuda")
    pages = (n + 63) // 64
    table = rng.permutation(pages).astype(np.int32)[None]
    pos, seq = H.i32_t(rng.permutation(n)), H.i32_t(np.zeros(n))
    few, st1 = evict_in_calls(x, U, clip, pos, seq, table, 64, max(1, 2000 // hk))
    many, st2 = evict_in_calls(x, U, clip, pos, seq, table, 64, None)
    assert st1 == 0 and st2 == 0 and torch.equal(few, many)


def test_rows_with_nan_and_infinity_leave_the_others_alone():
    rng = np.random.default_rng(8)
    hk, n, g = 8, 300, 32
    x = H.bf16_t(kv_bits(rng, n, hk))
    U, clip = H.f32_t(rotation(rng, hk)), torch.full((hk, 2), 0.9, device="cuda")
    table, pos, seq = np.arange(5, dtype=np.int32)[None], H.i32_t(np.arange(n)), H.i32_t(np.zeros(n))
    clean, _ = evict_in_calls(x, U, clip, pos, seq, table, g, None)
    bad = [3, 17, 40, 41, 299]
    x[3, 0, 0, 5], x[17], x[40, :, 1, 0], x[41, 2, 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[299, :, :, ::2] = 3e38
    for per_call in (None, 7):
        pool, status = evict_in_calls(x, U, clip, pos, seq, table, g, per_call)
        assert status == 0
        a, b = (p.view(5, hk, -1).cpu().numpy() for p in (clean, pool))
        for t in sorted(set(range(n)) - set(bad)):
            for w in (0, 1):
                at = np.concatenate([I.pair_bytes(4, g, w, t % 64).ravel(), I.code_bytes(4, g, w, t % 64)[0]])
                assert np.array_equal(a[t // 64][:, at], b[t // 64][:, at]), (t, w)


@pytest.mark.parametrize("hq,hk,g", [(4, 1, 32), (16, 2, 128)])
def test_a_sequence_with_nan_leaves_the_others_alone(hq, hk, g):
    c = Cache(40, [500, 700, 130, 64], hq, hk, g)
    want = c.want()
    pool = c.pool.reshape(c.num_pages, hk, -1)
    nan = np.full(2 * (D // g), 0x7E00, np.uint16).view(np.uint8)
    for page in c.table[1, :3]:
        for w in (0, 1):
            pool[page][:, I.pair_bytes(4, g, w, 9).ravel()] = nan
    c.q[1, 1], c.kv[1, 7] = 0x7FC0, 0x7F80
    out = c.decode()
    keep = [0, 2, 3]
    check(out[keep], *[x[keep] for x in want])
    assert out[1].isnan().any()


def test_many_tokens_from_rows_at_an_eight_byte_address():
    rng = np.random.default_rng(41)
    hk, n = 8, 280
    x, U = H.bf16_t(kv_bits(rng, n, hk)), H.f32_t(rotation(rng, hk))
    moved = torch.zeros(x.numel() + 4, dtype=torch.bfloat16, device="cuda")[4:].view(x.shape)
    moved.copy_(x)
    assert moved.data_ptr() % 16 == 8
    clip = torch.full((hk, 2), 0.9, device="cuda")
    table, pos, seq = np.arange(5, dtype=np.int32)[None], H.i32_t(np.arange(n)), H.i32_t(np.zeros(n))
    a, _ = evict_in_calls(x, U, clip, pos, seq, table, 32, None)
    b, status = evict_in_calls(moved, U, clip, pos, seq, table, 32, None)
    assert status == 0 and torch.equal(a, b)
