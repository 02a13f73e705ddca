"""Stored tokens read, gathered and copied on the GPU against the oracle: the
values are single roundings and the moves are byte copies, so everything is
compared for equality.  The last test runs the 4-bit calls together."""
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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def random_pool(rng, pages, hk, bits, g):
    """Random codes, random finite pairs."""
    ng = D // g
    pool = rng.integers(0, 256, (pages, hk, I.block_bytes(bits, g))).astype(np.uint8)
    for w in (0, 1):
        at = int(I.pair_bytes(bits, g, w, 0)[0, 0])
        sz = rng.standard_normal((pages, hk, 128 * ng)).astype(np.float16) * np.float16(3)
        pool[:, :, at:at + 256 * ng] = sz.view(np.uint8)
    return pool.ravel()


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("g,hk,n", [(32, 1, 1), (64, 3, 63), (128, 2, 65), (32, 8, 200)])
def test_read_is_exact(bits, g, hk, n):
    rng = np.random.default_rng(n + bits)
    pool, table = random_pool(rng, 9, hk, bits, g), rng.permutation(9)[:8].astype(np.int32).reshape(2, 4)
    seq, pos = rng.integers(0, 2, n).astype(np.int32), rng.integers(0, 256, n).astype(np.int32)
    if n > 100:                                            # runs inside and across pages, from any slot
        pos[:100], seq[:100] = np.arange(61, 161), 1
    want = np.zeros((n, hk, 2, D))
    for i in range(n):
        for h in range(hk):
            for w in (0, 1):
                want[i, h, w] = I.values(pool, table, seq[i], pos[i:i + 1], h, w, hk, bits, g)[0]
    sh, status = O.make_shape(hk, hk, quant_group=g), torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((n + 1, hk, 2, D), 7.0, dtype=dtype, device="cuda")
        O.oscar_history_read(sh, bits, H.i32_t(seq), H.i32_t(pos), H.u8_t(pool), H.i32_t(table), 2, 4, 9, out, dev_status=status)
        ref = torch.from_numpy(want).cuda()
        # s c is exact in fp32 and one addition rounds: the fp32 value of the exact sum
        assert torch.equal(out[:n], ref.float().to(dtype)) and (out[n] == 7).all()
    assert int(status) == 0


@pytest.mark.parametrize("bits", [2, 4])
def test_read_leaves_rows_of_bad_tokens(bits):
    rng = np.random.default_rng(2)
    pool, table = random_pool(rng, 3, 2, bits, 32), np.array([[0, 9], [-1, 2]], np.int32)
    seq = np.array([0, 2, -1, 0, 0, 1, 1, 1], np.int32)
    pos = np.array([5, 5, 5, 128, 64, 3, -1, 70], np.int32)
    ok = np.array([1, 0, 0, 0, 0, 0, 0, 1], bool)
    out, status = torch.full((8, 2, 2, D), 7.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_history_read(O.make_shape(2, 2), bits, H.i32_t(seq), H.i32_t(pos), H.u8_t(pool), H.i32_t(table), 2, 2, 3, out,
                         dev_status=status)
    assert int(status) == O.OSCAR_STATUS_BAD_POS | O.OSCAR_STATUS_BAD_PAGE
    out = out.cpu().numpy()
    assert (out[~ok] == 7).all()
    for i in np.nonzero(ok)[0]:
        for h in range(2):
            for w in (0, 1):
                want = I.values(pool, table, seq[i], pos[i:i + 1], h, w, 2, bits, 32)[0]
                assert np.array_equal(out[i, h, w], want.astype(np.float32))


@pytest.mark.parametrize("bits,g,hk,boost", [(2, 32, 2, True), (2, 64, 1, False), (2, 128, 3, True), (4, 32, 2, False),
                                              (4, 64, 1, False), (4, 128, 3, False)])
def test_gather_moves_the_kept_tokens(bits, g, hk, boost):
    rng = np.random.default_rng(bits + g + hk)
    hist = [300, 64, 1, 129]
    need = [(h + 63) // 64 for h in hist]
    keeps = [np.sort(rng.permutation(300)[:131]), np.arange(64), np.zeros(0, int), np.array([128, 5, 5, 64, 127])]
    fresh = [3, 1, 1, 1]
    pages = sum(need) + sum(fresh) + 2
    ids = rng.permutation(pages)
    src, dst = np.full((4, 5), -1, np.int32), np.full((4, 3), -1, np.int32)
    at = 0
    for t, counts in ((src, need), (dst, fresh)):
        for b, n in enumerate(counts):
            t[b, :n] = ids[at:at + n]
            at += n
    keep = np.full((4, 140), -1, np.int32)                 # what lies behind a row's list is not read
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = k
    n_keep = np.array([len(k) for k in keeps], np.int32)
    pool = random_pool(rng, pages, hk, bits, g)
    rec = rng.integers(0, 256, pages * hk * O.BOOST_BLOCK_BYTES).astype(np.uint8)
    want = I.gather(pool, src, dst, keep, n_keep, hk, bits, g)
    wrec = rec.copy().reshape(pages, hk, 64, 16)
    for b, k in enumerate(keeps):
        for i, x in enumerate(k):
            wrec[dst[b, i // 64], :, i % 64] = rec.reshape(pages, hk, 64, 16)[src[b, x // 64], :, x % 64]
    dev, drec, status = H.u8_t(pool), H.u8_t(rec), torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_history_gather(O.make_shape(hk, hk, quant_group=g), bits, dev, H.i32_t(src), H.i32_t(dst), H.i32_t(keep),
                           H.i32_t(n_keep), pages, boost=drec if boost else None, dev_status=status)
    assert int(status) == 0
    assert np.array_equal(dev.cpu().numpy(), want)
    assert np.array_equal(drec.cpu().numpy(), wrec.ravel() if boost else rec)


@pytest.mark.parametrize("bits", [2, 4])
def test_gather_skips_and_reports_bad_entries(bits):
    rng = np.random.default_rng(9)
    pool = random_pool(rng, 6, 1, bits, 32)
    src = np.array([[0, 7], [1, 2]], np.int32)             # page 7 does not exist
    dst = np.array([[3, 4], [5, -1]], np.int32)
    keep = np.array([[3, 64, -1, 128, 9, 10, 11, 12] + [0] * 62, list(range(70))], np.int32)
    n_keep = np.array([8, 70], np.int32)                   # row 1: tokens 64.. would go to page -1
    want = pool.copy()
    ok = [(0, i, x) for i, x in enumerate(keep[0][:8]) if x in (3, 9, 10, 11, 12)]
    for b, i, x in ok:
        k = np.zeros((2, 8), int)
        k[0, i] = x
        one = I.gather(want, src, np.array([[3], [5]]), k, [i + 1, 0], 1, bits, 32)
        for w in (0, 1):                                   # slot i of page 3 only
            base = 3 * I.block_bytes(bits, 32)
            a = np.concatenate([base + np.unique(I.code_bytes(bits, 32, w, i)[0]), base + I.pair_bytes(bits, 32, w, i).ravel()])
            want[a] = one[a]
    want = I.gather(want, src, dst, keep, [0, 64], 1, bits, 32)
    dev, status = H.u8_t(pool), torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_history_gather(O.make_shape(1, 1), bits, dev, H.i32_t(src), H.i32_t(dst), H.i32_t(keep), H.i32_t(n_keep), 6,
                           dev_status=status)
    assert int(status) == O.OSCAR_STATUS_BAD_POS | O.OSCAR_STATUS_BAD_PAGE
    assert np.array_equal(dev.cpu().numpy(), want)
    status.zero_()
    O.oscar_history_gather(O.make_shape(1, 1), bits, dev, H.i32_t(src), H.i32_t(dst), H.i32_t(keep), H.i32_t([-1, 200]), 6,
                           dev_status=status)              # lengths outside the lists: none, and all that fit
    assert int(status) & O.OSCAR_STATUS_BAD_POS
    assert np.array_equal(dev.cpu().numpy(), I.gather(want, src, dst, keep, [0, 64], 1, bits, 32))


@pytest.mark.parametrize("page_bytes,n,n_pools", [(16, 1, 1), (6144, 3, 2), (81920, 5, 36), (10240 + 16, 40, 1), (16400, 2, 128)])
def test_pages_copy(page_bytes, n, n_pools):
    rng = np.random.default_rng(n)
    pages = 2 * n + 3
    ids = rng.permutation(pages).astype(np.int32)
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    pools = [rng.integers(0, 256, pages * page_bytes).astype(np.uint8) for _ in range(n_pools)]
    dev, status = [H.u8_t(p) for p in pools], torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_pages_copy_device(page_bytes, H.i32_t(src), H.i32_t(dst), dev, pages, dev_status=status)
    assert int(status) == 0
    for p, q in zip(pools, dev):
        p = p.reshape(pages, page_bytes)
        p[dst] = p[src]
        assert np.array_equal(q.cpu().numpy(), p.ravel())


def test_pages_copy_reports_bad_pages_and_keeps_equal_ones():
    pool = torch.arange(4 * 64, device="cuda").to(torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = pool.clone()
    want[192:256] = want[0:64]
    O.oscar_pages_copy_device(64, H.i32_t([-1, 1, 0, 2, 4]), H.i32_t([1, 4, 3, 2, 1]), [pool], 4, dev_status=status)
    assert int(status) == O.OSCAR_STATUS_BAD_PAGE and torch.equal(pool, want)


def test_copies_in_a_graph_follow_the_index_arrays():
    pool = torch.randint(0, 256, (6, 256), dtype=torch.uint8, device="cuda")
    src, dst = H.i32_t([0, 1]), H.i32_t([4, 5])
    O.oscar_pages_copy_device(256, src, dst, [pool], 6)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        O.oscar_pages_copy_device(256, src, dst, [pool], 6)
    src.copy_(H.i32_t([2, 3]))
    dst.copy_(H.i32_t([0, 5]))
    want = pool.clone()
    want[0], want[5] = pool[2], pool[3]
    g.replay()
    assert torch.equal(pool, want)


def test_prompt_fork_compaction_and_decode_together():
    """A prompt's history quantised in one call, read back; a second sequence
    forks it inside a page (copy-on-write plan of the host allocator, one
    launch for two layers' pools) and goes on with its own tokens; then both
    are compacted to a part of their tokens and decoded: equal to the oracle's
    attention over the kept tokens."""
    rng = np.random.default_rng(31)
    hq, hk, g, n0, own = 8, 2, 32, 200, 50
    sh = O.make_shape(hq, hk, quant_group=g)
    pages, mp = 24, 5
    P = O.Pages(pages)
    U = np.linalg.qr(rng.standard_normal((hk, 2, D, D)))[0].astype(np.float32)
    clip = np.full((hk, 2), 0.97, np.float32)
    toks = [S.bf16_bits(rng.standard_normal((n, hk, 2, D))) for n in (n0, own, own)]
    f = lambda bits: S.bf16_to_f32(bits).astype(np.float64)  # noqa: E731
    table = np.full((2, mp), -1, np.int32)
    pool = torch.zeros(pages * hk * O.block_bytes_int4(sh), dtype=torch.uint8, device="cuda")
    other = torch.zeros_like(pool)                         # a second layer with the same page table
    want = np.zeros(pool.numel(), np.uint8)
    dU, dclip = H.f32_t(U), H.f32_t(clip)

    def evict(bits, seq, pos):
        src, dst = P.prepare_write(seq, pos // 64, table)
        if src.size:
            O.oscar_pages_copy_device(hk * O.block_bytes_int4(sh), H.i32_t(src), H.i32_t(dst), [pool, other], pages)
            v = want.reshape(pages, -1)
            v[dst] = v[src]
        for p in (pool, other):
            O.oscar_evict_quantize_int4(sh, H.bf16_t(bits), H.i32_t(seq), H.i32_t(pos), dU, dclip, p, H.i32_t(table), 2, mp, pages)
        I.evict(want, f(bits), U, clip, table, seq, pos, g)

    evict(toks[0], np.zeros(n0, np.int32), np.arange(n0, dtype=np.int32))
    rows = torch.empty(n0, hk, 2, D, device="cuda")
    O.oscar_history_read(sh, 4, H.i32_t(np.zeros(n0)), H.i32_t(np.arange(n0)), pool, H.i32_t(table), 2, mp, pages, rows)
    ref = np.stack([np.stack([I.values(want, table, 0, np.arange(n0), h, w, hk, 4, g) for w in (0, 1)], 1) for h in range(hk)], 1)
    assert np.array_equal(rows.cpu().numpy(), ref.astype(np.float32))
    table[1] = table[0]                                     # the fork: shared pages, one more reference each
    P.retain(table[0][table[0] >= 0])
    for s in (0, 1):
        evict(toks[1 + s], np.full(own, s, np.int32), np.arange(n0, n0 + own, dtype=np.int32))
    assert torch.equal(pool, other) and np.array_equal(pool.cpu().numpy(), want)

    keeps = [np.sort(rng.permutation(n0 + own)[:n]) for n in (131, 64)]
    keep = np.zeros((2, 140), np.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = k
    n_keep = np.array([131, 64], np.int32)
    fresh = np.full((2, mp), -1, np.int32)
    fresh[0, :3], fresh[1, :1] = P.alloc(3), P.alloc(1)
    O.oscar_history_gather(sh, 4, pool, H.i32_t(table), H.i32_t(fresh), H.i32_t(keep), H.i32_t(n_keep), pages)
    before, free = want.copy(), P.free_count()
    for b in (0, 1):
        P.release(table[b][table[b] >= 0])
    assert P.free_count() > free
    kv, q = S.bf16_bits(rng.standard_normal((2, S.NSLOT, hk, 2, D))), S.bf16_bits(rng.standard_normal((2, hq, D)))
    out = torch.empty(2, hq, D, device="cuda")
    ws = torch.empty(O.oscar_decode_workspace_bytes_int4(sh, 2, mp), dtype=torch.uint8, device="cuda")
    O.oscar_decode_attn_int4(sh, H.bf16_t(q), H.bf16_t(kv), H.i32_t([320, 320]), pool, H.i32_t(fresh), mp, pages, H.i32_t(n_keep),
                             dU, 1 / np.sqrt(D), out, ws)
    kept = I.gather(before, table, fresh, keep, n_keep, hk, 4, g)
    ref, mag = I.decode(f(q), f(kv), [320, 320], kept, fresh, n_keep, U, 1 / np.sqrt(D), g)
    tol = mag[..., 1:] * (4 * mag[..., :1] / np.log(2) * 2.0 ** -19 + 2.0 ** -15)
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("bits", [2, 4])
def test_offsets_past_32_bits(bits):
    """Reads, compaction and copies at the end of a pool of 4.9 GB."""
    hk, g, n, rng = 8, 32, 10, np.random.default_rng(bits)
    page = hk * I.block_bytes(bits, g)
    pages = 4_900_000_000 // page
    base = pages - n
    assert base * page > 1 << 32
    sh, small = O.make_shape(hk, hk, quant_group=g), H.u8_t(random_pool(rng, n, hk, bits, g))
    big = torch.zeros(pages, page, dtype=torch.uint8, device="cuda")
    big[base:] = small.view(n, page)
    src, dst = np.array([[3, 1, 4]], np.int32), np.array([[0, 5]], np.int32)
    keep = np.sort(rng.permutation(192)[:100]).astype(np.int32)[None]
    pos = rng.permutation(192).astype(np.int32)
    outs = []
    for pool, up, np_ in ((small, 0, n), (big.view(-1), base, pages)):
        out = torch.zeros(192, hk, 2, D, device="cuda")
        O.oscar_history_read(sh, bits, H.i32_t(np.zeros(192)), H.i32_t(pos), pool, H.i32_t(src + up), 1, 3, np_, out)
        O.oscar_history_gather(sh, bits, pool, H.i32_t(src + up), H.i32_t(dst + up), H.i32_t(keep), H.i32_t([100]), np_)
        O.oscar_pages_copy_device(page, H.i32_t([1 + up, 2 + up]), H.i32_t([8 + up, 9 + up]), [pool], np_)
        outs.append(out)
    assert torch.equal(*outs) and outs[0].any()
    assert torch.equal(big[base:], small.view(n, page)) and not big[:base:997].any()


def test_all_calls_on_a_side_stream():
    """Each call given a stream orders with what that stream does, not the current one."""
    rng = np.random.default_rng(5)
    hk, g, n = 2, 32, 6
    sh, page = O.make_shape(hk, hk, quant_group=g), hk * I.block_bytes(4, g)
    host = random_pool(rng, n, hk, 4, g)
    src, dst, keep, nk = H.i32_t([[0, 1]]), H.i32_t([[2, 3]]), H.i32_t(np.arange(0, 128, 2)[None]), H.i32_t([64])
    zero, pos, cs, cd = H.i32_t(np.zeros(64)), H.i32_t(np.arange(64)), H.i32_t([2]), H.i32_t([5])
    held, moved = H.u8_t(host), H.i32_t([[5, -1]])
    pool, out = torch.zeros_like(held), torch.zeros(64, hk, 2, D, device="cuda")
    big = torch.zeros(1 << 28, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(8):
            big.add_(1)                                    # keeps the side stream busy before the pool is filled
        pool.copy_(held)
    O.oscar_history_gather(sh, 4, pool, src, dst, keep, nk, n, stream=st)
    O.oscar_pages_copy_device(page, cs, cd, [pool], n, stream=st)
    O.oscar_history_read(sh, 4, zero, pos, pool, moved, 1, 2, n, out, stream=st)
    st.synchronize()
    ref = np.stack([np.stack([I.values(host, np.array([[0, 1]]), 0, np.arange(0, 128, 2), h, w, hk, 4, g) for w in (0, 1)], 1)
                    for h in range(hk)], 1)
    assert np.array_equal(out.cpu().numpy(), ref.astype(np.float32))
