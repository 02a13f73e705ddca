"""NaN and infinity in the 4-bit decode: what the definition makes of them is
what comes out, whichever partial of the history or window holds them.

Expected: out = softmax(q . k) . v over a context of a NaN or +infinite logit is
NaN in every dimension; a token of logit -infinity has weight 0; a non-finite
value makes the dimensions that it enters non-finite (a stored history value
enters all of them, through R^T).  Rows that hold none of it are as without it.
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
from test_gpu_int4 import Cache, check, f64  # noqa: E402

D = 128
NAN16, INF16 = 0x7FC0, 0x7F80                              # bf16
SHAPES = [(1, 1, 32), (4, 1, 32), (16, 2, 128), (8, 2, 64)]
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def set_pair(c, b, x, kv, which, k, s=None, z=None):
    """The stored scale or zero (fp16) of group k of a history token."""
    at = int(c.table[b, x // 64]) * c.hk + kv
    pool = c.pool.reshape(c.num_pages * c.hk, -1)[at]
    w = pool[I.pair_bytes(4, c.g, which, x % 64)[k]].copy().view(np.float16)
    w[0], w[1] = w[0] if s is None else s, w[1] if z is None else z
    pool[I.pair_bytes(4, c.g, which, x % 64)[k]] = w.view(np.uint8)


def expect(c, want, nan_rows, dtype):
    """nan_rows: set of (sequence, query head) that are NaN throughout; the others as `want` of the clean cache."""
    out = c.decode(dtype=dtype)
    bad = np.zeros((c.B, c.hq), bool)
    for b, h in nan_rows:
        bad[b, h] = True
    assert out.isnan().cpu().numpy()[bad].all(), np.argwhere(bad & ~out.isnan().all(-1).cpu().numpy())
    ok = torch.from_numpy(~bad).cuda()
    assert out[ok].isfinite().all()
    ref, mag = want
    check(out[ok], ref[~bad], mag[~bad], dtype=dtype)


def heads(c, b, kv):
    G = c.hq // c.hk
    return {(b, h) for h in range(kv * G, (kv + 1) * G)}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hk,g", SHAPES)
@pytest.mark.parametrize("bad", [NAN16, INF16])
def test_a_query_with_nan_or_infinity_gives_nan_and_leaves_the_other_heads(hq, hk, g, bad, dtype):
    c = Cache(50, [10, 700, 0, 130], hq, hk, g)
    c.len[2] = 40
    want = c.want()
    rows = {(0, hq - 1), (1, 0), (2, 0)}
    for i, (b, h) in enumerate(sorted(rows)):
        c.q[b, h, 5 * i + 1] = bad
    expect(c, want, rows, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hk,g", SHAPES)
@pytest.mark.parametrize("hist", [[10, 10], [64, 640], [300, 3000]])
def test_a_nan_key_of_the_history_gives_nan(hq, hk, g, hist, dtype):
    c = Cache(51, hist + [77], hq, hk, g)
    want = c.want()
    set_pair(c, 0, 9, hk - 1, 0, 0, s=np.nan)
    set_pair(c, 1, hist[1] - 1, 0, 0, D // g - 1, z=np.nan)
    expect(c, want, heads(c, 0, hk - 1) | heads(c, 1, 0), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 10, 200])
def test_an_infinite_key_zero_gives_nan_or_drops_the_token(n, dtype):
    """z = +-infinity: the logit of a head is +infinity (its row is NaN) or
    -infinity (that token has weight 0), by the sign of its sum of q' over the group."""
    for sign in (1, -1):
        c, d = (Cache(56, [n, n, 90], 4, 1, 32) for _ in range(2))
        qsum = (f64(c.q[0]) @ oracle.get().build_R(c.U[0, 0].astype(np.float64)))[:, 32:64].sum(1)
        up = {(0, h) for h in range(4) if qsum[h] * sign > 0}
        assert (np.abs(qsum) > 1e-2).all() and 0 < len(up) < 4
        x, last = n // 2, n - 1
        set_pair(c, 0, x, 0, 0, 1, z=sign * np.inf)
        # d is without the token: the last one takes its place, one fewer
        pool = d.pool.reshape(d.num_pages, -1)
        src, dst = pool[d.table[0, last // 64]].copy(), pool[d.table[0, x // 64]]
        for w in (0, 1):
            dst[I.code_bytes(4, 32, w, x % 64)[0]] = src[I.code_bytes(4, 32, w, last % 64)[0]]
            dst[I.pair_bytes(4, 32, w, x % 64)] = src[I.pair_bytes(4, 32, w, last % 64)]
        d.hist[0] = last
        expect(c, d.want(), up, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hk,g", SHAPES)
def test_nan_rows_of_the_window(hq, hk, g, dtype):
    """A NaN key makes its KV head's rows NaN; a NaN value its own dimension
    only; a key whose logit is -infinity has weight 0."""
    for n in (1, 17, 320):
        c = Cache(53, [200, 0, 200, 64], hq, hk, g)
        c.len[:3] = n
        want = c.want()
        c.kv[0, n - 1, 0, 0, 3] = NAN16
        c.kv[1, n // 2, hk - 1, 0, 127] = NAN16
        expect(c, want, heads(c, 0, 0) | heads(c, 1, hk - 1), dtype)
        c = Cache(53, [200, 0, 200, 64], hq, hk, g)
        c.len[:3] = n
        c.kv[2, n // 2, 0, 1, 11] = NAN16
        out = c.decode(dtype=dtype).isnan().cpu().numpy()
        exp = np.zeros_like(out)
        for b, h in heads(c, 2, 0):
            exp[b, h, 11] = True
        assert np.array_equal(out, exp)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("which", ["s", "z"])
@pytest.mark.parametrize("hist", [10, 700])
def test_a_nan_value_of_the_history_reaches_every_dimension(hist, which, dtype):
    c = Cache(54, [hist, 100], 8, 2, 64)
    want = c.want()
    set_pair(c, 0, hist // 2, 1, 1, 1, **{which: np.nan})
    expect(c, want, heads(c, 0, 1), dtype)


def test_what_an_eviction_stores_for_a_nan_row_is_seen_by_the_decode():
    """A row with NaN is quantised to pairs that the decode does not lose, in a history of that row alone and among others."""
    c = Cache(55, [1, 64, 5], 4, 1, 32, extra=1)
    d = c.device()
    rng = np.random.default_rng(1)
    rows = S.bf16_bits(rng.standard_normal((3, 1, 2, D)))
    rows[0, 0, 0, 7], rows[1, 0, 0, :] = NAN16, INF16
    pos = np.array([0, 63, 4], np.int32)
    clip = torch.full((1, 2), 0.95, device="cuda")
    O.oscar_evict_quantize_int4(c.sh, H.bf16_t(rows), H.i32_t(np.arange(3)), H.i32_t(pos), d["U"], clip, d["pool"], d["table"], c.B,
                                c.max_pages, c.num_pages)
    out = c.decode()
    assert out[:2].isnan().all() and out[2].isfinite().all()


@pytest.mark.parametrize("hq,hk,g", SHAPES[1:])
def test_a_query_that_overflows_leaves_the_other_heads(hq, hk, g):
    """1e38 along a column of U_K: the rotated query passes fp32's range, to infinity or NaN."""
    c = Cache(57, [700, 20], hq, hk, g)
    for b in (0, 1):
        c.q[b, 1] = S.bf16_bits(1e38 * np.sign(c.U[0, 0, :, 5]))
    want, mag = c.want()
    keep = np.arange(hq) != 1
    out = c.decode()[:, torch.from_numpy(keep).cuda()]
    check(out, want[:, keep], mag[:, keep])


@pytest.mark.parametrize("g", [32, 128])
@pytest.mark.parametrize("per_call", [None, 7])            # tensor cores; one vector per block
def test_rows_that_are_not_finite_stand_for_no_finite_value(g, per_call):
    """Whatever codes and pairs such a vector gets, what is read back of it is NaN or
    infinite throughout, and finite of every other vector."""
    from test_gpu_int4 import evict_in_calls, kv_bits, rotation
    rng = np.random.default_rng(58)
    hk, n = 8, 300
    x = H.bf16_t(kv_bits(rng, n, hk))
    nan, inf = float("nan"), float("inf")
    bad = torch.zeros(n, hk, 2, dtype=torch.bool, device="cuda")
    for at, v in (((3, 0, 0, 5), nan), ((17,), inf), ((40, slice(None), 1, 0), -inf), ((41, 2, 0), nan), ((299, 1, 1), 3e38), ((64, 7, 0, 127), inf)):
        x[at] = v
        bad[at[:3]] = True
    table, pos, seq = np.arange(5, dtype=np.int32)[None], H.i32_t(np.arange(n)), H.i32_t(np.zeros(n))
    pool, status = evict_in_calls(x, H.f32_t(rotation(rng, hk)), torch.full((hk, 2), 0.9, device="cuda"), pos, seq, table, g, per_call)
    out = torch.zeros(n, hk, 2, D, device="cuda")
    O.oscar_history_read(O.make_shape(hk, hk, quant_group=g), 4, seq, pos, pool, H.i32_t(table), 1, 5, 5, out)
    assert status == 0
    assert torch.equal(out.isfinite().all(-1), ~bad) and torch.equal(out.isfinite().any(-1), ~bad)
