"""The bound that the bulk 4-bit eviction (csrc/evict_bulk.cu) puts on its
tensor-core product y = x . R: a decision is retaken from exact sums only where
an error of that size could change it, so no product may be further off.

The bound follows from how one MMA adds: the sixteen products and the
accumulator are exact, are aligned to the largest of them, cut off there, added, and
the sum is cut off to 24 bits.  With u = 2^-23 of the largest addend each of
them loses at most u / 4 (two bits more than fp32's 24 are kept) and the result at most
u of itself: checked here on single MMAs, then the whole product on rows made to
lose the most, and the stored bytes of those rows.
"""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest

from bit_kv_cache_evict_gb300 import synth as S

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gpu_harness as H  # noqa: E402
import oracle  # noqa: E402
from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from oracle import int4 as I  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))
D = 128


@pytest.fixture(scope="module")
def probe():
    out = os.path.join(tempfile.mkdtemp(), "bulk_product.so")
    subprocess.run([B.nvcc_path(), *B.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-cudart",
                    "shared", os.path.join(HERE, "cuda", "bulk_product.cu"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.run_product.argtypes = [ctypes.c_int, ctypes.c_int] + [ctypes.c_void_p] * 4
    lib.run_sums.argtypes = [ctypes.c_int] + [ctypes.c_void_p] * 4
    return lib


def sums(probe, a, b, c):
    """One MMA's c + sum a b, and the exact sum and the exact addends, for rows of 16."""
    a, b, c = np.float16(a), np.float16(b), np.float32(c)
    ta, tb, tc = (torch.from_numpy(v).cuda() for v in (a, b, c))
    d = torch.zeros(len(c), device="cuda")
    assert probe.run_sums(len(c), *(t.data_ptr() for t in (ta, tb, tc, d))) == 0
    terms = np.concatenate([a.astype(np.float64) * b.astype(np.float64), c.astype(np.float64)[:, None]], 1)
    return d.cpu().numpy().astype(np.float64), terms


def test_one_mma_keeps_two_bits_more_than_fp32_of_every_addend(probe):
    rng = np.random.default_rng(0)
    rows = []
    for _ in range(40000):                                 # one large addend of either kind, the others around its last bits
        top, big = rng.uniform(1, 2), rng.integers(0, 17)
        scale = 2.0 ** -rng.uniform(18, 28) if rng.random() < 0.8 else 2.0 ** -rng.uniform(0, 12, 16)
        prod = top * scale * rng.uniform(1, 2, 16) * (1 if rng.random() < 0.7 else rng.choice([-1.0, 1.0], 16))
        a = 2.0 ** np.clip(np.floor(np.log2(np.abs(prod))) / 2, -14, 0).round()   # (both factors stay normal fp16 values)
        b = prod / a
        c = top * rng.uniform(1, 2) * 2.0 ** -rng.uniform(0, 26) * rng.choice([-1.0, 1.0])
        if big == 16:
            c = top * rng.choice([-1.0, 1.0])
        else:
            a[big], b[big] = 1.0, top
        rows.append((a, b, c))
    d, terms = sums(probe, *(np.stack([r[i] for r in rows]) for i in range(3)))
    most, exact = np.abs(terms).max(1), terms.sum(1)
    lost = np.abs(d - exact)
    ratio = lost / (2.0 ** -23 * (17 / 4 * most + np.abs(exact)))
    print("single MMAs: largest loss / bound %.3f" % ratio.max())
    assert ratio.max() <= 1.0


def matrices():
    """Orthogonal ones, as a calibration gives; times 37.5; a signed permutation; and one
    whose R is close to a permutation, so that one channel is nearly all of a column."""
    rng = np.random.default_rng(3)
    U = np.linalg.qr(rng.standard_normal((2, D, D)))[0]
    perm = np.eye(D)[rng.permutation(D)] * rng.choice([-1.0, 1.0], D)
    turn = np.linalg.qr(np.eye(D) + 0.01 * rng.standard_normal((D, D)))[0]
    H = oracle.get().build_R(np.eye(D))
    return np.stack([U[0], U[1] * 37.5, perm, turn @ H.T]).astype(np.float32)


def rows_for(R, rng, n):
    """Rows for one matrix R: random ones, with outlier channels, along R's columns, and one
    dominant channel with 127 whose products with a column all lie near the
    last bits of the dominant one's, with its sign."""
    cols = R[:, np.arange(n) % D].T
    kinds = [rng.standard_normal((n, D)), rng.standard_normal((n, D)), cols * np.exp2(rng.uniform(-3, 3, (n, 1))), np.sign(cols)]
    kinds[1][:, [5, 90]] *= 300
    for part in (1, 4, 16, 64):                            # the small products' spread inside a row
        c = np.exp2(rng.uniform(-29, -20, (n, 1))) * rng.uniform(1 / part, 1, (n, D))
        at = rng.integers(0, D, n)
        i = np.arange(n)
        for a in (at, np.zeros(n, int)):                   # the dominant channel anywhere; in the first step, so that every later one adds to it
            x = c * cols[i, a][:, None] / np.where(np.abs(cols) < 1e-4, np.inf, cols)
            x[i, a] = 1.0
            kinds.append(x)
    return S.bf16_bits(np.concatenate(kinds))


def test_no_product_is_further_off_than_its_bound(probe):
    U, rng, n = matrices(), np.random.default_rng(5), 1024
    R = [oracle.get().build_R(u.astype(np.float64)) for u in U]
    x = np.stack([rows_for(r, rng, n) for r in R])
    x = x[:, :x.shape[1] // 16 * 16]
    tx, tU = H.bf16_t(x), H.f32_t(U)
    y, bound = torch.zeros(x.shape, device="cuda"), torch.zeros(x.shape[:2], device="cuda")
    assert probe.run_product(len(U), x.shape[1] // 16, *(t.data_ptr() for t in (tU, tx, y, bound))) == 0
    y, bound = y.cpu().numpy().astype(np.float64), bound.cpu().numpy().astype(np.float64)
    f = S.bf16_to_f32(x).astype(np.float64)
    for m, r in enumerate(R):
        ratio = np.abs(y[m] - f[m] @ r).max(1) / bound[m]
        kinds = ratio.reshape(-1, n).max(1)
        print("matrix %d: largest error / bound by kind of row: %s" % (m, " ".join("%.3f" % k for k in kinds)))
        assert kinds.max() <= 1.0
        # the bound is no larger than it says: 1.6 2^-20 |x| of the largest column
        assert (bound[m] <= 2.0 * 2.0 ** -20 * np.linalg.norm(f[m], axis=1) * np.linalg.norm(r, axis=0).max()).all()


@pytest.mark.parametrize("g", [32, 64, 128])
def test_those_rows_are_stored_as_by_the_kernel_for_few_tokens(g):
    from test_gpu_int4 import evict_in_calls
    U, rng = matrices(), np.random.default_rng(6)
    x = np.stack([rows_for(oracle.get().build_R(u.astype(np.float64)), rng, 400) for u in U], 1)
    n = len(x)
    assert 4 * n >= 4096
    rows, dU = H.bf16_t(x.reshape(n, 2, 2, D)), H.f32_t(U.reshape(2, 2, D, D))
    clip = torch.tensor([[0.95, 1.0], [0.9, 0.6]], device="cuda")
    table = rng.permutation((n + 63) // 64).astype(np.int32)[None]
    pos, seq = H.i32_t(np.arange(n)), H.i32_t(np.zeros(n))
    few, st1 = evict_in_calls(rows, dU, clip, pos, seq, table, g, 1000)
    many, st2 = evict_in_calls(rows, dU, clip, pos, seq, table, g, None)
    assert st1 == 0 and st2 == 0
    # A row along a column of a permutation's R has rotated values that are exactly 0.  Both kernels decide
    # from values within 2^-36 |x| of the exact ones, so either sign of a zero z is such a value's rounding: 0 and
    # -0 count as the same there.
    for pool in (few, many):
        blocks = pool.view(-1, I.block_bytes(4, g))
        for w in (0, 1):
            at = int(I.pair_bytes(4, g, w, 0)[0, 0])
            pairs = blocks[:, at:at + 256 * (D // g)].contiguous().view(torch.int16)
            pairs[pairs == -32768] = 0
            blocks[:, at:at + 256 * (D // g)] = pairs.view(torch.uint8)
    assert torch.equal(few, many), int((few != many).sum())
