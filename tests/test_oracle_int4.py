"""Pins of the 4-bit oracle (oracle/int4.py): its layout covers every byte
once, on-grid values come back exactly, the quantiser's error bound, and its
attention against a direct softmax."""
import numpy as np
import pytest

import oracle
from oracle import int4 as I

D = 128


@pytest.mark.parametrize("g", [32, 64, 128])
def test_layout_covers_a_block_once(g):
    used = np.zeros(I.block_bytes(4, g) * 2, np.int64)      # nibbles
    for w in (0, 1):
        for t in range(64):
            at, shift = I.code_bytes(4, g, w, t)
            np.add.at(used, 2 * at + shift // 4, 1)
            p = I.pair_bytes(4, g, w, t).ravel()
            used[2 * p] += 1
            used[2 * p + 1] += 1
    assert (used == 1).all()


def test_layout_of_hand_computed_positions():
    # K: position 77 = group block 2, index 13: a = 1, i = 2, high nibble
    at, shift = I.code_bytes(4, 32, 0, 5)
    assert at[77] == 5 * 64 + 16 * 1 + 4 * 2 + 2 and shift[77] == 4
    at, shift = I.code_bytes(4, 32, 1, 5)
    assert at[77] == 4096 + 1024 + 38 * 64 + 5 and shift[77] == 4 and at[76] == at[77] and shift[76] == 0
    assert I.block_bytes(4, 32) == 10240 and I.block_bytes(4, 64) == 9216 and I.block_bytes(4, 128) == 8704


@pytest.mark.parametrize("g", [32, 64, 128])
def test_on_grid_values_come_back(g):
    rng = np.random.default_rng(3)
    c = rng.integers(0, 16, D)
    c[::g], c[1::g] = 0, 15
    codes, s, z, u, _, _ = I.quantize(c * 0.25 - 1.5, g, 1.0)
    assert np.array_equal(codes, c) and (s == 0.25).all() and (z == -1.5).all() and np.array_equal(u, c)


def test_error_is_at_most_half_a_step_plus_the_rounding_of_s_and_z():
    rng = np.random.default_rng(4)
    for g in (32, 64, 128):
        for clip in (0.8, 1.0):
            y = rng.standard_normal(D) * 3
            codes, s, z, u, sp, zp = I.quantize(y, g, clip)
            sr, zr = np.repeat(s.astype(float), g), np.repeat(z.astype(float), g)
            t = np.repeat(clip * np.abs(y.reshape(-1, g)).max(1), g)
            y = np.clip(y, -t, t) if clip < 1 else y
            # s and z are each within half an fp16 step: 15 s and z move by 15 s 2^-11 and |z| 2^-11
            assert (np.abs(codes * sr + zr - y) <= sr / 2 + 2.0 ** -11 * (15 * sr + np.abs(zr))).all()


def test_equal_values_give_codes_zero():
    codes, s, z, u, _, _ = I.quantize(np.full(D, 0.75), 32, 0.9)
    assert (codes == 0).all() and (s == 0).all() and (z == np.float16(0.675)).all() and (u == 0).all()


def test_store_and_values_round_trip():
    rng = np.random.default_rng(5)
    hk, g = 2, 64
    pool = rng.integers(0, 256, 3 * hk * I.block_bytes(4, g)).astype(np.uint8)
    before = pool.copy()
    table = np.array([[2, 0]])
    codes = rng.integers(0, 16, D).astype(np.uint8)
    s, z = np.array([0.5, 2.0], np.float16), np.array([-1.0, 3.0], np.float16)
    I.store(pool, 0 * hk + 1, g, 1, 9, codes, s, z)
    v = I.values(pool, table, 0, [64 + 9], 1, 1, hk, 4, g)[0]
    assert np.array_equal(v, codes * np.repeat([0.5, 2.0], 64) + np.repeat([-1.0, 3.0], 64))
    assert (pool != before).sum() <= 64 + 8


def test_two_bit_values_match_the_c_oracle():
    orc = oracle.get()
    rng = np.random.default_rng(6)
    hk, g = 1, 32
    sh = oracle.Shape(D, g, 64, 256, 64, 1, 1)
    pool = np.zeros(2 * hk * I.block_bytes(2, g), np.uint8)
    table = np.array([[1, 0]], np.int32)
    rows = rng.standard_normal((3, hk, 2, D))
    bits = (np.float32(rows).view(np.uint32) >> 16).astype(np.uint16)
    U = np.linalg.qr(rng.standard_normal((hk, 2, D, D)))[0]
    pos = np.array([0, 63, 64], np.int32)
    orc.evict(sh, bits, np.zeros(3, np.int32), pos, U, np.full((hk, 2), 0.9), pool, table, 2)
    for i in range(3):
        for w in (0, 1):
            y = orc.f64_from_bf16(bits[i, 0, w]) @ orc.build_R(U[0, w])
            codes, s, z = orc.quantize_vec(y, g, 0.9)[:3]
            want = orc.dequantize_vec(codes, s, z, g)
            assert np.array_equal(I.values(pool, table, 0, [pos[i]], 0, w, hk, 2, g)[0], want)


def test_decode_is_softmax_over_the_concatenation():
    rng = np.random.default_rng(7)
    hk, g, n, m = 1, 32, 70, 5
    U = np.linalg.qr(rng.standard_normal((hk, 2, D, D)))[0]
    pool = np.zeros(2 * hk * I.block_bytes(4, g), np.uint8)
    table = np.array([[1, 0]], np.int32)
    rows = rng.standard_normal((n, hk, 2, D))
    I.evict(pool, rows, U, np.ones((hk, 2)), table, np.zeros(n, int), np.arange(n), g)
    kv, q = rng.standard_normal((1, 8, hk, 2, D)), rng.standard_normal((1, 2, D))
    out, _ = I.decode(q, kv, [m], pool, table, [n], U, 0.1, g)
    # 4-bit errors are at most half a step of about 4 / 15 per rotated value: near attention over the rows themselves
    k, v = np.concatenate([rows[:, 0, 0], kv[0, :m, 0, 0]]), np.concatenate([rows[:, 0, 1], kv[0, :m, 0, 1]])
    for h in range(2):
        p = np.exp(0.1 * k @ q[0, h])
        assert np.abs(out[0, h] - p @ v / p.sum()).max() < 0.2
    assert (I.decode(q, kv, [0], pool, table, [0], U, 0.1, g)[0] == 0).all()


def test_gather_moves_whole_vectors():
    rng = np.random.default_rng(8)
    for bits, g in ((2, 64), (4, 128)):
        hk = 2
        pool = rng.integers(0, 256, 4 * hk * I.block_bytes(bits, g)).astype(np.uint8)
        src, dst = np.array([[3, 0]]), np.array([[1]])
        keep = np.array([[70, 3, 3, 64]])
        out = I.gather(pool, src, dst, keep, [4], hk, bits, g)
        for h in range(hk):
            for w in (0, 1):
                a, b = I.raw(pool, src, 0, keep[0], h, w, hk, bits, g), I.raw(out, dst, 0, np.arange(4), h, w, hk, bits, g)
                assert np.array_equal(a[0], b[0]) and np.array_equal(a[1].view(np.uint16), b[1].view(np.uint16))
        bb = hk * I.block_bytes(bits, g)
        same = np.ones(4, bool)
        same[1] = False
        assert np.array_equal(out.reshape(4, bb)[same], pool.reshape(4, bb)[same])


def test_decode_of_the_window_alone_is_exact():
    rng = np.random.default_rng(9)
    hk, g, m = 2, 32, 6
    U = np.linalg.qr(rng.standard_normal((hk, 2, D, D)))[0]
    kv, q = rng.standard_normal((1, 8, hk, 2, D)), rng.standard_normal((1, 4, D))
    out, _ = I.decode(q, kv, [m], np.zeros(hk * I.block_bytes(4, g), np.uint8), np.array([[0]]), [0], U, 0.3, g)
    for h in range(4):
        p = np.exp(0.3 * kv[0, :m, h // 2, 0] @ q[0, h])
        assert np.allclose(out[0, h], p @ kv[0, :m, h // 2, 1] / p.sum(), rtol=0, atol=1e-13)
