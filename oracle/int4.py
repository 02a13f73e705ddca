"""Float64 oracle of the 4-bit history and of the calls that read, gather and
copy stored tokens (numpy; block layouts written from include/oscar.h).

TEST INFRASTRUCTURE ONLY: imported by tests/; the product library never
imports it.

The 4-bit history is the 2-bit method with 16 levels (the pages describe two
bits): group clip t = c max|y|, s = fp16((max - min) / 15), z = fp16(min) of
the clipped group, code = clamp(rne((y - z) / s), 0, 15), 0 where s = 0;
value = s code + z.  A block is a K half and a V half: codes, then the
(s, z) pairs.
"""
from __future__ import annotations

import numpy as np

D, PAGE = 128, 64


def block_bytes(bits: int, g: int) -> int:
    return (4096 if bits == 2 else 8192) + 512 * (D // g)


def code_bytes(bits: int, g: int, which: int, t: int):
    """Byte offset inside a block and bit shift of the 128 codes of token
    slot t (which: 0 = K, 1 = V), in stored order."""
    p = np.arange(D)
    if bits == 2:
        return (t * 32 + p % 32 if which == 0 else 2048 + (p % 32) * 64 + t), 2 * (p // 32)
    half = 4096 + 256 * (D // g)
    if which == 0:
        group, index = p // 32, p % 32
        return t * 64 + 16 * (index // 8) + 4 * group + (index % 8) // 2, 4 * (p % 2)
    return half + (p // 2) * 64 + t, 4 * (p % 2)


def pair_bytes(bits: int, g: int, which: int, t: int) -> np.ndarray:
    """Byte offsets [128/g][4] of the (fp16 s, fp16 z) pairs of token slot t."""
    ng = D // g
    if bits == 2:
        base = 4096 + which * 256 * ng
    else:
        base = 4096 + which * (4096 + 256 * ng)
    return base + t * 4 * ng + 4 * np.arange(ng)[:, None] + np.arange(4)[None, :]


def quantize(y: np.ndarray, g: int, clip: float):
    """Codes [128], s and z as fp16 arrays [128/g], u [128], and the values
    (s, z) before rounding, of one rotated vector (float64)."""
    y = np.asarray(y, np.float64).reshape(-1, g)
    c = float(np.float32(clip))
    if c < 1.0:
        t = c * np.abs(y).max(1, keepdims=True)
        y = np.clip(y, -t, t)
    lo, hi = y.min(1), y.max(1)
    s, z = ((hi - lo) / 15.0).astype(np.float16), lo.astype(np.float16)
    sf, zf = s.astype(np.float64)[:, None], z.astype(np.float64)[:, None]
    u = np.where(sf > 0, (y - zf) / np.where(sf > 0, sf, 1.0), 0.0)
    return np.clip(np.rint(u), 0, 15).astype(np.uint8).ravel(), s, z, u.ravel(), (hi - lo) / 15.0, lo


def store(pool: np.ndarray, block: int, g: int, which: int, t: int, codes: np.ndarray, s: np.ndarray, z: np.ndarray):
    """Write one 4-bit vector into slot t of block number `block` (pool: flat uint8)."""
    base = block * block_bytes(4, g)
    at, shift = code_bytes(4, g, which, t)
    for nib in (0, 4):
        m = shift == nib
        keep = pool[base + at[m]] & (0xF0 if nib == 0 else 0x0F)
        pool[base + at[m]] = keep | (codes[m] << nib)
    pool[base + pair_bytes(4, g, which, t)] = np.stack([s, z], 1).view(np.uint8).reshape(-1, 4)


def evict(pool, rows, U, clip, table, seq, pos, g):
    """rows: float64 [n][hk][2][d]; writes the pool in place.  Returns
    (u, s_pre, z_pre) per [n][hk][2]."""
    import oracle
    orc = oracle.get()
    n, hk = rows.shape[:2]
    R = [[orc.build_R(np.asarray(U[h, w], np.float64)) for w in (0, 1)] for h in range(hk)]
    aux = (np.zeros((n, hk, 2, D)), np.zeros((n, hk, 2, D // g)), np.zeros((n, hk, 2, D // g)))
    for i in range(n):
        page = int(table[seq[i], pos[i] // PAGE])
        for h in range(hk):
            for w in (0, 1):
                codes, s, z, u, sp, zp = quantize(rows[i, h, w] @ R[h][w], g, clip[h, w])
                store(pool, page * hk + h, g, w, int(pos[i]) % PAGE, codes, s, z)
                for a, v in zip(aux, (u, sp, zp)):
                    a[i, h, w] = v
    return aux


def raw(pool, table, b, pos, h, which, hk, bits, g):
    """Codes [n][128] and pairs fp16 [n][128/g][2] of the history positions
    `pos` of sequence b."""
    bb, ng = block_bytes(bits, g), D // g
    codes, pairs = np.zeros((len(pos), D), np.uint8), np.zeros((len(pos), ng, 2), np.float16)
    for i, x in enumerate(np.asarray(pos)):
        base = (int(table[b, x // PAGE]) * hk + h) * bb
        at, shift = code_bytes(bits, g, which, int(x) % PAGE)
        codes[i] = (pool[base + at] >> shift.astype(np.uint8)) & (3 if bits == 2 else 15)
        pairs[i] = np.ascontiguousarray(pool[base + pair_bytes(bits, g, which, int(x) % PAGE)]).view(np.float16)
    return codes, pairs


def values(pool, table, b, pos, h, which, hk, bits, g) -> np.ndarray:
    """float64 [n][128] stored-order values s c + z."""
    codes, pairs = raw(pool, table, b, pos, h, which, hk, bits, g)
    p = np.repeat(pairs.astype(np.float64), g, axis=1)
    return codes * p[..., 0] + p[..., 1]


def decode(q, bf16_kv, bf16_len, pool, table, hist_len, U, sm_scale, g, bits=4):
    """Attention of q [B][Hq][d] over BF16 slots and history tokens mapped
    back by R^T (all float64).  Returns (out, magnitude): magnitude[b, h] =
    (the largest sum of |q_j k_j| sm_scale over a token's terms in the domain
    the product is taken in, the largest |value|)."""
    import oracle
    orc = oracle.get()
    B, Hq, _ = q.shape
    hk = bf16_kv.shape[2]
    out, mag = np.zeros((B, Hq, D)), np.zeros((B, Hq, 2))
    R = [[orc.build_R(np.asarray(U[h, w], np.float64)) for w in (0, 1)] for h in range(hk)]
    for b in range(B):
        n, m = int(hist_len[b]), int(bf16_len[b])
        for kv in range(hk):
            ks = values(pool, table, b, np.arange(n), kv, 0, hk, bits, g)
            vs = values(pool, table, b, np.arange(n), kv, 1, hk, bits, g)
            k = np.concatenate([ks @ R[kv][0].T, bf16_kv[b, :m, kv, 0]])
            v = np.concatenate([vs @ R[kv][1].T, bf16_kv[b, :m, kv, 1]])
            for h in range(kv * (Hq // hk), (kv + 1) * (Hq // hk)):
                if n + m == 0:
                    continue
                x = sm_scale * (k @ q[b, h])
                e = np.exp(x - x.max())
                out[b, h] = (e / e.sum()) @ v
                terms = [np.abs(ks) @ np.abs(q[b, h] @ R[kv][0]), np.abs(bf16_kv[b, :m, kv, 0]) @ np.abs(q[b, h])]
                mag[b, h] = sm_scale * max(t.max(initial=0.0) for t in terms), max(np.abs(vs).max(initial=0.0), np.abs(v).max())
    return out, mag


def gather(pool, src_table, dst_table, keep, n_keep, hk, bits, g):
    """The kept tokens' codes and pairs into a copy of the pool."""
    out = pool.copy()
    bb = block_bytes(bits, g)
    for b in range(src_table.shape[0]):
        for i in range(int(n_keep[b])):
            x = int(keep[b, i])
            for h in range(hk):
                s0 = (int(src_table[b, x // PAGE]) * hk + h) * bb
                d0 = (int(dst_table[b, i // PAGE]) * hk + h) * bb
                for w in (0, 1):
                    sa, da = pair_bytes(bits, g, w, x % PAGE), pair_bytes(bits, g, w, i % PAGE)
                    out[d0 + da] = pool[s0 + sa]
                    sa = np.unique(code_bytes(bits, g, w, x % PAGE)[0])
                    da = np.unique(code_bytes(bits, g, w, i % PAGE)[0])
                    out[d0 + da] = pool[s0 + sa]
    return out
