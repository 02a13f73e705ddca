"""Histories of 2 or 4 bits with shared first pages, on host and device, and the float64
attention over them with every token's weight (written from include/oscar.h's layouts)."""
from __future__ import annotations

import numpy as np

from bit_kv_cache_evict_gb300 import oscar as O
from bit_kv_cache_evict_gb300 import synth as S
from oracle import int4 as I

D = 128
SCALE = 1 / np.sqrt(D)
NSLOT = S.NSLOT


def f64(bits):
    return S.bf16_to_f32(bits).astype(np.float64)


def unpack(pool, hk, bits, g):
    """float64 [pages][hk][2][64][128]: the values s code + z of every slot, in stored order."""
    pool = pool.reshape(-1, hk, I.block_bytes(bits, g))
    out = np.empty((pool.shape[0], hk, 2, 64, D))
    for w in (0, 1):
        for t in range(64):
            at, shift = I.code_bytes(bits, g, w, t)
            code = (pool[:, :, at] >> shift.astype(np.uint8)) & (3 if bits == 2 else 15)
            pairs = np.ascontiguousarray(pool[:, :, I.pair_bytes(bits, g, w, t).ravel()]).view(np.float16).astype(np.float64)
            s, z = np.repeat(pairs[..., 0::2], g, -1), np.repeat(pairs[..., 1::2], g, -1)
            out[:, :, w, t] = code * s + z
    return out


class Scene:
    """Histories of the given lengths; groups: the group of each sequence (-1: none), which share `shared` pages."""

    def __init__(self, seed, bits, hist, hq, hk, g, groups=None, shared=0, std=1.0, wide=1):
        import oracle
        self.rng = rng = np.random.default_rng(seed)
        self.bits, self.hq, self.hk, self.g, self.B = bits, hq, hk, g, len(hist)
        self.hist = np.array(hist, np.int32)
        self.group = np.full(self.B, -1, np.int32) if groups is None else np.array(groups, np.int32)
        self.n_groups = int(max(self.group.max(), 0)) + 1
        self.group_pages = np.full(self.n_groups, shared, np.int32)
        self.sh = O.make_shape(hq, hk, quant_group=g)
        need = (self.hist + 63) // 64
        self.max_pages = max(int(need.max()), shared, 1) + wide
        pre = np.minimum(need, np.where(self.group >= 0, shared, 0))
        self.num_pages = self.n_groups * shared + int((need - pre).sum()) + 2
        ids = rng.permutation(self.num_pages)
        self.table = np.full((self.B, self.max_pages), -1, np.int32)
        at = self.n_groups * shared
        for b in range(self.B):
            self.table[b, :pre[b]] = ids[self.group[b] * shared:][:pre[b]]
            self.table[b, pre[b]:need[b]] = ids[at:at + need[b] - pre[b]]
            at += need[b] - pre[b]
        self.spare = ids[at:]
        self.U = np.linalg.qr(rng.standard_normal((hk, 2, D, D)))[0].astype(np.float32)
        self.R = [[oracle.get().build_R(self.U[h, w].astype(np.float64)) for w in (0, 1)] for h in range(hk)]
        bb, ng = I.block_bytes(bits, g), D // g
        pool = rng.integers(0, 256, (self.num_pages, hk, bb)).astype(np.uint8)
        half = 2.0 * std
        for w in (0, 1):
            base = I.pair_bytes(bits, g, w, 0).ravel()[0]
            lo = -half * rng.uniform(0.8, 1.2, (self.num_pages, hk, 64 * ng))
            hi = half * rng.uniform(0.8, 1.2, lo.shape)
            sz = np.stack([(hi - lo) / (2 ** bits - 1), lo], -1).astype(np.float16)
            pool[:, :, base:base + 256 * ng] = sz.view(np.uint8).reshape(self.num_pages, hk, 256 * ng)
        self.pool = pool.ravel()
        self.q = S.bf16_bits(rng.standard_normal((self.B, hq, D)))
        self.kv = S.bf16_bits(rng.standard_normal((self.B, NSLOT, hk, 2, D)) * std)
        self.len = np.where(self.hist > 0, NSLOT, rng.integers(0, NSLOT + 1, self.B)).astype(np.int32)

    def pairs(self, page, h, w, t):
        """View of the pairs fp16 [128 / g][2] of a slot, to be written through set_pairs."""
        return np.ascontiguousarray(self.pool.reshape(self.num_pages, self.hk, -1)[page, h][I.pair_bytes(self.bits, self.g, w, t)]).view(np.float16)

    def set_pairs(self, page, h, w, t, v):
        self.pool.reshape(self.num_pages, self.hk, -1)[page, h][I.pair_bytes(self.bits, self.g, w, t)] = np.ascontiguousarray(v, np.float16).view(np.uint8)

    def poison(self):
        """NaN pairs in every slot behind the histories and in unused pages, NaN in the unused BF16 slots."""
        live = np.zeros((self.num_pages, 64), bool)
        for b in range(self.B):
            for i in range((int(self.hist[b]) + 63) // 64):
                live[self.table[b, i], :min(64, int(self.hist[b]) - 64 * i)] = True
        nan = np.full((D // self.g, 2), np.nan, np.float16)
        for p, t in zip(*np.nonzero(~live)):
            for h in range(self.hk):
                for w in (0, 1):
                    self.set_pairs(p, h, w, t, nan)
        for b in range(self.B):
            self.kv[b, self.len[b]:] = 0x7FC0
        return self

    def want(self, skip_pages=()):
        """float64: out [B][hq][d]; weights of the history [B][64 max_pages] and of the slots [B][320], summed over the
        heads; per (b, head) the largest sum of |q_j k_j| / sqrt(d) of a token's terms and the largest |value|; and the
        sums over the heads of p times that logit magnitude, for both kinds of tokens."""
        vals = unpack(self.pool, self.hk, self.bits, self.g)
        G = self.hq // self.hk
        q, kv = f64(self.q), f64(np.where(self.kv == 0x7FC0, 0, self.kv))
        out, mag = np.zeros((self.B, self.hq, D)), np.zeros((self.B, self.hq, 2))
        w, sw = np.zeros((self.B, 64 * self.max_pages)), np.zeros((self.B, NSLOT))
        we, swe = np.zeros_like(w), np.zeros_like(sw)
        for b in range(self.B):
            n, m = int(self.hist[b]), int(self.len[b])
            t = np.arange(n)
            page = self.table[b, t // 64]
            on = ~np.isin(page, skip_pages) & (page >= 0) & (page < self.num_pages)
            for h in range(self.hk):
                ks, vs = (vals[page[on], h, i, t[on] % 64] for i in (0, 1))
                k = np.concatenate([ks @ self.R[h][0].T, kv[b, :m, h, 0]])
                v = np.concatenate([vs @ self.R[h][1].T, kv[b, :m, h, 1]])
                for x in range(h * G, (h + 1) * G):
                    if len(k) == 0:
                        continue
                    a = SCALE * (k @ q[b, x])
                    e = np.exp(a - a.max())
                    p = e / e.sum()
                    out[b, x] = p @ v
                    terms = SCALE * np.concatenate([np.abs(ks) @ np.abs(q[b, x] @ self.R[h][0]), np.abs(kv[b, :m, h, 0]) @ np.abs(q[b, x])])
                    mag[b, x] = terms.max(), max(np.abs(vs).max(initial=0.0), np.abs(v).max())
                    n_on = int(on.sum())
                    w[b, t[on]] += p[:n_on]
                    sw[b, :m] += p[n_on:]
                    we[b, t[on]] += p[:n_on] * mag[b, x, 0]
                    swe[b, :m] += p[n_on:] * mag[b, x, 0]
        return out, w, sw, mag, we, swe

    def device(self):
        import gpu_harness as H
        self.d = {k: H.i32_t(getattr(self, k)) for k in ("table", "hist", "len", "group", "group_pages")}
        self.d.update(pool=H.u8_t(self.pool), U=H.f32_t(self.U), q=H.bf16_t(self.q), kv=H.bf16_t(self.kv))
        return self.d


def out_tolerance(want, mag, bits, bf16, fp16_shared=False):
    """Elementwise bound on an output's error.  A base-2 logit is a sum of products with q' to 22 bits: within A 2^-19
    of the exact one, A the sum of its terms' sizes (8 truncated accumulations 2^-23, q' 2^-22, the fp32 sums 2^-21);
    for 2 bits A 2^-18 (operands that are subnormal patterns keep up to four bits fewer of a product: 2^-20 more).
    Shared pages of a bf16 output: q' and k rounded to fp16, 2^-11 each.  A weight is then off by twice that times ln 2,
    relatively, and 4 (> 2 x 2 ln 2) covers numerator and sum.  The value sums: W to 22 bits and fp32 sums over at most
    2^7 steps per warp, 2^-15 of the largest value; shared pages of a bf16 output: P and v rounded to fp16, 2^-11 each.  A bf16 output: 2^-8."""
    logit = mag[..., :1] / np.log(2) * (2.0 ** -18 if bits == 2 else 2.0 ** -19)
    vals = 2.0 ** -15
    if fp16_shared:
        logit = logit + mag[..., :1] / np.log(2) * 2.0 ** -10
        vals += 2.0 ** -10
    return mag[..., 1:] * (4 * logit + vals) + 1e-30 + (np.abs(want) * 2.0 ** -8 if bf16 else 0)


def weight_tolerance(w, we, old, hq, bits):
    """Bound on a score's error: every head's p as above (and 2^-20 for its exponential and the division), the fp32 sum over hq heads and the old score."""
    return 4 * we / np.log(2) * (2.0 ** -18 if bits == 2 else 2.0 ** -19) + w * (2.0 ** -20 + hq * 2.0 ** -24) + (w + np.abs(old)) * 2.0 ** -22 + 1e-30
