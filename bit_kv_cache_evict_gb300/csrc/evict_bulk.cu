// evict_bulk.cu -- eviction of many tokens at once into the 4-bit history (a
// prompt's history): the same codes and pairs as evict4_kernel
// (evict4.cu), with the rotation on tensor cores.
//
// The mathematics.  A vector's decisions (s, z, codes) have to be those of the
// exact rotated values, while a tensor-core product gives y within some
// bound delta.  So every decision is taken from the product first, together with a
// test whether an error of delta could change it; the few that could (about
// one group in 25 for s or z, one code in 10^4) are taken again from exactly
// summed values.
//   Product: y = x . R, R = U . Hadamard . bit-reversal / sqrt(d) formed once
// per block in fixed point and kept as fp16 parts h1 + h2 (22 bits) and
// a remainder r3 of 16 bits, all scaled by a power of two; x (bf16) is scaled per row into
// fp16, exactly but for elements below 2^-31 of the row's largest (2^-35 |x| |R_j| of y in all).
//   delta.  One MMA aligns its sixteen exact products and the accumulator to
// the largest of them, cuts each off two bits below fp32's last (2^-25 of the largest),
// adds, and cuts the sum off to 24 bits: it loses at most (17 / 4) 2^-23 M + 2^-23
// |sum|, M the largest addend (tests/test_gpu_evict4_product.py measures
// single MMAs against this: at most 0.79 of it).  A chain of eight k-steps would
// lose 8 (17 / 4 + 1) 2^-23 |x| |R_j| in all, as M can be as large as the whole
// (measured: 1.6 times the 1.5 2^-20 that was once allowed).  So each k-step s
// is summed from zero: M and the sum are at most |x_s| |R_sj|
// (Cauchy-Schwarz, over the step's indices), and the sum of those over the steps
// at most |x| |R_j| (the same again): 5.25 2^-23.  The seven rounded
// fp32 additions lose at most 2^-24 of a partial sum each: 3.5 2^-23; r3 is below
// 3.5 2^-23 of R (two of 24 bits cut off, and the pair's low part).  In all 12.25 2^-23 and
// less than 0.05 2^-23 for h2's own product: delta = 1.6 2^-20 |x| max_j |R_j|
// is 12.8 2^-23 (measured: errors up to 0.40 delta on rows made for it).
//   Exact value of one element: x (h1 + h2) as an error-free product, x r3 exact
// in fp32 (8 x 16 bits), added by the warp as pairs: the value of R to about
// 2^-38.
//
// What bounds it: 512 bytes read and 160 written per token and KV head
// (12 us for 15,104 tokens of eight KV heads), 256 tensor-core products per
// 16 vectors, and their decisions: 4,800 instructions in all.  Measured 125 us
// for that case (GB300; 0.65 TB/s; the per-vector kernel: 1832 us; 120 with the
// products in chains, see delta): 9 us for
// R, then per 16-token tile a third of the time in the products (at half of
// mma.sync's rate), a sixth in the exact sums, an eighth in the codes; the
// schedulers issue in 52 % of the cycles, the tensor cores run in 22 %.  The kernel's
// code is larger than the instruction caches hold: loops are kept rolled and
// warps in step (below) for that reason.  (16 warps of 128 registers instead of
// 12 of 168 cost 3 us, groups of four warps 7, two barriers fewer per tile 5.)
#include <algorithm>
#include <climits>

#include "pairs.cuh"

namespace oscar {

namespace {

constexpr int kBulkWarps = 12;
constexpr int kBulkThreads = 32 * kBulkWarps;
constexpr int kGroupWarps = 6;              // warps that go through a tile together
constexpr int kTile = 16;                   // tokens of a warp's tile (MMA rows)
constexpr int kXPitch = kD * 2 + 16;        // bytes of a staged row: ldmatrix rows on distinct banks
constexpr int kStgPitch = kD / 2 + 4;       // bytes of a staged code row

// Fragment words of a k-step: [16 n-tiles][32 lanes], and four more, so that the
// eight k-steps that a team of bulk_exact reads lie on distinct banks (without
// them that phase took 66 of 302 thousand cycles, with them 30).
constexpr int kStepWords = 16 * 32 + 4;

struct BulkSmem {
    static constexpr int kFrag = 0;                                  // [2 parts][8 k-steps][kStepWords] uint2
    static constexpr int kR3 = kFrag + 2 * 8 * kStepWords * 8;       // [8][kStepWords] float4
    static constexpr int kX = kR3 + 8 * kStepWords * 16;             // [warp][16][kXPitch]
    static constexpr int kStg = kX + kBulkWarps * kTile * kXPitch;   // [warp][16][kStgPitch]: byte j = positions 2j, 2j + 1
    static constexpr int kSz = kStg + kBulkWarps * kTile * kStgPitch;  // [warp][16][4] (s, z) word per 32-position block
    static constexpr int kDst = kSz + kBulkWarps * kTile * 16;       // [warp][16] destination half, [warp][16] slot
    static constexpr int kCol = kDst + kBulkWarps * kTile * 16;      // [128] column sums of squares, then scalars
    static constexpr int kList = kCol + (kD + 4) * 4;                // open groups of the round
    static constexpr int kBytes = kList + kBulkWarps * kTile * 4 * 8;
};
static_assert(BulkSmem::kBytes <= 227 * 1024, "one block per SM");

__device__ __forceinline__ float pow2f_bits(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Place of k-step ks's fragment word pair (position p, quad member tq).  The quad
// member is exchanged by the n-tile's low bits, so that the 32 positions that
// a warp of bulk_matrix stores lie on distinct banks (8-way conflicts without).
__device__ __forceinline__ int frag_at(int ks, int p, int tq) {
    return ks * kStepWords + (p >> 3) * 32 + 4 * (p & 7) + (tq ^ ((p >> 3) & 3));
}

// R of this block's (KV head, K|V) into shared memory.  Row a of U times the
// Hadamard matrix in fixed point, as two 32-bit integers (2^-44 of the largest
// |U|; the additions are exact), then times 1 / sqrt(d) as a pair.  (64-bit
// integers took 25 us: their conversions run on the slow 64-bit pipe.)  A warp takes
// the four rows of one fragment word pair (16 ks + 2 tq, + 1, + 8, + 9) at a time, eight
// lanes to a row, lane c of them inputs 4 c + 32 j + k: four of the seven butterfly
// stages stay in the lane.  Returns the exponent q of the scale (stored = R 2^q) and the largest
// column norm of the stored matrix.
__device__ __forceinline__ void bulk_matrix(const float* U, uint8_t* smem, int& q, float& norm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kTurns = (kD / 4 + kBulkWarps - 1) / kBulkWarps;
    // every load first, for the largest entry too
    float4 u[kTurns][4];
    float mx = 0.f;
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const int w = warp + kBulkWarps * t, i = lane >> 3;
        const float* row = U + (size_t)(16 * (w >> 2) + 2 * (w & 3) + (i & 1) + 8 * (i >> 1)) * kD + 4 * (lane & 7);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            u[t][j] = w < kD / 4 ? __ldg(reinterpret_cast<const float4*>(row + 32 * j)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float* col = reinterpret_cast<float*>(smem + BulkSmem::kCol);
    int* umax = reinterpret_cast<int*>(col + kD);
    if (threadIdx.x < kD) col[threadIdx.x] = 0.f;
    if (threadIdx.x == 0) *umax = 0;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kTurns; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            mx = fmaxf(mx, fmaxf(fmaxf(fabsf(u[t][j].x), fabsf(u[t][j].y)), fmaxf(fabsf(u[t][j].z), fabsf(u[t][j].w))));
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, m));
    if (lane == 0) atomicMax(umax, __float_as_int(mx));
    __syncthreads();
    const int e = min(60, max(-60, ((*umax >> 23) & 0xff) - 127));
    q = 10 - e;  // |R| <= 128 |U| / sqrt(128) < 2^(e + 4.5): stored below 2^14.5
    const float up = pow2f_bits(21 - e);  // |U| 2^(21 - e) < 2^22: sums of 128 below 2^29
    // R 2^q = v 2^(e - 21 + q) / sqrt(128) = v 2^-11 / sqrt(128)
    const float kc_hi = __uint_as_float(0x3db504f3u), kc_lo = __uint_as_float(0x30cfe77au), down = pow2f_bits(-11);
    uint2* frag = reinterpret_cast<uint2*>(smem + BulkSmem::kFrag);
    float4* r3 = reinterpret_cast<float4*>(smem + BulkSmem::kR3);
    // [high, low][4 rows][128 outputs]; output o at o ^ ((o >> 5) & 3), so that the outputs of 32 neighbouring
    // positions lie on distinct banks
    int* sums = reinterpret_cast<int*>(smem + BulkSmem::kX + warp * kTile * kXPitch);
    static_assert(2 * 4 * kD * 4 <= kTile * kXPitch, "the sums fit in the warp's rows");
    float sq[4] = {0.f, 0.f, 0.f, 0.f};
    // (Rolled, the loads moving up by a turn: this code runs three times per warp and
    // would otherwise wait on its own instruction fetches.)
#pragma unroll 1
    for (int w = warp; w < kD / 4; w += kBulkWarps) {
        const int ks = w >> 2, tq = w & 3;
        int v[2][16];  // input = v[0] + v[1] 2^-22
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x[4] = {u[0][j].x * up, u[0][j].y * up, u[0][j].z * up, u[0][j].w * up};
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 1.5 2^23 added rounds to an integer, in the low bits
                const float m0 = __fadd_rn(x[k], 12582912.f);
                const float m1 = __fadd_rn(__fsub_rn(x[k], __fsub_rn(m0, 12582912.f)) * 4194304.f, 12582912.f);
                v[0][4 * j + k] = __float_as_int(m0) - 0x4b400000;
                v[1][4 * j + k] = __float_as_int(m1) - 0x4b400000;
            }
        }
#pragma unroll
        for (int t = 0; t + 1 < kTurns; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) u[t][j] = u[t + 1][j];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 1; m < 16; m <<= 1)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!(i & m)) {
                        const int x = v[h][i], y = v[h][i | m];
                        v[h][i] = x + y;
                        v[h][i | m] = x - y;
                    }
#pragma unroll 1
        for (int m = 1; m < 8; m <<= 1) {
            const int sign = (lane & m) ? -1 : 1;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i) v[h][i] = v[h][i] * sign + __shfl_xor_sync(kFull, v[h][i], m);
        }
        __syncwarp();  // (the last turn's sums are read)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<int4*>(sums + (4 * h + (lane >> 3)) * kD + 32 * j + 4 * (lane & 7)) =
                    make_int4(v[h][4 * j + j], v[h][4 * j + (1 ^ j)], v[h][4 * j + (2 ^ j)], v[h][4 * j + (3 ^ j)]);
        __syncwarp();
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            const int p = 32 * k + lane, l = bitrev5(lane);  // stored position p is output 4 l + bitrev2(k)
            const int* from = sums + 4 * l + (bitrev2(k) ^ (l >> 3));
            uint32_t h1[4], h2[4];
            float r[4], ss = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int va = from[i * kD], vb = from[(4 + i) * kD];
                const float hi = __int2float_rn(va);
                const float lo = __int2float_rn((va - __float2int_rn(hi)) * 4194304 + vb) * (1.f / 4194304.f);
                float ph = __fmul_rn(hi, kc_hi);
                float pe = __fmaf_rn(lo, kc_hi, __fmaf_rn(hi, kc_lo, __fmaf_rn(hi, kc_hi, -ph)));
                ph = __fmul_rn(ph, down);
                pe = __fmul_rn(pe, down);
                // h1 + h2: the leading 22 bits (down to 2^-24), so that their fp32 sum is exact
                const float lead = __uint_as_float(__float_as_uint(ph) & 0xfffffffcu);
                const __half f1 = __float2half_rn(lead);
                const float r1 = __half2float(f1);
                const __half f2 = __float2half_rn(__fsub_rn(lead, r1));
                h1[i] = __half_as_ushort(f1);
                h2[i] = __half_as_ushort(f2);
                // 16 bits, so that its products with bf16 are exact too
                r[i] = __uint_as_float(
                    __float_as_uint(__fadd_rn(__fsub_rn(__fsub_rn(ph, r1), __half2float(f2)), pe)) & 0xffffff00u);
                ss = fmaf(ph, ph, ss);
            }
            const int at = frag_at(ks, p, tq);
            frag[at] = make_uint2(h1[0] | (h1[1] << 16), h1[2] | (h1[3] << 16));
            frag[8 * kStepWords + at] = make_uint2(h2[0] | (h2[1] << 16), h2[2] | (h2[3] << 16));
            r3[at] = make_float4(r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) sq[j] += j == k ? ss : 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) atomicAdd(col + 32 * k + lane, sq[k]);
    __syncthreads();
    float c2 = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) c2 = fmaxf(c2, col[lane + 32 * i]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) c2 = fmaxf(c2, __shfl_xor_sync(kFull, c2, m));
    norm = sqrtf(c2) * 1.001f;
}

// Exact value of stored position p of a staged row, by teams of eight lanes
// (each team its own row and position; every lane of the warp takes part):
// lane ks of a team sums k indices 16 ks .. 16 ks + 15.
__device__ __noinline__ df bulk_exact(const uint8_t* smem, const uint8_t* xrow, int p, float down) {
    const int ks = threadIdx.x & 7;
    const uint2* f1 = reinterpret_cast<const uint2*>(smem + BulkSmem::kFrag);
    const uint2* f2 = f1 + 8 * kStepWords;
    const float4* f3 = reinterpret_cast<const float4*>(smem + BulkSmem::kR3);
    const uint4 xa = *reinterpret_cast<const uint4*>(xrow + 32 * ks), xb = *reinterpret_cast<const uint4*>(xrow + 32 * ks + 16);
    const uint32_t xl[4] = {xa.x, xa.y, xa.z, xa.w}, xh[4] = {xb.x, xb.y, xb.z, xb.w};  // k = 2 tq, + 1; 8 + 2 tq, + 1
    float s[4], c[4];  // four chains
#pragma unroll
    for (int tq = 0; tq < 4; ++tq) {  // fragment word pair of quad member tq
        const int at = frag_at(ks, p, tq);
        const uint2 u1 = f1[at], u2 = f2[at];
        const float4 r = f3[at];
        const float x[4] = {bf16_lo(xl[tq]), bf16_hi(xl[tq]), bf16_lo(xh[tq]), bf16_hi(xh[tq])};
        const float h[4] = {half_lo(u1.x) + half_lo(u2.x), half_hi(u1.x) + half_hi(u2.x), half_lo(u1.y) + half_lo(u2.y),
                            half_hi(u1.y) + half_hi(u2.y)};  // exact: 22 bits
        const float q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float pr = __fmul_rn(x[k], h[k]), pe = __fmaf_rn(x[k], h[k], -pr);  // exact product
            if (tq == 0) {
                s[k] = pr;
                c[k] = __fmaf_rn(x[k], q[k], pe);
            } else {
                const df t = two_sum(s[k], pr);
                s[k] = t.hi;
                c[k] = __fadd_rn(__fmaf_rn(x[k], q[k], c[k]), __fadd_rn(pe, t.lo));
            }
        }
    }
    const df s01 = two_sum(s[0], s[1]), s23 = two_sum(s[2], s[3]), sa = two_sum(s01.hi, s23.hi);
    const float rest = __fadd_rn(__fadd_rn(__fadd_rn(c[0], c[1]), __fadd_rn(c[2], c[3])), __fadd_rn(s01.lo, s23.lo));
    df y = two_sum(sa.hi, __fadd_rn(sa.lo, rest));
#pragma unroll
    for (int m = 1; m < 8; m <<= 1)
        y = df_add(y, df{__shfl_xor_sync(kFull, y.hi, m), __shfl_xor_sync(kFull, y.lo, m)});
    return {__fmul_rn(y.hi, down), __fmul_rn(y.lo, down)};
}

// c max|y| of exact extremes, and the extremes clipped by it.
__device__ __forceinline__ df bulk_clip(float cr, df& hi, df& lo) {
    if (!(cr < 1.f)) return {INFINITY, 0.f};
    const df nlo = df_neg(lo), a = df_less(hi, nlo) ? nlo : hi;
    const float th = __fmul_rn(cr, a.hi);
    const df t = fast_two_sum(th, __fmaf_rn(cr, a.lo, __fmaf_rn(cr, a.hi, -th))), nt = df_neg(t);
    if (df_less(t, hi)) hi = t;
    if (df_less(lo, nt)) lo = nt;
    return t;
}

__device__ __forceinline__ uint32_t bulk_pair(df hi, df lo) {
    return (uint32_t)df_to_f16(df_div15(df_add(hi, df_neg(lo)))) | ((uint32_t)df_to_f16(lo) << 16);
}

// A whole group from exact values: extremes, pair and codes of its 32-position
// blocks b0 .. b0 + nb - 1, written over the staged ones.  For groups whose
// extremes are not single elements within the bound.
__device__ __noinline__ void bulk_group_exact(uint8_t* smem, const uint8_t* xrow, uint8_t* stg, uint32_t* sz, int b0, int nb,
                                              float cr, float down) {
    const int lane = threadIdx.x & 31;
    df v[4], hi{-INFINITY, 0.f}, lo{INFINITY, 0.f};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        v[b] = {0.f, 0.f};
        if (b >= nb) continue;
        for (int e = 0; e < 8; ++e) {  // team j takes element 8 j + e
            const df y = bulk_exact(smem, xrow, 32 * (b0 + b) + 8 * (lane >> 3) + e, down);
            if ((lane & 7) == e) v[b] = y;
        }
        if (df_less(hi, v[b])) hi = v[b];
        if (df_less(v[b], lo)) lo = v[b];
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const df h{__shfl_xor_sync(kFull, hi.hi, m), __shfl_xor_sync(kFull, hi.lo, m)};
        const df l{__shfl_xor_sync(kFull, lo.hi, m), __shfl_xor_sync(kFull, lo.lo, m)};
        if (df_less(hi, h)) hi = h;
        if (df_less(l, lo)) lo = l;
    }
    const df t = bulk_clip(cr, hi, lo), nt = df_neg(t);
    const uint32_t w = bulk_pair(hi, lo);
    const float sf = half_lo(w), zf = half_hi(w);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (b >= nb) continue;
        df y = v[b];
        if (df_less(t, y)) y = t;
        else if (df_less(y, nt)) y = nt;
        const uint32_t code = sf != 0.f ? (uint32_t)code4_of(y, sf, zf) : 0u;
        const uint32_t other = __shfl_xor_sync(kFull, code, 1);
        if (!(lane & 1)) stg[16 * (b0 + b) + (lane >> 1)] = (uint8_t)(code | (other << 4));
        if (lane == 0) sz[b0 + b] = w;
    }
    __syncwarp();
}

__device__ __forceinline__ void bulk_ldsm(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}

// n-tiles whose products run side by side, and whose operands are loaded ahead
// (15,104 tokens of eight KV heads, us: 2, 4: 124.5; 2, 8: 124.6; 4, 4: 124.8; 4, 8: 126).
constexpr int kSide = 2, kAhead = 4;

// y = x . R of a warp's tile of 16 staged rows: acc[n][e] is stored position
// 8 n + 2 tq + (e & 1) of row gID + 8 (e >> 1), delta[r] the bound of its error for row gID + 8 r.
__device__ __forceinline__ void bulk_product(const uint8_t* smem, const uint8_t* xs, float rdown, float rnorm,
                                             float (&acc)[16][4], float (&delta)[2]) {
    const int lane = threadIdx.x & 31;
    const uint2* frag = reinterpret_cast<const uint2*>(smem + BulkSmem::kFrag);
    // -- rows scaled by 2^k, k from the largest element
    const uint8_t* xfrag = xs + ((lane & 7) + 8 * ((lane >> 3) & 1)) * kXPitch + 16 * (lane >> 4);
    float mx[2] = {0.f, 0.f}, n2[2] = {0.f, 0.f}, fdown[2], up[2];
#pragma unroll 2
    for (int ks = 0; ks < 8; ++ks) {
        uint32_t a[4];
        bulk_ldsm(a, xfrag + 32 * ks);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            mx[e & 1] = fmaxf(mx[e & 1], fmaxf(fabsf(bf16_lo(a[e])), fabsf(bf16_hi(a[e]))));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(kFull, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(kFull, mx[r], 2));
        // largest |x| 2^k below 2^15; or k = 110, where every bf16 value (a multiple of 2^-133) is a multiple of 2^-23
        const int k = min(110, 14 - ((int)(__float_as_uint(mx[r]) >> 23) - 127));
        up[r] = pow2f_bits(k);
        fdown[r] = pow2f_bits(-k) * rdown;  // accumulator -> y
    }

    // -- y: n-tile n = stored positions 8 n .. 8 n + 7; rows gID (entries
    //    0, 1) and gID + 8 (2, 3).  A k-step's sum starts from zero, x . h2
    //    then x . h1, and is added to acc in fp32 (for the bound's sake, see above).  (A
    //    loop, not unrolled: with every product unrolled the kernel waited on
    //    instruction fetches for half of its time.)
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    uint32_t raw[4], a[4];
    auto scale = [&](bool sum) {  // raw to fp16; the sum of squares
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v0 = bf16_lo(raw[e]) * up[e & 1], v1 = bf16_hi(raw[e]) * up[e & 1];
            if (sum) n2[e & 1] = fmaf(v0, v0, fmaf(v1, v1, n2[e & 1]));
            a[e] = pack_f16x2_rn(v0, v1);
        }
    };
    auto operand = [&](int ks, int n, int part) {  // (frag_at)
        return frag[(part * 8 + ks) * kStepWords + n * 32 + (lane ^ (n & 3))];
    };
    bulk_ldsm(raw, xfrag);
    uint2 b[kAhead][2];  // operands of the next kAhead n-tiles: h1, h2
#pragma unroll
    for (int n = 0; n < kAhead; ++n)
#pragma unroll
        for (int part = 0; part < 2; ++part) b[n][part] = operand(0, n, part);
    scale(true);
#pragma unroll 1
    for (int ks = 0; ks < 8; ++ks) {  // (the next step's operands are loaded and made while the products run)
        const int next = (ks + 1) & 7;
        bulk_ldsm(raw, xfrag + 32 * next);
        float t[2][kSide][4];  // the sums of kSide n-tiles, and of the kSide before them
#pragma unroll
        for (int n0 = 0; n0 < 16 + kSide; n0 += kSide) {
            const int now = (n0 / kSide) & 1;
            if (n0 < 16) {
#pragma unroll
                for (int i = 0; i < kSide; ++i) {
                    uint2& u = b[(n0 + i) % kAhead][1];
                    mma_f16_16816_zero(t[now][i], a[0], a[1], a[2], a[3], u.x, u.y);
                    u = operand(n0 + i + kAhead < 16 ? ks : next, (n0 + i + kAhead) & 15, 1);
                }
#pragma unroll
                for (int i = 0; i < kSide; ++i) {
                    uint2& u = b[(n0 + i) % kAhead][0];
                    mma_f16_16816(t[now][i], a[0], a[1], a[2], a[3], u.x, u.y);
                    u = operand(n0 + i + kAhead < 16 ? ks : next, (n0 + i + kAhead) & 15, 0);
                }
            }
            if (n0 > 0) {
#pragma unroll
                for (int i = 0; i < kSide; ++i) {
                    float(&y)[4] = acc[n0 - kSide + i];
                    const float(&u)[4] = t[now ^ 1][i];
                    const float2 y0 = add2(make_float2(y[0], y[1]), make_float2(u[0], u[1]));
                    const float2 y1 = add2(make_float2(y[2], y[3]), make_float2(u[2], u[3]));
                    y[0] = y0.x;
                    y[1] = y0.y;
                    y[2] = y1.x;
                    y[3] = y1.y;
                }
            }
        }
        scale(ks < 7);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        n2[r] += __shfl_xor_sync(kFull, n2[r], 1);
        n2[r] += __shfl_xor_sync(kFull, n2[r], 2);
        delta[r] = 1.6f * 9.5367431640625e-7f * sqrtf(n2[r]) * 1.001f * rnorm * fdown[r];
    }
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] *= fdown[e >> 1];
}

// Block = one (KV head, K|V), blockIdx.x / pairs of the blocks that share it;
// its warps take tiles of 16 listed tokens in turn.
__global__ void __launch_bounds__(kBulkThreads, 1) evict_bulk_kernel(EvictParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gID = lane >> 2, tq = lane & 3;
    const int pairs = 2 * p.hk, pair = blockIdx.x % pairs, kv = pair >> 1, which = pair & 1;
    const int step = gridDim.x / pairs * kBulkWarps, tiles = (p.n_tok + kTile - 1) / kTile;
    int q;
    float rnorm;
    bulk_matrix(p.U + ((size_t)kv * 2 + which) * kD * kD, smem, q, rnorm);
    const float cr = __ldg(p.clip + kv * 2 + which), rdown = pow2f_bits(-q);
    const int nb = 1 << p.gshift;  // 32-position blocks per group
    uint8_t* xs = smem + BulkSmem::kX + warp * kTile * kXPitch;
    uint8_t* stg = smem + BulkSmem::kStg + warp * kTile * kStgPitch;
    uint32_t* sz = reinterpret_cast<uint32_t*>(smem + BulkSmem::kSz) + warp * kTile * 4;
    uint8_t** dst = reinterpret_cast<uint8_t**>(smem + BulkSmem::kDst) + warp * kTile;
    int* slots = reinterpret_cast<int*>(smem + BulkSmem::kDst + kBulkWarps * kTile * 8) + warp * kTile;
    // the group's open quantisation groups: row of the block, 32-position block, positions of the extremes
    ushort4* list = reinterpret_cast<ushort4*>(smem + BulkSmem::kList) + warp / kGroupWarps * (kGroupWarps * kTile * 4);
    int* n_list = reinterpret_cast<int*>(smem + BulkSmem::kCol) + kD + 1 + warp / kGroupWarps;

    // Lane r < 16 (and 16 + r) looks token r of a tile up, in steps a tile
    // apart so that nothing waits for a load: its indices two tiles ahead; the
    // checks, the row's request into L2 and the page's load one tile ahead;
    // the row's copy at the end of the tile before.
    struct Token {
        int row, seq, pos;
    };
    auto fetch = [&](int tile) {
        Token k{-1, -1, 0};
        const int i = tile * kTile + (lane & 15);
        if (i < p.n_tok) {
            k.row = p.src_row ? __ldg(p.src_row + i) : i;
            k.seq = __ldg(p.dst_seq + i);
            k.pos = __ldg(p.dst_pos + i);
        }
        return k;
    };
    struct Place {
        int row, page, slot;  // row -1: skipped; page kNone: no destination
    };
    constexpr int kNone = INT_MIN;
    auto locate = [&](int tile, const Token& k) {
        Place at{-1, kNone, k.pos % kPage};
        if (tile * kTile + (lane & 15) < p.n_tok) {
            if (k.row < 0 || k.row >= p.src_rows) {
                report(p.status, OSCAR_STATUS_BAD_POS);
            } else {
                at.row = k.row;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.src_kv + ((size_t)k.row * pairs + pair) * kD + 64 * (lane >> 4)));
                if (k.pos < 0 || k.pos >= p.max_pages * kPage || k.seq < 0 || k.seq >= p.batch)
                    report(p.status, OSCAR_STATUS_BAD_POS);
                else
                    at.page = __ldg(p.page_table + (size_t)k.seq * p.max_pages + k.pos / kPage);
            }
        }
        return at;
    };
    auto copy_rows = [&](int row) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // two rows of 16 chunks at a time
            const int r = 2 * c + (lane >> 4), ch = lane & 15;
            const int rr = __shfl_sync(kFull, row, r);
            uint8_t* to = xs + r * kXPitch + 16 * ch;
            if (rr >= 0)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)),
                             "l"(p.src_kv + ((size_t)rr * pairs + pair) * kD + 8 * ch)
                             : "memory");
            else
                *reinterpret_cast<uint4*>(to) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Two groups of six warps, each going through a tile together (its own
    // barrier): left to themselves the warps spread over the loop's code and
    // wait for instruction fetches half of the time, and in one group the
    // tensor cores idle while the codes are made.
    auto group_sync = [&]() {
        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / kGroupWarps), "r"(32 * kGroupWarps) : "memory");
    };
    const int first = blockIdx.x / pairs * kBulkWarps, rounds = (tiles - first + step - 1) / step;
    Place now = locate(first + warp, fetch(first + warp));
    Token next = fetch(first + warp + step);
    copy_rows(now.row);
    for (int round = 0; round < rounds; ++round) {
        const int tile = first + warp + round * step;
        group_sync();
        if (lane == 0 && warp % kGroupWarps == 0) *n_list = 0;  // (added to after a further barrier)
        const int row = now.row;
        if (lane < kTile) {  // (the last tile's stores have read dst and slots)
            const bool ok = now.page >= 0 && now.page < p.num_pages;
            if (!ok && now.page != kNone) report(p.status, OSCAR_STATUS_BAD_PAGE);
            dst[lane] = ok ? p.pool + ((size_t)now.page * p.hk + kv) * p.block_bytes + which * half_bytes4(p.gshift) : nullptr;
            slots[lane] = now.slot;
        }
        now = locate(tile + step, next);
        next = fetch(tile + 2 * step);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        if (p.new_kv) {  // fused ring append: overwrite the rows just read
#pragma unroll 1
            for (int r = 0; r < kTile; ++r) {
                const int rr = __shfl_sync(kFull, row, r);
                if (rr >= 0)
                    reinterpret_cast<uint2*>(const_cast<__nv_bfloat16*>(p.src_kv) + ((size_t)rr * pairs + pair) * kD)[lane] =
                        __ldg(reinterpret_cast<const uint2*>(p.new_kv + ((size_t)(tile * kTile + r) * pairs + pair) * kD) + lane);
            }
        }

        float acc[16][4], delta[2];
        bulk_product(smem, xs, rdown, rnorm, acc, delta);

        // -- extremes, clip threshold and pair of every group (by 32-position block)
        float gmx[2][4], gmn[2][4], clip[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float h = acc[4 * b][2 * r], l = h;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h = fmaxf(h, fmaxf(acc[4 * b + i][2 * r], acc[4 * b + i][2 * r + 1]));
                    l = fminf(l, fminf(acc[4 * b + i][2 * r], acc[4 * b + i][2 * r + 1]));
                }
                h = fmaxf(h, __shfl_xor_sync(kFull, h, 1));
                l = fminf(l, __shfl_xor_sync(kFull, l, 1));
                gmx[r][b] = fmaxf(h, __shfl_xor_sync(kFull, h, 2));
                gmn[r][b] = fminf(l, __shfl_xor_sync(kFull, l, 2));
            }
            if (p.gshift >= 1) {
                gmx[r][0] = gmx[r][1] = fmaxf(gmx[r][0], gmx[r][1]);
                gmx[r][2] = gmx[r][3] = fmaxf(gmx[r][2], gmx[r][3]);
                gmn[r][0] = gmn[r][1] = fminf(gmn[r][0], gmn[r][1]);
                gmn[r][2] = gmn[r][3] = fminf(gmn[r][2], gmn[r][3]);
            }
            if (p.gshift >= 2) {
                gmx[r][0] = gmx[r][1] = gmx[r][2] = gmx[r][3] = fmaxf(gmx[r][0], gmx[r][2]);
                gmn[r][0] = gmn[r][1] = gmn[r][2] = gmn[r][3] = fminf(gmn[r][0], gmn[r][2]);
            }
        }
        // Clip threshold and pair of every group, and whether an error of delta
        // leaves it open (bit 4 r + b; the same in a group's blocks and in a quad)
        uint32_t open = 0;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float d = delta[r];
                const float t = cr < 1.f ? cr * fmaxf(gmx[r][b], -gmn[r][b]) : INFINITY;
                const float hi = fminf(gmx[r][b], t), lo = fmaxf(gmn[r][b], -t);
                const float sp = (hi - lo) * (1.f / 15.f), es = d * (2.f / 15.f) + sp * 4.8e-7f, ez = d + fabsf(lo) * 2.4e-7f;
                const uint32_t w0 = pack_f16x2_rn(sp - es, lo - ez), w1 = pack_f16x2_rn(sp + es, lo + ez);
                clip[r][b] = t;
                if (tq == 0) sz[(gID + 8 * r) * 4 + b] = w0;
                // (NaN bounds leave it open as well)
                if (!(sp - es <= sp + es && lo - ez <= lo + ez) || w0 != w1) open |= 1u << (4 * r + b);
            }
        // Candidates for the extremes of the open groups: elements within 2 delta of
        // them; count (bits 0-7) and sum of positions per row and block, then per group
        const uint32_t some = __reduce_or_sync(kFull, open);
        uint32_t cx[2][4], cn[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float d2 = 2.02f * delta[r];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                cx[r][b] = cn[r][b] = 0;
                if (!((some >> (4 * r + b)) & 1u)) continue;  // warp-uniform
                const float bx = gmx[r][b] - d2, bn = gmn[r][b] + d2;
                uint32_t x = 0, n = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float y = acc[4 * b + i][2 * r + e];
                        const uint32_t one = 1u + ((uint32_t)(32 * b + 8 * i + 2 * tq + e) << 8);
                        if (!(y < bx)) x += one;
                        if (!(y > bn)) n += one;
                    }
                x += __shfl_xor_sync(kFull, x, 1);
                n += __shfl_xor_sync(kFull, n, 1);
                cx[r][b] = x + __shfl_xor_sync(kFull, x, 2);
                cn[r][b] = n + __shfl_xor_sync(kFull, n, 2);
            }
            if (p.gshift >= 1) {
                cx[r][0] += cx[r][1];
                cx[r][2] += cx[r][3];
                cn[r][0] += cn[r][1];
                cn[r][2] += cn[r][3];
            }
            if (p.gshift >= 2) {
                cx[r][0] += cx[r][2];
                cn[r][0] += cn[r][2];
            }
        }
        uint32_t whole[2] = {0u, 0u};  // bit 4 gID + b: the group of (row gID + 8 r, block b) is taken from exact values as a whole
        group_sync();  // (the list's counter is zero)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (!((some >> (4 * r + b)) & 1u) || (b & (nb - 1))) continue;  // warp-uniform
                const bool mine = ((open >> (4 * r + b)) & 1u) && tq == 0;
                const bool single = (cx[r][b] & 0xffu) == 1u && (cn[r][b] & 0xffu) == 1u;
                whole[r] |= (__ballot_sync(kFull, mine && !single) & 0x11111111u) << b;
                if (mine && single)
                    list[atomicAdd(n_list, 1)] =
                        make_ushort4((unsigned short)(warp * kTile + gID + 8 * r), (unsigned short)b,
                                     (unsigned short)(cx[r][b] >> 8), (unsigned short)(cn[r][b] >> 8));
            }
        // The group's warps share the list (a tile opens about three groups,
        // some six or more): half warps take an entry each, a team of eight
        // lanes per extreme.
        group_sync();
        const int entries = *n_list;
        for (int e0 = 2 * (warp % kGroupWarps); e0 < entries; e0 += 2 * kGroupWarps) {
            const ushort4 en = list[min(e0 + (lane >> 4), entries - 1)];
            const df y = bulk_exact(smem, smem + BulkSmem::kX + en.x * kXPitch, (lane & 8) ? en.w : en.z, rdown);
            const df o{__shfl_xor_sync(kFull, y.hi, 8), __shfl_xor_sync(kFull, y.lo, 8)};
            df hi = (lane & 8) ? o : y, lo = (lane & 8) ? y : o;
            (void)bulk_clip(cr, hi, lo);
            const uint32_t w = bulk_pair(hi, lo);
            if ((lane & 15) < nb) reinterpret_cast<uint32_t*>(smem + BulkSmem::kSz)[en.x * 4 + en.y + (lane & 15)] = w;
        }
        group_sync();

        // -- codes: byte 4 n + tq of a row; an undecided code's bit 2 n + e in `late`
        uint32_t late[2] = {0u, 0u};
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t w = sz[(gID + 8 * r) * 4 + b];
                const float sf = half_lo(w), zf = half_hi(w), t = clip[r][b];
                const float inv = sf != 0.f ? __fdividef(1.f, sf) : 0.f;
                // u = y / s - z / s, two elements an instruction: off by delta / s, by the rounding of z / s (|z| is at most
                // |x| |R|, so a tenth of that) and by that of three fp32 operations on |u| < 16
                const float nz = -zf * inv, edge = 0.5f - (delta[r] * inv * 1.01f + fabsf(nz) * 1.2e-7f + 8e-6f);
                const float2 inv2 = make_float2(inv, inv), nz2 = make_float2(nz, nz), round2 = make_float2(12582912.f, 12582912.f);
                // u of the clip thresholds and of the codes' range, as one pair of bounds (s = 0: every code 0)
                const float ulo = sf != 0.f ? fmaxf(0.f, (-t - zf) * inv) : 0.f, uhi = sf != 0.f ? fminf(15.f, (t - zf) * inv) : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = 4 * b + i;
                    float2 u = fma2(make_float2(acc[n][2 * r], acc[n][2 * r + 1]), inv2, nz2);
                    u = make_float2(fminf(fmaxf(u.x, ulo), uhi), fminf(fmaxf(u.y, ulo), uhi));
                    const float2 m = add2(u, round2);  // 1.5 2^23: rounds u to an integer, in the low bits
                    const float2 off = sub2(u, sub2(m, round2));
                    if (!(fabsf(off.x) < edge)) late[r] |= 1u << (2 * n);
                    if (!(fabsf(off.y) < edge)) late[r] |= 2u << (2 * n);
                    stg[(gID + 8 * r) * kStgPitch + 4 * n + tq] = (uint8_t)(__float_as_uint(m.x) + (__float_as_uint(m.y) << 4));
                }
            }
        __syncwarp();
        for (;;) {
            const uint32_t who = __ballot_sync(kFull, (late[0] | late[1]) != 0u);
            if (!who) break;
            const int src = __ffs(who) - 1;
            const int r = late[0] ? 0 : 1;
            int item = 64 * r + __ffs(r ? late[1] : late[0]) - 1;  // (of each lane; the chosen lane's is taken)
            item = __shfl_sync(kFull, item, src);
            const int rr = item >> 6, n = (item & 63) >> 1, e = item & 1, g = src >> 2;
            if (lane == src) {
                if (rr) late[1] &= late[1] - 1;
                else late[0] &= late[0] - 1;
            }
            const int row16 = g + 8 * rr, pos = 8 * n + 2 * (src & 3) + e, b0 = (n >> 2) & ~(nb - 1);
            if ((whole[rr] >> (4 * g + b0)) & 1u) continue;  // taken as a whole below
            const df y = bulk_exact(smem, xs + row16 * kXPitch, pos, rdown);
            float t = 0.f, d = 0.f;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b == b0) t = rr ? clip[1][b] : clip[0][b];
            t = __shfl_sync(kFull, t, src);
            d = __shfl_sync(kFull, rr ? delta[1] : delta[0], src);
            if (!(fabsf(y.hi) < t - 2.f * d)) {  // at the clip threshold: its exact value is needed too
                whole[rr] |= 1u << (4 * g + b0);
                continue;
            }
            if (lane == src) {
                const uint32_t w = sz[row16 * 4 + (n >> 2)];
                const uint32_t code = (uint32_t)code4_of(y, half_lo(w), half_hi(w));
                uint8_t* at = stg + row16 * kStgPitch + (pos >> 1);
                *at = (uint8_t)(e ? (*at & 0x0f) | (code << 4) : (*at & 0xf0) | code);
            }
            __syncwarp();
        }
#pragma unroll 1
        for (int r = 0; r < 2; ++r)
            for (uint32_t m = r ? whole[1] : whole[0]; m; m &= m - 1) {
                const int bit = __ffs(m) - 1, row16 = (bit >> 2) + 8 * r;
                bulk_group_exact(smem, xs + row16 * kXPitch, stg + row16 * kStgPitch, sz + row16 * 4, bit & 3, nb, cr, rdown);
            }
        __syncwarp();
        copy_rows(now.row);  // the next tile's (these rows have been read for the last time)

        // -- stores
        if (which == 0) {  // 16-byte chunk a of a token: word k = bytes 16 k + 4 a .. + 3
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                const int t = 8 * it + gID;
                const uint32_t* w = reinterpret_cast<const uint32_t*>(stg + t * kStgPitch) + tq;
                if (dst[t])
                    *reinterpret_cast<uint4*>(dst[t] + slots[t] * (kD / 2) + 16 * tq) = make_uint4(w[0], w[4], w[8], w[12]);
            }
        } else {  // plane j, four tokens at a time
            const int t0 = 4 * tq;
            uint8_t* const d0 = dst[t0];
            const int s0 = slots[t0];
            const bool joined = d0 && (s0 & 3) == 0 && dst[t0 + 1] == d0 && dst[t0 + 2] == d0 && dst[t0 + 3] == d0 &&
                                slots[t0 + 1] == s0 + 1 && slots[t0 + 2] == s0 + 2 && slots[t0 + 3] == s0 + 3;
#pragma unroll
            for (int it = 0; it < 2; ++it) {  // planes 4 (gID + 8 it) .. + 3
                const int j4 = gID + 8 * it;
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const uint32_t*>(stg + (t0 + i) * kStgPitch)[j4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w01 = __byte_perm(v[0], v[1], 0x0040u + 0x0011u * i), w23 = __byte_perm(v[2], v[3], 0x0040u + 0x0011u * i);
                    const uint32_t w = __byte_perm(w01, w23, 0x5410u);
                    const int plane = (4 * j4 + i) * kPage;
                    if (joined) {
                        *reinterpret_cast<uint32_t*>(d0 + plane + s0) = w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (dst[t0 + k]) dst[t0 + k][plane + slots[t0 + k]] = (uint8_t)(w >> (8 * k));
                    }
                }
            }
        }
        if (lane < kTile && dst[lane]) {
            const int ng = sz_pairs(p.gshift);
            const uint32_t* w = sz + lane * 4;
            uint8_t* to = dst[lane] + kCodes4 + slots[lane] * 4 * ng;
            if (ng == 4) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            else if (ng == 2) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[2]);
            else *reinterpret_cast<uint32_t*>(to) = w[0];
        }
    }
}

}  // namespace

cudaError_t launch_evict_bulk(const EvictParams& p, cudaStream_t st) {
    static int sms[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (sms[dev & 63] == 0) {
        e = cudaFuncSetAttribute(evict_bulk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BulkSmem::kBytes);
        if (e != cudaSuccess) return e;
        e = cudaDeviceGetAttribute(&sms[dev & 63], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
    }
    const int pairs = 2 * p.hk, tiles = (p.n_tok + kTile - 1) / kTile;
    const int share = std::max(1, std::min((tiles + kBulkWarps - 1) / kBulkWarps, sms[dev & 63] / pairs));
    e = launch_pdl(evict_bulk_kernel, dim3(pairs * share), dim3(kBulkThreads), BulkSmem::kBytes, st, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace oscar
