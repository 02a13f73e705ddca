// int4.cu -- split-K decode attention over the 4-bit history (blocks of
// oscar_evict_quantize_int4), between prep_kernel and bf16_kernel of the
// decode chain (decode.cu), which are those of the 2-bit history: rotated
// query fragments and plan before, un-rotation and log-sum-exp merge after.
//
// The mathematics.  A stored value is s c + z (c in 0..15, one fp16 pair per
// token and quantisation group b):
//   logit_t = sum_b s_tb D_tb + z_tb Q_b,  D_tb = sum_{j in b} c_tj q'_j,
//                                          Q_b = sum_{j in b} q'_j;
//   o'_j    = sum_t W_tb(j) (c_tj - 8) + sum_t p_t z'_tb,  W_tb = p_t s_tb,
//                                          z' = z + 8 s.
// D and the W products are tensor-core products (mma.sync m16n8k16, fp16 in,
// fp32 sums) with the codes as the A operand, exact in fp16; q' (times 2^e,
// from prep) and W (times 2^w) enter as fp16 high and low parts, 22 bits.
// The V codes are centred so that a flat softmax over a long history does
// not subtract two sums far larger than their difference (7.5 s against the
// values' 4.6 s, both times sum p, where the result is of the order of 4.6 s
// sqrt(sum p^2)), and their products are summed page by page (page_values).
// A logit has 128 terms and no such difference: K codes stay as they are.
//
// Operands of V, by the method of Kim, Henry, Fahim and Hassan Awadalla, "Who
// Says Elephants Can't Run" (2022): a 16-bit pattern 0x6400 | c is the fp16 1024 + c and
// 0x6400 | 16 c is 1024 + 16 c: one AND-OR on the code word in place and one
// fp16 add (-1032) or fused multiply-add (/ 16, -72) give c - 8 exactly; a
// shift by 8 serves the other two nibbles of each half: nine instructions
// for a word of eight codes, against seven for the K codes' in_place4.
//
// 2^w: W is scaled by a power of two per warp and item, from the largest V
// scale seen so far, so that its fp16 parts keep 22 bits whatever the
// values' size; a page with a larger scale rescales the sums.
//
// What bounds it: 160 bytes and 4 d G flops per (token, KV head) make it a
// stream of the pages, so K and V halves travel separately (each consumer
// warp owns a ring of halves and gives one back as soon as it has read it).
// Measured (GB300, copy peak 6.79 TB/s): batch 64, 4K-32K, four heads per KV
// head, groups of 32: 275 us for 1.44 GB, 5.2 TB/s; 32 x 32K, eight heads,
// groups of 128: 266 us for 1.13 GB, 4.2 TB/s.  The first is bound by its
// instructions (about 350 per 16-token tile, issued in 63 % of the cycles by
// 12 consumer warps per SM), the second by its products (tensor pipe 44 %) and
// their latency (issue 52 %).  The code of a page is kept small and free of
// divergent branches for the same reason: with separate code for partial pages,
// every tile unrolled and the waits polled lane by lane it took 295 and 282 us.
#include <algorithm>
#include <type_traits>

#include "splitk.cuh"

namespace oscar {

namespace {

static_assert(kPartsPerItem4 == kConsumerWarps, "a partial per consumer warp");
constexpr int kThreads4 = (kConsumerWarps + 1) * 32;
constexpr int kHalfMax = kCodes4 + kPage * 16;  // bytes of a half at g = 32

struct PageInfo {  // one per page of a consumer warp; 16 bytes
    int item, bk, page, valid_flags;  // (sequence, KV head) and page of its history (-1: none): kModeWeights
};

template <Mode MODE>
using Params4 = std::conditional_t<MODE == kModePlain, DecodeParams4, DecodeParamsX>;

// A probability or V-scale row of the value phase: the page's 64 tokens in 16
// groups of four; k-step m of lane quad member tq covers group 4 tq + m (whose V
// codes are bytes 16 tq + 4 m .. + 3 of every plane, so that one 16-byte load
// per plane serves the four k-steps).  Group q lies at 20 (q / 4) + 4 (q % 4): the
// skew of 20 keeps the lanes of a load on distinct banks and every k-step or
// tile at a constant offset from the lane's own place; inside a group the
// order is pv_slot (tokens 0, 2 | 1, 3: the two B-operand pairs).
constexpr int kRow4 = 80;
__device__ __forceinline__ int row_pos(int t) { return 20 * (t >> 4) + 4 * ((t >> 2) & 3) + pv_slot(t & 3); }

template <int NT, int GS>
struct Int4Smem {
    static constexpr int G4 = NT * 4;
    // halves per consumer warp: three (one being read, two in flight); with
    // the larger scratch of eight heads two where three blocks share an SM,
    // four where two do
    static constexpr int kBlocks = int4_blocks_per_sm(NT, GS);
    static constexpr int NSW = NT == 1 ? 3 : kBlocks == 3 ? 2 : 4;
    // per-warp scratch (NB groups per vector).  Logit phase: K s [64][NB] | K z
    // [64][NB].  Value phase: V s 2^w [NB][kRow4] (token order row_pos) | V z'
    // [64][NB], then P [G4][kRow4] over the z'.
    static constexpr int kWVs = 0, kWVz = 4 * kRow4 * 4, kWP = kWVz;
    static constexpr int kWarp1 = 2 * kPage * 16, kWarp2 = kWP + G4 * kRow4 * 4;
    static constexpr int kWarpBytes = kWarp1 > kWarp2 ? kWarp1 : kWarp2;
    static constexpr int kStage = 0;
    static constexpr int kInfo = kStage + kConsumerWarps * NSW * kHalfMax;  // [4][2] PageInfo
    static constexpr int kWarp = kInfo + kConsumerWarps * 2 * 16;
    // two item buffers: q' fragments [NT][8][32] uint2, group sums [G4] float4, 2^-e
    static constexpr int kQbSum = NT * 8 * 32 * 8, kQbKinv = kQbSum + G4 * 16, kQbBytes = kQbKinv + 16;
    static constexpr int kQb = kWarp + kConsumerWarps * kWarpBytes;
    // full / empty per half, qfull[2], qempty[2]
    static constexpr int kBars = kQb + 2 * kQbBytes;
    static constexpr int kBytes = kBars + (2 * kConsumerWarps * NSW + 4) * 8;
    static_assert(kWarp % 16 == 0 && kWarpBytes % 16 == 0 && kQb % 16 == 0 && kQbBytes % 16 == 0 && kBars % 8 == 0,
                  "16-byte vectors and bulk copies");
    static_assert(kBlocks * (kBytes + 1024) <= 228 * 1024, "blocks per SM");
};

// Ring position: half `slot` of NSW, in its `phase`-th use.
template <int NSW>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step() {
        if (++slot == NSW) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// mbar_wait_bounded by a whole warp: one branch per poll, the same for every lane
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    return __all_sync(kFull, mbar_wait_bounded(bar, parity, kWaitPolls));
}

__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
    return r;
}

// Eight codes of a word as four f16x2 operand registers of c - 8: nibble n
// of the low and of the high half.
__device__ __forceinline__ void unpack4(uint32_t x, uint32_t (&r)[4]) {
    const uint32_t y = x >> 8;
    const uint32_t n0 = and_or(x, 0x000f000fu, 0x64006400u), n1 = and_or(x, 0x00f000f0u, 0x64006400u);
    const uint32_t n2 = and_or(y, 0x000f000fu, 0x64006400u), n3 = and_or(y, 0x00f000f0u, 0x64006400u);
    // 0xE408 = -1032, 0x2C00 = 1/16, 0xD480 = -72
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r[0]) : "r"(n0), "r"(0xE408E408u));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[1]) : "r"(n1), "r"(0x2C002C00u), "r"(0xD480D480u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r[2]) : "r"(n2), "r"(0xE408E408u));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[3]) : "r"(n3), "r"(0x2C002C00u), "r"(0xD480D480u));
}

// N consecutive floats of shared memory (N = 1, 2, 4; aligned to them).
template <int N>
__device__ __forceinline__ void load_n(const float* at, float (&v)[N]) {
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4*>(at);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else if constexpr (N == 2) {
        const float2 x = *reinterpret_cast<const float2*>(at);
        v[0] = x.x; v[1] = x.y;
    } else {
        v[0] = *at;
    }
}
template <int N>
__device__ __forceinline__ void store_n(float* at, const float (&v)[N]) {
    if constexpr (N == 4) *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
    else if constexpr (N == 2) *reinterpret_cast<float2*>(at) = make_float2(v[0], v[1]);
    else *at = v[0];
}

// The K codes stay uncentred and in place: a 16-bit pattern below 0x0400 is an
// fp16 of value pattern 2^-24, so a nibble at bits 4-7 reads c 2^-20; three
// shifts and four ANDs for eight codes.
constexpr float kInPlaceUp = 1048576.f;  // 2^20
__device__ __forceinline__ void in_place4(uint32_t x, uint32_t (&r)[4]) {
    r[0] = (x << 4) & 0x00f000f0u;
    r[1] = x & 0x00f000f0u;
    r[2] = (x >> 4) & 0x00f000f0u;
    r[3] = (x >> 8) & 0x00f000f0u;
}

// The (s, z) words of token t of a half, one per quantisation group.
template <int NB>
__device__ __forceinline__ void load_pairs(const uint8_t* half, int t, uint32_t (&w)[NB]) {
    const uint8_t* at = half + kCodes4 + t * 4 * NB;
    if constexpr (NB == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(at);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (NB == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    }
}

__device__ __forceinline__ float pow2_bits(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// State of one consumer warp inside an item.  NB = 4 >> GS quantisation groups
// per vector, of 4 / NB 32-position blocks each.
template <int NT, int GS>
struct WarpState {
    float m_run[NT], l_run[NT], zacc[NT][4 >> GS];  // per head of the lane: max, sum, sum p z' per group (lane partials)
    // [M tile][row gID: columns 2tq, 2tq+1; row gID+8]; up to four heads: columns = (hi, lo) of head tq; eight: heads 2tq, 2tq+1
    float acc[8][4];
    int wexp;                                       // 2^wexp scales W; kNoScale before the first page
};
constexpr int kNoScale = 64;

// How the products of a page are laid out in the code: kTiles token tiles of 16
// per turn of a loop (less code to fetch, against less to schedule), kSide of them
// (logits) and kSideV M tiles (values) side by side, so that their chains of
// products interleave and share the B fragments.  32 x 32K, eight KV heads, us, as (kTiles, kSide,
// kSideV) for groups of 32, 64, 128:
//            1,1,1          2,2,2          4,2,1          4,4,2
// 4 heads    275 239 226    283 232 216    291 229 213    289 247 219
// 8 heads    422 370 315    411 358 318    435 333 295    407 345 300
template <int NT, int GS>
struct Shape {
    static constexpr int kTiles = NT == 1 && GS == 0 ? 1 : 4, kSide = GS > 0 ? 2 : NT == 1 ? 1 : 4, kSideV = GS > 0 ? 1 : NT;
};

// K half of a page: logits (base 2) of the lane's tokens 16m + gID and
// 16m + gID + 8.  Up to four heads: lg[m][0], lg[m][1] = the two tokens of
// head tq; eight heads: (token a, heads 2tq, 2tq+1), (token b, the same).
template <int NT, int GS>
__device__ __forceinline__ void page_logits(const uint8_t* half, int valid, uint8_t* wbuf, const uint2* qf,
                                            const float (&qsv)[NT][4 >> GS], float kq, float (&lg)[4][2 * NT]) {
    constexpr int NB = 4 >> GS;
    const int lane = threadIdx.x & 31, gID = lane >> 2, tq = lane & 3;
    float* ksS = reinterpret_cast<float*>(wbuf);  // [64][NB]
    float* kzS = ksS + kPage * NB;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int t = lane + 32 * it;
        float sv[NB], zv[NB];
        uint32_t w[NB];
        load_pairs<NB>(half, t, w);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float s = half_lo(w[b]);
            sv[b] = s * (kq * kInPlaceUp);
            zv[b] = half_hi(w[b]);
        }
        store_n<NB>(ksS + t * NB, sv);
        store_n<NB>(kzS + t * NB, zv);
    }
    __syncwarp();
    constexpr int kTiles = Shape<NT, GS>::kTiles, kSide = Shape<NT, GS>::kSide;
#pragma unroll 1
    for (int m0 = 0; m0 < 4; m0 += kTiles) {
        float cur[kTiles][2 * NT];
#pragma unroll
        for (int m1 = 0; m1 < kTiles; m1 += kSide) {
            uint32_t wa[kSide][4], wb[kSide][4];
            float acc[kSide][NB][4];
#pragma unroll
            for (int i = 0; i < kSide; ++i) {
                const int ta = 16 * (m0 + m1 + i) + gID;
                const uint4 xa = *reinterpret_cast<const uint4*>(half + ta * (kD / 2) + 16 * tq);
                const uint4 xb = *reinterpret_cast<const uint4*>(half + (ta + 8) * (kD / 2) + 16 * tq);
                wa[i][0] = xa.x; wa[i][1] = xa.y; wa[i][2] = xa.z; wa[i][3] = xa.w;
                wb[i][0] = xb.x; wb[i][1] = xb.y; wb[i][2] = xb.z; wb[i][3] = xb.w;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][b][e] = 0.f;
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t ra[kSide][4], rb[kSide][4];
#pragma unroll
                for (int i = 0; i < kSide; ++i) {
                    in_place4(wa[i][b], ra[i]);
                    in_place4(wb[i][b], rb[i]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {  // eight heads: the high, then the low parts
                        const uint2 q = qf[(nt * 8 + 2 * b + h) * 32 + lane];
#pragma unroll
                        for (int i = 0; i < kSide; ++i)
                            mma_f16_16816(acc[i][b >> GS], ra[i][2 * h], rb[i][2 * h], ra[i][2 * h + 1], rb[i][2 * h + 1], q.x, q.y);
                    }
            }
#pragma unroll
            for (int i = 0; i < kSide; ++i) {
                const int m = m1 + i, ta = 16 * (m0 + m) + gID;
                float sa[NB], za[NB], sb[NB], zb[NB];
                load_n<NB>(ksS + ta * NB, sa);
                load_n<NB>(ksS + (ta + 8) * NB, sb);
                load_n<NB>(kzS + ta * NB, za);
                load_n<NB>(kzS + (ta + 8) * NB, zb);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float x = 0.f, y = 0.f;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        x = fmaf(sa[b], NT == 1 ? acc[i][b][0] + acc[i][b][1] : acc[i][b][j], fmaf(za[b], qsv[j][b], x));
                        y = fmaf(sb[b], NT == 1 ? acc[i][b][2] + acc[i][b][3] : acc[i][b][2 + j], fmaf(zb[b], qsv[j][b], y));
                    }
                    cur[m][j] = x;
                    cur[m][NT == 1 ? 1 : 2 + j] = y;
                }
            }
        }
        // the tiles move up: tile m ends in lg[m] after the last turn
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int e = 0; e < 2 * NT; ++e) lg[m][e] = m + kTiles < 4 ? lg[(m + kTiles) & 3][e] : cur[(m + kTiles) & (kTiles - 1)][e];
    }
    if (valid < kPage) {  // whatever the slots behind the last token hold, NaN included
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (16 * m + gID >= valid) lg[m][j] = -INFINITY;
                if (16 * m + gID + 8 >= valid) lg[m][NT == 1 ? 1 : 2 + j] = -INFINITY;
            }
    }
}

// Online softmax of a page's logits: lg becomes p, l_run advances, alpha is
// the factor that the older sums take.  Returns whether any lane's is not 1.
template <int NT, int GS>
__device__ __forceinline__ bool page_softmax(float (&lg)[4][2 * NT], WarpState<NT, GS>& st, float (&alpha)[NT]) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < NT; ++j) {  // j: token pair entries (NT == 1: 0 and 1; NT == 2: j and 2 + j)
        const int e1 = NT == 1 ? 1 : 2 + j;
        float mx = fmaxf(lg[0][j], lg[0][e1]);
#pragma unroll
        for (int m = 1; m < 4; ++m) mx = fmaxf(mx, fmaxf(lg[m][j], lg[m][e1]));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
        const float m_new = fmaxf(st.m_run[j], mx);
        alpha[j] = 1.f;
        if (__any_sync(kFull, m_new > st.m_run[j])) {
            any = true;
            alpha[j] = (m_new > st.m_run[j]) ? ex2(st.m_run[j] - m_new) : 1.f;
            st.l_run[j] *= alpha[j];
            st.m_run[j] = m_new;
        }
        const float sub = (m_new == -INFINITY) ? 0.f : m_new;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            lg[m][j] = ex2(lg[m][j] - sub);
            lg[m][e1] = ex2(lg[m][e1] - sub);
            st.l_run[j] += lg[m][j] + lg[m][e1];
        }
    }
    return any;
}

// V half of a page: the scales, the rescaling of the sums, sum p z', and the
// products W . (c - 8).
template <int NT, int GS>
__device__ __forceinline__ void page_values(const uint8_t* half, int valid, uint8_t* wbuf, const float (&p)[4][2 * NT],
                                            const float (&alpha)[NT], bool any, const SplitSel& take_lo,
                                            WarpState<NT, GS>& st) {
    using SM = Int4Smem<NT, GS>;
    constexpr int NB = 4 >> GS;
    const int lane = threadIdx.x & 31, gID = lane >> 2, tq = lane & 3;
    float* vsS = reinterpret_cast<float*>(wbuf + SM::kWVs);  // [NB][kRow4]
    float* vzS = reinterpret_cast<float*>(wbuf + SM::kWVz);  // [64][NB]
    float* pS = reinterpret_cast<float*>(wbuf + SM::kWP);
    // -- pairs; the largest scale of the page picks 2^w: s 2^w < 2^14
    uint32_t w[2][NB];
    uint32_t smax = 0;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int t = lane + 32 * it;
        load_pairs<NB>(half, t, w[it]);
        if (valid < kPage && t >= valid)
#pragma unroll
            for (int b = 0; b < NB; ++b) w[it][b] = 0u;
#pragma unroll
        for (int b = 0; b < NB; ++b) smax = max(smax, w[it][b] & 0x7fffu);
    }
    smax = __reduce_max_sync(kFull, smax);
    const int wexp = 13 - (max((int)(smax >> 10), 1) - 15);
    if (any || wexp < st.wexp) {  // warp-uniform
        float down = 1.f;
        if (wexp < st.wexp) {
            down = st.wexp == kNoScale ? 0.f : pow2_bits(wexp - st.wexp);  // (no sums before the first page)
            st.wexp = wexp;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int b = 0; b < NB; ++b) st.zacc[j][b] *= alpha[j];
        // column 2tq + e: up to four heads, both columns belong to head tq; eight: heads 2tq, 2tq + 1
        const float f0 = alpha[0] * down, f1 = alpha[NT - 1] * down;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            st.acc[mt][0] *= f0;
            st.acc[mt][1] *= f1;
            st.acc[mt][2] *= f0;
            st.acc[mt][3] *= f1;
        }
    }
    const float up = pow2_bits(st.wexp);
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int t = lane + 32 * it, ps = row_pos(lane) + 40 * it;
        float z[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float s = half_lo(w[it][b]);
            z[b] = fmaf(8.f, s, half_hi(w[it][b]));
            vsS[b * kRow4 + ps] = s * up;
        }
        store_n<NB>(vzS + t * NB, z);
    }
    __syncwarp();
    // -- sum p z'
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int ta = 16 * m + gID;
        float zA[NB], zB[NB];
        load_n<NB>(vzS + ta * NB, zA);
        load_n<NB>(vzS + (ta + 8) * NB, zB);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                st.zacc[j][b] = fmaf(p[m][j], zA[b], fmaf(p[m][NT == 1 ? 1 : 2 + j], zB[b], st.zacc[j][b]));
    }
    __syncwarp();  // z' read: P takes its place
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float* row = pS + (NT == 1 ? tq : 2 * tq + j) * kRow4 + row_pos(gID) + 20 * m;
            row[0] = p[m][j];
            row[8] = p[m][NT == 1 ? 1 : 2 + j];
        }
    __syncwarp();
    // -- products: M tile mt = planes 8 mt + gID (rows gID: position
    //    16 mt + 2 gID, rows gID + 8: the next one), k-step m = token group
    //    4 tq + m.  W of group b and k-step m: B registers (b0, b1), eight
    //    heads also their low parts
    auto weights = [&](int b, int m, uint32_t (&r)[2 * NT]) {
        const int chunk = 20 * tq + 4 * m;
        const float4 pp = *reinterpret_cast<const float4*>(pS + (NT == 1 ? gID >> 1 : gID) * kRow4 + chunk);
        const float4 sg = *reinterpret_cast<const float4*>(vsS + b * kRow4 + chunk);
        const float2 p0 = make_float2(pp.x, pp.y), p1 = make_float2(pp.z, pp.w);
        const float2 s0 = make_float2(sg.x, sg.y), s1 = make_float2(sg.z, sg.w);
        if constexpr (NT == 1) {
            r[0] = split_w_pair_f16(p0, s0, take_lo);
            r[1] = split_w_pair_f16(p1, s1, take_lo);
        } else {
            split_both(mul2(p0, s0), r[0], r[2]);
            split_both(mul2(p1, s1), r[1], r[3]);
        }
    };
    // One block (two M tiles) at a time, summed over the page from zero and then
    // added to the running sums in fp32: the tensor core truncates its
    // accumulator at every step, always toward zero, which over the
    // hundreds of steps of an item shrinks a flat softmax's small result by
    // 10^-5; four steps from zero and one rounded addition do not.
    const uint8_t* vb = half + gID * kPage + 16 * tq;
    uint32_t r[4][2 * NT];  // the block's group's W
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (GS == 0 || (b & ((1 << GS) - 1)) == 0)
#pragma unroll
            for (int m = 0; m < 4; ++m) weights(b >> GS, m, r[m]);
        constexpr int kSideV = Shape<NT, GS>::kSideV;
#pragma unroll
        for (int k0 = 0; k0 < 2; k0 += kSideV) {
            uint4 v[kSideV];
            float t[kSideV][4];
#pragma unroll
            for (int k = 0; k < kSideV; ++k) {
                v[k] = *reinterpret_cast<const uint4*>(vb + (2 * b + k0 + k) * 8 * kPage);
                t[k][0] = t[k][1] = t[k][2] = t[k][3] = 0.f;
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t c[kSideV][4];
#pragma unroll
                for (int k = 0; k < kSideV; ++k) unpack4(m == 0 ? v[k].x : m == 1 ? v[k].y : m == 2 ? v[k].z : v[k].w, c[k]);
#pragma unroll
                for (int k = 0; k < kSideV; ++k) mma_f16_16816(t[k], c[k][0], c[k][1], c[k][2], c[k][3], r[m][0], r[m][1]);
                if constexpr (NT == 2)
#pragma unroll
                    for (int k = 0; k < kSideV; ++k) mma_f16_16816(t[k], c[k][0], c[k][1], c[k][2], c[k][3], r[m][2], r[m][3]);
            }
#pragma unroll
            for (int k = 0; k < kSideV; ++k) {
                float(&acc)[4] = st.acc[2 * b + k0 + k];
                const float2 a0 = add2(make_float2(acc[0], acc[1]), make_float2(t[k][0], t[k][1]));
                const float2 a1 = add2(make_float2(acc[2], acc[3]), make_float2(t[k][2], t[k][3]));
                acc[0] = a0.x;
                acc[1] = a0.y;
                acc[2] = a1.x;
                acc[3] = a1.y;
            }
        }
    }
}

// Persistent blocks: the producer warp takes split-K items from the work
// counter and streams their pages, page i of an item to consumer warp i % 4,
// as two halves (K, then V) into the warp's ring; in each round of four
// pages the four K halves go first.  A consumer warp writes its own partial
// state at an item's end and goes on with the next item: a merge of the four
// in shared memory cost about four pages' time per item.  Every wait is bounded: on a timeout the
// block reports OSCAR_STATUS_TIMEOUT, lets its copies land and exits.
template <int NT, int GS, Mode MODE>
__global__ void __launch_bounds__(kThreads4, int4_blocks_per_sm(NT, GS)) int4_kernel(Params4<MODE> p) {
    extern __shared__ __align__(128) uint8_t smem[];
    using SM = Int4Smem<NT, GS>;
    constexpr int NSW = SM::NSW, NB = 4 >> GS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars);  // [warp][NSW]
    uint64_t* empty = full + kConsumerWarps * NSW;
    uint64_t* qfull = empty + kConsumerWarps * NSW;
    uint64_t* qempty = qfull + 2;
    PageInfo* info = reinterpret_cast<PageInfo*>(smem + SM::kInfo);  // [warp][2]
    constexpr uint32_t half_bytes = kCodes4 + kPage * 4 * NB;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kConsumerWarps * NSW; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&qfull[s], 1);
            mbar_init(&qempty[s], kConsumerWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();     // q' fragments, plan and counter come from prep_kernel
    pdl_trigger();  // the BF16 segment kernel may take SMs as this grid retires

    if (warp == kConsumerWarps) {
        // ------------------------------ producer ------------------------------
        const int pps = p.counter[kPlanPps], tail_pg = p.counter[kPlanTail];  // from prep_kernel
        const int total_long = __ldg(p.item_start + p.B);
        const int total = total_long + __ldg(p.item_start2 + p.B);
        Ring<NSW> ring;       // the same for the four warps: every round gives each two halves
        uint32_t halves = 0;  // halves issued to each warp
        uint32_t round = 0, pitem = 0;
        bool ok = true;
        // wait until the ring's slot is free in the four warps (lane w polls
        // warp w's barrier, so that one wait covers the round)
        auto wait_free = [&]() -> bool {
            if (halves < (uint32_t)NSW) return true;
            const bool w = lane >= kConsumerWarps ||
                           mbar_wait_bounded(&empty[lane * NSW + ring.slot], ring.phase ^ 1u, kWaitPolls);
            return __all_sync(kFull, w);
        };
        for (;;) {
            int item = 0;
            if (lane == 0) item = atomicAdd(p.counter, 1);
            item = __shfl_sync(kFull, item, 0);
            if (item >= total) {  // an end marker for each consumer warp
                ok = wait_free();
                if (ok && lane < kConsumerWarps) {
                    info[lane * 2 + (round & 1u)].item = -1;
                    mbar_arrive(&full[lane * NSW + ring.slot]);
                }
                break;
            }
            const bool is_long = item < total_long;
            const int32_t* starts = is_long ? p.item_start : p.item_start2;
            const int rel = is_long ? item : item - total_long;
            const int b = find_seq(starts, p.B, rel);
            const int s0 = __ldg(starts + b);
            const int splits = (__ldg(starts + b + 1) - s0) / p.hk;
            const int kv = (rel - s0) / splits;
            const int split = (rel - s0) % splits;
            int hist = min(max(__ldg(p.hist_len + b), 0), p.max_pages * kPage);
            const int32_t* table = p.page_table + (size_t)b * p.max_pages;
            if constexpr (MODE == kModeShared) {  // the pages behind the shared ones
                const int skip = __ldg(p.skip + b);
                hist -= skip * kPage;
                table += skip;
            }
            const int seq_pages = (hist + kPage - 1) / kPage;
            const SeqSplits sp = seq_splits(seq_pages, pps, tail_pg);
            const int pg0 = is_long ? split * pps : sp.long_pages + split * kShortItemPages;
            const int npg = is_long ? min(pps, sp.long_pages - pg0) : min(kShortItemPages, seq_pages - pg0);
            const int rounds = (npg + kConsumerWarps - 1) / kConsumerWarps;
            {   // the item's q' data into its buffer, once item k - 2 has left it
                const uint32_t qs = pitem & 1u;
                if (pitem >= 2) {
                    const bool w = mbar_wait_bounded(&qempty[qs], ((pitem >> 1) - 1) & 1u, kWaitPolls);
                    if (!__all_sync(kFull, w)) {
                        ok = false;
                        break;
                    }
                }
                if (lane == 0) {
                    const size_t bk = (size_t)b * p.hk + kv;
                    uint8_t* qb = smem + SM::kQb + qs * SM::kQbBytes;
                    mbar_arrive_expect_tx(&qfull[qs], SM::kQbBytes);
                    bulk_g2s(qb, p.qfrag + bk * NT * 8 * 32 * 2, NT * 8 * 32 * 8, &qfull[qs]);
                    bulk_g2s(qb + SM::kQbSum, p.qsum + bk * SM::G4 * 4, SM::G4 * 16, &qfull[qs]);
                    bulk_g2s(qb + SM::kQbKinv, p.qkinv + bk * 4, 16, &qfull[qs]);
                }
                __syncwarp();
                ++pitem;
            }
            int pid = -1;
            for (int r = 0; r < rounds && ok; ++r, ++round) {
                if ((r & 7) == 0) {  // page ids of the next eight rounds, one per lane
                    const int pl = 4 * r + lane;
                    pid = pl < npg ? __ldg(table + pg0 + pl) : -1;
                }
                // lane w < 4 serves warp w: page 4 r + w of the item
                const int pl = 4 * r + (lane & 3);
                const int page = __shfl_sync(kFull, pid, (4 * r + (lane & 3)) & 31);
                bool pad = pl >= npg;
                if (!pad && (page < 0 || page >= p.num_pages)) {
                    if (lane < kConsumerWarps) report(p.status, OSCAR_STATUS_BAD_PAGE);
                    pad = true;
                }
                const uint8_t* src = p.pool + ((size_t)(pad ? 0 : page) * p.hk + kv) * p.block_bytes;
                if (!(ok = wait_free())) break;
                if (lane < kConsumerWarps) {
                    const int flags = (r == 0 ? kFlagFirst : 0) | (r == rounds - 1 ? kFlagLast : 0) | (pad ? kFlagPad : 0);
                    PageInfo& pi = info[lane * 2 + (round & 1u)];
                    pi.item = item;
                    if constexpr (MODE == kModeWeights) {
                        pi.bk = b * p.hk + kv;
                        pi.page = pl < npg ? pg0 + pl : -1;
                    }
                    pi.valid_flags = (pad ? 0 : min(kPage, hist - (pg0 + pl) * kPage)) | (flags << 8);
                    uint64_t* bar = &full[lane * NSW + ring.slot];
                    if (pad) {
                        mbar_arrive(bar);
                    } else {
                        mbar_arrive_expect_tx(bar, half_bytes);
                        bulk_g2s(smem + SM::kStage + (lane * NSW + ring.slot) * kHalfMax, src, half_bytes, bar);
                    }
                }
                __syncwarp();
                ring.step();
                ++halves;
                if (!(ok = wait_free())) break;
                if (lane < kConsumerWarps) {
                    uint64_t* bar = &full[lane * NSW + ring.slot];
                    if (pad) {
                        mbar_arrive(bar);
                    } else {
                        mbar_arrive_expect_tx(bar, half_bytes);
                        bulk_g2s(smem + SM::kStage + (lane * NSW + ring.slot) * kHalfMax, src + half_bytes, half_bytes, bar);
                    }
                }
                __syncwarp();
                ring.step();
                ++halves;
            }
            if (!ok) break;
        }
        if (!ok) {
            if (lane == 0) report(p.status, OSCAR_STATUS_TIMEOUT);
            // let issued copies land before the block can exit: the last use of every slot
            for (int s = 0; s < NSW; ++s) {
                if ((uint32_t)s >= halves) break;
                // slots at or past the ring position were last used a turn earlier
                const uint32_t ph = s < ring.slot ? ring.phase : ring.phase ^ 1u;
                if (lane < kConsumerWarps) (void)mbar_wait_bounded(&full[lane * NSW + s], ph, kWaitPolls);
                __syncwarp();
            }
            for (uint32_t k = pitem > 2 ? pitem - 2 : 0; k < pitem; ++k)
                (void)mbar_wait_bounded(&qfull[k & 1u], (k >> 1) & 1u, kWaitPolls);
        }
        return;
    }

    // ------------------------------- consumers ---------------------------------
    const int gID = lane >> 2, tq = lane & 3;
    uint8_t* wbuf = smem + SM::kWarp + warp * SM::kWarpBytes;
    const uint8_t* stages = smem + SM::kStage + warp * NSW * kHalfMax;
    full += warp * NSW;
    empty += warp * NSW;
    const SplitSel take_lo = split_sel(gID & 1);

    auto give_up = [&]() {
        if (lane == 0) report(p.status, OSCAR_STATUS_TIMEOUT);
    };

    WarpState<NT, GS> st;
    float qsv[NT][NB];  // group sums of q'
    float kq = 1.f;
    uint32_t citem = 0, cur_qs = 0;
    const uint2* qf = nullptr;
    Ring<NSW> ring;

    for (uint32_t j = 0;; ++j) {
        if (!warp_wait(&full[ring.slot], ring.phase)) return give_up();
        const int4 sraw = *reinterpret_cast<const int4*>(&info[warp * 2 + (j & 1u)]);
        const int item = sraw.x, flags = sraw.w >> 8, valid = sraw.w & 0xff;
        if (item < 0) break;
        if (flags & kFlagFirst) {
            cur_qs = citem & 1u;
            if (!warp_wait(&qfull[cur_qs], (citem >> 1) & 1u)) return give_up();
            ++citem;
            const uint8_t* qb = smem + SM::kQb + cur_qs * SM::kQbBytes;
            qf = reinterpret_cast<const uint2*>(qb);
            kq = *reinterpret_cast<const float*>(qb + SM::kQbKinv);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 q4 = reinterpret_cast<const float4*>(qb + SM::kQbSum)[NT == 1 ? tq : 2 * tq + n];
                const float q1[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    qsv[n][b] = q1[b << GS];
#pragma unroll
                    for (int i = 1; i < 1 << GS; ++i) qsv[n][b] += q1[(b << GS) + i];
                }
                st.m_run[n] = -INFINITY;
                st.l_run[n] = 0.f;
#pragma unroll
                for (int b = 0; b < NB; ++b) st.zacc[n][b] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.acc[mt][e] = 0.f;
            st.wexp = kNoScale;
        }
        const uint8_t* half = stages + ring.slot * kHalfMax;
        if (flags & kFlagPad) {  // no page: give both halves back
            if constexpr (MODE == kModeWeights) {
                if (sraw.z >= 0) {  // a page that cannot be read: its tokens have weight 0
                    float none[4][2 * NT];
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int e = 0; e < 2 * NT; ++e) none[m][e] = -INFINITY;
                    store_logits<NT>(page_logits_at(p, sraw.y, sraw.z), p.G, none);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[ring.slot]);
            ring.step();
            if (!warp_wait(&full[ring.slot], ring.phase)) return give_up();
        } else {
            float lg[4][2 * NT], alpha[NT];
            page_logits<NT, GS>(half, valid, wbuf, qf, qsv, kq, lg);
            if constexpr (MODE == kModeWeights) store_logits<NT>(page_logits_at(p, sraw.y, sraw.z), p.G, lg);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[ring.slot]);
            ring.step();
            const bool any = page_softmax<NT, GS>(lg, st, alpha);
            if (!warp_wait(&full[ring.slot], ring.phase)) return give_up();
            page_values<NT, GS>(stages + ring.slot * kHalfMax, valid, wbuf, lg, alpha, any, take_lo, st);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[ring.slot]);
        ring.step();

        if (!(flags & kFlagLast)) continue;
        if (lane == 0) mbar_arrive(&qempty[cur_qs]);  // done with the item's q' data
        // this warp's partial state: part[4 item + warp] = o' [G][d], m [G], l [G]
        float* part = p.part + ((size_t)item * kConsumerWarps + warp) * p.part_stride;
        const float down = st.wexp == kNoScale ? 0.f : pow2_bits(-st.wexp);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int head = NT == 1 ? tq : 2 * tq + n;
            float l = st.l_run[n];
            l += __shfl_xor_sync(kFull, l, 4);
            l += __shfl_xor_sync(kFull, l, 8);
            l += __shfl_xor_sync(kFull, l, 16);
            float z[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                z[b] = st.zacc[n][b];
                z[b] += __shfl_xor_sync(kFull, z[b], 4);
                z[b] += __shfl_xor_sync(kFull, z[b], 8);
                z[b] += __shfl_xor_sync(kFull, z[b], 16);
            }
            if (head >= p.G) continue;
            float* o = part + (size_t)head * kD;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                const float a = NT == 1 ? st.acc[mt][0] + st.acc[mt][1] : st.acc[mt][n];
                const float c = NT == 1 ? st.acc[mt][2] + st.acc[mt][3] : st.acc[mt][2 + n];
                *reinterpret_cast<float2*>(o + 16 * mt + 2 * gID) =
                    make_float2(fmaf(a, down, z[mt >> (1 + GS)]), fmaf(c, down, z[mt >> (1 + GS)]));
            }
            if (gID == 0) {
                part[(size_t)p.G * kD + head] = st.m_run[n];
                part[(size_t)p.G * kD + p.G + head] = l;
            }
        }
    }
}

template <int NT, int GS, Mode MODE>
cudaError_t launch(const Params4<MODE>& p, cudaStream_t st, bool& attr_set) {
    if (!attr_set) {
        const cudaError_t e = set_smem(int4_kernel<NT, GS, MODE>, Int4Smem<NT, GS>::kBytes);
        if (e != cudaSuccess) return e;
        attr_set = true;
    }
    // no more blocks than items (of four pages at least)
    const int64_t items = (int64_t)p.B * p.hk * ((p.max_pages + 3) / 4);
    const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(p.blocks, items));
    const cudaError_t e =
        launch_pdl(int4_kernel<NT, GS, MODE>, dim3(blocks), dim3(kThreads4), Int4Smem<NT, GS>::kBytes, st, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <Mode MODE>
cudaError_t launch_mode(const Params4<MODE>& p, cudaStream_t st, int dev) {
    static bool attr_set[64][6];
    bool(&at)[6] = attr_set[dev & 63];
    if (p.NT == 1) {
        if (p.gshift == 0) return launch<1, 0, MODE>(p, st, at[0]);
        return p.gshift == 1 ? launch<1, 1, MODE>(p, st, at[1]) : launch<1, 2, MODE>(p, st, at[2]);
    }
    if (p.gshift == 0) return launch<2, 0, MODE>(p, st, at[3]);
    return p.gshift == 1 ? launch<2, 1, MODE>(p, st, at[4]) : launch<2, 2, MODE>(p, st, at[5]);
}

}  // namespace

cudaError_t launch_int4(const DecodeParams4& p, cudaStream_t st, int dev) { return launch_mode<kModePlain>(p, st, dev); }
cudaError_t launch_int4(const DecodeParamsX& p, Mode mode, cudaStream_t st, int dev) {
    return mode == kModeWeights ? launch_mode<kModeWeights>(p, st, dev) : launch_mode<kModeShared>(p, st, dev);
}

}  // namespace oscar
