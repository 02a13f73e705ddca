// evict4.cu -- eviction into the 4-bit history, a few tokens at a time (a
// decode step's); calls with many tokens go to evict_bulk.cu.
//
// As in evict.cu the rotation, the Hadamard transform and the group statistics
// run on float pairs; 16 levels, and every decision (the clip threshold c
// max|y|, s and z to fp16, the codes) is taken from the pairs: codes and
// pairs are those of a float64 evaluation except where that lies within
// 2^-36 |x| of a border (the arithmetic replayed on the host over random and
// aligned rows: at most 2^-39.5 |x|; if every rounding were of one sign, 2^-29).
//
// The sum y = x . U takes four instructions a term instead of the ten of a
// compensated product and sum: the accumulator starts at M = 1.5 2^E, far
// enough above every partial sum that it never leaves [2^E, 2^(E+1)), so its
// steps are multiples of one unit, and
//   n = fma(x, u, acc),  d = n - acc (exact),  lo += fma(x, u, -d) (exact to 2^-49 2^E)
// keep what each step rounds away.  E comes from sum|x| of the warp's terms and
// |u| < 2 (an orthogonal U has |u| <= 1); a matrix with a larger entry is
// summed the long way.  1024 vectors took 13.2 us with compensated sums
// and loads where they are used, 9.3 now; what is left is the chain of one
// vector (about 6,000 cycles), as the U of a KV head comes from L2. (Blocks of
// two or four tokens that share the rows of U were slower: 16.7 and 20 us.)
//
// Block = one vector: W warps sum 128 / W terms each, DEPTH rows of U in flight
// per warp; warp 0 adds the partial sums and finishes the vector.
#include "pairs.cuh"

namespace oscar {

namespace {
// Codes and pairs of one vector into its slot of a half.  Value k of the lane is
// in-group index j = bitrev5(lane) of 32-position block bitrev2(k); its
// nibble partner (j ^ 1) is lane ^ 16.
__device__ __forceinline__ void store4(const EvictParams& p, const df (&yn)[4], const df (&hi)[4],
                                       const df (&lo)[4], uint8_t* half, int slot, int which) {
    const int lane = threadIdx.x & 31;
    uint32_t w[4], nib = 0;  // (s, z) words in block order; nibble of block b in byte b
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int b = bitrev2(k);
        const unsigned short sb = df_to_f16(df_div15(df_add(hi[k], df_neg(lo[k])))), zb = df_to_f16(lo[k]);
        const float sf = __half2float(__ushort_as_half(sb)), zf = __half2float(__ushort_as_half(zb));
        const int code = sf != 0.f ? code4_of(yn[k], sf, zf) : 0;
        nib |= (uint32_t)code << (8 * b);
        w[b >> p.gshift] = (uint32_t)sb | ((uint32_t)zb << 16);
    }
    const uint32_t other = __shfl_xor_sync(kFull, nib, 16);
    const uint32_t bytes = lane < 16 ? nib | (other << 4) : other | (nib << 4);  // byte b: byte j / 2 of block b
    if (which == 0) {  // word (a, b) of the token: bytes j / 2 = 4 a .. 4 a + 3 of block b
        uint32_t word = 0;
        const int a = (lane >> 2) & 3, b = lane & 3;
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
            const uint32_t v = __shfl_sync(kFull, bytes, bitrev5(2 * (4 * a + i4)));
            word |= ((v >> (8 * b)) & 0xffu) << (8 * i4);
        }
        if (lane < 16) *reinterpret_cast<uint32_t*>(half + slot * (kD / 2) + 4 * lane) = word;
    } else {  // plane 16 b + j / 2: the pair of lanes stores two blocks each
        const int jj = bitrev5(lane & 15) >> 1, b0 = (lane >> 4) * 2;
#pragma unroll
        for (int b = 0; b < 2; ++b)
            half[(16 * (b0 + b) + jj) * kPage + slot] = (uint8_t)(bytes >> (8 * (b0 + b)));
    }
    if (lane == 0) {
        const int ng = sz_pairs(p.gshift);
        uint8_t* sz = half + kCodes4 + slot * 4 * ng;
        if (ng == 4) *reinterpret_cast<uint4*>(sz) = make_uint4(w[0], w[1], w[2], w[3]);
        else if (ng == 2) *reinterpret_cast<uint2*>(sz) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(sz) = w[0];
    }
}

template <int W, int DEPTH>
__global__ void __launch_bounds__(32 * W) evict4_kernel(EvictParams p) {
    constexpr int kTerms = kD / W;
    __shared__ df part[W][kD];
    pdl_wait();     // launched early (programmatic serialization): the previous kernel's results first
    pdl_trigger();  // the decode's query preparation reads nothing that this kernel writes (but what came before it)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pairs = 2 * p.hk, pair = blockIdx.x % pairs, i = blockIdx.x / pairs;
    const float* Um = p.U + (size_t)pair * kD * kD + (size_t)kTerms * warp * kD;
    // -- every load that depends on nothing, before anything waits: the first
    //    rows of U, the clip ratio, the token's row and destination (a round
    //    trip to L2 costs about 900 cycles: with the loads where they are
    //    used, four rows of U at a time, one token took 11,600 cycles of which
    //    8,000 were such waits)
    float4 u[DEPTH];
#pragma unroll
    for (int a = 0; a < DEPTH; ++a) u[a] = __ldg(reinterpret_cast<const float4*>(Um + (size_t)a * kD) + lane);
    const float cr = __ldg(p.clip + pair);
    const int row = p.src_row ? __ldg(p.src_row + i) : i, seq = __ldg(p.dst_seq + i), pos = __ldg(p.dst_pos + i);
    if (row < 0 || row >= p.src_rows) {
        if (threadIdx.x == 0) report(p.status, OSCAR_STATUS_BAD_POS);
        return;
    }
    uint8_t* half = nullptr;
    int bad = OSCAR_STATUS_BAD_POS;
    if (pos >= 0 && pos < p.max_pages * kPage && seq >= 0 && seq < p.batch) {
        const int page = __ldg(p.page_table + (size_t)seq * p.max_pages + pos / kPage);
        bad = OSCAR_STATUS_BAD_PAGE;
        if (page >= 0 && page < p.num_pages)
            half = p.pool + ((size_t)page * p.hk + (pair >> 1)) * p.block_bytes + (pair & 1) * half_bytes4(p.gshift);
    }
    const size_t xrow = ((size_t)row * pairs + pair) * kD;
    // lane a holds term a of the warp's share
    const float x = lane < kTerms ? __bfloat162float(p.src_kv[xrow + kTerms * warp + lane]) : 0.f;

    // -- y = x . U over the warp's terms
    float sum = fabsf(x);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(kFull, sum, m);
    // |partial sum| < 2 sum < 2^(exponent + 2) = 2^(E - 1)
    const int E = min(126, max(-100, (int)(__float_as_uint(sum) >> 23) - 127 + 3));
    const float M = __uint_as_float(((uint32_t)(127 + E) << 23) | 0x400000u);
    float acc[4] = {M, M, M, M}, c[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t bits = 0;  // bit 30: an entry of 2 or more (the top exponent bit)
#pragma unroll
    for (int a = 0; a < kTerms; ++a) {
        const float4 v = u[a % DEPTH];
        if (a + DEPTH < kTerms) u[a % DEPTH] = __ldg(reinterpret_cast<const float4*>(Um + (size_t)(a + DEPTH) * kD) + lane);
        const float uu[4] = {v.x, v.y, v.z, v.w};
        bits |= __float_as_uint(v.x) | __float_as_uint(v.y);
        bits |= __float_as_uint(v.z) | __float_as_uint(v.w);
        const float xa = __shfl_sync(kFull, x, a);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float n = __fmaf_rn(xa, uu[k], acc[k]);
            const float d = __fsub_rn(n, acc[k]);
            c[k] = __fadd_rn(c[k], __fmaf_rn(xa, uu[k], -d));
            acc[k] = n;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = __fsub_rn(acc[k], M);  // exact
    if (__any_sync(kFull, bits & 0x40000000u)) {  // the long way: error-free products and sums
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = c[k] = 0.f;
#pragma unroll 1
        for (int a = 0; a < kTerms; ++a) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(Um + (size_t)a * kD) + lane);
            const float uu[4] = {v.x, v.y, v.z, v.w};
            const float xa = __shfl_sync(kFull, x, a);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float pr = __fmul_rn(xa, uu[k]);
                const float pe = __fmaf_rn(xa, uu[k], -pr);
                const df t = two_sum(acc[k], pr);
                acc[k] = t.hi;
                c[k] = __fadd_rn(c[k], __fadd_rn(pe, t.lo));
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) part[warp][4 * lane + k] = two_sum(acc[k], c[k]);
    __syncthreads();  // all warps have read the source row and written partials
    if (warp != 0) return;
    if (p.new_kv)  // fused ring append: overwrite the row just read
        *(reinterpret_cast<uint2*>(const_cast<__nv_bfloat16*>(p.src_kv) + xrow) + lane) =
            __ldg(reinterpret_cast<const uint2*>(p.new_kv + ((size_t)i * pairs + pair) * kD) + lane);
    if (!half) {
        if (lane == 0) report(p.status, bad);
        return;
    }
    df y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        y[k] = part[0][4 * lane + k];
#pragma unroll
        for (int w = 1; w < W; ++w) y[k] = df_add(y[k], part[w][4 * lane + k]);
    }
    {  // Walsh-Hadamard transform (unnormalised), Sylvester order: in-lane stages, then partner lane l ^ m
        const df t0 = df_add(y[0], y[1]), t1 = df_add(y[0], df_neg(y[1]));
        const df t2 = df_add(y[2], y[3]), t3 = df_add(y[2], df_neg(y[3]));
        y[0] = df_add(t0, t2);
        y[2] = df_add(t0, df_neg(t2));
        y[1] = df_add(t1, t3);
        y[3] = df_add(t1, df_neg(t3));
    }
#pragma unroll 1
    for (int m = 1; m < 32; m <<= 1) {
        const bool upper = (lane & m) != 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const df o{__shfl_xor_sync(kFull, y[k].hi, m), __shfl_xor_sync(kFull, y[k].lo, m)};
            y[k] = upper ? df_add(o, df_neg(y[k])) : df_add(y[k], o);
        }
    }
    // times 1 / sqrt(d) as a pair; extremes of every group (exact on the pairs: the
    // high parts first, then the low parts of the lanes that hold the extreme)
    const float kc_hi = __uint_as_float(0x3db504f3u), kc_lo = __uint_as_float(0x30cfe77au);
    df yn[4], lo[4], hi[4];
    float mx[4], mn[4], mxl[4], mnl[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float ph = __fmul_rn(y[k].hi, kc_hi);
        float e = __fmaf_rn(y[k].hi, kc_hi, -ph);
        e = __fmaf_rn(y[k].hi, kc_lo, e);
        e = __fmaf_rn(y[k].lo, kc_hi, e);
        yn[k] = fast_two_sum(ph, e);
        mx[k] = mn[k] = yn[k].hi;
    }
#pragma unroll 1
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mx[k] = fmaxf(mx[k], __shfl_xor_sync(kFull, mx[k], m));
            mn[k] = fminf(mn[k], __shfl_xor_sync(kFull, mn[k], m));
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        mxl[k] = yn[k].hi == mx[k] ? yn[k].lo : -INFINITY;
        mnl[k] = yn[k].hi == mn[k] ? yn[k].lo : INFINITY;
    }
#pragma unroll 1
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mxl[k] = fmaxf(mxl[k], __shfl_xor_sync(kFull, mxl[k], m));
            mnl[k] = fminf(mnl[k], __shfl_xor_sync(kFull, mnl[k], m));
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        hi[k] = {mx[k], mxl[k]};
        lo[k] = {mn[k], mnl[k]};
    }
    // value k's 32-position block is bitrev2(k): groups of 64 are k = {0, 2}, {1, 3}
    if (p.gshift >= 1) {
        df_group_extremes(hi[0], hi[2], lo[0], lo[2]);
        df_group_extremes(hi[1], hi[3], lo[1], lo[3]);
    }
    if (p.gshift >= 2) {
        df_group_extremes(hi[0], hi[1], lo[0], lo[1]);
        hi[2] = hi[3] = hi[0];
        lo[2] = lo[3] = lo[0];
    }
    if (cr < 1.f) {  // clip by +-t, t = c max|y| = c max(max, -min)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const df nlo = df_neg(lo[k]), a = df_less(hi[k], nlo) ? nlo : hi[k];
            const float th = __fmul_rn(cr, a.hi);
            const df t = fast_two_sum(th, __fmaf_rn(cr, a.lo, __fmaf_rn(cr, a.hi, -th))), nt = df_neg(t);
            if (df_less(t, yn[k])) yn[k] = t;
            else if (df_less(yn[k], nt)) yn[k] = nt;
            if (df_less(t, hi[k])) hi[k] = t;
            if (df_less(lo[k], nt)) lo[k] = nt;
        }
    }
    store4(p, yn, hi, lo, half, pos % kPage, pair & 1);
}

template <int W, int DEPTH>
cudaError_t launch(const EvictParams& p, cudaStream_t st) {
    static bool carveout_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!carveout_set[dev & 63]) {  // the largest split, as every kernel of the step (launch_evict)
        e = cudaFuncSetAttribute(evict4_kernel<W, DEPTH>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 (int)cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        carveout_set[dev & 63] = true;
    }
    e = launch_pdl(evict4_kernel<W, DEPTH>, dim3(p.n_tok * 2 * p.hk), dim3(32 * W), 0, st, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Calls with this many vectors (tokens x KV heads x 2) take the bulk kernel: it
// starts with 9 us of forming R in every block and then needs 0.5 ns per
// vector, this kernel 5 ns.  (GB300, us here and there, a graph of 20 calls:
//                2048 vectors   4096         6000         8192
//   1 KV head    15.7  22.8     24.9  23.5   34.0  23.5   44.5  24.3
//   8            16.2  22.1     25.3  23.5   30.4  23.4*  45.1  24.0
//   40           16.4  21.2     25.7  21.7   30.6  21.6*  46.0  22.4
//   80           16.5  38.2     25.8  38.2   36.0  38.9   46.0  38.8
// (*) 5120 vectors.  With 80 heads 160 (KV head, K|V) pairs make two waves of bulk
// blocks: from 77 heads up the border would lie near 6800.
// 15,104 tokens of eight heads: 1830 and 124.)
constexpr int kBulkVectors = 4096;

}  // namespace

cudaError_t launch_evict4(const EvictParams& p, cudaStream_t st) {
    const int vecs = p.n_tok * p.hk * 2;
    if (vecs == 0) return cudaSuccess;
    if (vecs >= kBulkVectors && ((uintptr_t)p.src_kv & 15) == 0) return launch_evict_bulk(p, st);  // (16-byte row copies)
    // As many rows of U in flight as keep the call's blocks on the GPU at once: 2,
    // 4 or 8 blocks per SM (16 vectors: 4.8, 4.9, 5.3 us; 256: 5.6, 6.7, 8.0; 512: 10.5,
    // 7.0, 9.0; 1024: 20, 12.0, 9.3)
    if (vecs <= 304) return launch<8, 16>(p, st);
    return vecs <= 608 ? launch<8, 8>(p, st) : launch<4, 8>(p, st);
}

}  // namespace oscar
