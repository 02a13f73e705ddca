// history.cu -- stored history tokens read back as rows, gathered into fresh
// pages (compaction after tokens are dropped), and whole pages copied in
// every layer's pool.  Memory-bound: each byte is read once and written
// once.
//
// A block's K codes and its (s, z) pairs are token-major (a token's bytes
// are contiguous); its V codes are byte planes of 64 tokens, so a token's V
// codes are one byte in each of 32 (2-bit) or 64 (4-bit) planes.  Both kernels
// that move tokens therefore take 64 tokens together, so that the 32-byte
// sectors of a plane are used whole.
//
// Measured (GB300, copy peak 6.79 TB/s): 32,448 tokens of eight KV heads read
// as bf16 in 33.5 us (5.2 TB/s of 160 + 512 bytes per token and head); half of
// eight 32K histories kept, 81 us (4.1 TB/s of 2 x 160 bytes; a random half of
// a page's V plane costs its whole sectors, so 400 bytes move: 5.1 TB/s);
// 2048 pages copied in 50.7 us (6.6 TB/s).
#include "oscar_common.cuh"

namespace oscar {

namespace {

constexpr int kHistThreads = 256;

// Byte offsets inside a (page, KV head) block and code bytes of a vector.
template <int BITS>
struct Layout {
    static constexpr int kVec = BITS * kD / 8;        // code bytes of a vector = V code planes
    __device__ static __forceinline__ int k_pairs() { return BITS == 2 ? kKScale : kCodes4; }
    __device__ static __forceinline__ int v_codes(int gshift) { return BITS == 2 ? kVCodes : half_bytes4(gshift); }
    __device__ static __forceinline__ int v_pairs(int gshift) {
        return BITS == 2 ? v_scale_off(gshift) : half_bytes4(gshift) + kCodes4;
    }
};

// Where a token is stored: its KV head's block of its page (null: the token
// is skipped) and its slot.
struct Source {
    const uint8_t* blk;
    int slot;
};

__device__ __forceinline__ Source find_token(const uint8_t* pool, const int32_t* table_row, int max_pages, int num_pages,
                                             int pos, int hk, int kv, int block_bytes, int32_t* status) {
    if (pos < 0 || pos >= max_pages * kPage) {
        report(status, OSCAR_STATUS_BAD_POS);
        return {nullptr, 0};
    }
    const int page = __ldg(table_row + pos / kPage);
    if (page < 0 || page >= num_pages) {
        report(status, OSCAR_STATUS_BAD_PAGE);
        return {nullptr, 0};
    }
    return {pool + ((size_t)page * hk + kv) * block_bytes, pos % kPage};
}

// The V codes of four listed tokens: neighbours at a slot divisible by four
// (one word per plane), or each by itself (a byte per plane and token).
struct Quad {
    const uint8_t* at[4];  // plane 0 of each token's byte; null: skipped
    bool joined;
    __device__ __forceinline__ Quad(const Source* src, int v_codes) {
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = src[i].blk ? src[i].blk + v_codes + src[i].slot : nullptr;
        joined = at[0] && (src[0].slot & 3) == 0 && at[1] == at[0] + 1 && at[2] == at[0] + 2 && at[3] == at[0] + 3;
    }
    // planes p0 .. p0 + N - 1, all loads issued before any is used; bytes of skipped tokens 0
    template <int N>
    __device__ __forceinline__ void load(int p0, uint32_t (&w)[N]) const {
        if (joined) {
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = *reinterpret_cast<const uint32_t*>(at[0] + (p0 + j) * kPage);
            return;
        }
        uint32_t v[4][N];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) v[i][j] = at[i] ? at[i][(p0 + j) * kPage] : 0u;
#pragma unroll
        for (int j = 0; j < N; ++j)
            w[j] = __byte_perm(__byte_perm(v[0][j], v[1][j], 0x0040u), __byte_perm(v[2][j], v[3][j], 0x0040u), 0x5410u);
    }
};

// ---------------------------------------------------------------------------
// read: stored tokens as rows
// ---------------------------------------------------------------------------
// Eight neighbouring positions 32 k + 8 a .. + 7 from their codes: 4 bits: one
// word (low nibble first); 2 bits: slot k of the eight bytes of w0, w1.  The
// code bytes go into the mantissa of 2^23 (exact, and off the conversion
// unit).
template <int BITS>
__device__ __forceinline__ void eight_values(uint32_t w0, uint32_t w1, int k, uint32_t sz, float (&v)[8]) {
    const float s = half_lo(sz), z = half_hi(sz);
    const uint32_t a = BITS == 4 ? w0 & 0x0f0f0f0fu : (w0 >> (2 * k)) & 0x03030303u;         // codes 0 2 4 6 | 0 1 2 3
    const uint32_t b = BITS == 4 ? (w0 >> 4) & 0x0f0f0f0fu : (w1 >> (2 * k)) & 0x03030303u;  // codes 1 3 5 7 | 4 5 6 7
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t from = BITS == 4 ? ((i & 1) ? b : a) : (i < 4 ? a : b);
        const int byte = BITS == 4 ? i >> 1 : i & 3;
        const float c = __uint_as_float(__byte_perm(from, 0x4b000000u, 0x7440u + byte)) - 8388608.f;
        v[i] = fmaf(s, c, z);
    }
}

template <typename T>
__device__ __forceinline__ void store_eight(T* out, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                                                    pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
    } else {
        reinterpret_cast<float4*>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// Block = kTok listed tokens of one KV head (64: 33.5 us for 32,448 tokens of
// eight heads; 32: 36.8, the look-up of the tokens then weighs more).  Thread (token, c) makes the eight values of
// positions 8 c .. 8 c + 7, so that a row is stored by 16 neighbouring lanes: K
// straight from global memory, V through shared memory, where the plane
// bytes are laid token by token.  Every load of a thread is issued before the
// first is used.
constexpr int kTok = 64;

template <int BITS, typename T>
__global__ void __launch_bounds__(kHistThreads) read_kernel(HistoryReadParams p) {
    using L = Layout<BITS>;
    constexpr int kRow = L::kVec + 4;  // bytes of a staged token: words of distinct tokens on distinct banks
    constexpr int kPlanes = L::kVec * (kTok / 4) / kHistThreads;  // planes per thread: 4 (4 bits), 2
    __shared__ Source src[kTok];
    __shared__ __align__(16) uint8_t vS[kTok * kRow];
    const int t0 = blockIdx.x * kTok, kv = blockIdx.y;
    pdl_wait();
    if (threadIdx.x < kTok) {
        Source s{nullptr, 0};
        const int i = t0 + threadIdx.x;
        if (i < p.n_tok) {
            const int seq = __ldg(p.seq + i);
            if (seq < 0 || seq >= p.batch) report(p.status, OSCAR_STATUS_BAD_POS);
            else s = find_token(p.pool, p.page_table + (size_t)seq * p.max_pages, p.max_pages, p.num_pages,
                                __ldg(p.pos + i), p.hk, kv, p.block_bytes, p.status);
        }
        src[threadIdx.x] = s;
    }
    __syncthreads();
    const int quad = threadIdx.x % (kTok / 4), plane = threadIdx.x / (kTok / 4) * kPlanes;
    uint32_t vw[kPlanes];
    Quad(src + 4 * quad, L::v_codes(p.gshift)).load(plane, vw);
    const int c = threadIdx.x & 15, k = c >> 2, a = c & 3, ng = sz_pairs(p.gshift);
    constexpr int kIt = kTok / 16;
    uint32_t kw[kIt][2], ksz[kIt], vsz[kIt];
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
        const Source s = src[16 * it + (threadIdx.x >> 4)];
        kw[it][0] = kw[it][1] = ksz[it] = vsz[it] = 0u;
        if (!s.blk) continue;
        const uint8_t* codes = s.blk + s.slot * L::kVec;
        if constexpr (BITS == 4) {
            kw[it][0] = *reinterpret_cast<const uint32_t*>(codes + 16 * a + 4 * k);
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(codes + 8 * a);
            kw[it][0] = x.x;
            kw[it][1] = x.y;
        }
        const int at = (s.slot * ng + (k >> p.gshift)) * 4;
        ksz[it] = *reinterpret_cast<const uint32_t*>(s.blk + L::k_pairs() + at);
        vsz[it] = *reinterpret_cast<const uint32_t*>(s.blk + L::v_pairs(p.gshift) + at);
    }
#pragma unroll
    for (int j = 0; j < kPlanes; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) vS[(4 * quad + e) * kRow + plane + j] = (uint8_t)(vw[j] >> (8 * e));
    T* out[kIt];
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
        const int t = 16 * it + (threadIdx.x >> 4);
        out[it] = src[t].blk ? static_cast<T*>(p.out) + ((size_t)(t0 + t) * p.hk + kv) * 2 * kD + 8 * c : nullptr;
        float v[8];
        eight_values<BITS>(kw[it][0], kw[it][1], k, ksz[it], v);
        if (out[it]) store_eight(out[it], v);
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
        const uint32_t* row = reinterpret_cast<const uint32_t*>(vS + (16 * it + (threadIdx.x >> 4)) * kRow);
        float v[8];
        // 4 bits: planes 4 c .. 4 c + 3; 2 bits: planes 8 a .. 8 a + 7
        eight_values<BITS>(BITS == 4 ? row[c] : row[2 * a], BITS == 4 ? 0u : row[2 * a + 1], k, vsz[it], v);
        if (out[it]) store_eight(out[it] + kD, v);
    }
}

// ---------------------------------------------------------------------------
// gather: kept tokens into fresh pages
// ---------------------------------------------------------------------------
// Block = one destination page of one sequence, `heads` of its KV heads in turn
// (the tokens' pages and slots are the same for all, so they are looked up
// once); all loads of a thread come first.
template <int BITS>
__global__ void __launch_bounds__(kHistThreads, 6) gather_kernel(HistoryGatherParams p) {
    using L = Layout<BITS>;
    constexpr int kPlanes = L::kVec / 4;                     // V planes per warp pair: 16 (4 bits), 8
    constexpr int kChunks = L::kVec / 16;                    // 16-byte chunks of a token's K codes
    __shared__ Source src[kPage];                            // KV head 0's block
    const int turns = (p.hk + p.heads - 1) / p.heads, kv0 = blockIdx.x % turns * p.heads;
    const int pg = blockIdx.x / turns % p.dst_max_pages, b = blockIdx.x / turns / p.dst_max_pages;
    const int most = min(p.keep_stride, p.dst_max_pages * kPage);
    pdl_wait();
    // (the three index loads are independent: one round trip, then the page)
    int n_keep = __ldg(p.n_keep + b);
    const int dst_page = __ldg(p.dst_table + (size_t)b * p.dst_max_pages + pg);
    const int i0 = pg * kPage + (threadIdx.x & (kPage - 1));
    const int pos = i0 < p.keep_stride ? __ldg(p.keep + (size_t)b * p.keep_stride + i0) : -1;
    if (n_keep < 0 || n_keep > most) {
        if (threadIdx.x == 0) report(p.status, OSCAR_STATUS_BAD_POS);
        n_keep = min(max(n_keep, 0), most);
    }
    const int n = min(kPage, n_keep - pg * kPage);
    if (n <= 0) return;
    if (dst_page < 0 || dst_page >= p.num_pages) {
        if (threadIdx.x == 0) report(p.status, OSCAR_STATUS_BAD_PAGE);
        return;
    }
    if (threadIdx.x < kPage) {
        Source s{nullptr, 0};
        if ((int)threadIdx.x < n)
            s = find_token(p.pool, p.src_table + (size_t)b * p.src_max_pages, p.src_max_pages, p.num_pages, pos, p.hk, 0,
                           p.block_bytes, p.status);
        src[threadIdx.x] = s;
    }
    __syncthreads();
    const int ng = sz_pairs(p.gshift), vc = L::v_codes(p.gshift);
    // V code planes: lane = token, kPlanes planes per warp and half page.  A
    // byte of 32 kept tokens per access: their source slots span few sectors,
    // and the 32 bytes stored are one.
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vt = 32 * (warp & 1) + lane, plane = (warp >> 1) * kPlanes;
    const uint8_t* vfrom = src[vt].blk ? src[vt].blk + vc + src[vt].slot + plane * kPage : nullptr;
    // K codes: token-major, 16 bytes per thread
    const int kt = threadIdx.x / kChunks, kc = threadIdx.x % kChunks;
    const uint8_t* kfrom = kt < kPage && src[kt].blk ? src[kt].blk + src[kt].slot * L::kVec + 16 * kc : nullptr;
    // pairs of K and V: words threadIdx.x and threadIdx.x + 256 of the 128 ng
    const uint8_t* zfrom[2];
    int zto[2];
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int i = threadIdx.x + kHistThreads * it, which = i >= kPage * ng, r = i - which * kPage * ng, t = r / ng;
        const int at = which ? L::v_pairs(p.gshift) : L::k_pairs();
        zfrom[it] = i < 2 * kPage * ng && src[t].blk ? src[t].blk + at + (src[t].slot * ng + r % ng) * 4 : nullptr;
        zto[it] = at + r * 4;
    }
    const int kv1 = min(kv0 + p.heads, p.hk);
    for (int kv = kv0; kv < kv1; ++kv) {
        const size_t head = (size_t)kv * p.block_bytes;
        uint8_t* dst = p.pool + (size_t)dst_page * p.hk * p.block_bytes + head;
        uint8_t vw[kPlanes];
        uint4 kw;
        uint32_t zw[2];
        if (vfrom)
#pragma unroll
            for (int j = 0; j < kPlanes; ++j) vw[j] = vfrom[head + j * kPage];
        if (kfrom) kw = *reinterpret_cast<const uint4*>(kfrom + head);
#pragma unroll
        for (int it = 0; it < 2; ++it)
            if (zfrom[it]) zw[it] = *reinterpret_cast<const uint32_t*>(zfrom[it] + head);
        if (vfrom)
#pragma unroll
            for (int j = 0; j < kPlanes; ++j) dst[vc + (plane + j) * kPage + vt] = vw[j];
        if (kfrom) *reinterpret_cast<uint4*>(dst + kt * L::kVec + 16 * kc) = kw;
#pragma unroll
        for (int it = 0; it < 2; ++it)
            if (zfrom[it]) *reinterpret_cast<uint32_t*>(dst + zto[it]) = zw[it];
        if (p.boost && threadIdx.x < kPage && src[threadIdx.x].blk) {
            const size_t page = (size_t)(src[threadIdx.x].blk - p.pool) / ((size_t)p.hk * p.block_bytes);
            *reinterpret_cast<uint4*>(p.boost + ((size_t)dst_page * p.hk + kv) * kBoostBlock + threadIdx.x * kBoostRecord) =
                *reinterpret_cast<const uint4*>(p.boost + (page * p.hk + kv) * kBoostBlock +
                                                src[threadIdx.x].slot * kBoostRecord);
        }
    }
}

// ---------------------------------------------------------------------------
// page copies
// ---------------------------------------------------------------------------
// Block = one 16 KB piece of one (pair, pool).
constexpr int kCopyPiece = 16384;

__global__ void __launch_bounds__(kHistThreads) pages_copy_kernel(PagesCopyParams p) {
    const int piece = blockIdx.x % p.pieces, pair = blockIdx.x / p.pieces % p.n;
    uint8_t* pool = p.pool[blockIdx.x / p.pieces / p.n];
    pdl_wait();
    const int s = __ldg(p.src + pair), d = __ldg(p.dst + pair);
    if (s < 0 || s >= p.num_pages || d < 0 || d >= p.num_pages) {
        if (threadIdx.x == 0) report(p.status, OSCAR_STATUS_BAD_PAGE);
        return;
    }
    if (s == d) return;
    const size_t at = (size_t)piece * kCopyPiece;
    const int words = (int)(min((size_t)kCopyPiece, p.page_bytes - at) / 16);
    const uint4* from = reinterpret_cast<const uint4*>(pool + (size_t)s * p.page_bytes + at);
    uint4* to = reinterpret_cast<uint4*>(pool + (size_t)d * p.page_bytes + at);
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = threadIdx.x + kHistThreads * i;
        if (c < words) v[i] = from[c];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = threadIdx.x + kHistThreads * i;
        if (c < words) to[c] = v[i];
    }
}
static_assert(kCopyPiece == kHistThreads * 16 * 4, "four vectors per thread");

}  // namespace

// Launched with programmatic serialization, like the rest of the chain: the
// blocks may be placed while an eviction's last blocks run, and wait for its
// completion first.
template <typename P>
static cudaError_t launch_history(void (*kernel)(P), dim3 grid, const P& p, cudaStream_t st) {
    const cudaError_t e = launch_pdl(kernel, grid, dim3(kHistThreads), 0, st, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_history_read(const HistoryReadParams& p, cudaStream_t st) {
    const dim3 grid((p.n_tok + kTok - 1) / kTok, p.hk);
    if (p.bits4) return launch_history(p.out_bf16 ? read_kernel<4, __nv_bfloat16> : read_kernel<4, float>, grid, p, st);
    return launch_history(p.out_bf16 ? read_kernel<2, __nv_bfloat16> : read_kernel<2, float>, grid, p, st);
}

cudaError_t launch_history_gather(const HistoryGatherParams& p, cudaStream_t st) {
    HistoryGatherParams q = p;
    // Four KV heads per block once that still leaves as many blocks as the GPU
    // holds (912).  Pages x KV heads, us with one head and with four: 16256 89.1,
    // 81.8; 8128 47.0, 44.0; 7616 (nearly all tokens kept) 38.8, 35.9; 4064 as 508 x 8
    // 25.6, 25.0 and as 2032 x 2 26.2, 24.6; 2048 15.0, 15.4.
    q.heads = (int64_t)p.batch * p.dst_max_pages * p.hk >= 4 * 912 ? 4 : 1;
    const dim3 grid(p.batch * p.dst_max_pages * ((p.hk + q.heads - 1) / q.heads));
    return launch_history(p.bits4 ? gather_kernel<4> : gather_kernel<2>, grid, q, st);
}

int64_t pages_copy_pieces(size_t page_bytes) { return (int64_t)((page_bytes + kCopyPiece - 1) / kCopyPiece); }

cudaError_t launch_pages_copy(const PagesCopyParams& p, int n_pools, cudaStream_t st) {
    return launch_history(pages_copy_kernel, dim3(p.pieces * p.n * n_pools), p, st);
}

}  // namespace oscar
