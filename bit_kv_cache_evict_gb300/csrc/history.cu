// history.cu -- stored history tokens read back as rows, gathered into fresh
// pages (compaction after tokens are dropped), and whole pages copied in
// every layer's pool.  Memory-bound: each byte is read once and written
// once.
//
// A block's K codes and its (s, z) pairs are token-major (a token's bytes
// are contiguous); its V codes are byte planes of 64 tokens, so a token's V
// codes are one byte in each of 32 (2-bit) or 64 (4-bit) planes.  Both kernels
// that move tokens therefore take the 64 tokens of a block of work together
// and move plane bytes four tokens at a time: one word where the four
// tokens are neighbours in their page, four bytes otherwise.
#include "splitk.cuh"

namespace oscar {

namespace {

constexpr int kTok = 64;         // tokens per thread block
constexpr int kHistThreads = 256;

// Byte offsets inside a (page, KV head) block and code bytes of a vector.
template <int BITS>
struct Layout {
    static constexpr int kVec = BITS * kD / 8;        // code bytes of a vector = V code planes
    static constexpr int kChunk = kVec / 4;           // code bytes of 32 of its positions, four runs of eight
    __device__ static __forceinline__ int k_pairs() { return BITS == 2 ? kKScale : kCodes4; }
    __device__ static __forceinline__ int v_codes(int gshift) { return BITS == 2 ? kVCodes : half_bytes4(gshift); }
    __device__ static __forceinline__ int v_pairs(int gshift) {
        return BITS == 2 ? v_scale_off(gshift) : half_bytes4(gshift) + kCodes4;
    }
};

// Where a token is stored: the page's first block (KV head 0), or null for a
// token that is skipped, and its slot.
struct Source {
    const uint8_t* page;
    int slot;
};

__device__ __forceinline__ Source find_token(const uint8_t* pool, const int32_t* table_row, int max_pages, int num_pages,
                                             int pos, size_t page_bytes, int32_t* status) {
    if (pos < 0 || pos >= max_pages * kPage) {
        report(status, OSCAR_STATUS_BAD_POS);
        return {nullptr, 0};
    }
    const int page = __ldg(table_row + pos / kPage);
    if (page < 0 || page >= num_pages) {
        report(status, OSCAR_STATUS_BAD_PAGE);
        return {nullptr, 0};
    }
    return {pool + (size_t)page * page_bytes, pos % kPage};
}

// Byte `plane` of the V codes of the four tokens of a quad, as one word
// (bytes of skipped tokens 0).  `off`: the KV head's V codes inside a page.
// joined: the four are neighbours at a slot divisible by four.
__device__ __forceinline__ uint32_t load_quad(const Source* src, bool joined, size_t off, int plane) {
    if (joined) return *reinterpret_cast<const uint32_t*>(src[0].page + off + plane * kPage + src[0].slot);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (src[i].page) w |= (uint32_t)src[i].page[off + plane * kPage + src[i].slot] << (8 * i);
    return w;
}

__device__ __forceinline__ bool quad_joined(const Source* src) {
    return src[0].page && (src[0].slot & 3) == 0 && src[1].page == src[0].page && src[2].page == src[0].page &&
           src[3].page == src[0].page && src[1].slot == src[0].slot + 1 && src[2].slot == src[0].slot + 2 &&
           src[3].slot == src[0].slot + 3;
}

// ---------------------------------------------------------------------------
// read: stored tokens as rows
// ---------------------------------------------------------------------------
// Eight neighbouring positions 32 k + 8 a .. + 7 from their codes: 4 bits: one
// word (low nibble first); 2 bits: slot k of the eight bytes of w0, w1.
template <int BITS>
__device__ __forceinline__ void eight_values(uint32_t w0, uint32_t w1, int k, float s, float z, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t c = BITS == 4 ? (w0 >> (4 * i)) & 15u : ((i < 4 ? w0 : w1) >> (8 * (i & 3) + 2 * k)) & 3u;
        v[i] = fmaf(s, (float)c, z);
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

// Block = 64 listed tokens of one KV head.  Thread (token, a) turns the codes
// of positions 32 k + 8 a .. + 7 (k = 0..3) into four runs of eight values: K
// straight from global memory, V through shared memory, where the plane
// bytes are laid token by token.
template <int BITS, typename T>
__global__ void __launch_bounds__(kHistThreads) read_kernel(HistoryReadParams p) {
    using L = Layout<BITS>;
    constexpr int kRow = L::kVec + 4;  // bytes of a staged token: words of distinct tokens on distinct banks
    __shared__ Source src[kTok];
    __shared__ __align__(16) uint8_t vS[kTok * kRow];
    const int t0 = blockIdx.x * kTok, kv = blockIdx.y;
    const size_t page_bytes = (size_t)p.hk * p.block_bytes, head = (size_t)kv * p.block_bytes;
    if (threadIdx.x < kTok) {
        Source s{nullptr, 0};
        const int i = t0 + threadIdx.x;
        if (i < p.n_tok) {
            const int seq = __ldg(p.seq + i);
            if (seq < 0 || seq >= p.batch) report(p.status, OSCAR_STATUS_BAD_POS);
            else s = find_token(p.pool, p.page_table + (size_t)seq * p.max_pages, p.max_pages, p.num_pages,
                                __ldg(p.pos + i), page_bytes, p.status);
        }
        src[threadIdx.x] = s;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < L::kVec * (kTok / 4); i += kHistThreads) {
        const int quad = i & 15, plane = i >> 4;
        const Source* q = src + 4 * quad;
        const uint32_t w = load_quad(q, quad_joined(q), head + L::v_codes(p.gshift), plane);
#pragma unroll
        for (int e = 0; e < 4; ++e) vS[(4 * quad + e) * kRow + plane] = (uint8_t)(w >> (8 * e));
    }
    const int t = threadIdx.x >> 2, a = threadIdx.x & 3;
    const Source s = src[t];
    T* out = static_cast<T*>(p.out) + ((size_t)(t0 + t) * p.hk + kv) * 2 * kD + 8 * a;
    const int ng = sz_pairs(p.gshift);
    if (s.page) {
        const uint8_t* blk = s.page + head;
        const uint32_t* sz = reinterpret_cast<const uint32_t*>(blk + L::k_pairs() + s.slot * 4 * ng);
        uint32_t w[4];
        const uint8_t* at = blk + s.slot * L::kVec + a * L::kChunk;
        if constexpr (BITS == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(at);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            w[0] = x.x; w[1] = x.y;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t z = sz[k >> p.gshift];
            float v[8];
            eight_values<BITS>(BITS == 4 ? w[k] : w[0], w[1], k, half_lo(z), half_hi(z), v);
            store_eight(out + 32 * k, v);
        }
    }
    __syncthreads();
    if (s.page) {
        const uint32_t* sz = reinterpret_cast<const uint32_t*>(s.page + head + L::v_pairs(p.gshift) + s.slot * 4 * ng);
        const uint32_t* row = reinterpret_cast<const uint32_t*>(vS + t * kRow);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t z = sz[k >> p.gshift];
            float v[8];
            // 4 bits: planes 16 k + 4 a .. + 3; 2 bits: planes 8 a .. + 7
            eight_values<BITS>(BITS == 4 ? row[4 * k + a] : row[2 * a], row[2 * a + 1], k, half_lo(z), half_hi(z), v);
            store_eight(out + kD + 32 * k, v);
        }
    }
}

// ---------------------------------------------------------------------------
// gather: kept tokens into fresh pages
// ---------------------------------------------------------------------------
// Block = one destination page of one sequence and KV head.
template <int BITS>
__global__ void __launch_bounds__(kHistThreads) gather_kernel(HistoryGatherParams p) {
    using L = Layout<BITS>;
    __shared__ Source src[kTok];
    const int kv = blockIdx.x % p.hk;
    const int pg = blockIdx.x / p.hk % p.dst_max_pages, b = blockIdx.x / p.hk / p.dst_max_pages;
    const int most = min(p.keep_stride, p.dst_max_pages * kPage);
    int n_keep = __ldg(p.n_keep + b);
    if (n_keep < 0 || n_keep > most) {
        if (threadIdx.x == 0) report(p.status, OSCAR_STATUS_BAD_POS);
        n_keep = min(max(n_keep, 0), most);
    }
    const int n = min(kTok, n_keep - pg * kPage);
    if (n <= 0) return;
    const int dst_page = __ldg(p.dst_table + (size_t)b * p.dst_max_pages + pg);
    if (dst_page < 0 || dst_page >= p.num_pages) {
        if (threadIdx.x == 0) report(p.status, OSCAR_STATUS_BAD_PAGE);
        return;
    }
    const size_t page_bytes = (size_t)p.hk * p.block_bytes, head = (size_t)kv * p.block_bytes;
    if (threadIdx.x < kTok) {
        Source s{nullptr, 0};
        if ((int)threadIdx.x < n)
            s = find_token(p.pool, p.src_table + (size_t)b * p.src_max_pages, p.src_max_pages, p.num_pages,
                           __ldg(p.keep + (size_t)b * p.keep_stride + pg * kPage + threadIdx.x), page_bytes, p.status);
        src[threadIdx.x] = s;
    }
    __syncthreads();
    uint8_t* dst = p.pool + (size_t)dst_page * page_bytes + head;
    // K codes: token-major, 16 bytes at a time
    for (int i = threadIdx.x; i < kTok * (L::kVec / 16); i += kHistThreads) {
        const int t = i / (L::kVec / 16), c = i % (L::kVec / 16);
        if (src[t].page)
            *reinterpret_cast<uint4*>(dst + t * L::kVec + 16 * c) =
                *reinterpret_cast<const uint4*>(src[t].page + head + src[t].slot * L::kVec + 16 * c);
    }
    // pairs of K and V: words
    const int ng = sz_pairs(p.gshift);
    for (int i = threadIdx.x; i < kTok * 2 * ng; i += kHistThreads) {
        const int which = i >= kTok * ng, r = i - which * kTok * ng, t = r / ng;
        const int at = (which ? L::v_pairs(p.gshift) : L::k_pairs()) + 4 * (r % ng);
        if (src[t].page)
            *reinterpret_cast<uint32_t*>(dst + at + t * 4 * ng) =
                *reinterpret_cast<const uint32_t*>(src[t].page + head + at + src[t].slot * 4 * ng);
    }
    // V code planes, four tokens at a time
    const int vc = L::v_codes(p.gshift);
    for (int i = threadIdx.x; i < L::kVec * (kTok / 4); i += kHistThreads) {
        const int quad = i & 15, plane = i >> 4;
        const Source* q = src + 4 * quad;
        const uint32_t w = load_quad(q, quad_joined(q), head + vc, plane);
        uint8_t* to = dst + vc + plane * kPage + 4 * quad;
        if (q[0].page && q[1].page && q[2].page && q[3].page) {
            *reinterpret_cast<uint32_t*>(to) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (q[e].page) to[e] = (uint8_t)(w >> (8 * e));
        }
    }
    if (p.boost && threadIdx.x < kTok) {
        const Source s = src[threadIdx.x];
        if (s.page) {
            const size_t page = (size_t)(s.page - p.pool) / page_bytes;
            *reinterpret_cast<uint4*>(p.boost + ((size_t)dst_page * p.hk + kv) * kBoostBlock + threadIdx.x * kBoostRecord) =
                *reinterpret_cast<const uint4*>(p.boost + (page * p.hk + kv) * kBoostBlock + s.slot * kBoostRecord);
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

cudaError_t launch_history_read(const HistoryReadParams& p, cudaStream_t st) {
    const dim3 grid((p.n_tok + kTok - 1) / kTok, p.hk);
    if (p.bits4) {
        if (p.out_bf16) read_kernel<4, __nv_bfloat16><<<grid, kHistThreads, 0, st>>>(p);
        else read_kernel<4, float><<<grid, kHistThreads, 0, st>>>(p);
    } else {
        if (p.out_bf16) read_kernel<2, __nv_bfloat16><<<grid, kHistThreads, 0, st>>>(p);
        else read_kernel<2, float><<<grid, kHistThreads, 0, st>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_history_gather(const HistoryGatherParams& p, cudaStream_t st) {
    const int grid = p.batch * p.dst_max_pages * p.hk;
    if (p.bits4) gather_kernel<4><<<grid, kHistThreads, 0, st>>>(p);
    else gather_kernel<2><<<grid, kHistThreads, 0, st>>>(p);
    return cudaGetLastError();
}

int64_t pages_copy_pieces(size_t page_bytes) { return (int64_t)((page_bytes + kCopyPiece - 1) / kCopyPiece); }

cudaError_t launch_pages_copy(const PagesCopyParams& p, int n_pools, cudaStream_t st) {
    pages_copy_kernel<<<p.pieces * p.n * n_pools, kHistThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace oscar
