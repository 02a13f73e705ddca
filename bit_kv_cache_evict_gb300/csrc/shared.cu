// shared.cu -- the shared pages of oscar_decode_attn_shared: groups of sequences
// whose histories begin with the same pages attend them once for all.
//
// The rows (member, head) of a group and KV head are stacked: logits S = Q' K^T and
// outputs O = P V of up to 256 rows against each 64-token page are products on
// the 5th-generation tensor cores (tcgen05.mma, operands in shared memory, S, P
// and O in tensor memory), flash-attention style over a run of pages.  A page is
// read and dequantised once for all rows: K and V values s c + z become fp16
// operands with one rounding (fma.rn.f16x2), in the swizzled layout that the
// products read.  The order of the 128 positions inside a product of logits and of the
// 64 tokens inside a product of values is the one in which the codes unpack; Q'
// (prep_kernel) and P are laid out in the same order.
//
// group_kernel  makes the plan: members of each group, its split of the pages.
// shared_kernel a block per item (group, KV head, up to 256 rows, run of pages):
//               a producer warp (bulk copies of the packed pages), four warps
//               that dequantise, a warp that issues the products, and four
//               warps of softmax per 128 rows (a thread per row).
// Partials (o', m, l) per row and run join the split-K partials of the members' own
// pages in merge_kernel.
//
// PARTS = 1 (bf16 output): Q', K, V and P as fp16, off by 2^-11 at most per rounding.  PARTS = 2
// (fp32 output): each as two fp16 parts, three products, 22 bits, and the value
// products of each page are summed from zero and added in fp32 registers, as
// the tensor core truncates its accumulator (int4.cu, page_values).
#include <algorithm>

#include "oscar_common.cuh"
#include "splitk.cuh"

namespace oscar {

namespace {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kMinMembers = 2;  // smaller groups attend by themselves

// One block.  skip[b]: pages of sequence b that its group attends; sref[b]: its
// partials (first, splits, members, index); the groups' items.
__global__ void __launch_bounds__(kPlanThreads) group_kernel(DecodeParamsX p, int rows) {
    extern __shared__ int32_t gsm[];
    int32_t* count = gsm;                 // [n_groups] members
    int32_t* first = gsm + p.n_groups;    // [n_groups] first member's place
    __shared__ int32_t chunk_group[kPlanThreads], chunk_index[kPlanThreads];
    __shared__ int sh_pps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int g = threadIdx.x; g < p.n_groups; g += kPlanThreads) count[g] = 0;
    pdl_wait();
    pdl_trigger();
    auto pages_of = [&](int g) { return min(max(__ldg(p.group_pages + g), 0), p.max_pages); };
    // members in order of their sequences, by warp 0 (one order, whatever the launch)
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int g = b < p.B ? __ldg(p.prefix_group + b) : -1;
        if (g >= p.n_groups) {
            report(p.status, OSCAR_STATUS_BAD_POS);
            g = -1;
        }
        if (g >= 0) {
            const int raw = __ldg(p.group_pages + g), pages = pages_of(g);
            if (raw != pages) report(p.status, OSCAR_STATUS_BAD_POS);
            const int hist = min(max(__ldg(p.hist_len + b), 0), p.max_pages * kPage);
            if (pages == 0 || hist / kPage < pages) g = -1;  // (a history that ends inside the prefix goes by itself)
        }
        chunk_group[threadIdx.x] = g;
        __syncthreads();
        if (warp == 0) {
            for (int i = 0; i < kPlanThreads && b0 + i < p.B; i += 32) {
                const int gg = chunk_group[i + lane];
                const unsigned peers = __match_any_sync(kFull, gg);
                const int rank = __popc(peers & ((1u << lane) - 1u));
                int base = 0;
                if (gg >= 0) base = count[gg];
                chunk_index[i + lane] = base + rank;
                __syncwarp();
                if (gg >= 0 && rank == 0) count[gg] = base + __popc(peers);
                __syncwarp();
            }
        }
        __syncthreads();
        if (b < p.B) p.sref[b] = make_int4(0, 0, chunk_group[threadIdx.x], chunk_index[threadIdx.x]);
    }
    __syncthreads();
    auto tiles_of = [&](int g) {  // row tiles of a group; 0: it is not attended together
        const int n = count[g];
        return n >= kMinMembers ? (n * p.G + rows - 1) / rows : 0;
    };
    if (warp == 0) {
        // Pages per item: the smallest number that leaves at most one item for each
        // block; where even whole groups are more, a quarter of a block's share.
        auto sum_over = [&](auto f) {
            long n = 0;
            for (int g = lane; g < p.n_groups; g += 32) n += f(g);
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) n += __shfl_xor_sync(kFull, n, m);
            return n;
        };
        auto items_at = [&](int pps) {
            return sum_over([&](int g) { return (long)tiles_of(g) * ((pages_of(g) + pps - 1) / pps); }) * p.hk;
        };
        int lo = kMinSharedPages, hi = max(lo, p.max_pages);
        int pps;
        if (items_at(hi) <= p.shared_blocks) {
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                if (items_at(mid) <= p.shared_blocks) hi = mid;
                else lo = mid + 1;
            }
            pps = lo;
        } else {
            const long total = sum_over([&](int g) { return (long)tiles_of(g) * pages_of(g); }) * p.hk;
            pps = (int)max((long)kMinItemPages4, min((long)p.max_pages, total / (4 * p.shared_blocks)));
        }
        int run_member = 0, run_part = 0, run_item = 0;
        for (int g0 = 0; g0 < p.n_groups; g0 += 32) {
            const int g = g0 + lane;
            const int tiles = g < p.n_groups ? tiles_of(g) : 0;
            const int members = tiles ? count[g] : 0, pages = tiles ? pages_of(g) : 0;
            const int splits = (pages + pps - 1) / pps;
            int m = members, pt = splits * members * p.hk, it = splits * tiles * p.hk;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int a = __shfl_up_sync(kFull, m, d), b = __shfl_up_sync(kFull, pt, d), c = __shfl_up_sync(kFull, it, d);
                if (lane >= d) {
                    m += a;
                    pt += b;
                    it += c;
                }
            }
            if (g < p.n_groups) {
                first[g] = run_member + m - members;
                SharedGroup gi;
                gi.pages = pages;
                gi.members = members;
                gi.first_member = first[g];
                gi.splits = splits;
                gi.first_part = run_part + pt - splits * members * p.hk;
                gi.first_item = run_item + it - splits * tiles * p.hk;
                gi.tiles = tiles;
                gi.pad = 0;
                p.groups[g] = gi;
            }
            run_member += __shfl_sync(kFull, m, 31);
            run_part += __shfl_sync(kFull, pt, 31);
            run_item += __shfl_sync(kFull, it, 31);
        }
        if (lane == 0) {
            p.counter[kSharedItems] = run_item;
            sh_pps = pps;
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += kPlanThreads) {
        const int4 r = p.sref[b];
        const int g = r.z;
        int4 out = make_int4(0, 0, 0, 0);
        int skip = 0;
        if (g >= 0 && tiles_of(g) > 0) {
            const SharedGroup gi = p.groups[g];
            p.member[gi.first_member + r.w] = b;
            out = make_int4(gi.first_part, gi.splits, gi.members, r.w);
            skip = gi.pages;
        }
        p.sref[b] = out;
        p.skip[b] = skip;
    }
}

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// D[128 x N] (+)= A B^T, A and B K-major in shared memory (128-byte swizzle), 16 deep
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
                 : "memory");
}
// the same with A in tensor memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
                 : "memory");
}
// Instruction descriptor: fp16 operands, fp32 sums, both K-major, M = 128.
__host__ __device__ constexpr uint32_t tc_idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24); }
// Shared-memory descriptor of a K-major operand whose rows are 128 bytes (64 fp16),
// swizzled by 16-byte chunk ^ row % 8; groups of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
// The loaded registers pass through the wait, so that nothing reads them before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------------------
// dequantisation
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t masked(uint32_t x, uint32_t mask) {  // (x & mask) | 1024.0 in both halves
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(0x64006400u));
    return r;
}
// Codes at bits P.. of the halves of x (mask: the field), as fp16 integers, exact: the
// pattern 0x6400 | c 2^P is 1024 + c 2^P.
template <int P>
__device__ __forceinline__ uint32_t code_at(uint32_t x, uint32_t field) {
    constexpr uint32_t down = (uint32_t)((15 - P) << 10) * 0x10001u;            // 2^-P
    constexpr uint32_t off = (uint32_t)(0x8000 | ((25 - P) << 10)) * 0x10001u;  // -2^(10 - P)
    return h2_fma(masked(x, field << P), down, off);
}
// Two values s c + z (s, z per half) as fp16: hi, and with PARTS = 2 the remainder
// of the fp32 value in lo.
template <int PARTS>
__device__ __forceinline__ void value_pair(uint32_t s, uint32_t c, uint32_t z, uint32_t& hi, uint32_t& lo) {
    if constexpr (PARTS == 1) {
        hi = h2_fma(s, c, z);
    } else {
        const float x = fmaf(half_lo(s), half_lo(c), half_lo(z)), y = fmaf(half_hi(s), half_hi(c), half_hi(z));
        hi = pack_f16x2_rn(x, y);
        lo = pack_f16x2_rn(x - half_lo(hi), y - half_hi(hi));
    }
}

// ---------------------------------------------------------------------------
// kernel
// ---------------------------------------------------------------------------
template <int BITS, int PARTS>
struct SharedSmem {
    static constexpr int T = PARTS == 1 ? 2 : 1;        // 128-row tiles of an item
    static constexpr int kRaw = BITS == 4 ? 2 * (kCodes4 + kPage * 16) : 4096 + 512 * 4;
    static constexpr int kRawStages = PARTS == 1 ? 4 : 2;
    static constexpr int kStages = 2;                   // dequantised pages
    static constexpr int kOperand = kPage * kD * 2;     // fp16 K (or V) of a page
    static constexpr int kQTile = 128 * kD * 2;
    static constexpr int kQ = 0;                        // [T][PARTS] tiles, each two atoms [128 rows][128 bytes]
    static constexpr int kK = kQ + T * PARTS * kQTile;  // [kStages][PARTS], each two atoms [64 rows][128 bytes]
    static constexpr int kV = kK + kStages * PARTS * kOperand;  // [kStages][PARTS] [128 rows][128 bytes]
    static constexpr int kRawAt = kV + kStages * PARTS * kOperand;
    static constexpr int kPairs = kRawAt + kRawStages * kRaw;  // [4 warps][s, z][4 groups][64] fp16
    static constexpr int kBars = kPairs + 4 * 2 * 4 * kPage * 2;
    static constexpr int kNumBars = 2 * kRawStages + 4 * kStages + T * 4 + T + 1;
    static constexpr int kBytes = kBars + kNumBars * 8 + 32;
    static constexpr int kAlloc = kBytes + 1024;        // the swizzled operands start on 1024 bytes
    static_assert(kAlloc <= 227 * 1024, "shared memory of a block");
    static constexpr int kSoftWarps = 4 * T;
    static constexpr int kThreads = (kSoftWarps + 4 + 2) * 32;
    // tensor memory, columns: PARTS = 1: per tile S [2][64] (P in the first 32 columns
    // of its S) and O [128]; PARTS = 2: S [2][64], P [2][64] (hi, lo), O [2][128]
    static constexpr int kTileCols = 256;
    static constexpr int kColP = PARTS == 1 ? 0 : 128, kColO = PARTS == 1 ? 128 : 256;
    static constexpr int kCols = 512;
};

// log2 of the factor that P carries, so that small weights are not subnormal
// fp16, and how far a row's logits may pass the subtracted maximum before its
// sums are rescaled: P stays below 2^(kShift + kSlack + 1)
constexpr float kShift = 6.f, kSlack = 8.f;

template <int BITS, int PARTS>
__global__ void __launch_bounds__(SharedSmem<BITS, PARTS>::kThreads, 1) shared_kernel(DecodeParamsX p) {
    using SM = SharedSmem<BITS, PARTS>;
    constexpr int T = SM::T, NS = SM::kStages, NR = SM::kRawStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + SM::kBars);
    uint64_t* raw_empty = raw_full + NR;
    uint64_t* k_full = raw_empty + NR;
    uint64_t* k_empty = k_full + NS;
    uint64_t* v_full = k_empty + NS;
    uint64_t* v_empty = v_full + NS;
    uint64_t* s_full = v_empty + NS;   // [T][2]
    uint64_t* p_full = s_full + 2 * T; // [T][2]
    uint64_t* o_done = p_full + 2 * T; // [T]
    uint64_t* drain = o_done + T;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* dead = reinterpret_cast<volatile int*>(tmem_at + 1);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NR; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2 * T; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        for (int i = 0; i < T; ++i) mbar_init(&o_done[i], 1);
        mbar_init(drain, 1);
        fence_mbar_init();
        *dead = 0;
    }
    if (warp == 0) tmem_alloc(tmem_at, SM::kCols);
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_at;
    pdl_wait();     // plan and Q' rows
    pdl_trigger();

    const int total = __ldg(p.counter + kSharedItems);
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // by a whole warp
        if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
        if (__all_sync(kFull, mbar_wait_bounded(bar, parity, kWaitPolls))) return true;
        if (lane == 0) {
            report(p.status, OSCAR_STATUS_TIMEOUT);
            *dead = 1;
        }
        return false;
    };
    bool ok = true;
    uint32_t done = 0;          // pages of earlier items (rings of the pages)
    uint32_t tile_done[T] = {};  // the same of each row tile's barriers (an item may have one tile only)

    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        // ---- the item: group, KV head, row tile, run of pages
        int lo = 0, hi = p.n_groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(&p.groups[mid].first_item) <= item) lo = mid;
            else hi = mid;
        }
        const SharedGroup gi = p.groups[lo];
        const int rel = item - gi.first_item;
        const int split = rel % gi.splits, kv = rel / gi.splits % p.hk, rt = rel / gi.splits / p.hk;
        const int pg0 = (int)((long)gi.pages * split / gi.splits), pg1 = (int)((long)gi.pages * (split + 1) / gi.splits);
        const int32_t* members = p.member + gi.first_member;
        const int32_t* table = p.page_table + (size_t)__ldg(members) * p.max_pages;
        const int row0 = rt * T * 128, rows_left = gi.members * p.G - row0;
        const int tiles = T == 2 && rows_left > 128 ? 2 : 1;
        int n = 0;  // pages that can be read
        for (int q0 = pg0; q0 < pg1; q0 += 32) {
            const int q = q0 + lane;
            const int id = q < pg1 ? __ldg(table + q) : -1;
            n += __popc(__ballot_sync(kFull, id >= 0 && id < p.num_pages));
        }

        // ---- Q' rows into their tiles (zeros behind the last row)
        if (warp < SM::kSoftWarps) {
            for (int i = threadIdx.x; i < tiles * 128 * 16; i += SM::kSoftWarps * 32) {
                const int r = i >> 4, c = i & 15, t = r >> 7, rr = r & 127;
                const int row = row0 + r;
                uint8_t* to = smem + SM::kQ + t * PARTS * SM::kQTile + (c >> 3) * (128 * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
                uint4 v[PARTS];
#pragma unroll
                for (int part = 0; part < PARTS; ++part) v[part] = make_uint4(0u, 0u, 0u, 0u);
                if (row < gi.members * p.G) {
                    const size_t at = ((size_t)__ldg(members + row / p.G) * p.hk + kv) * p.G + row % p.G;
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
                        v[part] = __ldg(reinterpret_cast<const uint4*>(p.qrow + ((size_t)part * p.B * p.hq + at) * kD) + c);
                }
#pragma unroll
                for (int part = 0; part < PARTS; ++part) *reinterpret_cast<uint4*>(to + part * SM::kQTile) = v[part];
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncthreads();

        if (warp < SM::kSoftWarps) {
            // ------------------------------ softmax ------------------------------
            const int t = warp >> 2;
            if (t < tiles) {
                const int r = row0 + t * 128 + (warp & 3) * 32 + lane;
                const bool row_on = r < gi.members * p.G;
                const int b = row_on ? __ldg(members + r / p.G) : 0, head = row_on ? r % p.G : 0;
                const float kq = row_on ? __ldg(p.qkinv + ((size_t)b * p.hk + kv) * 4) : 1.f;  // 2^-e of the Q' rows
                const uint32_t lanes = tmem + t * SM::kTileCols + ((uint32_t)((warp & 3) * 32) << 16);
                float m_run = -INFINITY, l0 = 0.f, l1 = 0.f;
                float o[PARTS == 2 ? kD : 1];
                if constexpr (PARTS == 2)
#pragma unroll
                    for (int d = 0; d < kD; ++d) o[d] = 0.f;
                const uint32_t g0 = T == 2 ? tile_done[t] : done;
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t g = g0 + j, buf = g & 1u;
                    if (!(ok = wait(&s_full[2 * t + buf], (g >> 1) & 1u))) break;
                    tc_after();
                    const uint32_t sa = lanes + buf * 64;
                    uint32_t s[2][32];
                    tmem_ld32(s[0], sa);
                    tmem_ld32(s[1], sa + 32);
                    tmem_wait_ld(s[0]);
                    tmem_wait_ld(s[1]);
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fmaxf(__uint_as_float(s[0][i]), __uint_as_float(s[1][i])));
                    mx *= kq;
                    float alpha = 1.f;
                    const bool over = PARTS == 2 ? mx > m_run : mx > m_run + kSlack;
                    const bool any = __any_sync(kFull, over);
                    if (any) {
                        const float m_new = fmaxf(m_run, mx);
                        alpha = m_new > m_run ? ex2(m_run - m_new) : 1.f;
                        m_run = m_new;
                        l0 *= alpha;
                        l1 *= alpha;
                    }
                    const float off = finite_max(m_run) - kShift;
                    const float2 kk = make_float2(kq, kq), oo = make_float2(-off, -off);
                    float2 sum = make_float2(0.f, 0.f);
                    uint32_t ph[2][16], pl[PARTS == 2 ? 2 : 1][16];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            // tokens i .. i + 3; stored (0, 2), (1, 3)
                            const float2 x = fma2(make_float2(__uint_as_float(s[h][i]), __uint_as_float(s[h][i + 2])), kk, oo);
                            const float2 y = fma2(make_float2(__uint_as_float(s[h][i + 1]), __uint_as_float(s[h][i + 3])), kk, oo);
                            const float2 pa = make_float2(ex2(x.x), ex2(x.y)), pb = make_float2(ex2(y.x), ex2(y.y));
                            sum = add2(sum, add2(pa, pb));
                            ph[h][i / 2] = pack_f16x2_rn(pa.x, pa.y);
                            ph[h][i / 2 + 1] = pack_f16x2_rn(pb.x, pb.y);
                            if constexpr (PARTS == 2) {
                                pl[h][i / 2] = pack_f16x2_rn(pa.x - half_lo(ph[h][i / 2]), pa.y - half_hi(ph[h][i / 2]));
                                pl[h][i / 2 + 1] = pack_f16x2_rn(pb.x - half_lo(ph[h][i / 2 + 1]), pb.y - half_hi(ph[h][i / 2 + 1]));
                            }
                        }
                    l0 += sum.x;
                    l1 += sum.y;
                    if constexpr (PARTS == 1) {
                        if (any && j > 0) {  // rescale O, once the products of the page before are in it
                            if (!(ok = wait(&o_done[t], (g - 1) & 1u))) break;
                            tc_after();
#pragma unroll
                            for (int c = 0; c < kD; c += 32) {
                                uint32_t v[32];
                                tmem_ld32(v, lanes + SM::kColO + c);
                                tmem_wait_ld(v);
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                                tmem_st32(lanes + SM::kColO + c, v);
                            }
                        }
                        tmem_st16(sa, ph[0]);
                        tmem_st16(sa + 16, ph[1]);
                    } else {
                        const uint32_t pa = lanes + SM::kColP + buf * 64;
                        tmem_st16(pa, ph[0]);
                        tmem_st16(pa + 16, ph[1]);
                        tmem_st16(pa + 32, pl[0]);
                        tmem_st16(pa + 48, pl[1]);
                    }
                    tmem_wait_st();
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * t + buf]);
                    if constexpr (PARTS == 2) {
                        // the page before: its products, in its own maximum's units, then this page's
                        if (j > 0) {
                            if (!(ok = wait(&o_done[t], (g - 1) & 1u))) break;
                            tc_after();
#pragma unroll
                            for (int c = 0; c < kD; c += 32) {
                                uint32_t v[32];
                                tmem_ld32(v, lanes + SM::kColO + (buf ^ 1u) * kD + c);
                                tmem_wait_ld(v);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[c + i] = (o[c + i] + __uint_as_float(v[i])) * alpha;
                            }
                        }
                    }
                }
                // ---- the row's partial
                if (ok && n > 0) {
                    // (a parity tells two neighbouring phases apart: the one before the last comes first;
                    // inside the loop S of page j is there only once the products of page j - 2 are done)
                    if (PARTS == 1 && n > 1) ok = wait(&o_done[t], (g0 + n - 2) & 1u);
                    ok = ok && wait(&o_done[t], (g0 + n - 1) & 1u);
                    tc_after();
                }
                if (ok) {
                    const float l = l0 + l1;
                    float* part = p.sh_part + ((size_t)gi.first_part + ((size_t)kv * gi.splits + split) * gi.members + (row_on ? r / p.G : 0)) * p.part_stride;
#pragma unroll
                    for (int c = 0; c < kD; c += 32) {
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0u;
                        if (n > 0) {
                            tmem_ld32(v, lanes + SM::kColO + (PARTS == 2 ? ((g0 + n - 1) & 1u) * kD : 0) + c);
                            tmem_wait_ld(v);
                        }
                        if constexpr (PARTS == 2)
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(o[c + i] + __uint_as_float(v[i]));
                        if (row_on)
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<uint4*>(part + head * kD + c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                    if (row_on) {
                        part[p.G * kD + head] = l == 0.f ? -INFINITY : finite_max(m_run) - kShift;
                        part[p.G * kD + p.G + head] = l;
                    }
                }
                tc_before();
            }
        } else if (warp < SM::kSoftWarps + 4) {
            // --------------------------- dequantisation ---------------------------
            const int wq = warp - SM::kSoftWarps;
            const int ng = 4 >> p.gshift;
            uint16_t* sS = reinterpret_cast<uint16_t*>(smem + SM::kPairs) + wq * (2 * 4 * kPage);  // [4 groups][64] s, then z
            uint16_t* zS = sS + 4 * kPage;
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t g = done + j, st = g % NS, rs = g % NR;
                if (!(ok = wait(&raw_full[rs], (g / NR) & 1u))) break;
                const uint8_t* blk = smem + SM::kRawAt + rs * SM::kRaw;
                if (g >= NS && !(ok = wait(&k_empty[st], ((g / NS) - 1) & 1u))) break;
                uint8_t* kS = smem + SM::kK + st * PARTS * SM::kOperand;
                const int a = lane & 3, t8 = (((lane >> 2) & 1) << 2) | (lane >> 3);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = 16 * wq + 8 * u + t8;
                    uint32_t w[4], sz[4];
                    if constexpr (BITS == 4) {
                        const uint4 x = *reinterpret_cast<const uint4*>(blk + t * 64 + 16 * a);
                        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(blk + t * 32 + 8 * a);
                        w[0] = x.x; w[1] = x.y; w[2] = x.x >> 8; w[3] = x.y >> 8;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sz[k] = *reinterpret_cast<const uint32_t*>(blk + (BITS == 4 ? kCodes4 : kKScale) + (t * ng + (k >> p.gshift)) * 4);
                    uint8_t* row = kS + t * 128;
                    auto chunk = [&](auto kk) {
                        constexpr int k = decltype(kk)::value;
                        const uint32_t s2 = __byte_perm(sz[k], 0u, 0x1010), z2 = __byte_perm(sz[k], 0u, 0x3232);
                        uint32_t c[4], hi[4], lo[4];
                        if constexpr (BITS == 4) {
                            const uint32_t y = w[k] >> 8;
                            c[0] = code_at<0>(w[k], 0x000f000fu);
                            c[1] = code_at<4>(w[k], 0x000f000fu);
                            c[2] = code_at<0>(y, 0x000f000fu);
                            c[3] = code_at<4>(y, 0x000f000fu);
                        } else {
                            c[0] = code_at<2 * k>(w[0], 0x00030003u);
                            c[1] = code_at<2 * k>(w[2], 0x00030003u);
                            c[2] = code_at<2 * k>(w[1], 0x00030003u);
                            c[3] = code_at<2 * k>(w[3], 0x00030003u);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) value_pair<PARTS>(s2, c[i], z2, hi[i], lo[i]);
                        uint8_t* to = row + (k >> 1) * (kPage * 128) + (((4 * (k & 1) + a) ^ (t & 7)) << 4);
                        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        if constexpr (PARTS == 2) *reinterpret_cast<uint4*>(to + SM::kOperand) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    };
                    chunk(std::integral_constant<int, 0>{});
                    chunk(std::integral_constant<int, 1>{});
                    chunk(std::integral_constant<int, 2>{});
                    chunk(std::integral_constant<int, 3>{});
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_full[st]);
                // V: the pairs first, by group and in the tokens' order of the products
                if (g >= NS && !(ok = wait(&v_empty[st], ((g / NS) - 1) & 1u))) break;
                uint8_t* vS = smem + SM::kV + st * PARTS * SM::kOperand;
                const uint8_t* vh = blk + (BITS == 4 ? half_bytes4(p.gshift) : kVCodes);
                const uint8_t* vp = blk + (BITS == 4 ? half_bytes4(p.gshift) + kCodes4 : v_scale_off(p.gshift));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = lane + 32 * u, at = (t & ~3) | pv_slot(t & 3);
                    if constexpr (BITS == 4) {  // warp wq: positions 32 wq .. + 31, one group
                        const uint32_t x = *reinterpret_cast<const uint32_t*>(vp + (t * ng + (wq >> p.gshift)) * 4);
                        sS[at] = (uint16_t)x;
                        zS[at] = (uint16_t)(x >> 16);
                    } else {
                        for (int k = 0; k < ng; ++k) {
                            const uint32_t x = *reinterpret_cast<const uint32_t*>(vp + (t * ng + k) * 4);
                            sS[k * kPage + at] = (uint16_t)x;
                            zS[k * kPage + at] = (uint16_t)(x >> 16);
                        }
                    }
                }
                __syncwarp();
                const int tc = lane & 3, jj = lane >> 2;
                // one row (stored position pos) of 16 tokens from the codes at bits P of the plane words x
                auto v_row = [&](auto pp, int pos, const uint4& x, const uint32_t (&s)[8], const uint32_t (&z)[8]) {
                    constexpr int P = decltype(pp)::value;
                    constexpr uint32_t field = BITS == 4 ? 0x000f000fu : 0x00030003u;
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        value_pair<PARTS>(s[2 * i], code_at<P>(w[i], field), z[2 * i], hi[2 * i], lo[2 * i]);
                        value_pair<PARTS>(s[2 * i + 1], code_at<P>(w[i] >> 8, field), z[2 * i + 1], hi[2 * i + 1], lo[2 * i + 1]);
                    }
                    uint8_t* row = vS + pos * 128;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint8_t* to = row + (((2 * tc + h) ^ (pos & 7)) << 4);
                        *reinterpret_cast<uint4*>(to) = make_uint4(hi[4 * h], hi[4 * h + 1], hi[4 * h + 2], hi[4 * h + 3]);
                        if constexpr (PARTS == 2) *reinterpret_cast<uint4*>(to + SM::kOperand) = make_uint4(lo[4 * h], lo[4 * h + 1], lo[4 * h + 2], lo[4 * h + 3]);
                    }
                };
                auto pairs_of = [&](int k, uint32_t (&s)[8], uint32_t (&z)[8]) {
                    const uint4* sp = reinterpret_cast<const uint4*>(sS + k * kPage + 16 * tc);
                    const uint4* zp = reinterpret_cast<const uint4*>(zS + k * kPage + 16 * tc);
                    const uint4 s0 = sp[0], s1 = sp[1], z0 = zp[0], z1 = zp[1];
                    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
                    z[0] = z0.x; z[1] = z0.y; z[2] = z0.z; z[3] = z0.w; z[4] = z1.x; z[5] = z1.y; z[6] = z1.z; z[7] = z1.w;
                };
                uint32_t s[8], z[8];
                if constexpr (BITS == 4) {
                    pairs_of(0, s, z);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int plane = 16 * wq + 8 * u + jj;
                        const uint4 x = *reinterpret_cast<const uint4*>(vh + plane * kPage + 16 * tc);
                        v_row(std::integral_constant<int, 0>{}, 2 * plane, x, s, z);
                        v_row(std::integral_constant<int, 4>{}, 2 * plane + 1, x, s, z);
                    }
                } else {
                    const int plane = 8 * wq + jj;
                    const uint4 x = *reinterpret_cast<const uint4*>(vh + plane * kPage + 16 * tc);
                    auto slot = [&](auto ii) {
                        constexpr int i = decltype(ii)::value;
                        pairs_of(i >> p.gshift, s, z);
                        v_row(std::integral_constant<int, 2 * i>{}, 32 * i + plane, x, s, z);
                    };
                    slot(std::integral_constant<int, 0>{});
                    slot(std::integral_constant<int, 1>{});
                    slot(std::integral_constant<int, 2>{});
                    slot(std::integral_constant<int, 3>{});
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&v_full[st]);
                    mbar_arrive(&raw_empty[rs]);
                }
            }
        } else if (warp == SM::kSoftWarps + 4) {
            // ------------------------------ products ------------------------------
            const uint32_t qa = smem_u32(smem + SM::kQ), ka = smem_u32(smem + SM::kK), va = smem_u32(smem + SM::kV);
            bool issued = false;
            auto values_of = [&](int j) {  // O (+)= P V of page j
                const uint32_t g = done + j, st = g % NS;
                for (int t = 0; t < tiles; ++t) {
                    const uint32_t gt = (T == 2 ? tile_done[t] : done) + j, buf = gt & 1u;
                    if (!wait(&p_full[2 * t + buf], (gt >> 1) & 1u)) return false;
                    if (t == 0 && !wait(&v_full[st], (g / NS) & 1u)) return false;
                    tc_after();
                    if (lane == 0) {
                        const uint32_t tt = tmem + t * SM::kTileCols;
                        const uint32_t pa = tt + SM::kColP + buf * 64, o = tt + SM::kColO + (PARTS == 2 ? buf * kD : 0);
#pragma unroll
                        for (int pr = 0; pr < (PARTS == 1 ? 1 : 3); ++pr)  // hi hi, lo hi, hi lo
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc_mma_ts(o, pa + (pr == 1 ? 32 : 0) + 8 * k, tc_desc(va + (st * PARTS + (pr == 2)) * SM::kOperand + 32 * k),
                                          tc_idesc(kD), (PARTS == 1 && j > 0) || pr > 0 || k > 0);
                        tc_commit(&o_done[t]);
                    }
                    __syncwarp();
                }
                if (lane == 0) tc_commit(&v_empty[st]);
                __syncwarp();
                return true;
            };
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t g = done + j, st = g % NS;
                if (!(ok = wait(&k_full[st], (g / NS) & 1u))) break;
                for (int t = 0; t < tiles && ok; ++t) {
                    const uint32_t gt = (T == 2 ? tile_done[t] : done) + j, buf = gt & 1u;
                    // S takes the place of the P of two pages before: its products are to be done
                    if (PARTS == 1 && j >= 2 && !(ok = wait(&o_done[t], gt & 1u))) break;
                    tc_after();
                    if (lane == 0) {
                        const uint32_t s = tmem + t * SM::kTileCols + buf * 64;
#pragma unroll
                        for (int pr = 0; pr < (PARTS == 1 ? 1 : 3); ++pr)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                tc_mma_ss(s, tc_desc(qa + (t * PARTS + (pr == 1)) * SM::kQTile + (k >> 2) * (128 * 128) + 32 * (k & 3)),
                                          tc_desc(ka + (st * PARTS + (pr == 2)) * SM::kOperand + (k >> 2) * (kPage * 128) + 32 * (k & 3)),
                                          tc_idesc(kPage), pr > 0 || k > 0);
                        tc_commit(&s_full[2 * t + buf]);
                    }
                    issued = true;
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) tc_commit(&k_empty[st]);
                __syncwarp();
                if (j > 0) ok = values_of(j - 1);
            }
            if (ok && n > 0) ok = values_of(n - 1);
            if (!ok && issued) {  // whatever was issued ends before the block does
                if (lane == 0) tc_commit(drain);
                __syncwarp();
                (void)mbar_wait_bounded(drain, 0, kWaitPolls);
            }
        } else {
            // ------------------------------ producer ------------------------------
            int j = 0;  // pages issued
            for (int q0 = pg0; q0 < pg1 && ok; q0 += 32) {
                const int q = q0 + lane;
                const int id = q < pg1 ? __ldg(table + q) : -1;
                const bool good = id >= 0 && id < p.num_pages;
                if (q < pg1 && !good) report(p.status, OSCAR_STATUS_BAD_PAGE);
                const unsigned have = __ballot_sync(kFull, good);
                for (unsigned left = have; left && ok; left &= left - 1) {
                    const int page = __shfl_sync(kFull, id, __ffs(left) - 1);
                    const uint32_t g = done + j, rs = g % NR;
                    if (g >= NR && !(ok = wait(&raw_empty[rs], ((g / NR) - 1) & 1u))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&raw_full[rs], p.block_bytes);
                        bulk_g2s(smem + SM::kRawAt + rs * SM::kRaw, p.pool + ((size_t)page * p.hk + kv) * p.block_bytes, p.block_bytes, &raw_full[rs]);
                    }
                    __syncwarp();
                    ++j;
                }
            }
            if (!ok)  // copies in flight land before the block ends
                for (uint32_t g = done + j > NR ? done + j - NR : 0; g < done + j; ++g)
                    (void)mbar_wait_bounded(&raw_full[g % NR], (g / NR) & 1u, kWaitPolls);
        }
        __syncthreads();
        if (*dead) break;
        done += n;
#pragma unroll
        for (int t = 0; t < T; ++t)
            if (t < tiles) tile_done[t] += n;
    }
    tc_before();
    __syncthreads();
    if (warp == 0) tmem_free(tmem, SM::kCols);
}

template <int BITS, int PARTS>
cudaError_t launch_parts(const DecodeParamsX& p, cudaStream_t st, int dev) {
    using SM = SharedSmem<BITS, PARTS>;
    static bool set[64];
    if (!set[dev & 63]) {
        const cudaError_t e = set_smem(shared_kernel<BITS, PARTS>, SM::kAlloc);
        if (e != cudaSuccess) return e;
        set[dev & 63] = true;
    }
    return launch_pdl(shared_kernel<BITS, PARTS>, dim3(p.shared_blocks), dim3(SM::kThreads), SM::kAlloc, st, p);
}

}  // namespace

cudaError_t launch_shared_plan(const DecodeParamsX& p, cudaStream_t st, int dev) {
    static bool set[64];
    if (!set[dev & 63]) {
        const cudaError_t e = set_smem(group_kernel, 2 * kMaxSharedGroups * 4, false);
        if (e != cudaSuccess) return e;
        set[dev & 63] = true;
    }
    return launch_pdl(group_kernel, dim3(1), dim3(kPlanThreads), (size_t)2 * p.n_groups * 4, st, p, p.out_bf16 ? 256 : 128);
}

cudaError_t launch_shared(const DecodeParamsX& p, int bits, cudaStream_t st, int dev) {
    if (bits == 4) return p.out_bf16 ? launch_parts<4, 1>(p, st, dev) : launch_parts<4, 2>(p, st, dev);
    return p.out_bf16 ? launch_parts<2, 1>(p, st, dev) : launch_parts<2, 2>(p, st, dev);
}

}  // namespace oscar
