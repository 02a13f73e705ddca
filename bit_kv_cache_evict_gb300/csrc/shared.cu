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
//               four warps of softmax per 128 rows (a thread per row), with an fp32
//               output four that add up the products of values, eight warps that
//               dequantise, two that issue the products (of logits, of values) and two that
//               copy (the packed pages, q').
// Partials (o', m, l) per row and run join the split-K partials of the members' own
// pages in merge_kernel.
//
// PARTS = 1 (bf16 output): Q', K, V and P as fp16, off by 2^-11 at most per rounding.  PARTS = 2
// (fp32 output): each as two fp16 parts, three products, 22 bits (a weight down to 2^-40 of
// the largest of its run of pages so far), and the value
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
// Which groups attend together, where the caller leaves it to the library.  A page of a
// KV head costs the members' own kernels 0.28 us of an SM per sequence (64 x 28K, 32:8
// heads: 504 us without sharing, 88 us of it not the prefix), shared_kernel about 0.8 us
// for up to 128 rows and 1.06 for 256 with a bf16 output, 1.8 for 128 rows with fp32: as
// many sequences as this.
__device__ __forceinline__ int shared_cost(int members, int G, int rows) {
    const int n = members * G;
    if (rows == 256) return n <= 128 ? 3 : (n + 255) / 256 * 4;
    return (n + 127) / 128 * (G == 8 ? 5 : 6);
}
// and 8 us for its start and end and its partials' merge, of all groups together: the
// pages of a KV head and sequence that take as long.  Eight members, 16K tokens: 44 us,
// 53 each by itself; 4K: 36 and 29; pairs behind 16K in eight groups: 132 and 97.
constexpr long kMinSaved = 4300;

// One block.  skip[b]: pages of sequence b that its group attends; sref[b]: its
// partials (first, splits, members, index); qref[b]: its rows of q'; and the items.
__global__ void __launch_bounds__(kPlanThreads) group_kernel(DecodeParamsX p, int rows) {
    extern __shared__ int32_t gsm[];
    int32_t* count = gsm;                          // [n_groups] members; 0 for a group that is not attended together
    int32_t* pages = count + p.n_groups;           // [n_groups]
    int32_t* first_item = pages + p.n_groups;      // [n_groups]
    int32_t* first_part = first_item + p.n_groups;
    int32_t* first_tile = first_part + p.n_groups;
    int32_t* first_seq = first_tile + p.n_groups;  // whose page-table row tells the group's pages
    __shared__ int32_t chunk_group[kPlanThreads], chunk_index[kPlanThreads];
    __shared__ int sh_pps, sh_total;
    __shared__ unsigned long long sh_saved;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    int g_first = threadIdx.x < p.B ? __ldg(p.prefix_group + threadIdx.x) : -1;  // (one round trip for all three)
    int h_first = threadIdx.x < p.B ? __ldg(p.hist_len + threadIdx.x) : 0;
    for (int g = threadIdx.x; g < p.n_groups; g += kPlanThreads) {
        const int raw = __ldg(p.group_pages + g), n = min(max(raw, 0), p.max_pages);
        if (raw != n) report(p.status, OSCAR_STATUS_BAD_POS);
        count[g] = 0;
        pages[g] = n;
    }
    if (threadIdx.x == 0) sh_saved = 0;
    __syncthreads();
    // members in order of their sequences, by warp 0 (one order, whatever the launch)
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int g = b0 == 0 ? g_first : b < p.B ? __ldg(p.prefix_group + b) : -1;
        const int h = b0 == 0 ? h_first : b < p.B ? __ldg(p.hist_len + b) : 0;
        if (g >= p.n_groups) {
            report(p.status, OSCAR_STATUS_BAD_POS);
            g = -1;
        }
        // (a history that ends inside the prefix goes by itself)
        if (g >= 0 && (pages[g] == 0 || min(max(h, 0), p.max_pages * kPage) / kPage < pages[g])) g = -1;
        chunk_group[threadIdx.x] = g;
        __syncthreads();
        if (warp == 0) {
            for (int i = 0; i < kPlanThreads && b0 + i < p.B; i += 32) {
                const int gg = chunk_group[i + lane];
                const unsigned peers = __match_any_sync(kFull, gg);
                const int rank = __popc(peers & ((1u << lane) - 1u));
                const int base = gg >= 0 ? count[gg] : 0;
                chunk_index[i + lane] = base + rank;
                __syncwarp();
                if (gg >= 0 && rank == 0) count[gg] = base + __popc(peers);
                __syncwarp();
            }
        }
        __syncthreads();
        if (b < p.B) p.sref[b] = make_int4(0, 0, chunk_group[threadIdx.x], chunk_index[threadIdx.x]);
    }
    for (int g = threadIdx.x; g < p.n_groups; g += kPlanThreads) {
        const int gain = p.min_members > 0 ? count[g] - max(p.min_members, 2) + 1 : count[g] - shared_cost(count[g], p.G, rows);
        if (gain <= 0) count[g] = 0;
        else atomicAdd(&sh_saved, (unsigned long long)gain * pages[g] * p.hk);
    }
    __syncthreads();
    if (p.min_members == 0 && sh_saved < kMinSaved)
        for (int g = threadIdx.x; g < p.n_groups; g += kPlanThreads) count[g] = 0;
    __syncthreads();
    auto row_tiles = [&](int g, int of) { return (count[g] * p.G + of - 1) / of; };
    if (warp == 0) {
        // Pages per item: the smallest number that leaves at most one item for each
        // block; where even whole groups (or the longest runs) are more, a quarter of a block's share.
        auto items_at = [&](int pps) {  // (each group's share is cut off far above what it is compared with)
            unsigned n = 0;
            for (int g = lane; g < p.n_groups; g += 32)
                n += (unsigned)min((long)row_tiles(g, rows) * ((pages[g] + pps - 1) / pps) * p.hk, 1l << 16);
            return __reduce_add_sync(kFull, n);
        };
        int lo = kMinSharedPages, hi = min(max(lo, p.max_pages), kMaxSharedRun);
        int pps;
        if (items_at(hi) <= (unsigned)p.shared_blocks) {
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                if (items_at(mid) <= (unsigned)p.shared_blocks) hi = mid;
                else lo = mid + 1;
            }
            pps = lo;
        } else {
            long total = 0;
            for (int g = lane; g < p.n_groups; g += 32) total += (long)row_tiles(g, rows) * pages[g];
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) total += __shfl_xor_sync(kFull, total, m);
            pps = (int)max((long)kMinItemPages4, min((long)min(p.max_pages, kMaxSharedRun), total * p.hk / (4 * p.shared_blocks)));
        }
        int run_part = 0, run_item = 0, run_tile = 0;
        for (int g0 = 0; g0 < p.n_groups; g0 += 32) {
            const int g = g0 + lane;
            const bool on = g < p.n_groups && count[g] > 0;
            const int splits = on ? (pages[g] + pps - 1) / pps : 0;
            const int np = on ? splits * count[g] * p.hk : 0, ni = on ? splits * row_tiles(g, rows) * p.hk : 0;
            const int nt = on ? row_tiles(g, 128) * p.hk : 0;
            int pt = np, it = ni, qt = nt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(kFull, pt, d), y = __shfl_up_sync(kFull, it, d), z = __shfl_up_sync(kFull, qt, d);
                if (lane >= d) {
                    pt += x;
                    it += y;
                    qt += z;
                }
            }
            if (g < p.n_groups) {
                first_part[g] = run_part + pt - np;
                first_item[g] = run_item + it - ni;
                first_tile[g] = run_tile + qt - nt;
            }
            run_part += __shfl_sync(kFull, pt, 31);
            run_item += __shfl_sync(kFull, it, 31);
            run_tile += __shfl_sync(kFull, qt, 31);
        }
        if (lane == 0) {
            p.counter[kSharedItems] = run_item;
            sh_pps = pps;
            sh_total = run_item;
        }
    }
    __syncthreads();
    const int pps = sh_pps, total = sh_total;
    for (int b = threadIdx.x; b < p.B; b += kPlanThreads) {
        const int4 r = p.sref[b];
        const int g = r.z;
        int4 part = make_int4(0, 0, 0, 0), q = make_int4(-1, 0, 0, 0);
        int skip = 0;
        if (g >= 0 && count[g] > 0) {
            part = make_int4(first_part[g], (pages[g] + pps - 1) / pps, count[g], r.w);
            q = make_int4(first_tile[g], row_tiles(g, 128), r.w, 0);
            skip = pages[g];
            if (r.w == 0) first_seq[g] = b;
        }
        p.sref[b] = part;
        p.qref[b] = q;
        p.skip[b] = skip;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < total; i += kPlanThreads) {
        int lo = 0, hi = p.n_groups;  // the last group that starts at or before item i and has items
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_item[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int splits = (pages[lo] + pps - 1) / pps, rel = i - first_item[lo];
        const int split = rel % splits, kv = rel / splits % p.hk, rt = rel / splits / p.hk;
        SharedItem it;
        it.seq = first_seq[lo];
        it.kv = kv;
        it.pg0 = (int)((long)pages[lo] * split / splits);
        it.pages = (int)((long)pages[lo] * (split + 1) / splits) - it.pg0;
        it.row0 = rt * rows;
        it.rows = min(rows, count[lo] * p.G - it.row0);
        it.qtile = first_tile[lo] + kv * row_tiles(lo, 128) + rt * (rows / 128);
        it.part0 = first_part[lo] + (kv * splits + split) * count[lo];
        p.items[i] = it;
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
__device__ __forceinline__ void tc_commit(uint32_t on, uint64_t* bar) {
    asm volatile("{ .reg .pred e; setp.ne.b32 e, %0, 0; @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1]; }" ::"r"(on),
                 "r"(smem_u32(bar))
                 : "memory");
}
// One lane of the warp, the same every time.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r;
}
// D[128 x N] (+)= A B^T, A and B K-major in shared memory (128-byte swizzle), 16 deep.  The
// whole warp calls, the elected lane issues: under a branch of one lane the
// operands are not uniform for the compiler and an issue took about 180 cycles.
__device__ __forceinline__ void tc_mma_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{ .reg .pred e, p; setp.ne.b32 e, %0, 0; setp.ne.b32 p, %5, 0; @e tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p; }" ::"r"(on),
                 "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}
// the same with A in tensor memory
__device__ __forceinline__ void tc_mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{ .reg .pred e, p; setp.ne.b32 e, %0, 0; setp.ne.b32 p, %5, 0; @e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p; }" ::"r"(on),
                 "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
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
constexpr int kDequantWarps = 8;

template <int BITS, int PARTS>
struct SharedSmem {
    static constexpr int T = PARTS == 1 ? 2 : 1;        // 128-row tiles of an item
    static constexpr int kRaw = BITS == 4 ? 2 * (kCodes4 + kPage * 16) : 4096 + 512 * 4;
    static constexpr int kRawStages = PARTS == 1 ? 4 : 2;
    static constexpr int kStages = 2;                   // dequantised pages
    static constexpr int kOperand = kPage * kD * 2;     // fp16 K (or V) of a page
    static constexpr int kQTile = kQTileBytes;
    static constexpr int kQ = 0;                        // [T][PARTS] tiles, each two atoms [128 rows][128 bytes]
    static constexpr int kK = kQ + T * PARTS * kQTile;  // [kStages][PARTS], each two atoms [64 rows][128 bytes]
    static constexpr int kV = kK + kStages * PARTS * kOperand;  // [kStages][PARTS] [128 rows][128 bytes]
    static constexpr int kRawAt = kV + kStages * PARTS * kOperand;
    static constexpr int kPairs = kRawAt + kRawStages * kRaw;  // [kDequantWarps][groups][s, z][64] fp16
    static constexpr int kPairGroups = BITS == 4 ? 1 : 4;      // groups that a warp's rows of V belong to, at most
    static constexpr int kPairBytes = kPairGroups * 2 * kPage * 2;
    static constexpr int kBars = kPairs + kDequantWarps * kPairBytes;
    static constexpr int kNumBars = 2 * kRawStages + 4 * kStages + T * 6 + 4 + 3;
    static constexpr int kAlpha = kBars + kNumBars * 8 + 32;    // PARTS = 2: [2][128] factors that a page's maxima give the sums so far
    static constexpr int kBytes = kAlpha + (PARTS == 2 ? 2 * 128 * 4 : 0);
    static constexpr int kAlloc = kBytes + 1024;        // the swizzled operands start on 1024 bytes
    static_assert(kAlloc <= 227 * 1024, "shared memory of a block");
    // warps by role, in whole warpgroups: softmax (four per tile), PARTS = 2: four that add up the
    // products of values, dequantisation, then one that issues the products of logits, one
    // those of values, one that copies pages and one that copies q'
    static constexpr int kSoftWarps = 4 * T;
    static constexpr int kRowWarps = 8;  // softmax and sums: the warps that a row's thread is in
    static constexpr int kMmaWarp = kRowWarps + kDequantWarps, kThreads = (kMmaWarp + 4) * 32;
    // registers per thread: of the launch, then of each role (their sum is within the launch's)
    static constexpr int kLaunchRegs = 96;
    static constexpr int kSoftRegs = PARTS == 1 ? 136 : 128, kSumRegs = PARTS == 1 ? 136 : 168;
    static constexpr int kDequantRegs = PARTS == 1 ? 80 : 72, kOtherRegs = 40;
    static_assert(4 * (kSoftRegs + kSumRegs) + kDequantWarps * kDequantRegs + 4 * kOtherRegs <= (kMmaWarp + 4) * kLaunchRegs, "registers");
    static_assert(kThreads * kLaunchRegs <= 65536, "registers of the SM");
    // tensor memory, columns: PARTS = 1: per tile S [2][64] (P in the first 32 columns
    // of its S) and O [128]; PARTS = 2: S [2][64], P [2][64] (hi, lo), O [2][128]
    static constexpr int kTileCols = 256;
    static constexpr int kColP = PARTS == 1 ? 0 : 128, kColO = PARTS == 1 ? 128 : 256;
    static constexpr int kCols = 512;
};

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// How far a row's logits may pass the subtracted maximum before its sums are
// rescaled (log2): P stays at 2^15 at most, and the weights of a page whose
// maximum is the one subtracted are fp16 normals down to 2^-14 of the largest,
// 2^-25 off at most below.  A warp rescales when one of its 32 rows asks for it, so
// with 8 every second page of logits of deviation 5 did, at 2000 cycles each.
constexpr float kSlack = 15.f;
// PARTS = 2 has no slack: what is subtracted lies this much below the maximum, so that P takes
// up to the same 2^15 and the two parts of a weight end 2^-40 below the largest.  (With
// a P of 1 at most, weights below 2^-25 of it were 0 in the products and counted in their sum: one
// token in front of 32K others lost the output up to 7e-4 of the largest value, now less than 3e-5.)
constexpr float kLift2 = 15.f;

// An item's record, its page-table row and the number of its pages that can be read.
struct Work {
    SharedItem it;
    const int32_t* table;
    int n;
};
__device__ __forceinline__ Work find_item(const DecodeParamsX& p, int item) {
    Work r;
    const int4 x = __ldg(reinterpret_cast<const int4*>(p.items + item)), y = __ldg(reinterpret_cast<const int4*>(p.items + item) + 1);
    r.it.seq = x.x; r.it.kv = x.y; r.it.pg0 = x.z; r.it.pages = x.w;
    r.it.rows = y.x; r.it.row0 = y.y; r.it.qtile = y.z; r.it.part0 = y.w;
    r.table = p.page_table + (size_t)r.it.seq * p.max_pages + r.it.pg0;
    r.n = 0;
    const int lane = threadIdx.x & 31;
    for (int q0 = 0; q0 < r.it.pages; q0 += 128) {
        int id[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = q0 + 32 * i + lane < r.it.pages ? __ldg(r.table + q0 + 32 * i + lane) : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.n += __popc(__ballot_sync(kFull, id[i] >= 0 && id[i] < p.num_pages));
    }
    return r;
}

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
    uint64_t* pv_done = p_full + 2 * T; // [T][2]
    uint64_t* a_full = pv_done + 2 * T; // [2] PARTS = 2: a page's factors
    uint64_t* o_free = a_full + 2;      // [2] PARTS = 2: its products and factors have been taken
    uint64_t* q_full = o_free + 2;
    uint64_t* drain = q_full + 1;      // [2] the two warps of the products
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drain + 2);
    volatile int* dead = reinterpret_cast<volatile int*>(tmem_at + 1);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);  // (uniform for the compiler)
    // The plan was complete before prep_kernel let this grid start; what prep_kernel makes,
    // q' and its scales, is waited for by the warps that read it.
    const int total = __ldg(p.counter + kSharedItems);
    if ((int)blockIdx.x >= total) {  // (this grid is not complete before prep_kernel is)
        if (threadIdx.x == 0) pdl_wait();
        return;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < NR; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], kDequantWarps);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&k_full[i], kDequantWarps);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], kDequantWarps);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2 * T; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&a_full[i], 4);
            mbar_init(&o_free[i], 4);
        }
        mbar_init(q_full, 1);
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        fence_mbar_init();
        *dead = 0;
    }
    if (warp == 0) tmem_alloc(tmem_at, SM::kCols);
    tc_before();
    block_sync();
    tc_after();
    const uint32_t tmem = *tmem_at;
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // by a whole warp
        if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
        if (__all_sync(kFull, mbar_wait_bounded(bar, parity, kWaitPolls))) return true;
        if (lane == 0) {
            report(p.status, OSCAR_STATUS_TIMEOUT);
            *dead = 1;
        }
        return false;
    };
    // The products of values of page g of tile t are done.  (A parity tells two
    // neighbouring phases of a barrier apart and no more: with a barrier for each of the
    // two buffers, the next phase of one needs the waiting warp itself.)
    auto wait_values = [&](int t, uint32_t g) { return wait(&pv_done[2 * t + (g & 1u)], (g >> 1) & 1u); };
    float* alphaS = reinterpret_cast<float*>(smem + SM::kAlpha);
    // The o' of a warp's 32 rows of tile t into their partials, by value(c, v): positions c .. c + 31
    // of the lane's row.  They go through the warp's quarter of the q' tile (no product reads that
    // any more), so that a store of the warp covers whole lines: 16 bytes of each of 32 rows
    // a store cost eight times the cycles.  Chunk c of row r lies at chunk c ^ (r & 15).
    const int gsh = 31 - __clz(p.G);  // G is a power of two
    auto store_rows = [&](const SharedItem& it, int t, auto value) {
        uint8_t* stage = smem + SM::kQ + t * PARTS * SM::kQTile + (warp & 3) * (SM::kQTile / 4);
        float* parts = p.sh_part + (size_t)it.part0 * p.part_stride;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 64 positions at a time
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                uint32_t v[32];
                value(64 * h + c, v);
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<uint4*>(stage + lane * 256 + ((((c + i) >> 2) ^ (lane & 15)) << 4)) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            __syncwarp();
            const int first = t * 128 + (warp & 3) * 32, c = lane & 15;
#pragma unroll 4
            for (int i = lane >> 4; i < 32; i += 2) {
                if (first + i >= it.rows) break;
                const int rw = it.row0 + first + i;
                const uint4 x = *reinterpret_cast<const uint4*>(stage + i * 256 + ((c ^ (i & 15)) << 4));
                *reinterpret_cast<uint4*>(parts + (size_t)(rw >> gsh) * p.part_stride + (rw & (p.G - 1)) * kD + 64 * h + 4 * c) = x;
            }
            __syncwarp();
        }
    };
    // Every role walks the block's items by itself; a barrier of the block ends an
    // item (with a timeout: the last one).
    bool ok = true;
    uint32_t items = 0;  // of this block so far
    uint32_t done = 0;   // pages of earlier items: the rings of the pages, and tile 0
    uint32_t done1 = 0;  // the same of tile 1, which an item may lack

    if (warp < SM::kSoftWarps) {
        // -------------------------------- softmax --------------------------------
        regs_up<SM::kSoftRegs>();
        pdl_wait();
        pdl_trigger();
        const int t = warp >> 2;
        for (int item = blockIdx.x; item < total; item += gridDim.x, ++items) {
            const Work wk = find_item(p, item);
            const SharedItem& it = wk.it;
            const int tiles = T == 2 && it.rows > 128 ? 2 : 1, n = wk.n;
            if (t < tiles) {
                const int r = t * 128 + (warp & 3) * 32 + lane, row = it.row0 + r;
                const bool row_on = r < it.rows;
                const float kq = row_on ? __ldg(p.qtile_kinv + (size_t)it.qtile * 128 + r) : 0.f;  // 2^-e of the row of q'
                const uint32_t lanes = tmem + t * SM::kTileCols + ((uint32_t)((warp & 3) * 32) << 16);
                float m_run = -INFINITY, l0 = 0.f, l1 = 0.f;
                const uint32_t g0 = t == 1 ? done1 : done;
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
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        mx4[i & 3] = fmaxf(mx4[i & 3], fmaxf(__uint_as_float(s[0][i]), __uint_as_float(s[1][i])));
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * kq - (PARTS == 2 ? kLift2 : 0.f);
                    float alpha = 1.f;
                    const bool any = __any_sync(kFull, PARTS == 2 ? mx > m_run : mx > m_run + kSlack);
                    if (any) {
                        const float m_new = fmaxf(m_run, mx);
                        alpha = m_new > m_run ? ex2(m_run - m_new) : 1.f;
                        m_run = m_new;
                        l0 *= alpha;
                        l1 *= alpha;
                    }
                    if constexpr (PARTS == 2) {
                        if (g >= 2 && !(ok = wait(&o_free[buf], ((g >> 1) - 1) & 1u))) break;
                        alphaS[buf * 128 + (warp & 3) * 32 + lane] = alpha;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&a_full[buf]);
                    }
                    const float off = finite_max(m_run);
                    const float2 kk = make_float2(kq, kq), oo = make_float2(-off, -off);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const uint32_t pa = PARTS == 1 ? sa : lanes + SM::kColP + buf * 64;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t ph[16], pl[PARTS == 2 ? 16 : 1];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            // tokens i .. i + 3; stored (0, 2), (1, 3)
                            const float2 x = fma2(make_float2(__uint_as_float(s[h][i]), __uint_as_float(s[h][i + 2])), kk, oo);
                            const float2 y = fma2(make_float2(__uint_as_float(s[h][i + 1]), __uint_as_float(s[h][i + 3])), kk, oo);
                            const float2 e0 = make_float2(ex2(x.x), ex2(x.y)), e1 = make_float2(ex2(y.x), ex2(y.y));
                            sum[(i >> 2) & 1] = add2(sum[(i >> 2) & 1], add2(e0, e1));
                            ph[i / 2] = pack_f16x2_rn(e0.x, e0.y);
                            ph[i / 2 + 1] = pack_f16x2_rn(e1.x, e1.y);
                            if constexpr (PARTS == 2) {
                                pl[i / 2] = pack_f16x2_rn(e0.x - half_lo(ph[i / 2]), e0.y - half_hi(ph[i / 2]));
                                pl[i / 2 + 1] = pack_f16x2_rn(e1.x - half_lo(ph[i / 2 + 1]), e1.y - half_hi(ph[i / 2 + 1]));
                            }
                        }
                        tmem_st16(pa + 16 * h, ph);
                        if constexpr (PARTS == 2) tmem_st16(pa + 32 + 16 * h, pl);
                    }
                    l0 += sum[0].x + sum[1].x;
                    l1 += sum[0].y + sum[1].y;
                    if constexpr (PARTS == 1) {
                        if (any && j > 0) {  // rescale O, once the products of the page before are in it
                            if (!(ok = wait_values(t, g - 1))) break;
                            tc_after();
#pragma unroll 1
                            for (int c = 0; c < kD; c += 32) {
                                uint32_t v[32];
                                tmem_ld32(v, lanes + SM::kColO + c);
                                tmem_wait_ld(v);
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                                tmem_st32(lanes + SM::kColO + c, v);
                            }
                        }
                    }
                    tmem_wait_st();
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * t + buf]);
                }
                // ---- the row's partial
                if constexpr (PARTS == 1) {
                    if (ok && n > 0) {
                        ok = wait_values(t, g0 + n - 1);
                        tc_after();
                    } else if (ok) {
                        ok = wait(q_full, items & 1u);  // (nothing else says that q' has landed, whose place is written below)
                    }
                    if (ok)
                        store_rows(it, t, [&](int c, uint32_t (&v)[32]) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = 0u;
                            if (n > 0) {
                                tmem_ld32(v, lanes + SM::kColO + c);
                                tmem_wait_ld(v);
                            }
                        });
                }
                if (ok && row_on) {
                    const float l = l0 + l1;
                    float* part = p.sh_part + ((size_t)it.part0 + (row >> gsh)) * p.part_stride;
                    const int head = row & (p.G - 1);
                    part[p.G * kD + head] = l == 0.f ? -INFINITY : finite_max(m_run);
                    part[p.G * kD + p.G + head] = l;
                }
                tc_before();
                fence_async();  // (the next item's q' is copied over the staged rows)
            }
            block_sync();
            if (*dead) break;
            done += n;
            if (tiles == 2) done1 += n;
        }
    } else if (warp < SM::kRowWarps) {
        // ------------------- sums of the products of values (PARTS = 2) ------------------
        // (Registers for the softmax's 64 logits and these 128 sums were 3300 cycles of one
        // warp per page.)
        if constexpr (PARTS == 2) {
            regs_up<SM::kSumRegs>();
            pdl_wait();
            for (int item = blockIdx.x; item < total; item += gridDim.x, ++items) {
                const Work wk = find_item(p, item);
                const int n = wk.n;
                const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
                float o[kD];
#pragma unroll
                for (int d = 0; d < kD; ++d) o[d] = 0.f;
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t g = done + j, buf = g & 1u;
                    if (!(ok = wait(&a_full[buf], (g >> 1) & 1u) && wait_values(0, g))) break;
                    tc_after();
                    const float alpha = alphaS[buf * 128 + (warp & 3) * 32 + lane];
                    const float2 aa = make_float2(alpha, alpha);
#pragma unroll
                    for (int c = 0; c < kD; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(v, lanes + SM::kColO + buf * kD + c);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 x = fma2(make_float2(o[c + i], o[c + i + 1]), aa, make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                            o[c + i] = x.x;
                            o[c + i + 1] = x.y;
                        }
                    }
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_free[buf]);
                }
                if (ok && n == 0) ok = wait(q_full, items & 1u);
                if (ok)
                    store_rows(wk.it, 0, [&](int c, uint32_t (&v)[32]) {
#pragma unroll
                        for (int d = 0; d < kD; d += 32)
                            if (d == c)
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(o[d + i]);
                    });
                fence_async();  // (as above)
                block_sync();
                if (*dead) break;
                done += n;
            }
        }
    } else if (warp < SM::kMmaWarp) {
        // ----------------------------- dequantisation -----------------------------
        regs_down<SM::kDequantRegs>();
        const int dw = warp - SM::kRowWarps;
        const int ng = 4 >> p.gshift;
        // K: a lane's token and 16-byte code chunk (lanes of a wavefront on distinct banks)
        const int ka = lane & 3, kt = 8 * dw + ((((lane >> 2) & 1) << 2) | (lane >> 3));
        // V: tokens 16 tc .. + 15; 4 bits: plane 8 dw + lane / 4, positions 2 plane, + 1, of group dw / 2;
        // 2 bits: plane 4 dw + lane / 4 % 4, positions 32 i + plane of slots i = i0, i0 + 1
        const int tc = lane & 3;
        const int plane = BITS == 4 ? 8 * dw + (lane >> 2) : 4 * dw + ((lane >> 2) & 3);
        const int i0 = BITS == 4 ? 0 : 2 * (lane >> 4);
        uint16_t* pairS = reinterpret_cast<uint16_t*>(smem + SM::kPairs + dw * SM::kPairBytes);  // [group][s, z][64]
        for (int item = blockIdx.x; item < total; item += gridDim.x) {
            const int n = find_item(p, item).n;
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t g = done + j, st = g % NS, rs = g % NR;
                if (!(ok = wait(&raw_full[rs], (g / NR) & 1u))) break;
                const uint8_t* blk = smem + SM::kRawAt + rs * SM::kRaw;
                if (g >= NS && !(ok = wait(&k_empty[st], ((g / NS) - 1) & 1u))) break;
                {
                    uint8_t* row = smem + SM::kK + st * PARTS * SM::kOperand + kt * 128;
                    uint32_t w[4], sz[4];
                    if constexpr (BITS == 4) {
                        const uint4 x = *reinterpret_cast<const uint4*>(blk + kt * 64 + 16 * ka);
                        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(blk + kt * 32 + 8 * ka);
                        w[0] = x.x; w[1] = x.y; w[2] = x.x >> 8; w[3] = x.y >> 8;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sz[k] = *reinterpret_cast<const uint32_t*>(blk + (BITS == 4 ? kCodes4 : kKScale) + (kt * ng + (k >> p.gshift)) * 4);
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
                        uint8_t* to = row + (k >> 1) * (kPage * 128) + (((4 * (k & 1) + ka) ^ (kt & 7)) << 4);
                        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        if constexpr (PARTS == 2) *reinterpret_cast<uint4*>(to + SM::kOperand) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    };
                    chunk(std::integral_constant<int, 0>{});
                    chunk(std::integral_constant<int, 1>{});
                    chunk(std::integral_constant<int, 2>{});
                    chunk(std::integral_constant<int, 3>{});
                }
                // V: its pairs go by group and in the tokens' order of the products
                const uint8_t* vh = blk + (BITS == 4 ? half_bytes4(p.gshift) : kVCodes);
                const uint8_t* vp = blk + (BITS == 4 ? half_bytes4(p.gshift) + kCodes4 : v_scale_off(p.gshift));
                uint4 x = *reinterpret_cast<const uint4*>(vh + plane * kPage + 16 * tc);
                if constexpr (BITS == 2) {
                    x.x >>= 2 * i0; x.y >>= 2 * i0; x.z >>= 2 * i0; x.w >>= 2 * i0;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = lane + 32 * u, at = (t & ~3) | pv_slot(t & 3);
                    for (int gr = 0; gr < (BITS == 4 ? 1 : ng); ++gr) {
                        const uint32_t y = *reinterpret_cast<const uint32_t*>(vp + (t * ng + (BITS == 4 ? (dw >> 1) >> p.gshift : gr)) * 4);
                        pairS[gr * 2 * kPage + at] = (uint16_t)y;
                        pairS[gr * 2 * kPage + kPage + at] = (uint16_t)(y >> 16);
                    }
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_full[st]);
                if (g >= NS && !(ok = wait(&v_empty[st], ((g / NS) - 1) & 1u))) break;
                uint8_t* vS = smem + SM::kV + st * PARTS * SM::kOperand;
                // one row (stored position pos) of 16 tokens from the codes at bits P of the plane words x
                auto v_row = [&](auto pp, int pos, const uint32_t (&s)[8], const uint32_t (&z)[8]) {
                    constexpr int P = decltype(pp)::value;
                    constexpr uint32_t field = BITS == 4 ? 0x000f000fu : 0x00030003u;
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint8_t* row = vS + pos * 128;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            value_pair<PARTS>(s[4 * h + 2 * i], code_at<P>(w[2 * h + i], field), z[4 * h + 2 * i], hi[2 * i], lo[2 * i]);
                            value_pair<PARTS>(s[4 * h + 2 * i + 1], code_at<P>(w[2 * h + i] >> 8, field), z[4 * h + 2 * i + 1], hi[2 * i + 1], lo[2 * i + 1]);
                        }
                        uint8_t* to = row + (((2 * tc + h) ^ (pos & 7)) << 4);
                        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        if constexpr (PARTS == 2) *reinterpret_cast<uint4*>(to + SM::kOperand) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                };
                auto pairs_of = [&](const uint16_t* at, uint32_t (&s)[8], uint32_t (&z)[8]) {
                    const uint4* sp = reinterpret_cast<const uint4*>(at + 16 * tc);
                    const uint4* zp = reinterpret_cast<const uint4*>(at + kPage + 16 * tc);
                    const uint4 s0 = sp[0], s1 = sp[1], z0 = zp[0], z1 = zp[1];
                    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
                    z[0] = z0.x; z[1] = z0.y; z[2] = z0.z; z[3] = z0.w; z[4] = z1.x; z[5] = z1.y; z[6] = z1.z; z[7] = z1.w;
                };
                uint32_t s[8], z[8];
                if constexpr (BITS == 4) {
                    pairs_of(pairS, s, z);
                    v_row(std::integral_constant<int, 0>{}, 2 * plane, s, z);
                    v_row(std::integral_constant<int, 4>{}, 2 * plane + 1, s, z);
                } else {
                    auto slot = [&](auto ii) {  // (x is shifted down by the half warp's first slot)
                        constexpr int i = decltype(ii)::value;
                        pairs_of(pairS + ((i + i0) >> p.gshift) * 2 * kPage, s, z);
                        v_row(std::integral_constant<int, 2 * i>{}, 32 * (i + i0) + plane, s, z);
                    };
                    slot(std::integral_constant<int, 0>{});
                    slot(std::integral_constant<int, 1>{});
                }
                fence_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&v_full[st]);
                    mbar_arrive(&raw_empty[rs]);
                }
            }
            block_sync();
            if (*dead) break;
            done += n;
        }
    } else {
        regs_down<SM::kOtherRegs>();  // (the warps of a warpgroup take the same instruction)
        const uint32_t on = elect_lane();
        if (warp == SM::kMmaWarp) {
            // --------------------------- products of logits ---------------------------
            // (The two kinds of products have a warp each: with one for both, its six waits
            // and 24 issues per page, one after the other, were the kernel's critical path.)
            const uint64_t qd = tc_desc(smem_u32(smem + SM::kQ)), kd = tc_desc(smem_u32(smem + SM::kK));
            for (int item = blockIdx.x; item < total; item += gridDim.x, ++items) {
                const Work wk = find_item(p, item);
                const int tiles = T == 2 && wk.it.rows > 128 ? 2 : 1, n = wk.n;
                bool issued = false;
                ok = wait(q_full, items & 1u);
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t g = done + j, st = g % NS;
                    if (!(ok = wait(&k_full[st], (g / NS) & 1u))) break;
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        if (t >= tiles || !ok) break;
                        const uint32_t gt = (t == 1 ? done1 : done) + j, buf = gt & 1u;
                        // S takes the place of the S, and P, of two pages before, whose products of values are to be done
                        if (gt >= 2 && !(ok = wait_values(t, gt - 2))) break;
                        tc_after();
                        const uint32_t s = tmem + t * SM::kTileCols + buf * 64;
#pragma unroll
                        for (int pr = 0; pr < (PARTS == 1 ? 1 : 3); ++pr)  // hi hi, lo hi, hi lo
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                tc_mma_ss(on, s, qd + (((t * PARTS + (pr == 1)) * SM::kQTile + (k >> 2) * (128 * 128) + 32 * (k & 3)) >> 4),
                                          kd + (((st * PARTS + (pr == 2)) * SM::kOperand + (k >> 2) * (kPage * 128) + 32 * (k & 3)) >> 4), tc_idesc(kPage),
                                          pr > 0 || k > 0);
                        tc_commit(on, &s_full[2 * t + buf]);
                        issued = true;
                    }
                    if (ok) tc_commit(on, &k_empty[st]);
                }
                if (!ok && issued) {  // whatever was issued ends before the block does
                    tc_commit(on, &drain[0]);
                    (void)mbar_wait_bounded(&drain[0], 0, kWaitPolls);
                }
                block_sync();
                if (*dead) break;
                done += n;
                if (tiles == 2) done1 += n;
            }
        } else if (warp == SM::kMmaWarp + 1) {
            // --------------------------- products of values ---------------------------
            const uint64_t vd = tc_desc(smem_u32(smem + SM::kV));
            for (int item = blockIdx.x; item < total; item += gridDim.x) {
                const Work wk = find_item(p, item);
                const int tiles = T == 2 && wk.it.rows > 128 ? 2 : 1, n = wk.n;
                bool issued = false;
                for (int j = 0; j < n && ok; ++j) {  // O (+)= P V
                    const uint32_t g = done + j, st = g % NS;
                    if (!(ok = wait(&v_full[st], (g / NS) & 1u))) break;
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        if (t >= tiles || !ok) break;
                        const uint32_t gt = (t == 1 ? done1 : done) + j, buf = gt & 1u;
                        if (!(ok = wait(&p_full[2 * t + buf], (gt >> 1) & 1u))) break;
                        if (PARTS == 2 && gt >= 2 && !(ok = wait(&o_free[buf], ((gt >> 1) - 1) & 1u))) break;
                        tc_after();
                        const uint32_t tt = tmem + t * SM::kTileCols;
                        const uint32_t pa = tt + SM::kColP + buf * 64, o = tt + SM::kColO + (PARTS == 2 ? buf * kD : 0);
#pragma unroll
                        for (int pr = 0; pr < (PARTS == 1 ? 1 : 3); ++pr)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc_mma_ts(on, o, pa + (pr == 1 ? 32 : 0) + 8 * k, vd + (((st * PARTS + (pr == 2)) * SM::kOperand + 32 * k) >> 4), tc_idesc(kD),
                                          (PARTS == 1 && j > 0) || pr > 0 || k > 0);
                        tc_commit(on, &pv_done[2 * t + buf]);
                        issued = true;
                    }
                    if (ok) tc_commit(on, &v_empty[st]);
                }
                if (!ok && issued) {
                    tc_commit(on, &drain[1]);
                    (void)mbar_wait_bounded(&drain[1], 0, kWaitPolls);
                }
                block_sync();
                if (*dead) break;
                done += n;
                if (tiles == 2) done1 += n;
            }
        } else {
            // --------------------------- copies: pages, and q' ------------------------
            if (warp == SM::kMmaWarp + 3) pdl_wait();
            for (int item = blockIdx.x; item < total; item += gridDim.x, ++items) {
                const Work wk = find_item(p, item);
                const SharedItem& it = wk.it;
                if (warp == SM::kMmaWarp + 2) {
                    int j = 0;  // pages issued
                    for (int q0 = 0; q0 < it.pages && ok; q0 += 32) {
                        const int id = q0 + lane < it.pages ? __ldg(wk.table + q0 + lane) : -1;
                        const bool good = id >= 0 && id < p.num_pages;
                        if (q0 + lane < it.pages && !good) report(p.status, OSCAR_STATUS_BAD_PAGE);
                        for (unsigned left = __ballot_sync(kFull, good); left && ok; left &= left - 1) {
                            const int page = __shfl_sync(kFull, id, __ffs(left) - 1);
                            const uint32_t g = done + j, rs = g % NR;
                            if (g >= NR && !(ok = wait(&raw_empty[rs], ((g / NR) - 1) & 1u))) break;
                            if (lane == 0) {
                                mbar_arrive_expect_tx(&raw_full[rs], p.block_bytes);
                                bulk_g2s(smem + SM::kRawAt + rs * SM::kRaw, p.pool + ((size_t)page * p.hk + it.kv) * p.block_bytes, p.block_bytes, &raw_full[rs]);
                            }
                            __syncwarp();
                            ++j;
                        }
                    }
                    if (!ok)  // copies in flight land before the block ends
                        for (uint32_t g = done + j > NR ? done + j - NR : 0; g < done + j; ++g)
                            (void)mbar_wait_bounded(&raw_full[g % NR], (g / NR) & 1u, kWaitPolls);
                } else {
                    // (rows behind the last one hold whatever the workspace does: no other row sees them)
                    const int tiles = T == 2 && it.rows > 128 ? 2 : 1;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(q_full, tiles * PARTS * kQTileBytes);
                        for (int t = 0; t < tiles; ++t)
                            bulk_g2s(smem + SM::kQ + t * PARTS * SM::kQTile, p.qtile + (size_t)(it.qtile + t) * 2 * kQTileBytes, PARTS * kQTileBytes, q_full);
                    }
                    __syncwarp();
                    ok = wait(q_full, items & 1u) && ok;  // (lands before the block ends, whoever else reads it)
                }
                block_sync();
                if (*dead) break;
                done += wk.n;
            }
        }
    }
    tc_before();
    block_sync();
    if (warp == 0) tmem_free(tmem, SM::kCols);
}

template <int BITS, int PARTS>
cudaError_t launch_parts(const DecodeParamsX& p, cudaStream_t st, int dev) {
    using SM = SharedSmem<BITS, PARTS>;
    static bool set[64];
    if (!set[dev & 63]) {
        // setmaxnreg moves registers between the roles and waits for ever where they are not there: the
        // shares were added up for a launch with kLaunchRegs
        cudaFuncAttributes a;
        cudaError_t e = cudaFuncGetAttributes(&a, shared_kernel<BITS, PARTS>);
        if (e == cudaSuccess && a.numRegs != SM::kLaunchRegs) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess) e = set_smem(shared_kernel<BITS, PARTS>, SM::kAlloc);
        if (e != cudaSuccess) return e;
        set[dev & 63] = true;
    }
    return launch_pdl(shared_kernel<BITS, PARTS>, dim3(p.shared_blocks), dim3(SM::kThreads), SM::kAlloc, st, p);
}

}  // namespace

cudaError_t launch_shared_plan(const DecodeParamsX& p, cudaStream_t st, int dev) {
    static bool set[64];
    if (!set[dev & 63]) {
        const cudaError_t e = set_smem(group_kernel, 6 * kMaxSharedGroups * 4, false);
        if (e != cudaSuccess) return e;
        set[dev & 63] = true;
    }
    return launch_pdl(group_kernel, dim3(1), dim3(kPlanThreads), (size_t)6 * p.n_groups * 4, st, p, p.out_bf16 ? 256 : 128);
}

cudaError_t launch_shared(const DecodeParamsX& p, int bits, cudaStream_t st, int dev) {
    if (bits == 4) return p.out_bf16 ? launch_parts<4, 1>(p, st, dev) : launch_parts<4, 2>(p, st, dev);
    return p.out_bf16 ? launch_parts<2, 1>(p, st, dev) : launch_parts<2, 2>(p, st, dev);
}

}  // namespace oscar
