// select.cu -- the history tokens that stay under a budget, by their scores:
// oscar_history_select.
//
// Of n tokens m = min(n, budget) stay: the newest min(protect, m), and the
// r = m - that many greatest scores of the others, ties to the lower position.
// The r-th greatest score is found digit by digit from the top (a radix select
// over 11 + 11 + 10 bits of the scores' order-preserving patterns, with
// histograms in shared memory); then every warp knows from prefix sums where its
// kept tokens go in the ascending list.  One pass over memory: the scores stay
// in shared memory.
//
// A cluster of thread blocks serves a sequence, each a contiguous part of it;
// they add their histograms through distributed shared memory.
#include <algorithm>
#include <cooperative_groups.h>

#include "oscar_common.cuh"

namespace cg = cooperative_groups;

namespace oscar {

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kPasses = 3;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 32768;  // scores that a block keeps in shared memory; longer parts are read again

// Scores in order as unsigned integers: -0 as 0, NaN above all.
__device__ __forceinline__ uint32_t score_key(float w) {
    const uint32_t b = __float_as_uint(w + 0.f);
    if (w != w) return 0xffffffffu;
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ int pass_shift(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__device__ __forceinline__ uint32_t pass_mask(int pass) { return pass == 2 ? 0x3ffu : 0x7ffu; }

struct SelShared {
    int hist[kPasses][kBins];
    int warp_sum[kSelWarps];
    int2 warp_count[kSelWarps];  // (greater than the threshold, equal to it)
    int2 count;                  // of the block, read by the others of the cluster
    int bin, above;
};

__global__ void __launch_bounds__(kSelThreads) select_kernel(HistorySelectParams p, int cached) {
    extern __shared__ __align__(16) float cacheS[];
    __shared__ SelShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int nblk = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / nblk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    int n = __ldg(p.hist_len + b), m = __ldg(p.budget + b);
    if (rank == 0 && threadIdx.x == 0 && (n < 0 || n > p.stride || m < 0)) report(p.status, OSCAR_STATUS_BAD_POS);
    n = min(max(n, 0), p.stride);
    m = min(max(m, 0), n);
    const int room = p.kept_weight ? min(p.keep_stride, p.kept_stride) : p.keep_stride;
    if (m > room) {
        if (rank == 0 && threadIdx.x == 0) report(p.status, OSCAR_STATUS_BAD_POS);
        m = room;
    }
    const int newest = min(p.protect, m), cand = n - newest;  // positions [cand, n) are protected
    int need = m - newest;                                    // of the cand others
    const float* w = p.weight + (size_t)b * p.stride;
    int32_t* keep = p.keep + (size_t)b * p.keep_stride;
    float* kept = p.kept_weight ? p.kept_weight + (size_t)b * p.kept_stride : nullptr;

    // this block's part: warps' contiguous runs of `run` tokens (a multiple of 32)
    const int run = ((cand + nblk * kSelWarps - 1) / (nblk * kSelWarps) + 31) & ~31;
    const int part0 = rank * kSelWarps * run;
    const int mine0 = warp * run;                             // offset of the warp's run in the part
    const bool choose = need > 0 && need < cand;              // (the same in every block of the cluster)
    const bool in_cache = choose && run * kSelWarps <= cached;
    auto score = [&](int off) {                               // score of token part0 + off < cand
        return in_cache ? cacheS[off] : __ldg(w + part0 + off);
    };
    uint32_t prefix = 0, known = 0;                           // the threshold's digits so far, and which bits they are
    if (choose) {
        for (int i = threadIdx.x; i < kPasses * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
        if (in_cache) {
#pragma unroll 8
            for (int off = threadIdx.x; off < run * kSelWarps; off += kSelThreads)
                cacheS[off] = part0 + off < cand ? __ldg(w + part0 + off) : 0.f;
        }
        for (int pass = 0; pass < kPasses; ++pass) {
            __syncthreads();
            const int shift = pass_shift(pass);
            const uint32_t mask = pass_mask(pass);
            for (int off = threadIdx.x; off < run * kSelWarps && part0 + off < cand; off += kSelThreads) {
                const uint32_t k = score_key(score(off));
                if ((k & known) == prefix) atomicAdd(&sh.hist[pass][(k >> shift) & mask], 1);
            }
            cluster.sync();
            // thread t: bins 2 (1023 - t) + 1 and 2 (1023 - t), from the top, over all blocks
            const int top = kBins - 2 - 2 * threadIdx.x;
            int c0 = 0, c1 = 0;
            for (int r = 0; r < nblk; ++r) {
                const int2 v = *reinterpret_cast<const int2*>(cluster.map_shared_rank(&sh.hist[pass][top], r));
                c0 += v.x;
                c1 += v.y;
            }
            int sum = c0 + c1;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(kFull, sum, d);
                if (lane >= d) sum += v;
            }
            if (lane == 31) sh.warp_sum[warp] = sum;
            __syncthreads();
            int before = lane < warp ? sh.warp_sum[lane] : 0;
            before = __reduce_add_sync(kFull, before);
            const int above = before + sum - c0 - c1;         // scores above this thread's bins
            if (above < need && above + c1 >= need) {
                sh.bin = top + 1;
                sh.above = above;
            } else if (above + c1 < need && above + c1 + c0 >= need) {
                sh.bin = top;
                sh.above = above + c1;
            }
            __syncthreads();
            prefix |= (uint32_t)sh.bin << shift;
            known |= mask << shift;
            need -= sh.above;
        }
    }
    // threshold `prefix`: every greater score stays, and the first `need` equal ones;
    // without a choice all or none do
    const bool all = need > 0 && !choose;
    int gt = 0, eq = 0;
    for (int off = mine0 + lane; off < mine0 + run; off += 32) {
        if (part0 + off >= cand) break;
        if (all) {
            ++gt;
        } else if (choose) {
            const uint32_t k = score_key(score(off));
            gt += k > prefix;
            eq += k == prefix;
        }
    }
    gt = __reduce_add_sync(kFull, gt);
    eq = __reduce_add_sync(kFull, eq);
    if (lane == 0) sh.warp_count[warp] = make_int2(gt, eq);
    __syncthreads();
    int gt0, eq0;  // before this warp, in the block; then in the sequence
    {
        const int2 c = sh.warp_count[lane];
        gt0 = __reduce_add_sync(kFull, lane < warp ? c.x : 0);
        eq0 = __reduce_add_sync(kFull, lane < warp ? c.y : 0);
        if (warp == 0) {
            const int g = __reduce_add_sync(kFull, c.x), e = __reduce_add_sync(kFull, c.y);
            if (lane == 0) sh.count = make_int2(g, e);
        }
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
        const int2 c = *cluster.map_shared_rank(&sh.count, r);
        gt0 += c.x;
        eq0 += c.y;
    }
    cluster.sync();  // no block leaves while another reads its shared memory
    const uint32_t below = (1u << lane) - 1u;
    if (all || choose) {
        for (int off = mine0 + lane; off - lane < mine0 + run && part0 + off - lane < cand; off += 32) {
            const bool in = part0 + off < cand;
            const float x = in ? score(off) : 0.f;
            const uint32_t k = score_key(x);
            const bool g = in && (all || k > prefix), e = in && !all && k == prefix;
            const uint32_t gm = __ballot_sync(kFull, g), em = __ballot_sync(kFull, e);
            const int eq_before = eq0 + __popc(em & below);
            if (g || (e && eq_before < need)) {
                const int to = gt0 + __popc(gm & below) + min(eq_before, need);
                keep[to] = part0 + off;
                if (kept) kept[to] = x;
            }
            gt0 += __popc(gm);
            eq0 += __popc(em);
        }
    }
    for (int i = rank * kSelThreads + threadIdx.x; i < newest; i += nblk * kSelThreads) {
        keep[m - newest + i] = cand + i;
        if (kept) kept[m - newest + i] = w[cand + i];
    }
    if (rank == 0 && threadIdx.x == 0) p.n_keep[b] = m;
}

}  // namespace

cudaError_t launch_history_select(const HistorySelectParams& p, cudaStream_t st) {
    static bool attr_set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!attr_set[dev & 63]) {
        e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
        if (e != cudaSuccess) return e;
        attr_set[dev & 63] = true;
    }
    // Blocks per sequence: one for every 4096 tokens, as far as the blocks of the
    // batch still run side by side (two per SM).
    int blocks = 1;
    while (blocks < kMaxCluster && p.stride > 4096 * blocks && (int64_t)p.batch * blocks * 2 <= 304) blocks *= 2;
    while (blocks < kMaxCluster && p.stride > kMaxCached * blocks) blocks *= 2;
    const int per_block = ((p.stride + blocks * kSelWarps - 1) / (blocks * kSelWarps) + 31) / 32 * 32 * kSelWarps;
    const int cached = std::min(per_block, kMaxCached);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.batch * blocks));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)cached * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, select_kernel, p, cached);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace oscar
