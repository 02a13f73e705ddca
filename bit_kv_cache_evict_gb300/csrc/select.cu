// select.cu -- the history tokens that stay under a budget, by their scores:
// oscar_history_select.
//
// Of n tokens m = min(n, budget) stay: the newest min(protect, m), and the
// r = m - that many greatest scores of the others, ties to the lower position.
// The r-th greatest score is found digit by digit from the top (a radix select
// over 11 + 11 + 10 bits of the scores' order-preserving patterns, with
// histograms in shared memory); then every warp knows from prefix sums where its
// kept tokens go in the ascending list.
//
// The bytes are few (4 per token read, 8 per kept token written: 2 MB, 0.3 us for
// eight histories of 32K), so the time is latency and instructions: the patterns
// are made once and stay in shared memory, four per access, and positions behind
// the last are the pattern 0, below every score's, so that no loop asks for the
// end.  A cluster of thread blocks serves a long sequence, each a contiguous part
// of it; a histogram is added up over the cluster in two steps, 64 sums that every
// block stores to every other, then 32 bins that a warp each reads (the whole of it
// read by every block took 4500 cycles a pass, these two about 1000).
#include <algorithm>
#include <cooperative_groups.h>

#include "oscar_common.cuh"

namespace cg = cooperative_groups;

namespace oscar {

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kPasses = 3;
constexpr int kMaxCluster = 16;   // 8 where the GPU has no room for clusters of 16
constexpr int kMaxCached = 32768;  // patterns that a block keeps in shared memory; longer parts are read again
constexpr int kRunStep = 128;      // a warp's run of tokens: whole steps of four per lane

// Scores in order as unsigned integers: -0 as 0, NaN above all.  No score has the pattern 0.
__device__ __forceinline__ uint32_t score_key(float w) {
    const uint32_t b = __float_as_uint(w + 0.f);
    if (w != w) return 0xffffffffu;
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float key_score(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

__device__ __forceinline__ int pass_shift(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__device__ __forceinline__ uint32_t pass_mask(int pass) { return pass == 2 ? 0x3ffu : 0x7ffu; }

static_assert(kMaxCluster <= 16, "a half warp's lanes store to the blocks");
struct SelShared {
    int hist[kPasses][kBins];
    int coarse[kPasses][kMaxCluster][kBins / 32];  // sums of 32 neighbouring bins, of every block
    int fine[kMaxCluster][32];                     // the 32 bins of one, of every block
    int2 warp_count[kSelWarps];       // (greater than the threshold, equal to it)
    int2 count;                       // of the block, read by the others of the cluster
    int bin, above;
};

// Of 32 lanes' numbers c, the highest bins first: the lane in whose bin the need-th
// greatest lies, and how many lie above it.  (Called by a whole warp.)
__device__ __forceinline__ int find_bin(int c, int need, int& above) {
    const int lane = threadIdx.x & 31;
    int sum = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kFull, sum, d);
        if (lane >= d) sum += v;
    }
    const int at = __ffs(__ballot_sync(kFull, sum >= need)) - 1;  // (there are that many)
    above = __shfl_sync(kFull, sum - c, at);
    return at;
}

// CLUSTER: several blocks per sequence; else one, with barriers and reads of its own only.
template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(HistorySelectParams p, int cached) {
    extern __shared__ __align__(16) uint32_t keyS[];
    __shared__ __align__(16) SelShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int nblk = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
    auto sync_all = [&]() {
        if constexpr (CLUSTER) cluster.sync();
        else __syncthreads();
    };
    auto of_block = [&](auto* at, int r) {
        if constexpr (CLUSTER) return cluster.map_shared_rank(at, r);
        else return at;
    };
    const int b = blockIdx.x / nblk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kPasses * kBins / 4; i += kSelThreads) reinterpret_cast<int4*>(&sh.hist[0][0])[i] = make_int4(0, 0, 0, 0);
    if constexpr (CLUSTER) cluster.barrier_arrive();  // (every block runs before another stores to it)
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

    // this block's part: warps' contiguous runs of `run` tokens
    const int run = ((cand + nblk * kSelWarps - 1) / (nblk * kSelWarps) + kRunStep - 1) / kRunStep * kRunStep;
    const int part0 = rank * kSelWarps * run, size = kSelWarps * run;
    const int mine0 = warp * run;                             // offset of the warp's run in the part
    const bool choose = need > 0 && need < cand;              // (the same in every block of the cluster)
    const bool all = need > 0 && !choose;
    const bool in_cache = choose && size <= cached;
    // patterns of tokens part0 + off .. + 3 (off a multiple of four)
    auto keys = [&](int off) {
        if (in_cache) return *reinterpret_cast<const uint4*>(keyS + off);
        uint32_t k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = part0 + off + i < cand ? score_key(__ldg(w + part0 + off + i)) : 0u;
        return make_uint4(k[0], k[1], k[2], k[3]);
    };
    if constexpr (CLUSTER) cluster.barrier_wait();
    uint32_t prefix = 0, known = 0;                           // the threshold's digits so far, and which bits they are
    if (choose) {
        if (in_cache) {
#pragma unroll 8
            for (int off = threadIdx.x; off < size; off += kSelThreads)
                keyS[off] = part0 + off < cand ? score_key(__ldg(w + part0 + off)) : 0u;
        }
        for (int pass = 0; pass < kPasses; ++pass) {
            __syncthreads();
            const int shift = pass_shift(pass);
            const uint32_t mask = pass_mask(pass);
            int* hist = sh.hist[pass];
#pragma unroll 2
            for (int off = 4 * threadIdx.x; off < size; off += 4 * kSelThreads) {
                const uint4 k = keys(off);
                if ((k.x & known) == prefix) atomicAdd(hist + ((k.x >> shift) & mask), 1);
                if ((k.y & known) == prefix) atomicAdd(hist + ((k.y >> shift) & mask), 1);
                if ((k.z & known) == prefix) atomicAdd(hist + ((k.z >> shift) & mask), 1);
                if ((k.w & known) == prefix) atomicAdd(hist + ((k.w >> shift) & mask), 1);
            }
            __syncthreads();
            {   // sums of 32 bins: a half warp each
                const int2 v = *reinterpret_cast<const int2*>(hist + 64 * warp + 2 * lane);
                int sum = v.x + v.y;
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
                if ((lane & 15) < nblk) of_block(&sh.coarse[pass][rank][2 * warp + (lane >> 4)], lane & 15)[0] = sum;
            }
            sync_all();
            // the 64 sums over all blocks, two a lane from the top; then the 32 bins of one: a
            // warp for each block's
            int above = 0, bins = 0;
            if (warp < nblk) {
                int2 c = make_int2(0, 0);
                for (int r = 0; r < nblk; ++r) {
                    const int2 v = *reinterpret_cast<const int2*>(&sh.coarse[pass][r][62 - 2 * lane]);
                    c.x += v.x;
                    c.y += v.y;
                }
                const int at = find_bin(c.x + c.y, need, above);
                const int upper = __shfl_sync(kFull, c.y, at);  // (the higher of the lane's two)
                const bool low = above + upper < need;
                if (low) above += upper;
                bins = 32 * (62 - 2 * at + (low ? 0 : 1));
                sh.fine[warp][lane] = *of_block(&sh.hist[pass][bins + 31 - lane], warp);
            }
            if (CLUSTER) __syncthreads();
            if (warp == 0) {
                int f = 0;
                for (int r = 0; r < nblk; ++r) f += sh.fine[r][lane];
                int fine;
                const int bin = bins + 31 - find_bin(f, need - above, fine);
                if (lane == 0) {
                    sh.bin = bin;
                    sh.above = above + fine;
                }
            }
            __syncthreads();
            prefix |= (uint32_t)sh.bin << shift;
            known |= mask << shift;
            need -= sh.above;
        }
    }
    // threshold `prefix`: every greater score stays, and the first `need` equal ones;
    // without a choice all or none do
    int gt = 0, eq = 0;
    if (all) {
        gt = lane == 0 ? max(0, min(run, cand - part0 - mine0)) : 0;
    } else if (choose) {
#pragma unroll 2
        for (int off = mine0 + 4 * lane; off < mine0 + run; off += kRunStep) {
            const uint4 k = keys(off);
            gt += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
            eq += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
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
        if (CLUSTER && warp == 0) {
            const int g = __reduce_add_sync(kFull, c.x), e = __reduce_add_sync(kFull, c.y);
            if (lane == 0) sh.count = make_int2(g, e);
        }
    }
    if constexpr (CLUSTER) {
        cluster.sync();
        const int2 c = lane < rank ? *cluster.map_shared_rank(&sh.count, lane) : make_int2(0, 0);
        gt0 += __reduce_add_sync(kFull, c.x);
        eq0 += __reduce_add_sync(kFull, c.y);
        cluster.barrier_arrive();  // (no block leaves while another reads its shared memory: see the end)
    }
    if (all) {
        for (int i = mine0 + lane; i < mine0 + gt; i += 32) {
            keep[part0 + i] = part0 + i;
            if (kept) kept[part0 + i] = __ldg(w + part0 + i);
        }
    } else if (choose) {
#pragma unroll 2
        for (int off0 = mine0; off0 < mine0 + run; off0 += kRunStep) {
            const int off = off0 + 4 * lane;
            const uint4 kv = keys(off);
            const uint32_t k[4] = {kv.x, kv.y, kv.z, kv.w};
            int g = 0, e = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g += k[i] > prefix;
                e += k[i] == prefix;
            }
            // both counts of the lanes below in one scan (at most 128 each)
            const int mine = g | (e << 16);
            int sum = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(kFull, sum, d);
                if (lane >= d) sum += v;
            }
            const int total = __shfl_sync(kFull, sum, 31), before = sum - mine;
            int gb = gt0 + (before & 0xffff), eb = eq0 + (before >> 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool is_g = k[i] > prefix, is_e = k[i] == prefix;
                if (is_g || (is_e && eb < need)) {
                    const int to = gb + min(eb, need);
                    keep[to] = part0 + off + i;
                    // (the pattern gives the score back, but for the sign of a zero and a NaN's bits)
                    if (kept) kept[to] = k[i] == 0x80000000u || k[i] == 0xffffffffu ? __ldg(w + part0 + off + i) : key_score(k[i]);
                }
                gb += is_g;
                eb += is_e;
            }
            gt0 += total & 0xffff;
            eq0 += total >> 16;
        }
    }
    for (int i = rank * kSelThreads + threadIdx.x; i < newest; i += nblk * kSelThreads) {
        keep[m - newest + i] = cand + i;
        if (kept) kept[m - newest + i] = w[cand + i];
    }
    if (rank == 0 && threadIdx.x == 0) p.n_keep[b] = m;
    if constexpr (CLUSTER) cluster.barrier_wait();
}

}  // namespace

cudaError_t launch_history_select(const HistorySelectParams& p, cudaStream_t st) {
    static int most_blocks[64];  // of a cluster on each device; 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    if (!most_blocks[dev & 63]) {
        e = cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        int clusters = 0;
        cfg.gridDim = dim3(kMaxCluster);
        cfg.dynamicSmemBytes = kMaxCached * 4;
        attr[0].val.clusterDim.x = kMaxCluster;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&clusters, select_kernel<true>, &cfg);
        if (e != cudaSuccess) (void)cudaGetLastError();  // (an answer too: none)
        most_blocks[dev & 63] = e == cudaSuccess && clusters > 0 ? kMaxCluster : kMaxCluster / 2;
    }
    const int most = most_blocks[dev & 63];
    // Blocks per sequence: one for every 4096 tokens, as far as the blocks of the
    // batch still run side by side (two per SM).
    int blocks = 1;
    while (blocks < most && p.stride > 4096 * blocks && (int64_t)p.batch * blocks * 2 <= 304) blocks *= 2;
    while (blocks < most && p.stride > kMaxCached * blocks) blocks *= 2;
    const int64_t per_block = (((int64_t)p.stride + blocks * kSelWarps - 1) / (blocks * kSelWarps) + kRunStep - 1) / kRunStep * kRunStep * kSelWarps;
    const int cached = (int)std::min<int64_t>(per_block, kMaxCached);
    cfg.gridDim = dim3((unsigned)(p.batch * blocks));
    cfg.dynamicSmemBytes = (size_t)cached * 4;
    attr[0].val.clusterDim.x = blocks;
    cfg.attrs = blocks > 1 ? attr : attr + 1;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, blocks > 1 ? select_kernel<true> : select_kernel<false>, p, cached);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace oscar
