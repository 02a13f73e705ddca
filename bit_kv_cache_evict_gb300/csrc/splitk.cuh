// splitk.cuh -- what the split-K history kernels (decode.cu: 2-bit codes,
// int4.cu: 4-bit codes) share: block roles and waits, the item lookup, the
// token order of the P.V products, operand splits and the launch helpers.
// Library-internal.
#pragma once

#include <algorithm>

#include "oscar_common.cuh"

namespace oscar {

// Blocks are four consumer warps and one producer warp.
constexpr int kConsumerWarps = 4;
// Poll budget of every bounded mbarrier wait: a try_wait suspends about 4 us
// when the phase is not complete (measured on GB300), so 2^18 polls give up
// after about a second, far beyond any legitimate wait (a page copy, or the
// other consumer warps finishing an item).
constexpr int kWaitPolls = 1 << 18;
constexpr int kFlagFirst = 1, kFlagLast = 2, kFlagPad = 4;


__device__ __forceinline__ int find_seq(const int32_t* item_start, int B, int item) {
    int lo = 0, hi = B;  // largest b with item_start[b] <= item
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(item_start + mid) <= item) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Position of token t (0..63) in the warp's probability and V-scale rows.
// The P.V products take the page's tokens in 16 groups of four: k-step m of
// lane quad tq covers group q = 4 tq + m (tokens 4q .. 4q+3, whose V codes
// are bytes 4q .. 4q+3 of every code plane, so one 16-byte load per plane
// serves all four k-steps).  Group q sits in 16-byte chunk 4 tq + (m ^ tq)
// of a row, which keeps the lanes of one shared-memory wavefront on
// distinct banks; inside a chunk the order is pv_slot (tokens 4q, 4q+2 |
// 4q+1, 4q+3 as the two B-operand pairs).
__device__ __forceinline__ int pv_pos(int t) {
    const int q = t >> 2, tq = q >> 2, m = q & 3;
    return 4 * (4 * tq + (m ^ tq)) + pv_slot(t & 3);
}
constexpr int kPvRow = 72;  // floats per probability / V-scale row (64 + 8: conflict-free stores)

// Split two fp32 values into f16x2 registers of their high parts (the
// values with the low 13 bits cleared, see split_pair_f16) and of the
// rounded remainders.
__device__ __forceinline__ void split_both(float2 w, uint32_t& hi, uint32_t& lo) {
    const float2 h = make_float2(__uint_as_float(__float_as_uint(w.x) & 0xffffe000u),
                                 __uint_as_float(__float_as_uint(w.y) & 0xffffe000u));
    hi = pack_f16x2_rn(h.x, h.y);
    const float2 r = sub2(w, h);
    lo = pack_f16x2_rn(r.x, r.y);
}

// ------------------------------------------------------------------
// host side
// ------------------------------------------------------------------
// Dynamic shared memory of a kernel, and the largest L1 / shared carveout:
// an SM changes its split only when idle, so every kernel of the chain asks
// for the same split and a programmatically launched kernel can start on SMs
// where its predecessor still runs.  (Not for the eight-head Lloyd-Max INT2
// kernel: its register spills go through L1, which the largest split leaves
// at 28 KB; it took 9 % longer with it.)
template <typename... Args>
inline cudaError_t set_smem(void (*kernel)(Args...), int bytes, bool max_carveout = true) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && max_carveout)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 (int)cudaSharedmemCarveoutMaxShared);
    return e;
}

// Launch with a programmatic dependency on the previous kernel in the stream
// (the kernel itself decides where it waits, see pdl_wait).
template <typename P>
inline cudaError_t launch_pdl(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const P& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Blocks per SM of the 4-bit history kernel: three (128 registers); two (168, and
// four page halves per warp instead of two) for eight query heads per KV head
// with four quantisation groups per vector, whose state would spill: 32 x
// 32K, 64 query heads, groups of 32: 437 us with three blocks, 407 with two;
// groups of 64: 333 and 339; groups of 128: 295 and 321.
__host__ __device__ constexpr int int4_blocks_per_sm(int nt, int gshift) { return nt == 2 && gshift == 0 ? 2 : 3; }

// the 4-bit history kernel (int4.cu), launched by launch_decode4 between prep_kernel and bf16_kernel
cudaError_t launch_int4(const DecodeParams4& p, cudaStream_t st, int dev);

}  // namespace oscar
