// splitk.cuh -- what the split-K history kernels (decode.cu: 2-bit codes,
// int4.cu: 4-bit codes) share: block roles and waits, the item lookup and
// operand splits.
// Library-internal.
#pragma once

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

// Blocks per SM of the 4-bit history kernel: three (128 registers); two (168, and
// four page halves per warp instead of two) for eight query heads per KV head
// with four quantisation groups per vector, whose state would spill: 32 x
// 32K, 64 query heads, groups of 32: 437 us with three blocks, 407 with two;
// groups of 64: 333 and 339; groups of 128: 295 and 321.
__host__ __device__ constexpr int int4_blocks_per_sm(int nt, int gshift) { return nt == 2 && gshift == 0 ? 2 : 3; }

// the 4-bit history kernel (int4.cu), launched by launch_decode4 between prep_kernel and bf16_kernel
cudaError_t launch_int4(const DecodeParams4& p, cudaStream_t st, int dev);

}  // namespace oscar
