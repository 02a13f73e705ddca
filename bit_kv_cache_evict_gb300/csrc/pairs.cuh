// pairs.cuh -- double-float arithmetic (unevaluated sums of two fp32) and the
// 4-bit quantiser's decisions on such pairs, shared by the eviction kernels.
// Library-internal.
#pragma once

#include "oscar_common.cuh"

namespace oscar {

struct df {  // unevaluated sum hi + lo
    float hi, lo;
};

__device__ __forceinline__ df two_sum(float a, float b) {
    float s = __fadd_rn(a, b);
    float bp = __fsub_rn(s, a);
    float e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bp)), __fsub_rn(b, bp));
    return {s, e};
}

__device__ __forceinline__ df fast_two_sum(float a, float b) {  // |a| >= |b|
    float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}

__device__ __forceinline__ df df_add(df a, df b) {
    df s = two_sum(a.hi, b.hi);
    float e = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
    return fast_two_sum(s.hi, e);
}

__device__ __forceinline__ df df_neg(df a) { return {-a.hi, -a.lo}; }

// exact order of normalised pairs: compare high parts, then low parts
__device__ __forceinline__ bool df_less(df a, df b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }

// a / 15 of a pair, to about 2^-46 (relative)
__device__ __forceinline__ df df_div15(df a) {
    const float q = __fdiv_rn(a.hi, 15.f);
    const float r = __fadd_rn(__fmaf_rn(-q, 15.f, a.hi), a.lo);  // the remainder of the division is exact
    return fast_two_sum(q, __fdiv_rn(r, 15.f));
}

// A pair rounded to fp16 once, to nearest even: first to fp32 by round to
// odd (toward zero, the last bit set when inexact), from which a second
// rounding to 11 bits cannot err.
__device__ __forceinline__ unsigned short df_to_f16(df a) {
    uint32_t b = __float_as_uint(a.hi);
    if (a.lo != 0.f && a.hi != 0.f) {
        if ((a.lo < 0.f) != (a.hi < 0.f)) --b;  // hi lies beyond the value: the next float toward zero
        b |= 1u;
    }
    return __half_as_ushort(__float2half_rn(__uint_as_float(b)));
}

// The 4-bit code of y: clamp(rne((y - z) / s), 0, 15), s > 0.  The fp32
// quotient is within 2e-6 of the exact one; where it lies within 2e-5 of a
// border k + 1/2, y - z is compared with (k + 1/2) s, which fp32 holds
// exactly (5 x 11 bits), so the decision is that of the pair.
__device__ __forceinline__ int code4_of(df y, float sf, float zf) {
    const df yz = df_add(y, df{-zf, 0.f});
    const float u = __fdiv_rn(__fadd_rn(yz.hi, yz.lo), sf);
    float c = rintf(u);
    const float f = floorf(u);
    if (fabsf(u - f - 0.5f) < 2e-5f) {
        const df r = df_add(yz, df{-__fmul_rn(f + 0.5f, sf), 0.f});
        const bool above = r.hi > 0.f || (r.hi == 0.f && r.lo > 0.f);
        const bool tie = r.hi == 0.f && r.lo == 0.f;
        c = (above || (tie && ((int)f & 1))) ? f + 1.f : f;
    }
    return (int)fminf(fmaxf(c, 0.f), 15.f);
}
// merge two blocks' (max, min) into both: the extremes of their union
__device__ __forceinline__ void df_group_extremes(df& hi_a, df& hi_b, df& lo_a, df& lo_b) {
    const df h = df_less(hi_a, hi_b) ? hi_b : hi_a;
    const df l = df_less(lo_b, lo_a) ? lo_b : lo_a;
    hi_a = hi_b = h;
    lo_a = lo_b = l;
}

}  // namespace oscar
