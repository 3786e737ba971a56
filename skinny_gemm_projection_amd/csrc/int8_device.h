// int8_device.h -- device helpers shared by the 8-bit integer kernels.
#pragma once

#include "sg_device.h"

namespace sg {

// bf16 pair of two fp32 values (round to nearest even), a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    bf16x2_t p;
    p[0] = (__bf16)a;
    p[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, p);
}

// silu(g) * u in fp32, off by at most 7 * 2^-24 relative for g >= -87 (below,
// the exponential falls out of the normal range and the result is 0).
//   e = exp(-|g|): the hardware's exponential (one step) of p = fl(-|g| log2 e)
//   and a first-order term for what p leaves of -|g|, below 2^-17: 3 * 2^-24 in
//   all (p stays finite, so that the largest gates give 0 too);
//   1 / (1 + exp(-g)) is 1 / (1 + e) or, for a negative gate, e / (1 + e), which
//   overflows nowhere; the quotient is the hardware's reciprocal corrected by its
//   exact remainder.  The sum, both products and the quotient round once.
// An infinite or NaN gate gives NaN.
// 64 rows of 18432 gated values take 6.9 us to quantise.  exp2(fl(-g log2 e)) and
// the bare reciprocal took 5.7, but their error grew with the gate, to 33 steps
// (2^-23) at -87.
__device__ __forceinline__ float gated_product(float g, float u) {
#pragma clang fp contract(off)
    constexpr float kLog2e = 0x1.715476p+0f, kLn2 = 0x1.62e43p-1f, kLn2Low = -0x1.05c61p-29f;
    const float a = -fabsf(g), p = fmaxf(a * kLog2e, -256.0f);
    float e = __builtin_amdgcn_exp2f(p);
    e = fmaf(e, fmaf(-p, kLn2Low, fmaf(-p, kLn2, a)), e);
    const float d = 1.0f + e, n = g < 0.0f ? g * e : g;
    const float r = __builtin_amdgcn_rcpf(d), y = n * r;
    return fmaf(fmaf(-d, y, n), r, y) * u;
}

}  // namespace sg
