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

// silu(g) * u in fp32.  The hardware's exponential and reciprocal are off by
// one step each (2^-23 relative), about what the other roundings here add up
// to; with the exact division instead, 64 rows of 18432 gated values took
// 7.4 us to quantise, most of it in the division's ten instructions.
__device__ __forceinline__ float gated_product(float g, float u) {
#pragma clang fp contract(off)
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

}  // namespace sg
