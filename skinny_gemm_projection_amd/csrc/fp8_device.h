// fp8_device.h -- device helpers of the e4m3 codes with a power-of-two scale a block.
#pragma once

#include "int8_device.h"

namespace sg {

// The scale of a block from the bits of its largest magnitude (a NaN is above
// infinity): the least power of two, from 2^-126 on, that is at least amax / 448 --
// its exponent, less 8, plus 1 where the mantissa is past 1.75 (448 = 1.75 * 2^8).
struct BlockScale {
    float unit, inv;  // the scale (NaN for a block that is not finite) and 1 / it
    bool bad;
};

__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
    const bool bad = amax_bits >= 0x7f800000u;
    const int e = max((int)((amax_bits + 0x1fffffu) >> 23) - 8, 1);
    return BlockScale{bad ? __builtin_nanf("") : as_f((uint32_t)e << 23),
                      as_f((uint32_t)(254 - e) << 23), bad};
}

// Codes of four values times inv, each rounded once (half to even); zeros for a bad block.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const BlockScale& s) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a * s.inv, b * s.inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c * s.inv, d * s.inv, v, true);
    return s.bad ? 0u : (uint32_t)v;
}

}  // namespace sg
