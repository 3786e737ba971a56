// tile_device.h -- device helpers shared by the kernels that multiply tiles of codes through
// LDS: loads that write LDS directly, waits, and outputs of four neighbours a lane.
#pragma once

#include <type_traits>

#include "int8_device.h"

namespace sg {

typedef __attribute__((address_space(3))) void lds_void_t;

// A buffer offset that reads zeros, also after a row offset is added: buffers
// here end below 2^31 and rows of one tile span less than 2^27 bytes.
constexpr uint32_t kPastEnd = 1u << 31;

// 64 lanes x 16 bytes from the buffer (each lane its own offset) to 1 KB of LDS.
template <int POLICY>
__device__ __forceinline__ void load_to_lds(rsrc_t r, uint4* lds, uint32_t offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 16, (int)offset, 0, 0, POLICY);
}

// Before a wave refills an LDS slot of its own: its reads of the slot are done.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Outputs y[m][n .. n+4) with the residual, one access each way also where rows
// of y are not 4-element aligned: global memory takes any alignment.  (333 x 5001
// x 2064: 10.9 us, as for 5008 columns; four scalar stores a lane 15.5, rows
// turned in LDS and stored an element a lane 12.3.)
template <class Ep>
__device__ __forceinline__ void finish4(const Ep& ep, int N, int m, int n, float (&y)[4]) {
    const int64_t at = (int64_t)m * ep.ld + n;
    if (n + 4 <= N) {
        if (ep.r) {
            uint2 r;
            __builtin_memcpy(&r, ep.r + at, 8);
            y[0] = as_f(r.x << 16) + y[0];
            y[1] = as_f(r.x & 0xffff0000u) + y[1];
            y[2] = as_f(r.y << 16) + y[2];
            y[3] = as_f(r.y & 0xffff0000u) + y[3];
        }
        if (ep.y_f32) {
            const float4 v = make_float4(y[0], y[1], y[2], y[3]);
            __builtin_memcpy(ep.y_f32 + at, &v, 16);
        }
        if (ep.y_bf16) {
            const uint2 v = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
            __builtin_memcpy(ep.y_bf16 + at, &v, 8);
        }
    } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (n + v >= N) break;
            float o = y[v];
            if (ep.r) o = bf16_to_f32(ep.r[at + v]) + o;
            if (ep.y_f32) ep.y_f32[at + v] = o;
            if (ep.y_bf16) ep.y_bf16[at + v] = f32_to_bf16(o);
        }
    }
}

template <int N>
__device__ __forceinline__ void wait_and_barrier() {
    // at most N loads of this wave outstanding, its LDS reads done, then all waves
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
}

template <int I, int END, class F>
__device__ __forceinline__ void unrolled(F f) {
    if constexpr (I < END) {
        f(std::integral_constant<int, I>{});
        unrolled<I + 1, END>(f);
    }
}

}  // namespace sg
