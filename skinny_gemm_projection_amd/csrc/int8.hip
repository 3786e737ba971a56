// int8.hip -- product of int8 codes with one scale per row of x (token) and
// per row of W (channel), on gfx950 matrix cores.
//
//   y[m,n] = float(sum_k xq[m,k] * wq[n,k]) * ws[n] * xs[m]  (+ r, in fp32)
//
// v_mfma_i32_16x16x64_i8 multiplies 16 rows of W by 16 rows of x over 64
// codes: lane (row = lane & 15, grp = lane >> 4) supplies the 16 codes
// k = 16*grp .. +16 of its row, one 16-byte load, and receives
// y[m = lane & 15][n = 4*grp .. +4], four neighbours of one row of y.  The
// int32 sums are exact, so no split of K changes a bit.
#include "launch.h"

namespace sg {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4_t mfma16(const uint4 w, const uint4 x, i32x4_t acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, w),
                                                 __builtin_bit_cast(i32x4_t, x), acc, 0, 0, 0);
}

__device__ __forceinline__ void store_scaled(const Int8Epilogue& ep, int64_t i, int acc, float ws,
                                             float xs) {
#pragma clang fp contract(off)  // the same roundings wherever an output is finished
    float v = (float)acc * ws * xs;
    if (ep.r) v += bf16_to_f32(ep.r[i]);
    if (ep.y_f32) ep.y_f32[i] = v;
    if (ep.y_bf16) ep.y_bf16[i] = f32_to_bf16(v);
}

// One wave: 16 rows of W times 16 * MT rows of x over all of K, both operands
// straight from memory.
template <int MT>
__global__ __launch_bounds__(kBlock) void int8_direct_kernel(const int8_t* __restrict__ xq,
                                                             const int8_t* __restrict__ wq, int M,
                                                             int N, int K, Int8Epilogue ep) {
    const int lane = threadIdx.x & (kWave - 1);
    const int n0 = (blockIdx.x * kWavesPerBlock + wave_id_in_block()) * 16;
    const int m0 = blockIdx.y * 16 * MT;
    if (n0 >= N) return;
    const int row = lane & 15, grp = lane >> 4;
    const rsrc_t rw = make_rsrc(wq + (int64_t)n0 * K, (uint32_t)min(16, N - n0) * (uint32_t)K);
    const rsrc_t rx = make_rsrc(xq + (int64_t)m0 * K, (uint32_t)min(16 * MT, M - m0) * (uint32_t)K);
    i32x4_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = i32x4_t{0, 0, 0, 0};
    for (int k0 = 0; k0 < K; k0 += 64) {
        const int k = k0 + 16 * grp;
        const bool in = k < K;  // K is a multiple of 16: a lane's codes are all in or all out
        const uint4 w = load16(rw, in ? (uint32_t)row * K + k : ~15u);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const uint4 x = load16(rx, in ? (uint32_t)(16 * t + row) * K + k : ~15u);
            acc[t] = mfma16(w, x, acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = m0 + 16 * t + row;
        if (m >= M) continue;
        const float xs = ep.xs[m];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int n = n0 + 4 * grp + v;
            if (n < N) store_scaled(ep, (int64_t)m * N + n, acc[t][v], ep.ws[n], xs);
        }
    }
}

}  // namespace

size_t int8_workspace_bytes(int, int, int) { return 0; }

hipError_t launch_gemm_int8(int M, int N, int K, const int8_t* xq, const int8_t* wq,
                            const Int8Epilogue& ep, void*, hipStream_t stream) {
    const int gx = (N + 16 * kWavesPerBlock - 1) / (16 * kWavesPerBlock);
    // grid.y: at most SG_INT8_MAX_M / 64 = 16384 tiles
    if (M <= 16)
        hipLaunchKernelGGL((int8_direct_kernel<1>), dim3(gx), dim3(kBlock), 0, stream, xq, wq, M, N,
                           K, ep);
    else
        hipLaunchKernelGGL((int8_direct_kernel<4>), dim3(gx, (M + 63) / 64), dim3(kBlock), 0,
                           stream, xq, wq, M, N, K, ep);
    return hipGetLastError();
}

}  // namespace sg
