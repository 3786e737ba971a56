// quant_fp8.hip -- e4m3 codes of rows (optionally of a gated product) with one
// scale for each block of 128 columns.
//
// Mathematics, per block of values v: scale = the least power of two, from 2^-126
// on, that is at least max |v| / 448, so that |v| / scale lies at most at 448,
// e4m3's largest value; code = v / scale rounded once, half to even.  A power of
// two makes that quotient exact: which code a value gets is decided by the value
// alone, and halfway cases are real ones.  (With scale = max |v| / 448 the rounding
// of the quotient decides them; rows of bf16 have many.)  A floating-point code
// loses nothing by the coarser scale but up to one binade below its normal range.
#include "fp8_device.h"
#include "launch.h"

namespace sg {

namespace {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}

template <bool F32, int POLICY>
__device__ __forceinline__ void load8(const rsrc_t rs, uint32_t piece, float (&v)[8]) {
    if constexpr (F32) {
        const uint4 a = load16<POLICY>(rs, piece * 32u), b = load16<POLICY>(rs, piece * 32u + 16u);
        v[0] = as_f(a.x), v[1] = as_f(a.y), v[2] = as_f(a.z), v[3] = as_f(a.w);
        v[4] = as_f(b.x), v[5] = as_f(b.y), v[6] = as_f(b.z), v[7] = as_f(b.w);
    } else {
        const uint4 u = load16<POLICY>(rs, piece * 16u);
        const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = as_f(d[i] << 16);
            v[2 * i + 1] = as_f(d[i] & 0xffff0000u);
        }
    }
}

template <bool CACHED>
__device__ __forceinline__ void store_codes(uint8_t* to, const uint2 c) {
    if constexpr (CACHED)
        *reinterpret_cast<uint2*>(to) = c;
    else
        __builtin_nontemporal_store(__builtin_bit_cast(uint64_t, c), reinterpret_cast<uint64_t*>(to));
}

// A wave takes 512 columns (8 a lane, so 16 lanes share a block) of R rows.
template <int R, bool F32, bool GATED>
__global__ __launch_bounds__(kBlock) void quant_fp8_kernel(const char* __restrict__ x, int M, int K,
                                                           int spans, uint8_t* codes,
                                                           float* scales) {
    const int64_t item = (int64_t)blockIdx.x * kWavesPerBlock + wave_id_in_block();
    const int64_t group = item / spans;
    const int span = (int)(item - group * spans);
    const int64_t r0 = group * R;
    if (r0 >= M) return;  // whole waves, no barrier follows
    const int lane = threadIdx.x & (kWave - 1);
    const int piece = span * kWave + lane;  // of 8 columns
    const int64_t half = (int64_t)K * (F32 ? 4 : 2), pitch = half * (GATED ? 2 : 1);
    // Of many rows values and codes pass the caches by: 8191 x 7168 bf16 34.9 -> 30.7 us
    // (the values alone 31.5).
    constexpr int kPolicy = R > 1 ? kStream : kCached;
    float t[R][8], u[GATED ? R : 1][8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint32_t bytes = r0 + i < M ? (uint32_t)half : 0u;
        const char* row = x + (r0 + i) * pitch;
        load8<F32, kPolicy>(make_rsrc(row, bytes), piece, t[i]);
        if constexpr (GATED) load8<F32, kPolicy>(make_rsrc(row + half, bytes), piece, u[i]);
    }
    float unit[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        uint32_t amax = 0;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            if constexpr (GATED) t[i][v] = gated_product(t[i][v], u[i][v]);
            amax = max(amax, as_u(t[i][v]) & 0x7fffffffu);  // a NaN is above infinity
        }
        amax = dpp_umax<0xB1>(amax);   // quad_perm [1,0,3,2]
        amax = dpp_umax<0x4E>(amax);   // quad_perm [2,3,0,1]
        amax = dpp_umax<0x141>(amax);  // row_half_mirror
        amax = dpp_umax<0x140>(amax);  // row_mirror
        const BlockScale s = block_scale(amax);
        unit[i] = s.unit;
        if (piece * 8 < K && r0 + i < M)
            store_codes<R == 1>(codes + (r0 + i) * K + piece * 8,
                                make_uint2(codes4(t[i][0], t[i][1], t[i][2], t[i][3], s),
                                           codes4(t[i][4], t[i][5], t[i][6], t[i][7], s)));
    }
    const int b = span * 4 + (lane >> 4);
    if ((lane & 15) == 0 && b * 128 < K) {
        float* to = scales + (int64_t)b * M + r0;
        if (r0 + R <= M) {
            __builtin_memcpy(to, unit, sizeof unit);  // one store at any alignment
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (r0 + i < M) to[i] = unit[i];
        }
    }
}

template <int R>
void launch(int M, int K, const char* x, bool f32, bool gated, uint8_t* codes, float* scales,
            hipStream_t stream) {
    const int spans = (K + 511) / 512;
    const int64_t waves = (int64_t)((M + R - 1) / R) * spans;
    const dim3 grid((uint32_t)((waves + kWavesPerBlock - 1) / kWavesPerBlock)), block(kBlock);
    if (f32 && gated)
        hipLaunchKernelGGL((quant_fp8_kernel<R, true, true>), grid, block, 0, stream, x, M, K, spans,
                           codes, scales);
    else if (f32)
        hipLaunchKernelGGL((quant_fp8_kernel<R, true, false>), grid, block, 0, stream, x, M, K,
                           spans, codes, scales);
    else if (gated)
        hipLaunchKernelGGL((quant_fp8_kernel<R, false, true>), grid, block, 0, stream, x, M, K,
                           spans, codes, scales);
    else
        hipLaunchKernelGGL((quant_fp8_kernel<R, false, false>), grid, block, 0, stream, x, M, K,
                           spans, codes, scales);
}

}  // namespace

hipError_t launch_quant_fp8(int M, int K, const void* x, bool f32, bool gated, uint8_t* codes,
                            float* scales, hipStream_t stream) {
    const char* xb = static_cast<const char*>(x);
    if (M >= 512)
        launch<4>(M, K, xb, f32, gated, codes, scales, stream);
    else
        launch<1>(M, K, xb, f32, gated, codes, scales, stream);
    return hipGetLastError();
}

}  // namespace sg
