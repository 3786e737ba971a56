// norm_quant.hip -- row operators in front of the integer projections: the
// root-mean-square norm with the residual addition and int8 output, and the
// int8 codes of rows (optionally of a gated product).
//
// Mathematics, per row of K values:
//   norm:  s = x + r, t = s * g, inv = 1 / sqrt(sum s^2 / K + eps);
//          h = bf16(s), y = bf16(t * inv)
//   codes: amax = max |t|, c = 127 / amax, code = rne(t * c), scale = amax / 127
//          (the norm's scale is amax * inv / 127: the rms cancels from the codes,
//          so they depend on no sum and one rounding of 127 / amax only).
// t * c + 1.5 * 2^23 is one fused multiply-add whose only rounding is the
// rounding to a whole number: the low byte of its bits is the code.
//
// A row stays in the registers of one workgroup (each thread holds P pieces of
// 8 values), so every value is read once and written once and the two row
// statistics cost one exchange through LDS.  Norms of rows past 32768 values are
// the exception: P = 8 spills 25 registers a thread to scratch.  1024 x 65536
// with residual and int8 output takes 116 us, 2048 x 32768, as many bytes, 98;
// one row of 65536 10.0, of 32768 4.9.
//
// Many rows are bound by HBM: 8191 x 7168 with residual, bf16 and int8 output
// (528 MB) takes 92 us, 5.7 TB/s; without the bf16 output 74 (5.5); bf16 output
// alone without a residual 44 (5.4); 5003 x 8192 bf16 codes (123 MB) 22.7 us, 5.4
// TB/s; a copy reaches 4.8 to 5.1.  One row takes 2.8 us, a launch and two memory
// latencies.  Gated rows are bound by the exponential and the quotient of each
// value too: 64 x 18432 from fp32 6.9 us (64 workgroups), from bf16 7.1; 4096 x
// 8192 from bf16 (168 MB) 35.3, 4.8 TB/s.
#include <math.h>

#include <type_traits>

#include "int8_device.h"
#include "launch.h"

namespace sg {

namespace {

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: x + kMagic is x rounded to a whole number
constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ void unpack8(const uint4 u, float (&v)[8]) {
    const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = as_f(d[i] << 16);
        v[2 * i + 1] = as_f(d[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float k) {
    const uint32_t ia = as_u(fmaf(a, k, kMagic)), ib = as_u(fmaf(b, k, kMagic));
    const uint32_t ic = as_u(fmaf(c, k, kMagic)), id = as_u(fmaf(d, k, kMagic));
    return (ia & 0xffu) | ((ib & 0xffu) << 8) | ((ic & 0xffu) << 16) | (id << 24);
}

__device__ __forceinline__ uint32_t dpp_max(uint32_t v, uint32_t o) { return v > o ? v : o; }

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    v = dpp_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
    v = dpp_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
    v = dpp_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));
    v = dpp_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
    const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32);
    const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
    return dpp_max(dpp_max(a, b), dpp_max(c, d));
}

// Row statistics over the W waves that share a row: the sum of squares and the
// largest |t| as a bit pattern (ordered like the values; a NaN is above
// infinity, so one comparison finds any value that is not finite).
template <int W>
__device__ __forceinline__ void row_stats(float& ss, uint32_t& amax) {
    ss = wave_sum(ss);
    amax = wave_umax(amax);
    if constexpr (W > 1) {
        __shared__ float2 part[W];
        if ((threadIdx.x & (kWave - 1)) == 0)
            part[wave_id_in_block()] = make_float2(ss, as_f(amax));
        __syncthreads();
        ss = 0.0f;
        amax = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float2 p = part[w];
            ss += p.x;
            amax = dpp_max(amax, as_u(p.y));
        }
    }
}

// Codes of the P pieces held in t and the factor of the row's scale: rows whose
// 127 / amax would overflow are first scaled up by 2^64 (exactly).
template <int THREADS, int P>
__device__ __forceinline__ float store_codes(float (&t)[P][8], uint32_t amax_bits, bool bad, int tid,
                                             int n8, int8_t* codes) {
    float amax = as_f(amax_bits), back = 1.0f;
    if (amax < 0x1p-100f) {
        amax *= 0x1p64f;
        back = 0x1p-64f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) t[p][i] *= 0x1p64f;
    }
    const float c = amax > 0.0f && !bad ? 127.0f / amax : 0.0f;
    const uint32_t keep = bad ? 0u : ~0u;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int i = p * THREADS + tid;
        uint2 w;
        w.x = code4(t[p][0], t[p][1], t[p][2], t[p][3], c) & keep;
        w.y = code4(t[p][4], t[p][5], t[p][6], t[p][7], c) & keep;
        if (i < n8) reinterpret_cast<uint2*>(codes)[i] = w;
    }
    return amax * back;
}

// THREADS threads hold one row, ROWS rows a workgroup.
template <int THREADS, int ROWS, int P>
__global__ __launch_bounds__(THREADS* ROWS) void rmsnorm_kernel(
    const uint16_t* x, const uint16_t* r, const uint16_t* __restrict__ g, float eps, int M, int K,
    uint16_t* h, uint16_t* y, int8_t* codes, float* scales) {  // h, y may be x or r
    static_assert(ROWS == 1 || THREADS == kWave, "several rows a workgroup: a wave each");
    const int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? wave_id_in_block() : 0);
    if (ROWS > 1 && row >= M) return;  // whole waves; no barrier follows for them
    const int tid = ROWS > 1 ? (threadIdx.x & (kWave - 1)) : threadIdx.x;
    const int n8 = K / 8;
    const uint32_t bytes = (uint32_t)K * 2u;
    const rsrc_t rx = make_rsrc(x + row * K, bytes);
    const rsrc_t rr = make_rsrc(r ? r + row * K : x, r ? bytes : 0u);
    const rsrc_t rg = make_rsrc(g, bytes);

    uint4 ux[P], ur[P], ug[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const uint32_t off = (uint32_t)(p * THREADS + tid) * 16u;
        ux[p] = load16(rx, off);
        ur[p] = load16(rr, off);  // zeros without a residual
        ug[p] = load16(rg, off);
    }
    float t[P][8];
    float ss = 0.0f;
    uint32_t amax = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        float s[8], b[8], w[8];
        unpack8(ux[p], s);
        unpack8(ur[p], b);
        unpack8(ug[p], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = r ? s[i] + b[i] : s[i];
            ss = fmaf(s[i], s[i], ss);
            t[p][i] = s[i] * w[i];
            amax = dpp_max(amax, as_u(t[p][i]) & 0x7fffffffu);
        }
        ux[p] = pack8(s);
    }
    row_stats<THREADS / kWave>(ss, amax);
    const bool bad = amax >= kInfBits || !(as_u(ss) < kInfBits);
    const float inv = bad ? __builtin_nanf("") : 1.0f / sqrtf(ss / (float)K + eps);
    if (h) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (p * THREADS + tid < n8)
                reinterpret_cast<uint4*>(h + row * K)[p * THREADS + tid] = ux[p];
    }
    if (y) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = t[p][i] * inv;
            if (p * THREADS + tid < n8)
                reinterpret_cast<uint4*>(y + row * K)[p * THREADS + tid] = pack8(v);
        }
    }
    if (codes) {
        const float m = store_codes<THREADS, P>(t, amax, bad, tid, n8, codes + row * K);
        if (tid == 0) scales[row] = m * inv / 127.0f;
    }
}

template <bool F32>
__device__ __forceinline__ void load8(const rsrc_t rs, uint32_t piece, float (&v)[8]) {
    if constexpr (F32) {
        const uint4 a = load16(rs, piece * 32u), b = load16(rs, piece * 32u + 16u);
        v[0] = as_f(a.x), v[1] = as_f(a.y), v[2] = as_f(a.z), v[3] = as_f(a.w);
        v[4] = as_f(b.x), v[5] = as_f(b.y), v[6] = as_f(b.z), v[7] = as_f(b.w);
    } else {
        unpack8(load16(rs, piece * 16u), v);
    }
}

template <int THREADS, int ROWS, int P, bool F32, bool GATED>
__global__ __launch_bounds__(THREADS* ROWS) void quant_int8_kernel(const char* __restrict__ x,
                                                                   int M, int K, int8_t* codes,
                                                                   float* scales) {
    static_assert(ROWS == 1 || THREADS == kWave, "several rows a workgroup: a wave each");
    const int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? wave_id_in_block() : 0);
    if (ROWS > 1 && row >= M) return;
    const int tid = ROWS > 1 ? (threadIdx.x & (kWave - 1)) : threadIdx.x;
    const int n8 = K / 8;
    const int64_t bytes = (int64_t)K * (F32 ? 4 : 2);
    const char* base = x + row * bytes * (GATED ? 2 : 1);
    const rsrc_t ra = make_rsrc(base, (uint32_t)bytes);
    const rsrc_t rb = make_rsrc(base + (GATED ? bytes : 0), (uint32_t)bytes);
    float t[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p) load8<F32>(ra, p * THREADS + tid, t[p]);
    if constexpr (GATED) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float u[8];
            load8<F32>(rb, p * THREADS + tid, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[p][i] = gated_product(t[p][i], u[i]);
        }
    }
    float ss = 0.0f;
    uint32_t amax = 0;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = dpp_max(amax, as_u(t[p][i]) & 0x7fffffffu);
    row_stats<THREADS / kWave>(ss, amax);
    const bool bad = amax >= kInfBits;
    const float m = store_codes<THREADS, P>(t, amax, bad, tid, n8, codes + row * K);
    if (tid == 0) scales[row] = bad ? __builtin_nanf("") : m / 127.0f;
}

constexpr int kFewRows = 256;

// How a row is spread: over one wave, 256 or 1024 threads, whichever is the
// first to hold it in at most 4 (1024 threads: 8) pieces a thread.  Fewer rows
// than compute units get 1024 threads, so that one load a thread brings the row.
template <class F>
void with_shape(int M, int n8, F f) {
#define SG_SHAPE(T, R, P)                                            \
    f(std::integral_constant<int, T>{}, std::integral_constant<int, R>{}, \
      std::integral_constant<int, P>{})
    if (M < kFewRows && n8 > 256 && n8 <= 1024) SG_SHAPE(1024, 1, 1);
    else if (n8 <= 64) SG_SHAPE(64, 4, 1);
    else if (n8 <= 128) SG_SHAPE(64, 4, 2);
    else if (n8 <= 256) SG_SHAPE(256, 1, 1);
    else if (n8 <= 512) SG_SHAPE(256, 1, 2);
    else if (n8 <= 1024) SG_SHAPE(256, 1, 4);
    else if (n8 <= 2048) SG_SHAPE(1024, 1, 2);
    else if (n8 <= 4096) SG_SHAPE(1024, 1, 4);
    else SG_SHAPE(1024, 1, 8);
#undef SG_SHAPE
}

}  // namespace

hipError_t launch_rmsnorm(int M, int K, const uint16_t* x, const uint16_t* r, const uint16_t* g,
                          float eps, uint16_t* h, uint16_t* y, int8_t* codes, float* scales,
                          hipStream_t stream) {
    with_shape(M, K / 8, [&](auto t, auto rows, auto p) {
        constexpr int T = decltype(t)::value, R = decltype(rows)::value, P = decltype(p)::value;
        hipLaunchKernelGGL((rmsnorm_kernel<T, R, P>), dim3((M + R - 1) / R), dim3(T * R), 0, stream,
                           x, r, g, eps, M, K, h, y, codes, scales);
    });
    return hipGetLastError();
}

hipError_t launch_quant_int8(int M, int K, const void* x, bool f32, bool gated, int8_t* codes,
                             float* scales, hipStream_t stream) {
    with_shape(M, K / 8, [&](auto t, auto rows, auto p) {
        constexpr int T = decltype(t)::value, R = decltype(rows)::value, P = decltype(p)::value;
        const dim3 grid((M + R - 1) / R), block(T * R);
        const char* xb = static_cast<const char*>(x);
        if (f32 && gated)
            hipLaunchKernelGGL((quant_int8_kernel<T, R, P, true, true>), grid, block, 0, stream, xb,
                               M, K, codes, scales);
        else if (f32)
            hipLaunchKernelGGL((quant_int8_kernel<T, R, P, true, false>), grid, block, 0, stream,
                               xb, M, K, codes, scales);
        else if (gated)
            hipLaunchKernelGGL((quant_int8_kernel<T, R, P, false, true>), grid, block, 0, stream,
                               xb, M, K, codes, scales);
        else
            hipLaunchKernelGGL((quant_int8_kernel<T, R, P, false, false>), grid, block, 0, stream,
                               xb, M, K, codes, scales);
    });
    return hipGetLastError();
}

}  // namespace sg
