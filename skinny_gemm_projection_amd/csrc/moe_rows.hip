// moe_rows.hip -- (token, slot) pairs sorted by expert, token rows laid out in that
// order, and expert outputs brought back to their tokens with the routing weights;
// the gradients of both.
//
// Pair p = t * topk + j belongs to expert ids[p].  The sort is a counting sort,
// stable in p:
//   offsets[e]   = number of pairs of experts below e,
//   positions[p] = offsets[ids[p]] + number of pairs q < p with ids[q] == ids[p],
//   sorted[positions[p]] = p,
// and pairs whose id is outside [0, E) are left out (position -1).  The place of a
// pair follows from the ids alone, no atomic decides an order.
//
//   gather:   rows[positions[t, j]] = x[t]
//   combine:  out[t] = (r[t] +) sum_j w[t, j] * rows[positions[t, j]]
//   combine's gradient: d_rows[positions[t, j]] = w[t, j] * d_out[t],
//                       d_w[t, j] = <d_out[t], rows[positions[t, j]]>
//   gather's gradient is combine without weights.
// A pair has one row and a row one pair, so no two threads write one place.  All
// row kernels go token by token: the token's own row is read (or written) once, and
// its topk rows elsewhere once each.
#include <algorithm>

#include "int8_device.h"
#include "launch.h"

namespace sg {

namespace {

// ------------------------------------------------------------------ sort

// Inclusive sum over the 64 lanes of a wave.
__device__ __forceinline__ int wave_scan(int v) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int u = __shfl_up(v, d, kWave);
        if (lane >= d) v += u;
    }
    return v;
}

// s[e] becomes the sum of s[0 .. e), e < n, and the sum of all is returned.
// Thread t owns the entries [t * per, (t + 1) * per).
template <int THREADS>
__device__ __forceinline__ int exclusive_scan(int32_t* s, int n) {
    __shared__ int32_t part[THREADS / kWave];
    const int per = (n + THREADS - 1) / THREADS;
    const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
    int sum = 0;
    for (int e = lo; e < hi; ++e) sum += s[e];
    const int inc = wave_scan(sum);
    if ((threadIdx.x & (kWave - 1)) == kWave - 1) part[threadIdx.x >> 6] = inc;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) {
        const int v = part[w];
        base += w < (int)(threadIdx.x >> 6) ? v : 0;
        total += v;
    }
    int run = base + inc - sum;
    for (int e = lo; e < hi; ++e) {
        const int v = s[e];
        s[e] = run;
        run += v;
    }
    __syncthreads();
    return total;
}

// counts[e] of the pairs [p0, p0 + count), which the given threads of one or more waves
// take in turn.  (A count: the order of the additions is free.)
__device__ __forceinline__ void count_pairs(const int32_t* __restrict__ ids, int64_t p0, int count,
                                            int E, int32_t* counts, int thread, int threads) {
    for (int c = thread; c < count; c += threads) {
        const int e = ids[p0 + c];
        if (e >= 0 && e < E) atomicAdd(&counts[e], 1);
    }
}

// Places of the pairs [p0, p0 + count) by one wave, 64 at a time: cursor[e] holds the next
// place of expert e, and the lanes of one expert are found by a ballot for each bit of
// the id.  LDS serves a wave in order, so every lane reads a cursor before it moves.
__device__ __forceinline__ void place_pairs(const int32_t* __restrict__ ids, int64_t p0, int count,
                                            int E, int bits, int32_t* cursor, int32_t* sorted,
                                            int32_t* positions) {
    const int lane = threadIdx.x & (kWave - 1);
    for (int c0 = 0; c0 < count; c0 += kWave) {
        const int c = c0 + lane;
        const int e = c < count ? ids[p0 + c] : -1;
        const bool ok = e >= 0 && e < E;
        uint64_t same = __ballot(ok);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        volatile int32_t* next = cursor;
        const int at = ok ? next[e] : 0;
        if (ok && rank == 0) next[e] = at + __popcll(same);
        if (c < count) {
            positions[p0 + c] = ok ? at + rank : -1;
            if (ok && sorted) sorted[at + rank] = (int32_t)(p0 + c);
        }
    }
}

constexpr int kSortMaxExperts = 4096;
constexpr int kSortManyWavesExperts = 1024;  // 16 waves in one workgroup: their counts take 68 KB
constexpr int kSortOneMax = 4096;      // pairs one workgroup sorts alone
constexpr int kSortChunk = 1024;       // pairs of a workgroup beyond, in two launches,
constexpr int kSortTwoMax = 1 << 16;   // up to so many pairs
constexpr int64_t kSortTwoWork = 1 << 27;  // and pairs * experts;
constexpr int kSortBigChunk = 4096;    // past them three launches

// The sort of one workgroup's pairs [p0, p0 + count): every wave counts its share of them,
// the shares' counts become first places, and every wave places its own.  before(e): the
// pairs of expert e in front of p0; base[e] comes in as the pairs of all experts below e.
// s: LDS for the waves' counts, [WAVES][E].
template <int WAVES, class Before>
__device__ __forceinline__ void sort_share(const int32_t* __restrict__ ids, int64_t p0, int count, int E,
                                           int bits, int32_t* s, const int32_t* base, Before before,
                                           int32_t* sorted, int32_t* positions) {
    const int wave = wave_id_in_block();
    const int share = (count + WAVES * kWave - 1) / (WAVES * kWave) * kWave;
    const int lo = min(count, wave * share), n = min(share, count - lo);
    for (int e = threadIdx.x; e < E; e += WAVES * kWave) {
        int run = base[e] + before(e);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int c = s[w * E + e];
            s[w * E + e] = run;
            run += c;
        }
    }
    __syncthreads();
    place_pairs(ids, p0 + lo, n, E, bits, s + wave * E, sorted, positions);
}

// Every wave's counts of its share, and the sum of all in total[e].
template <int WAVES>
__device__ __forceinline__ void count_shares(const int32_t* __restrict__ ids, int64_t p0, int count,
                                             int E, int32_t* s, int32_t* total) {
    const int wave = wave_id_in_block(), lane = threadIdx.x & (kWave - 1);
    const int share = (count + WAVES * kWave - 1) / (WAVES * kWave) * kWave;
    const int lo = min(count, wave * share), n = min(share, count - lo);
    for (int e = threadIdx.x; e < WAVES * E; e += WAVES * kWave) s[e] = 0;
    __syncthreads();
    count_pairs(ids, p0 + lo, n, E, s + wave * E, lane, kWave);
    __syncthreads();
    if (total) {
        for (int e = threadIdx.x; e < E; e += WAVES * kWave) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) sum += s[w * E + e];
            total[e] = sum;
        }
        __syncthreads();
    }
}

// LDS: counts of WAVES waves and their sums, (WAVES + 1) * E.
template <int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void moe_sort_one_kernel(const int32_t* __restrict__ ids,
                                                                    int P, int E, int bits,
                                                                    int32_t* offsets, int32_t* sorted,
                                                                    int32_t* positions) {
    extern __shared__ int32_t lds[];
    int32_t* base = lds + WAVES * E;
    count_shares<WAVES>(ids, 0, P, E, lds, base);
    const int total = exclusive_scan<WAVES * kWave>(base, E);
    for (int e = threadIdx.x; e < E; e += WAVES * kWave) offsets[e] = base[e];
    if (threadIdx.x == 0) offsets[E] = total;
    sort_share<WAVES>(ids, 0, P, E, bits, lds, base, [](int) { return 0; }, sorted, positions);
    if (sorted)
        for (int i = total + threadIdx.x; i < P; i += WAVES * kWave) sorted[i] = -1;
}

// counts[chunk][e] of the pairs of a chunk
__global__ __launch_bounds__(kBlock) void moe_count_kernel(const int32_t* __restrict__ ids, int P,
                                                           int chunk, int E, int32_t* counts) {
    __shared__ int32_t s[kSortMaxExperts];
    const int64_t p0 = (int64_t)blockIdx.x * chunk;
    for (int e = threadIdx.x; e < E; e += kBlock) s[e] = 0;
    __syncthreads();
    count_pairs(ids, p0, (int)min((int64_t)chunk, P - p0), E, s, threadIdx.x, kBlock);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kBlock) counts[(int64_t)blockIdx.x * E + e] = s[e];
}

// counts[chunk][e] becomes the sum over the chunks before, totals[e] that over all.
__global__ __launch_bounds__(kWave) void moe_scan_kernel(int32_t* counts, int chunks, int E,
                                                         int32_t* totals) {
    const int e = blockIdx.x * kWave + threadIdx.x;
    if (e >= E) return;
    int run = 0;
    int c = 0;
    for (; c + 8 <= chunks; c += 8) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = counts[(int64_t)(c + i) * E + e];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            counts[(int64_t)(c + i) * E + e] = run;
            run += v[i];
        }
    }
    for (; c < chunks; ++c) {
        const int v = counts[(int64_t)c * E + e];
        counts[(int64_t)c * E + e] = run;
        run += v;
    }
    totals[e] = run;
}

// The chunks' places.  SUMMED: counts are sums over the chunks before, with totals;
// otherwise each workgroup adds the few chunks' counts itself, which saves a launch.
// LDS: counts of the waves, the experts' first places and the pairs before, (waves + 2) * E.
template <bool SUMMED>
__global__ __launch_bounds__(kBlock) void moe_place_kernel(const int32_t* __restrict__ ids, int P,
                                                           int chunk, int chunks, int E, int bits,
                                                           const int32_t* __restrict__ counts,
                                                           const int32_t* __restrict__ totals,
                                                           int32_t* offsets, int32_t* sorted,
                                                           int32_t* positions) {
    extern __shared__ int32_t lds[];
    int32_t* base = lds + kWavesPerBlock * E;
    int32_t* before = base + E;
    const int b = blockIdx.x;
    for (int e = threadIdx.x; e < E; e += kBlock) {
        if constexpr (SUMMED) {
            base[e] = totals[e];
            before[e] = counts[(int64_t)b * E + e];
        } else {
            int all = 0, front = 0;
#pragma unroll 8
            for (int c = 0; c < chunks; ++c) {
                const int v = counts[(int64_t)c * E + e];
                all += v;
                front += c < b ? v : 0;
            }
            base[e] = all;
            before[e] = front;
        }
    }
    const int64_t p0 = (int64_t)b * chunk;
    const int count = (int)min((int64_t)chunk, P - p0);
    count_shares<kWavesPerBlock>(ids, p0, count, E, lds, nullptr);
    const int total = exclusive_scan<kBlock>(base, E);
    if (b == 0) {
        for (int e = threadIdx.x; e < E; e += kBlock) offsets[e] = base[e];
        if (threadIdx.x == 0) offsets[E] = total;
    }
    sort_share<kWavesPerBlock>(ids, p0, count, E, bits, lds, base, [&](int e) { return before[e]; }, sorted,
                               positions);
    if (sorted)  // behind the last valid pair
        for (int i = threadIdx.x; i < count; i += kBlock)
            if (p0 + i >= total) sorted[p0 + i] = -1;
}

// ------------------------------------------------------------------ rows

// Rows by expert are read once and written once, and there are topk of them to a token's
// own: they pass the caches by (non-temporal), which keep the rest.  4099 x 8 x 7168 laid
// out 122 -> 111 us, back 115 -> 111; both gradients of 2050 x 8 x 7168 162 -> 145.
__device__ __forceinline__ void store16_nt(char* to, const uint4 v) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(to));
}

constexpr int kSpan = kBlock * 16;  // bytes of a row a workgroup takes at once

// Workgroups (span, token): tokens go over y and z, whose sizes a launch limits.
constexpr int kTokensY = 32768;
__device__ __forceinline__ int64_t token_of() {
    return (int64_t)blockIdx.z * kTokensY + blockIdx.y;
}

// A workgroup brings one span of one token's row to its places.
__global__ __launch_bounds__(kBlock) void moe_gather_kernel(const char* __restrict__ x, int64_t pitch,
                                                            int T, int topk,
                                                            const int32_t* __restrict__ positions,
                                                            char* __restrict__ rows) {
    const int64_t t = token_of();
    const int64_t at = (int64_t)blockIdx.x * kSpan + threadIdx.x * 16;
    const int limit = T * topk;  // rows there are: a position past them is taken as left out
    if (t >= T || at >= pitch) return;
    const uint4 v = *reinterpret_cast<const uint4*>(x + t * pitch + at);
    for (int j = 0; j < topk; ++j) {
        const int pos = positions[t * topk + j];
        if (pos >= 0 && pos < limit) store16_nt(rows + pos * pitch + at, v);
    }
}

template <bool F32>
struct Piece {  // 16 bytes of a row
    static constexpr int N = F32 ? 4 : 8;
    static __device__ __forceinline__ void unpack(const uint4 u, float (&v)[N]) {
        const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                v[i] = as_f(d[i]);
            } else {
                v[2 * i] = as_f(d[i] << 16);
                v[2 * i + 1] = as_f(d[i] & 0xffff0000u);
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[N]) {
        if constexpr (F32)
            return make_uint4(as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3]));
        else
            return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                              pack_bf16(v[6], v[7]));
    }
};

constexpr int kAtOnce = 8;  // rows of a token requested before the first is added

// Sums in fp32, j ascending, each step one fused multiply-add (without weights an
// addition); the residual is added last and the result rounded once.  r and out have the
// rows' type, or with NARROW bf16 beside rows of fp32.
template <bool F32, bool NARROW>
__global__ __launch_bounds__(kBlock) void moe_combine_kernel(
    const char* __restrict__ rows, int64_t pitch, int T, int topk,
    const int32_t* __restrict__ positions, const float* __restrict__ w, const char* r,
    char* out) {  // out may be r
    static_assert(F32 || !NARROW, "bf16 rows have bf16 outputs");
    typedef Piece<F32> P;
    constexpr int kShrink = NARROW ? 2 : 1;
    const int64_t t = token_of();
    const int64_t at = (int64_t)blockIdx.x * kSpan + threadIdx.x * 16;
    const int limit = T * topk;
    if (t >= T || at >= pitch) return;
    // requested with the rows, not behind their sum
    const int64_t opitch = pitch / kShrink, oat = at / kShrink;
    const rsrc_t rr = make_rsrc(r + (r ? t : 0) * opitch, r ? (uint32_t)opitch : 0u);
    uint4 res = make_uint4(0, 0, 0, 0);
    if constexpr (NARROW) {
        const auto half = __builtin_amdgcn_raw_buffer_load_b64(rr, (uint32_t)oat, 0, 0);
        res = make_uint4(half[0] << 16, half[0] & 0xffff0000u, half[1] << 16, half[1] & 0xffff0000u);
    } else {
        res = load16(rr, (uint32_t)oat);
    }
    float acc[P::N] = {};
    for (int j0 = 0; j0 < topk; j0 += kAtOnce) {
        uint4 v[kAtOnce];
        float f[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int j = j0 + i;
            const int pos = j < topk ? positions[t * topk + j] : -1;
            const bool on = pos >= 0 && pos < limit;
            f[i] = on ? w ? w[t * topk + j] : 1.0f : 0.0f;
            // a left-out pair reads zeros through an empty buffer: no branch around a load
            v[i] = load16<kStream>(make_rsrc(rows + (on ? pos : 0) * pitch, on ? (uint32_t)pitch : 0u),
                          (uint32_t)at);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            float y[P::N];
            P::unpack(v[i], y);
#pragma unroll
            for (int k = 0; k < P::N; ++k) acc[k] = fmaf(f[i], y[k], acc[k]);
        }
    }
    if (r) {
        float y[P::N];
        P::unpack(res, y);
#pragma unroll
        for (int k = 0; k < P::N; ++k) acc[k] = y[k] + acc[k];
    }
    if constexpr (NARROW)
        *reinterpret_cast<uint2*>(out + t * opitch + oat) =
            make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
    else
        *reinterpret_cast<uint4*>(out + t * opitch + oat) = P::pack(acc);
}

// One workgroup a token.  The dot products of up to kAtOnce rows are held while the
// row is walked; d_rows may be rows (an element is read before it is written, by the
// same thread).
template <bool F32>
__global__ __launch_bounds__(kBlock) void moe_combine_grad_kernel(
    const char* __restrict__ d_out, const char* rows, int64_t pitch, int T, int topk,
    const int32_t* __restrict__ positions, const float* __restrict__ w, char* d_rows,
    float* __restrict__ d_w) {
    typedef Piece<F32> P;
    __shared__ float part[kWavesPerBlock][kAtOnce];
    const int64_t t = blockIdx.x;
    const int limit = T * topk;
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id_in_block();
    for (int j0 = 0; j0 < topk; j0 += kAtOnce) {
        int64_t base[kAtOnce];
        float f[kAtOnce], dot[kAtOnce];
        bool on[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int j = j0 + i;
            const int pos = j < topk ? positions[t * topk + j] : -1;
            on[i] = pos >= 0 && pos < limit;
            base[i] = on[i] ? pos * pitch : 0;
            f[i] = on[i] ? w[t * topk + j] : 0.0f;
            dot[i] = 0.0f;
        }
        for (int64_t at = threadIdx.x * 16; at < pitch; at += kSpan) {
            float g[P::N];
            P::unpack(*reinterpret_cast<const uint4*>(d_out + t * pitch + at), g);
            uint4 v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                v[i] = load16<kStream>(make_rsrc(rows + base[i], on[i] ? (uint32_t)pitch : 0u), (uint32_t)at);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (!on[i]) continue;
                float y[P::N], d[P::N];
                P::unpack(v[i], y);
#pragma unroll
                for (int k = 0; k < P::N; ++k) {
                    dot[i] = fmaf(g[k], y[k], dot[i]);
                    d[k] = f[i] * g[k];
                }
                store16_nt(d_rows + base[i] + at, P::pack(d));
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const float s = wave_sum(dot[i]);
            if (lane == 0) part[wave][i] = s;
        }
        __syncthreads();
        if (threadIdx.x < kAtOnce && j0 + (int)threadIdx.x < topk) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < kWavesPerBlock; ++v) s += part[v][threadIdx.x];
            d_w[t * topk + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

dim3 token_grid(int T, int64_t pitch) {
    return dim3((uint32_t)((pitch + kSpan - 1) / kSpan), (uint32_t)(T < kTokensY ? T : kTokensY),
                (uint32_t)((T + kTokensY - 1) / kTokensY));
}

}  // namespace

// One workgroup takes 8.2 us for 4096 pairs of 384 experts and 12.6 for 8192, two
// launches 10.8 and 9.9.  In two launches every workgroup adds the counts of all chunks
// itself: 12.3 us for 32768 pairs of 384 experts (three launches: 25.6) and 22.3 for 65536
// of 1024 (28.2), but 55.5 for 65536 of 4096 (38.3; for half of them 36.8 and 38.1).
int moe_sort_launches(int64_t P, int E) {
    return P <= kSortOneMax ? 1 : P <= kSortTwoMax && P * E <= kSortTwoWork ? 2 : 3;
}

// Never less for more pairs, so a workspace for the most of them serves all.
size_t moe_sort_workspace_bytes(int64_t P, int E) {
    if (P <= kSortOneMax) return 0;
    const int64_t small = (std::min<int64_t>(P, kSortTwoMax) + kSortChunk - 1) / kSortChunk;
    const int64_t big = (P + kSortBigChunk - 1) / kSortBigChunk;
    return (size_t)(std::max(small, big) + 1) * E * 4;
}

// One of the sorting kernels, with `per` ints of LDS for each of E experts.  The limit set is
// the kernel's own for as many experts as it takes, the same in every call: it belongs to
// the kernel, and a call for fewer experts may come between another thread's two steps.
template <class... P, class... A>
static hipError_t launch_sort(void (*kernel)(P...), int grid, int block, int per, int most_experts, int E,
                              hipStream_t stream, A... args) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             per * most_experts * 4);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(block), (size_t)per * E * 4, stream, args...);
    return hipGetLastError();
}

hipError_t launch_moe_sort(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* sorted,
                           int32_t* positions, void* ws, hipStream_t stream) {
    int bits = 0;
    while ((1 << bits) < E) ++bits;
    if (P <= kSortOneMax) {
        // 16 waves while their counts fit, and are needed
        if (E <= kSortManyWavesExperts && P > 4 * kWave)
            return launch_sort(moe_sort_one_kernel<16>, 1, 16 * kWave, 17, kSortManyWavesExperts, E, stream,
                               ids, P, E, bits, offsets, sorted, positions);
        return launch_sort(moe_sort_one_kernel<4>, 1, 4 * kWave, 5, kSortMaxExperts, E, stream, ids, P, E,
                           bits, offsets, sorted, positions);
    }
    const bool two = moe_sort_launches(P, E) == 2;
    const int chunk = two ? kSortChunk : kSortBigChunk, chunks = (P + chunk - 1) / chunk;
    constexpr int kPer = kWavesPerBlock + 2;
    int32_t* counts = static_cast<int32_t*>(ws);
    int32_t* totals = counts + (int64_t)chunks * E;
    hipLaunchKernelGGL(moe_count_kernel, dim3(chunks), dim3(kBlock), 0, stream, ids, P, chunk, E, counts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (two)
        return launch_sort(moe_place_kernel<false>, chunks, kBlock, kPer, kSortMaxExperts, E, stream, ids, P,
                           chunk, chunks, E, bits, counts, totals, offsets, sorted, positions);
    hipLaunchKernelGGL(moe_scan_kernel, dim3((E + kWave - 1) / kWave), dim3(kWave), 0, stream, counts,
                       chunks, E, totals);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    return launch_sort(moe_place_kernel<true>, chunks, kBlock, kPer, kSortMaxExperts, E, stream, ids, P,
                       chunk, chunks, E, bits, counts, totals, offsets, sorted, positions);
}

hipError_t launch_moe_gather(const void* x, int T, int topk, int64_t pitch, const int32_t* positions,
                             void* rows, hipStream_t stream) {
    hipLaunchKernelGGL(moe_gather_kernel, token_grid(T, pitch), dim3(kBlock), 0, stream,
                       static_cast<const char*>(x), pitch, T, topk, positions,
                       static_cast<char*>(rows));
    return hipGetLastError();
}

hipError_t launch_moe_combine(const void* rows, int T, int topk, int64_t pitch, bool f32, bool out_f32,
                              const int32_t* positions, const float* w, const void* r, void* out,
                              hipStream_t stream) {
    const auto kernel = !f32      ? moe_combine_kernel<false, false>
                        : out_f32 ? moe_combine_kernel<true, false>
                                  : moe_combine_kernel<true, true>;
    hipLaunchKernelGGL(kernel, token_grid(T, pitch), dim3(kBlock), 0, stream,
                       static_cast<const char*>(rows), pitch, T, topk, positions, w,
                       static_cast<const char*>(r), static_cast<char*>(out));
    return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const void* d_out, const void* rows, int T, int topk,
                                   int64_t pitch, bool f32, const int32_t* positions, const float* w,
                                   void* d_rows, float* d_w, hipStream_t stream) {
    const auto kernel = f32 ? moe_combine_grad_kernel<true> : moe_combine_grad_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)T), dim3(kBlock), 0, stream,
                       static_cast<const char*>(d_out), static_cast<const char*>(rows), pitch, T, topk,
                       positions, w, static_cast<char*>(d_rows), d_w);
    return hipGetLastError();
}

}  // namespace sg
