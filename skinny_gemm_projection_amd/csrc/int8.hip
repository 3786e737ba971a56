// int8.hip -- product of int8 codes with one scale per row of x (token) and
// per row of W (channel), on gfx950 matrix cores.
//
//   y[m,n] = float(sum_k xq[m,k] * wq[n,k]) * ws[n] * xs[m]  (+ r, in fp32)
//
// v_mfma_i32_16x16x64_i8 multiplies 16 rows of W by 16 rows of x over 64
// codes: lane (row = lane & 15, grp = lane >> 4) supplies 16 codes of its row,
// the same ones for W and x, and receives y[m = lane & 15][n = 4*grp .. +4],
// four neighbours of one row of y.  The int32 sums are exact, so no split of K
// changes a bit.
//
// Two kinds of kernel share the batch range:
//  * team kernels (up to 64 rows): a workgroup owns 16 or 32 rows of W and all
//    of K, its waves take windows of K in turn and add their sums in LDS.  Bound
//    by the weight stream from HBM, as far as the waits noted at the kernel let
//    it run, and, from about 16 rows, by the x rows that every workgroup reads
//    from L2.  2 x 8192 x 7168 takes 11.2 us (5.3 TB/s; a kernel that only reads
//    W 9.5), 16 x 7168 x 8192 with the residual 11.5, 4 x 36864 x 7168 40.7 (6.5
//    TB/s).
//  * int8_tile_kernel (beyond): a workgroup owns BM rows of x and BN rows of W,
//    both requested a few stages ahead; K may be split between workgroups, the
//    int32 partial tiles then go through the workspace to int8_reduce_kernel.
//    8192 x 8192 x 7168 takes 336 us (2.87 POP/s) on inputs that stay in the
//    caches and 354 to 388 on changing ones; all-zero codes take 271, so the rest
//    is the clock that the chip's power allows: the matrix cores are busy 70 % of
//    the cycles at about 1.8 GHz.
// All of them bring codes to LDS with loads that write it directly, 128-byte
// lines whole.
#include <type_traits>

#include "launch.h"
#include "tile_device.h"

namespace sg {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4_t mfma16(const uint4 w, const uint4 x, i32x4_t acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, w),
                                                 __builtin_bit_cast(i32x4_t, x), acc, 0, 0, 0);
}

// y of four neighbouring outputs: one rounding for the conversion and each product
__device__ __forceinline__ void scale4(const i32x4_t acc, const float4 ws, float xs, float (&y)[4]) {
#pragma clang fp contract(off)
    y[0] = (float)acc[0] * ws.x * xs;
    y[1] = (float)acc[1] * ws.y * xs;
    y[2] = (float)acc[2] * ws.z * xs;
    y[3] = (float)acc[3] * ws.w * xs;
}

// scales of channels n .. n+4 (zeros past N)
__device__ __forceinline__ float4 channel_scales(const float* ws, int N, int n) {
    if (n + 4 <= N) return make_float4(ws[n], ws[n + 1], ws[n + 2], ws[n + 3]);
    return make_float4(n < N ? ws[n] : 0.0f, n + 1 < N ? ws[n + 1] : 0.0f,
                       n + 2 < N ? ws[n + 2] : 0.0f, 0.0f);
}

// ---------------------------------------------------------------- team kernels

// Where a workgroup of the team kernels starts in K.  Rows whose pitch is a
// multiple of 4 KB have the same window in the same memory channels, and
// workgroups that all start at window 0 queue there together: such rows are
// started 7 windows apart and wrap around.  (16 x 7168 x 8192 takes 11.4 us
// against 14.1 without; other pitches lose about 1 %, so they start at 0.)
__device__ __forceinline__ int first_window(int K, int windows) {
    return K % 4096 == 0 ? (int)(blockIdx.x * 7u % (uint32_t)windows) : 0;
}

// Window of a slot: the slots behind the last are empty (past K).
__device__ __forceinline__ int window_of(int slot, int first, int windows) {
    const int t = slot + first;
    return slot >= windows ? windows : t >= windows ? t - windows : t;
}

// Sums of the S waves of a workgroup (RT * MT blocks of 16 x 16 each, in the
// LDS at sums + wave * stride) and the finished outputs.
template <int S, int RT, int MT>
__device__ __forceinline__ void finish_team(const uint4* sums, int stride, int M, int N, int n0,
                                            const Int8Epilogue& ep) {
    for (int e = threadIdx.x; e < RT * MT * kWave; e += S * kWave) {
        const int f = e >> 6, l = e & 63;
        const int m = (f % MT) * 16 + (l & 15), n = n0 + (f / MT) * 16 + 4 * (l >> 4);
        if (m >= M || n >= N) continue;
        i32x4_t a = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < S; ++s) a += __builtin_bit_cast(i32x4_t, sums[s * stride + e]);
        float y[4];
        scale4(a, channel_scales(ep.ws, N, n), ep.xs[m], y);
        finish4(ep, N, m, n, y);
    }
}

// S waves share 16 * RT rows of W and all of x; wave s takes the 128-code
// windows s, s + S, ... of K through D LDS slots of its own, W and x both: no
// barrier until the sums meet.  A slot is refilled as soon as it has been read,
// but only while there is more, and where those two paths meet the compiler
// waits for the stricter: before a slot is read a wave waits for every load it
// has out, the refill just requested among them (D = 2; D = 4: all, then all but
// 2, 1 and 0 slots' worth).  With two slots one window a wave is really in
// flight, and what overlaps is the waves of a compute unit.  A load instruction covers 8
// rows x 128 bytes, whole lines: with 64 bytes of 16 rows, the layout of the
// operand registers, reading W alone took 15 to 25 % longer (7168 x 8192 13.2
// against 10.7 us), and x came from L2 at 30 against 43 bytes a clock.  The
// 16-byte piece p of row r sits at place p ^ (r % 8) of the row.  W carries the
// non-temporal hint.
template <int S, int RT, int MT, int D>
__global__ __launch_bounds__(S* kWave) void int8_team_kernel(const int8_t* __restrict__ xq,
                                                             const int8_t* __restrict__ wq, int M,
                                                             int N, int K, Int8Epilogue ep) {
    static_assert(D == 2 || D == 4, "two or four slots");
    constexpr int kWin = 128, P = kWin / 16, kRows = 1024 / kWin;
    constexpr int kSlot = 16 * (RT + MT) * P;
    static_assert(kSlot >= RT * MT * kWave, "a wave's sums reuse its first slot");
    __shared__ uint4 slot0[S][kSlot], slot1[S][kSlot];
    __shared__ uint4 slot2[D > 2 ? S : 1][D > 2 ? kSlot : 1], slot3[D > 2 ? S : 1][D > 2 ? kSlot : 1];
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id_in_block();
    const int row = lane & 15, grp = lane >> 4;
    const int n0 = blockIdx.x * 16 * RT;
    const rsrc_t rw = make_rsrc(wq + (int64_t)n0 * K, (uint32_t)min(16 * RT, N - n0) * (uint32_t)K);
    const rsrc_t rx = make_rsrc(xq, (uint32_t)M * (uint32_t)K);

    i32x4_t acc[RT][MT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
    const int lrow = lane / P, kpos = ((lane % P) ^ lrow) * 16;
    const int rounds = max(1, (K + kWin * S - 1) / (kWin * S));  // every load issued is used
    const int windows = rounds * S, first = first_window(K, windows);
    auto load = [&](int round, uint4* slot) {
        const int k = window_of(round * S + wave, first, windows) * kWin + kpos;
        const uint32_t at = k < K ? (uint32_t)lrow * K + k : kPastEnd;
#pragma unroll
        for (int i = 0; i < 16 * RT / kRows; ++i)
            load_to_lds<kStream>(rw, slot + i * kWave, at + (uint32_t)(i * kRows * K));
#pragma unroll
        for (int i = 0; i < 16 * MT / kRows; ++i)
            load_to_lds<kCached>(rx, slot + 16 * RT * P + i * kWave, at + (uint32_t)(i * kRows * K));
    };
    auto multiply = [&](const uint4* slot) {
#pragma unroll
        for (int t = 0; t < kWin / 64; ++t) {
            const int p = (t * 4 + grp) ^ (row & 7);
            uint4 w[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) w[i] = slot[(i * 16 + row) * P + p];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const uint4 x = slot[((RT + j) * 16 + row) * P + p];
#pragma unroll
                for (int i = 0; i < RT; ++i) acc[i][j] = mfma16(w[i], x, acc[i][j]);
            }
        }
    };
    load(0, slot0[wave]);
    load(1, slot1[wave]);
    if constexpr (D > 2) load(2, slot2[wave]), load(3, slot3[wave]);
    for (int r = 0; r < rounds; r += D) {
        const bool more = r + D < rounds;
        multiply(slot0[wave]);
        if (more) reads_done(), load(r + D, slot0[wave]);
        multiply(slot1[wave]);
        if (more) reads_done(), load(r + D + 1, slot1[wave]);
        if constexpr (D > 2) {
            multiply(slot2[wave]);
            if (more) reads_done(), load(r + D + 2, slot2[wave]);
            multiply(slot3[wave]);
            if (more) reads_done(), load(r + D + 3, slot3[wave]);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            slot0[wave][(i * MT + j) * kWave + lane] = __builtin_bit_cast(uint4, acc[i][j]);
    __syncthreads();
    finish_team<S, RT, MT>(slot0[0], kSlot, M, N, n0, ep);
}

// The same for a few rows of x and very wide W (many workgroups a compute
// unit): x goes straight to the operand registers, which leaves the LDS to W,
// in 256-code windows, and twice as many workgroups resident.  (The waits before
// a slot is read cover W of the refill just requested here too.)  1 x 36864 x
// 7168 takes 43.0 us against 45.9 with x in LDS, 1 x 12304 x 2064 8.8 against
// 10.7; at 4096 x 7168 the other form is faster, 8.6 against 9.3.
template <int S>
__global__ __launch_bounds__(S* kWave) void int8_wide_kernel(const int8_t* __restrict__ xq,
                                                             const int8_t* __restrict__ wq, int M,
                                                             int N, int K, Int8Epilogue ep) {
    constexpr int kWin = 256;
    __shared__ uint4 slot0[S][kWin], slot1[S][kWin];
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id_in_block();
    const int row = lane & 15, grp = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const rsrc_t rw = make_rsrc(wq + (int64_t)n0 * K, (uint32_t)min(16, N - n0) * (uint32_t)K);
    const rsrc_t rx = make_rsrc(xq, (uint32_t)M * (uint32_t)K);

    i32x4_t acc = {0, 0, 0, 0};
    uint4 x0[4], x1[4];
    const int rounds = max(1, (K + kWin * S - 1) / (kWin * S));  // every load issued is used
    const int windows = rounds * S, first = first_window(K, windows);
    auto load = [&](int round, uint4* slot, uint4 (&x)[4]) {
        const int k = window_of(round * S + wave, first, windows) * kWin;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 4 rows x 256 bytes, piece p of row r at place p ^ r
            const int r = 4 * i + grp, kk = k + ((row ^ r) * 16);
            load_to_lds<kStream>(rw, slot + i * kWave, kk < K ? (uint32_t)r * K + kk : kPastEnd);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int kk = k + t * 64 + grp * 16;
            x[t] = load16(rx, kk < K ? (uint32_t)row * K + kk : kPastEnd);
        }
    };
    auto multiply = [&](const uint4* slot, const uint4 (&x)[4]) {
#pragma unroll
        for (int t = 0; t < 4; ++t) acc = mfma16(slot[row * 16 + ((t * 4 + grp) ^ row)], x[t], acc);
    };
    load(0, slot0[wave], x0);
    load(1, slot1[wave], x1);
    for (int r = 0; r < rounds; r += 2) {
        const bool more = r + 2 < rounds;
        multiply(slot0[wave], x0);
        if (more) reads_done(), load(r + 2, slot0[wave], x0);
        multiply(slot1[wave], x1);
        if (more) reads_done(), load(r + 3, slot1[wave], x1);
    }
    slot0[wave][lane] = __builtin_bit_cast(uint4, acc);
    __syncthreads();
    finish_team<S, 1, 1>(slot0[0], kWin, M, N, n0, ep);
}

// ---------------------------------------------------------------- tile kernel

// Schedules one step: FM + FN LDS reads (the next step's operands) and LOADS
// loads of a later stage, spread over the FM * FN products of this step.
template <int I, int FM, int FN, int LOADS>
__device__ __forceinline__ void interleave() {
    if constexpr (I < FM) {
        constexpr int kReads = (FM + FN) * (I + 1) / FM - (FM + FN) * I / FM;
        constexpr int kLoads = LOADS * (I + 1) / FM - LOADS * I / FM;
        if constexpr (kLoads > 0) __builtin_amdgcn_sched_group_barrier(0x10, kLoads, 0);  // loads
        __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);  // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x8, FN, 0);        // matrix instructions
        interleave<I + 1, FM, FN, LOADS>();
    }
}

enum TileOut { kTileFinal, kTilePartial, kTileGated };

// A stage is 128 codes of K: a whole line of every row, two matrix steps.
constexpr int kStageK = 128;
constexpr int kPieces = kStageK / 16;     // 16-byte pieces of a row
constexpr int kRowsPerLoad = 1024 / kStageK;  // a load instruction is 1 KB

// Geometry of a tile variant: WM x WN waves, each FM 16-row tiles of x times FN
// of W; NB stage buffers.  (More buffers for the small tiles, up to 8, changed
// nothing: 61 x 4096 x 7168 11.6 to 12.0 us.)
template <int WM_, int WN_, int FM_, int FN_, int NB_>
struct TileShape {
    static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_, NB = NB_;
    static constexpr int W = WM * WN, BM = WM * FM * 16, BN = WN * FN * 16;
    static constexpr int LX = BM / kRowsPerLoad / W, LW = BN / kRowsPerLoad / W;
    static_assert(LX * kRowsPerLoad * W == BM && LW * kRowsPerLoad * W == BN, "whole loads a wave");
    static_assert(NB >= 2 && NB <= 4, "two to four stage buffers");
    static constexpr int kStage = (BM + BN) * kPieces;  // 16-byte pieces
};

template <class T, int OUT>
__global__ __launch_bounds__(T::W* kWave, T::W == 8 ? 2 : 1) void int8_tile_kernel(
    const int8_t* __restrict__ xq, const int8_t* __restrict__ wq, int M, int N, int K, int tiles,
    int per_xcd, int group, int kc, int32_t* partial, Int8Epilogue ep) {
    constexpr int BM = T::BM, BN = T::BN, NB = T::NB, FM = T::FM, FN = T::FN, P = kPieces;
    // An array for each stage buffer: the compiler then knows that a load into one
    // of them does not delay reads of another.
    __shared__ uint4 b0[T::kStage], b1[T::kStage], b2[NB > 2 ? T::kStage : 1],
        b3[NB > 3 ? T::kStage : 1];
    auto buffer = [&](auto i) -> uint4* {
        constexpr int I = decltype(i)::value % NB;
        if constexpr (I == 0) return b0;
        if constexpr (I == 1) return b1;
        if constexpr (I == 2) return b2;
        if constexpr (I == 3) return b3;
    };
    __shared__ float sx[BM];
    __shared__ __attribute__((aligned(16))) float sw[BN];  // read four at a time
    __shared__ uint32_t touched[T::W][kWave];  // where the touching loads land; never read
    // Workgroups reach the 8 XCDs in turn: each XCD takes a run of consecutive
    // tiles, and a run goes down `group` tiles of x before the next tile of W,
    // so the tiles in flight on an XCD share rows of both through its L2.
    const int t = (blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;
    if (t >= tiles) return;
    // a gated tile is BN / 2 outputs wide: 16 gate rows, then their 16 up rows
    constexpr int BC = OUT == kTileGated ? BN / 2 : BN;
    const int nn = (N + BC - 1) / BC, nm = (M + BM - 1) / BM;
    const int first = t / (group * nn) * group, in = t - first * nn;
    const int rows = min(group, nm - first);
    const int m0 = (first + in % rows) * BM, n0 = in / rows * BC;
    const int kbeg = blockIdx.y * kc, kend = min(K, kbeg + kc);

    const int lane = threadIdx.x & (kWave - 1), w = wave_id_in_block();
    const rsrc_t rx = make_rsrc(xq + (int64_t)m0 * K, (uint32_t)min(BM, M - m0) * (uint32_t)K);
    const uint32_t wbytes = (uint32_t)min(BC, N - n0) * (uint32_t)K;
    const rsrc_t rw = make_rsrc(wq + (int64_t)n0 * K, wbytes);
    const rsrc_t ru = make_rsrc(wq + ((int64_t)n0 + (OUT == kTileGated ? ep.up : 0)) * K, wbytes);
    if constexpr (OUT != kTilePartial) {
        for (int i = threadIdx.x; i < BM; i += T::W * kWave) sx[i] = m0 + i < M ? ep.xs[m0 + i] : 0.0f;
        for (int i = threadIdx.x; i < BN; i += T::W * kWave) {
            if constexpr (OUT == kTileGated) {
                const int c = n0 + i / 32 * 16 + i % 16;
                sw[i] = c < N ? ep.ws[c + (i % 32 >= 16 ? ep.up : 0)] : 0.0f;
            } else {
                sw[i] = n0 + i < N ? ep.ws[n0 + i] : 0.0f;
            }
        }
    }
    // Piece p of row r sits at place p ^ (r % 8) of the row: 8 neighbouring rows
    // of one piece meet every bank once.
    const int lrow = lane / P, kpos = ((lane % P) ^ lrow) * 16;
    const uint32_t lbase = (uint32_t)lrow * K + kpos + kbeg;
    const int klen = kend - kbeg - kpos;
    // this lane's offset plus a scalar one for each load; past kend the lane reads zeros
    auto issue = [&](uint4* b, int k0) {
        const uint32_t base = k0 < klen ? lbase : kPastEnd;
#pragma unroll
        for (int i = 0; i < T::LX; ++i) {
            const int r = (w * T::LX + i) * kRowsPerLoad;
            load_to_lds<kCached>(rx, b + r * P, base + (uint32_t)(r * K + k0));
        }
#pragma unroll
        for (int i = 0; i < T::LW; ++i) {
            const int r = (w * T::LW + i) * kRowsPerLoad;
            const bool up = OUT == kTileGated && r % 32 >= 16;
            const int src = OUT == kTileGated ? r / 32 * 16 + r % 16 : r;
            load_to_lds<kCached>(up ? ru : rw, b + (BM + r) * P, base + (uint32_t)(src * K + k0));
        }
    };

    // With two buffers a stage is requested only one stage ahead, less than a
    // miss to HBM takes under load.  So every wave also reads one word of some
    // lines of the stage kAhead ahead, which brings them to L2: the workgroups
    // an XCD runs at once share rows (kShareW tiles of x along a tile of W,
    // kShareX the other way) and touch one part each; where fewer tiles share
    // (the last of 6 tiles of x stand in a group of 2), the other parts are not
    // touched.  On inputs larger than the
    // caches 8192 x 8192 x 7168 takes 359 against 383 us without, 1536 x 7168 x
    // 18432 183 against 219; with three or four buffers it cost 5 to 10 %.
    constexpr bool kTouch = NB == 2;
    constexpr int kAhead = 4, kShareX = 8, kShareW = 4, kTouches = kTouch ? 2 : 0;
    constexpr int kLinesX = BM / kShareX / T::W, kLinesW = BN / kShareW / T::W;  // a wave's
    const int line_x = (n0 / BC % kShareX * T::W + w) * kLinesX;
    const int line_w = (m0 / BM % kShareW * T::W + w) * kLinesW;
    const bool up_lines = OUT == kTileGated && line_w >= BC;
    const uint32_t tx = lane < kLinesX ? (uint32_t)(line_x + lane) * K + kbeg : kPastEnd;
    const uint32_t tw =
        lane < kLinesW ? (uint32_t)(line_w - (up_lines ? BC : 0) + lane) * K + kbeg : kPastEnd;
    auto touch = [&](int stage) {
        if constexpr (kTouch) {
            const int k0 = (stage + kAhead) * kStageK;
            const bool ok = k0 < kend - kbeg;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(up_lines ? ru : rw, (lds_void_t*)touched[w], 4,
                                                     (int)(ok ? tw + k0 : kPastEnd), 0, 0, kCached);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)touched[w], 4,
                                                     (int)(ok ? tx + k0 : kPastEnd), 0, 0, kCached);
        }
    };

    i32x4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
    const int row = lane & 15, grp = lane >> 4, wm = w / T::WN, wn = w % T::WN;
    const int xbase = (wm * FM * 16 + row) * P, wbase = (BM + wn * FN * 16 + row) * P;
    uint4 fw[2][FN], fx[2][FM];
    auto read = [&](const uint4* b, auto step, auto reg) {
        constexpr int R = decltype(reg)::value;
        const int p = (decltype(step)::value * 4 + grp) ^ (row & 7);
#pragma unroll
        for (int i = 0; i < FN; ++i) fw[R][i] = b[wbase + i * 16 * P + p];
#pragma unroll
        for (int j = 0; j < FM; ++j) fx[R][j] = b[xbase + j * 16 * P + p];
    };
    auto multiply = [&](auto reg) {
        constexpr int R = decltype(reg)::value;
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int i = 0; i < FN; ++i) acc[i][j] = mfma16(fw[R][i], fx[R][j], acc[i][j]);
    };
    std::integral_constant<int, 0> c0;
    std::integral_constant<int, 1> c1;

    // Stage s: wait until it has landed for every wave, refill the buffer of
    // stage s - 1 (all its reads are done) with stage s + NB - 1, read its
    // operands while the previous step's products run.  (Loads return in order:
    // the touching loads of a stage are behind its refill and may be out yet.)
    constexpr int kLoads = T::LX + T::LW, kOut = (NB - 2) * kLoads + kTouches;
    const int n = max(1, (kend - kbeg + kStageK - 1) / kStageK);
    auto stage = [&](auto i, int s) {  // s % NB == i
        constexpr int I = decltype(i)::value;
        const uint4* b = buffer(i);
        wait_and_barrier<kOut>();
        issue(buffer(std::integral_constant<int, I + NB - 1>{}), (s + NB - 1) * kStageK);
        touch(s);
        read(b, c0, c0);
        multiply(c1);
        interleave<0, FM, FN, kLoads + kTouches>();
        read(b, c1, c1);
        multiply(c0);
        interleave<0, FM, FN, 0>();
    };
    // stage 0: no products before it
    unrolled<0, NB - 1>([&](auto i) {
        issue(buffer(i), decltype(i)::value * kStageK);
        if constexpr (decltype(i)::value == 0) touch(-1);
    });
    wait_and_barrier<kOut>();
    issue(buffer(std::integral_constant<int, NB - 1>{}), (NB - 1) * kStageK);
    touch(0);
    read(b0, c0, c0);
    read(b0, c1, c1);
    multiply(c0);
    int s = 1;
    for (; s + NB <= n; s += NB)
        unrolled<1, NB + 1>([&](auto i) {
            constexpr int I = decltype(i)::value;
            stage(std::integral_constant<int, I % NB>{}, s + I - 1);
        });
    unrolled<1, NB>([&](auto i) {
        constexpr int I = decltype(i)::value;
        if (s + I - 1 < n) stage(i, s + I - 1);
    });
    multiply(c1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may outlive the workgroup's LDS

    if constexpr (OUT == kTilePartial) {
        int32_t* out = partial + ((int64_t)blockIdx.y * tiles + t) * (BM * BN);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
                if (m0 + (wm * FM + j) * 16 < M)
                    reinterpret_cast<i32x4_t*>(out)[((w * FN + i) * FM + j) * kWave + lane] = acc[i][j];
    } else {
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int ml = (wm * FM + j) * 16 + row, m = m0 + ml;
            if (m >= M) continue;
            const float xs = sx[ml];
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const int nl = (wn * FN + i) * 16 + grp * 4;
                const float4 s = *reinterpret_cast<const float4*>(&sw[nl]);
                float y[4];
                if constexpr (OUT == kTileGated) {
                    if (i % 2) continue;
                    const int c = n0 + nl / 32 * 16 + nl % 16;
                    if (c >= N) continue;
                    float u[4];
                    scale4(acc[i][j], s, xs, y);
                    scale4(acc[i + 1][j], *reinterpret_cast<const float4*>(&sw[nl + 16]), xs, u);
#pragma unroll
                    for (int v = 0; v < 4; ++v) y[v] = gated_product(y[v], u[v]);
                    *reinterpret_cast<float4*>(ep.y_f32 + (int64_t)m * ep.ld + c) =
                        make_float4(y[0], y[1], y[2], y[3]);
                } else {
                    if (n0 + nl >= N) continue;
                    scale4(acc[i][j], s, xs, y);
                    finish4(ep, N, m, n0 + nl, y);
                }
            }
        }
    }
}

// Sums the S partial tiles of int8_tile_kernel<T, kTilePartial> and finishes the
// outputs; a thread owns the four neighbours a lane of the tile kernel held.
template <class T>
__global__ __launch_bounds__(kBlock) void int8_reduce_kernel(const int32_t* __restrict__ partial,
                                                             int M, int N, int tiles, int group,
                                                             int S, Int8Epilogue ep) {
    constexpr int BM = T::BM, BN = T::BN, FM = T::FM, FN = T::FN;
    constexpr int kFrags = T::W * FM * FN;  // 16 x 16 blocks of a tile
    const int64_t e = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    const int t = (int)(e / (kFrags * kWave)), f = (int)(e / kWave) % kFrags, lane = (int)e & 63;
    if (t >= tiles) return;
    const int nn = (N + BN - 1) / BN, nm = (M + BM - 1) / BM;
    const int first = t / (group * nn) * group, in = t - first * nn;
    const int rows = min(group, nm - first);
    const int m0 = (first + in % rows) * BM, n0 = in / rows * BN;
    const int w = f / (FM * FN), i = f / FM % FN, j = f % FM;
    const int m = m0 + ((w / T::WN) * FM + j) * 16 + (lane & 15);
    const int n = n0 + ((w % T::WN) * FN + i) * 16 + (lane >> 4) * 4;
    if (m >= M || n >= N) return;
    const i32x4_t* p = reinterpret_cast<const i32x4_t*>(partial) +
                       ((int64_t)t * kFrags + f) * kWave + lane;
    const int64_t step = (int64_t)tiles * (BM * BN / 4);
    i32x4_t a = {0, 0, 0, 0};
    int s = 0;
    for (; s + 4 <= S; s += 4) {
        const i32x4_t q0 = p[s * step], q1 = p[(s + 1) * step], q2 = p[(s + 2) * step],
                      q3 = p[(s + 3) * step];
        a += (q0 + q1) + (q2 + q3);
    }
    for (; s < S; ++s) a += p[s * step];
    float y[4];
    scale4(a, channel_scales(ep.ws, N, n), ep.xs[m], y);
    finish4(ep, N, m, n, y);
}

template <class T, int OUT>
void launch_tile(int M, int N, int K, int S, int kc, int group, const int8_t* xq, const int8_t* wq,
                 int32_t* partial, const Int8Epilogue& ep, hipStream_t stream) {
    constexpr int BC = OUT == kTileGated ? T::BN / 2 : T::BN;
    const int tiles = ((M + T::BM - 1) / T::BM) * ((N + BC - 1) / BC);
    const int per = (tiles + kXcds - 1) / kXcds;
    hipLaunchKernelGGL((int8_tile_kernel<T, OUT>), dim3(per * kXcds, S), dim3(T::W * kWave), 0,
                       stream, xq, wq, M, N, K, tiles, per, group, kc, partial, ep);
}

template <class T>
void launch_split(int M, int N, int K, int S, int kc, int group, const int8_t* xq, const int8_t* wq,
                  void* ws, const Int8Epilogue& ep, hipStream_t stream) {
    int32_t* partial = static_cast<int32_t*>(ws);
    if (S <= 1) {
        launch_tile<T, kTileFinal>(M, N, K, 1, K, group, xq, wq, nullptr, ep, stream);
        return;
    }
    launch_tile<T, kTilePartial>(M, N, K, S, kc, group, xq, wq, partial, ep, stream);
    const int tiles = ((M + T::BM - 1) / T::BM) * ((N + T::BN - 1) / T::BN);
    const int64_t threads = (int64_t)tiles * (T::BM * T::BN / 4);
    hipLaunchKernelGGL((int8_reduce_kernel<T>), dim3((uint32_t)((threads + kBlock - 1) / kBlock)),
                       dim3(kBlock), 0, stream, partial, M, N, tiles, group, S, ep);
}

template <int S, int RT, int MT, int D>
void launch_team(int M, int N, int K, const int8_t* xq, const int8_t* wq, const Int8Epilogue& ep,
                 hipStream_t stream) {
    hipLaunchKernelGGL((int8_team_kernel<S, RT, MT, D>), dim3((N + 16 * RT - 1) / (16 * RT)),
                       dim3(S * kWave), 0, stream, xq, wq, M, N, K, ep);
}

// The team kernel for MT 16-row tiles of x, in the forms whose slots fit in LDS.
template <int MT>
void launch_team(int waves, int rt, int slots, int M, int N, int K, const int8_t* xq,
                 const int8_t* wq, const Int8Epilogue& ep, hipStream_t stream) {
    if constexpr (MT <= 3)
        if (rt == 2) return launch_team<8, 2, MT, 2>(M, N, K, xq, wq, ep, stream);
    if constexpr (MT == 1)
        if (slots == 4) return launch_team<8, 1, 1, 4>(M, N, K, xq, wq, ep, stream);
    if (waves == 4)
        launch_team<4, 1, MT, 2>(M, N, K, xq, wq, ep, stream);
    else
        launch_team<8, 1, MT, 2>(M, N, K, xq, wq, ep, stream);
}

// ---------------------------------------------------------------- choice

// Tile variants, BM x BN: 256 x 256, 128 x 256, 128 x 128, 64 x 128, 64 x 64.
typedef TileShape<2, 4, 8, 4, 2> Tile256;
typedef TileShape<2, 4, 4, 4, 3> Tile128w;
typedef TileShape<2, 4, 4, 2, 4> Tile128;
typedef TileShape<2, 2, 2, 4, 3> Tile64w;
typedef TileShape<2, 2, 2, 2, 4> Tile64;

template <class F>
void with_tile(int v, F f) {
    switch (v) {
        case 0: f(Tile256{}); break;
        case 1: f(Tile128w{}); break;
        case 2: f(Tile128{}); break;
        case 3: f(Tile64w{}); break;
        default: f(Tile64{}); break;
    }
}

struct TileCost {
    int bm, bn;
    int per_cu;      // workgroups a compute unit holds
    int group;       // tiles of x an XCD's run goes down before the next tile of W
    double full;     // ns per code of K of a round that fills every compute unit
    double single;   // of a round with at most one workgroup a compute unit
};
// Measured on MI355X (full: 8192 x 8192 x 7168 and 1024..2048 x 4096 x 4096;
// single: rounds of 64 to 256 tiles).
constexpr TileCost kTiles[] = {{256, 256, 1, 4, 12.0, 9.9},
                               {128, 256, 1, 8, 7.2, 6.2},
                               {128, 128, 1, 8, 4.1, 3.9},
                               {64, 128, 2, 8, 6.4, 3.6},
                               {64, 64, 2, 8, 4.1, 2.6}};
constexpr int kTileVariants = 5;
constexpr int kCus = 256;
constexpr int kTeamMaxM = 64;
constexpr double kStreamBytesPerUs = 5.6e6;  // W from HBM through the tile kernel

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// The variant with the least estimated time (us).  Team: 2 us, then 0.038 us
// per KB of W and 0.012 (0.016 past 48 rows) per KB of x that a compute unit
// takes in.  Tiles: 3 us, then rounds of workgroups at the measured cost per
// code, but no faster than W comes from HBM; a split adds the reduction's
// launch and its traffic.  Against every other form at 100 sizes drawn from 1 to
// 4096 rows, 16 to 40000 channels and 64 to 18432 codes the choice takes 4 %
// longer than the fastest on average, and by more than a tenth for 15.  Those
// are wide products of 10 to 30 rows, where the team estimate has no rounds and
// too little for x (13 x 28653 x 3488 27.6 us, 22.0 in tiles; 11 x 35161 x 528
// 13.5, 8.4 with 16 rows of W a workgroup), few rows and short K on the wide
// kernel (7 x 15100 x 112 4.7, 3.6 in tiles), and sizes just past a round of
// tiles (1177 x 2411 x 14672 100.8, 73.6 in large tiles split four ways).
Int8Plan int8_plan(int M, int N, int K) {
    Int8Plan best{};
    double least = 1e30;
    if (M <= kTeamMaxM) {
        for (int rt = 1; rt <= (M <= 48 ? 2 : 1); ++rt) {
            const double wgs = (double)ceil_div(N, 16 * rt);
            const double per = wgs > kCus ? wgs / kCus : 1.0;
            const double x = M <= 48 ? 0.012 : 0.016;
            double est = 2.0 + per * K * (0.038 * 16 * rt + x * M) / 1000.0;
            // two row tiles: idle compute units where they do not fill the GPU; at pitches
            // of a multiple of 4 KB faster (16 x 8192 x 8192 12.2 us, one tile 13.9)
            if (rt == 2) est *= K % 4096 == 0 ? 0.88 : wgs < kCus ? 1.04 : 1.0;
            if (est < least) {
                least = est;
                // 4 slots where a workgroup has a compute unit to itself; 4 waves where
                // 8 would have one window each
                best = Int8Plan{Int8Plan::kTeam, K <= 1024 ? 4 : 8, rt,
                                rt == 1 && M <= 16 && wgs <= kCus && K >= 4096 ? 4 : 2, 0, 1, K, 0, 0, 0};
            }
        }
        // The wide kernel against the team kernel of 16 and 32 rows, M = 1 / 8:
        //   6160 x 2064     6.1 / 6.5 us   against  6.4 / 6.9 and  6.5 / 6.8
        //   12304 x 2064    8.8 / 9.5              10.7 / 11.4    11.2 / 11.4
        //   8208 x 4096     8.6 / 9.5               9.4 / 9.6     10.1 / 10.1
        //   16400 x 7168   22.2 / 23.7             23.6 / 24.6    24.9 / 25.1
        //   36864 x 7168   43.0 / 45.7             45.9 / 49.0    47.3 / 48.0
        // and outside the rule:
        //   4096 x 4096     5.7 / 6.0               5.6 / 5.6      6.1 / 6.8
        //   6160 x 7168    10.5 / 11.9             10.4 / 11.4    10.4 / 10.6
        // It is not the fastest at 6160 x 4096 with 8 rows (8.2 against 7.1) and
        // would be between 8208 and 16400 rows of W past K = 4096 (12304 x 7168
        // 18.2 / 19.5 against 19.8 / 20.4 as planned).  The estimate that the
        // tiles below are held against stays the team kernel's.
        const int64_t wgs = ceil_div(N, 16);
        if (M <= 8 && (wgs > 4 * kCus || (wgs > 1.5 * kCus && K <= 4096)))
            best.kind = Int8Plan::kWide;
    }
    const double stream = (double)N * K / kStreamBytesPerUs;
    // us of rounds of tiles over n columns, kc codes each
    auto tiles_us = [&](int v, int64_t n, int S, int kc) {
        const TileCost& c = kTiles[v];
        const int64_t wgs = ceil_div(M, c.bm) * ceil_div(n, c.bn) * S, slots = (int64_t)kCus * c.per_cu;
        const int64_t rem = wgs % slots;
        return kc * (wgs / slots * c.full + (rem == 0 ? 0.0 : rem <= kCus ? c.single : c.full)) / 1000.0;
    };
    for (int v = 0; v < kTileVariants; ++v) {
        const TileCost& c = kTiles[v];
        const int64_t tiles = ceil_div(M, c.bm) * ceil_div(N, c.bn);
        for (int S = 1; S <= 16; ++S) {
            const int kc = S == 1 ? K : (int)ceil_div(ceil_div(K, S), kStageK) * kStageK;
            if (S > 1 && (kc < 4 * kStageK || (int64_t)(S - 1) * kc >= K)) break;
            double est = tiles_us(v, N, S, kc);
            est = 3.0 + (est > stream ? est : stream);
            const size_t ws = S > 1 ? (size_t)S * tiles * c.bm * c.bn * 4 : 0;
            if (S > 1) est += 3.0 + 8.0 * S * M * N / 4.0e6;
            if (est < least && ws <= ((size_t)1 << 30)) {
                least = est;
                best = Int8Plan{Int8Plan::kTile, 0, 0, 0, v, S, kc, ws, 0, 0};
            }
        }
    }
    // Whole rounds of the largest tiles, then a second launch over the columns
    // that would leave most of the GPU idle in a last round of theirs: 1000 x
    // 36864 x 7168 227 us against 254 in one launch, 5000 x 4096 x 4096 79
    // against 89, 1501 x 36864 x 7168 339 against 350.
    const TileCost& big = kTiles[0];
    const int64_t rounds = ceil_div(M, big.bm) * ceil_div(N, big.bn) / kCus;
    const int64_t cols = rounds * kCus / ceil_div(M, big.bm) * big.bn;
    if (rounds >= 1 && cols > 0 && cols < N)
        for (int v = 1; v < kTileVariants; ++v) {
            const double est = 6.0 + tiles_us(0, cols, 1, K) + tiles_us(v, N - cols, 1, K);
            if (est < least) {
                least = est;
                best = Int8Plan{Int8Plan::kTile, 0, 0, 0, 0, 1, K, 0, (int)cols, v};
            }
        }
    return best;
}

// The outputs and weights from column `cols` on.
static Int8Epilogue columns_from(const Int8Epilogue& ep, int cols) {
    Int8Epilogue e = ep;
    e.ws += cols;
    if (e.y_f32) e.y_f32 += cols;
    if (e.y_bf16) e.y_bf16 += cols;
    if (e.r) e.r += cols;
    return e;
}

hipError_t launch_gemm_int8(const Int8Plan& p, int M, int N, int K, const int8_t* xq,
                            const int8_t* wq, const Int8Epilogue& epilogue, void* ws,
                            hipStream_t stream) {
    Int8Epilogue ep = epilogue;
    ep.ld = N;
    if (p.kind == Int8Plan::kWide) {
        hipLaunchKernelGGL((int8_wide_kernel<4>), dim3((N + 15) / 16), dim3(4 * kWave), 0, stream, xq,
                           wq, M, N, K, ep);
    } else if (p.kind == Int8Plan::kTeam) {
        auto go = [&](auto mt) {
            launch_team<decltype(mt)::value>(p.waves, p.rt, p.slots, M, N, K, xq, wq, ep, stream);
        };
        if (M <= 16)
            go(std::integral_constant<int, 1>{});
        else if (M <= 32)
            go(std::integral_constant<int, 2>{});
        else if (M <= 48)
            go(std::integral_constant<int, 3>{});
        else
            go(std::integral_constant<int, 4>{});
    } else if (p.cols > 0) {
        launch_tile<Tile256, kTileFinal>(M, p.cols, K, 1, K, kTiles[0].group, xq, wq, nullptr, ep,
                                         stream);
        with_tile(p.rest, [&](auto shape) {
            launch_tile<decltype(shape), kTileFinal>(M, N - p.cols, K, 1, K, kTiles[p.rest].group, xq,
                                                     wq + (int64_t)p.cols * K, nullptr,
                                                     columns_from(ep, p.cols), stream);
        });
    } else {
        with_tile(p.tile, [&](auto shape) {
            launch_split<decltype(shape)>(M, N, K, p.S, p.kc, kTiles[p.tile].group, xq, wq, ws, ep,
                                          stream);
        });
    }
    return hipGetLastError();
}

bool int8_gated_ok(const Int8Plan& p) { return p.kind == Int8Plan::kTile && p.S == 1; }

hipError_t launch_gated_int8(const Int8Plan& p, int M, int F, int H, const int8_t* xq,
                             const int8_t* wq, const Int8Epilogue& epilogue, hipStream_t stream) {
    Int8Epilogue ep = epilogue;
    ep.ld = ep.up = F;
    const int half = p.cols / 2;  // gated tiles are half as wide in outputs
    with_tile(p.tile, [&](auto shape) {
        launch_tile<decltype(shape), kTileGated>(M, half > 0 ? half : F, H, 1, H, kTiles[p.tile].group,
                                                 xq, wq, nullptr, ep, stream);
    });
    if (half > 0)
        with_tile(p.rest, [&](auto shape) {
            launch_tile<decltype(shape), kTileGated>(M, F - half, H, 1, H, kTiles[p.rest].group, xq,
                                                     wq + (int64_t)half * H, nullptr,
                                                     columns_from(ep, half), stream);
        });
    return hipGetLastError();
}

}  // namespace sg
