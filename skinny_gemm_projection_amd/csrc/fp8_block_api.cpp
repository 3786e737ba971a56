// fp8_block_api.cpp -- the C ABI of the block-scaled FP8 operators and of the
// sort of tokens by expert (declared in include/skinny_gemm.h): argument checks,
// launches and launch counts, and the experts' step composed of them.  As for
// every other entry point, what the host can see is refused before anything is
// launched, and an accepted call only enqueues kernels on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>

#include "launch.h"
#include "plan_internal.h"
#include "skinny_gemm.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool gemm_sizes_ok(int32_t M, int32_t N, int32_t K) {
    return M >= 0 && M <= SG_INT8_MAX_M && N >= 0 && N <= (1 << 20) && K >= 0 && K <= SG_FP8_MAX_K;
}

bool pairs_ok(int32_t T, int32_t topk) {
    return T >= 0 && topk >= 1 && topk <= SG_MOE_MAX_TOPK && (int64_t)T * topk <= SG_MOE_MAX_PAIRS;
}

bool experts_ok(int32_t E) { return E >= 1 && E <= SG_MOE_MAX_EXPERTS; }

bool rows_ok(int32_t T, int32_t topk, int32_t K, int32_t f32) {
    return pairs_ok(T, topk) && K >= 1 && K <= SG_ROW_MAX_K && (f32 == 0 || f32 == 1);
}

int64_t pitch_of(int32_t K, int32_t f32) { return (int64_t)K * (f32 ? 4 : 2); }

// One counted and logged launch group; e is what its launcher returned.
sg_status done(hipError_t e, int kernel, int launches, const char* what, int a, int b, int c) {
    if (e != hipSuccess) return SG_ERR_HIP;
    for (int i = 0; i < launches; ++i) sg::count_launch(kernel);
    if (sg::launch_log_enabled())
        std::fprintf(stderr, "[skinny_gemm] %s %d %d %d launches=%d\n", what, a, b, c, launches);
    return SG_OK;
}

sg_status quant(int32_t M, int32_t K, const void* x, bool f32, bool gated, uint8_t* codes,
                float* scales, hipStream_t stream) {
    (void)hipGetLastError();
    return done(sg::launch_quant_fp8(M, K, x, f32, gated, codes, scales, stream), SG_KERNEL_QUANT_FP8,
                1, gated ? "quant_fp8 gated" : "quant_fp8", M, K, f32);
}

sg_status sort(int32_t T, int32_t topk, int32_t E, const int32_t* ids, int32_t* offsets,
               int32_t* sorted, int32_t* positions, void* ws, hipStream_t stream) {
    (void)hipGetLastError();
    const int32_t P = T * topk;
    return done(sg::launch_moe_sort(ids, P, E, offsets, sorted, positions, ws, stream),
                SG_KERNEL_MOE_SORT, sg::moe_sort_launches(P, E), "moe_sort", T, topk, E);
}

sg_status product(const sg::Fp8BlockPlan& plan, const sg::Fp8Product& a, void* ws,
                  hipStream_t stream) {
    (void)hipGetLastError();
    const sg_status st = done(sg::launch_fp8_block(plan, a, ws, stream), SG_KERNEL_FP8_BLOCK, 1,
                              a.offsets ? "fp8_block by expert" : "fp8_block", a.M, a.N, a.K);
    if (st == SG_OK && plan.workspace > 0) sg::count_launch(SG_KERNEL_REDUCE);
    return st;
}

// Byte offsets of the experts' step's intermediates in its workspace.
struct StepLayout {
    size_t q, sq, offsets, sorted, positions, sort, u, p, sp, y, total;
    sg::Fp8BlockPlan up, down;
    bool gated;  // the first product gives the gated product's codes itself
};

bool step_layout(int32_t T, int32_t topk, int32_t E, int32_t H, int32_t F, StepLayout* L) {
    if (!pairs_ok(T, topk) || !experts_ok(E) || H < 16 || H > SG_ROW_MAX_K || F < 16 ||
        F > SG_ROW_MAX_K || H % 16 != 0 || F % 16 != 0 || (int64_t)T * H >= ((int64_t)1 << 31))
        return false;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const size_t P = (size_t)T * topk, t = (size_t)T;
    const int rows = P > 0 ? (int)P : 1;
    // What follows is rounded to 4 bits, 2^-4 of a value: the FP8 instruction's sums do (with
    // fp32's the gate and up product of 2003 tokens, 48 experts, takes 1026 us, not 582).
    L->up = sg::fp8_grouped_plan(rows, E, 2 * F, H, false);
    L->gated = sg::fp8_gated_ok(L->up, F);
    L->down = sg::fp8_grouped_plan(rows, E, H, F, false);
    L->q = take(t * H);
    L->sq = take(t * ((H + 127) / 128) * 4);
    L->offsets = take(((size_t)E + 1) * 4);
    L->sorted = take(P * 4);
    L->positions = take(P * 4);
    L->sort = take(sg::moe_sort_workspace_bytes((int64_t)P, E));
    L->u = take(L->gated ? 0 : P * F * 8);
    L->p = take(P * F);
    L->sp = take(P * ((F + 127) / 128) * 4);
    L->y = take(P * H * 4);
    L->total = at;
    return true;
}

}  // namespace

extern "C" {

sg_status skinny_quant_fp8(int32_t M, int32_t K, const sg_bf16* x_bf16, const float* x_f32,
                           int32_t gated, uint8_t* codes, float* scales, void* stream) {
    if (M < 0 || M > SG_INT8_MAX_M || K < 1 || K > SG_FP8_MAX_K || (gated != 0 && gated != 1))
        return SG_ERR_SHAPE;
    if (K % 8 != 0) return SG_ERR_ALIGN;
    if (M == 0) return SG_OK;
    if ((x_bf16 != nullptr) == (x_f32 != nullptr) || !codes || !scales) return SG_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(x_f32, 16) || !aligned(codes, 8) || !aligned(scales, 4))
        return SG_ERR_ALIGN;
    const void* x = x_f32 ? static_cast<const void*>(x_f32) : x_bf16;
    return quant(M, K, x, x_f32 != nullptr, gated != 0, codes, scales,
                 static_cast<hipStream_t>(stream));
}

size_t skinny_gemm_fp8_block_workspace(int32_t M, int32_t N, int32_t K, int32_t with_f32) {
    if (!gemm_sizes_ok(M, N, K) || K % 16 != 0 || M == 0 || N == 0) return 0;
    return sg::fp8_block_plan(M, N, K, with_f32 != 0).workspace;
}

sg_status skinny_gemm_fp8_block(int32_t M, int32_t N, int32_t K, const uint8_t* x_codes,
                                const float* x_scales, const uint8_t* W_codes,
                                const float* W_scales, const sg_bf16* r, float* y_f32,
                                sg_bf16* y_bf16, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (!gemm_sizes_ok(M, N, K)) return SG_ERR_SHAPE;
    if (K % 16 != 0) return SG_ERR_ALIGN;
    if (M == 0 || N == 0) return SG_OK;
    if (!y_f32 && !y_bf16) return SG_ERR_NULL;
    if (K > 0 && (!x_codes || !x_scales || !W_codes || !W_scales)) return SG_ERR_NULL;
    if (!aligned(x_codes, 16) || !aligned(W_codes, 16) || !aligned(x_scales, 4) ||
        !aligned(W_scales, 4) || !aligned(r, 16) || !aligned(y_f32, 16) || !aligned(y_bf16, 16))
        return SG_ERR_ALIGN;
    const sg::Fp8BlockPlan plan = sg::fp8_block_plan(M, N, K, y_f32 != nullptr);
    if (plan.workspace > 0) {
        if (!workspace || workspace_bytes < plan.workspace) return SG_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return SG_ERR_ALIGN;
    }
    sg::Fp8Product a{x_codes, x_scales, W_codes, W_scales, M, N, K, M, y_f32, y_bf16, r};
    return product(plan, a, workspace, static_cast<hipStream_t>(stream));
}

size_t skinny_moe_sort_workspace(int32_t T, int32_t topk, int32_t E) {
    if (!pairs_ok(T, topk) || !experts_ok(E)) return 0;
    return sg::moe_sort_workspace_bytes((int64_t)T * topk, E);
}

sg_status skinny_moe_sort(int32_t T, int32_t topk, int32_t E, const int32_t* topk_ids,
                          int32_t* expert_offsets, int32_t* sorted_pairs, int32_t* positions,
                          void* workspace, size_t workspace_bytes, void* stream) {
    if (!pairs_ok(T, topk) || !experts_ok(E)) return SG_ERR_SHAPE;
    if (!expert_offsets || (T > 0 && (!topk_ids || !positions))) return SG_ERR_NULL;
    if (!aligned(topk_ids, 4) || !aligned(expert_offsets, 4) || !aligned(sorted_pairs, 4) ||
        !aligned(positions, 4))
        return SG_ERR_ALIGN;
    const size_t need = sg::moe_sort_workspace_bytes((int64_t)T * topk, E);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return SG_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return SG_ERR_ALIGN;
    }
    return sort(T, topk, E, topk_ids, expert_offsets, sorted_pairs, positions, workspace,
                static_cast<hipStream_t>(stream));
}

sg_status skinny_moe_gather(int32_t T, int32_t topk, int32_t K, const void* x, int32_t f32,
                            const int32_t* positions, void* rows, void* stream) {
    if (!rows_ok(T, topk, K, f32)) return SG_ERR_SHAPE;
    if (K % 8 != 0) return SG_ERR_ALIGN;
    if (T == 0) return SG_OK;
    if (!x || !positions || !rows) return SG_ERR_NULL;
    if (!aligned(x, 16) || !aligned(rows, 16) || !aligned(positions, 4)) return SG_ERR_ALIGN;
    (void)hipGetLastError();
    return done(sg::launch_moe_gather(x, T, topk, pitch_of(K, f32), positions, rows,
                                      static_cast<hipStream_t>(stream)),
                SG_KERNEL_MOE_ROWS, 1, "moe_gather", T, topk, K);
}

sg_status skinny_moe_combine(int32_t T, int32_t topk, int32_t K, const void* rows, int32_t f32,
                             const int32_t* positions, const float* weights, const void* r,
                             void* out, void* stream) {
    if (!rows_ok(T, topk, K, f32)) return SG_ERR_SHAPE;
    if (K % 8 != 0) return SG_ERR_ALIGN;
    if (T == 0) return SG_OK;
    if (!rows || !positions || !out) return SG_ERR_NULL;
    if (!aligned(rows, 16) || !aligned(r, 16) || !aligned(out, 16) || !aligned(positions, 4) ||
        !aligned(weights, 4))
        return SG_ERR_ALIGN;
    (void)hipGetLastError();
    return done(sg::launch_moe_combine(rows, T, topk, pitch_of(K, f32), f32 != 0, f32 != 0, positions,
                                       weights, r, out, static_cast<hipStream_t>(stream)),
                SG_KERNEL_MOE_ROWS, 1, "moe_combine", T, topk, K);
}

sg_status skinny_moe_combine_grad(int32_t T, int32_t topk, int32_t K, const void* d_out,
                                  const void* rows, int32_t f32, const int32_t* positions,
                                  const float* weights, void* d_rows, float* d_weights,
                                  void* stream) {
    if (!rows_ok(T, topk, K, f32)) return SG_ERR_SHAPE;
    if (K % 8 != 0) return SG_ERR_ALIGN;
    if (T == 0) return SG_OK;
    if (!d_out || !rows || !positions || !weights || !d_rows || !d_weights) return SG_ERR_NULL;
    if (!aligned(d_out, 16) || !aligned(rows, 16) || !aligned(d_rows, 16) || !aligned(positions, 4) ||
        !aligned(weights, 4) || !aligned(d_weights, 4))
        return SG_ERR_ALIGN;
    (void)hipGetLastError();
    return done(sg::launch_moe_combine_grad(d_out, rows, T, topk, pitch_of(K, f32), f32 != 0,
                                            positions, weights, d_rows, d_weights,
                                            static_cast<hipStream_t>(stream)),
                SG_KERNEL_MOE_ROWS, 1, "moe_combine_grad", T, topk, K);
}

sg_status grouped_skinny_gemm_fp8(int32_t rows, int32_t x_rows, int32_t E, int32_t N, int32_t K,
                                  const uint8_t* x_codes, const float* x_scales,
                                  const uint8_t* W_codes, const float* W_scales,
                                  const int32_t* expert_offsets, const int32_t* sorted_pairs,
                                  int32_t topk, float* y_f32, sg_bf16* y_bf16, void* stream) {
    if (rows < 0 || rows > SG_MOE_MAX_PAIRS || x_rows < 0 || x_rows > SG_MOE_MAX_PAIRS ||
        !experts_ok(E) || N < 0 || N > (1 << 20) || K < 0 || K > SG_FP8_MAX_K || topk < 1 ||
        topk > SG_MOE_MAX_TOPK)
        return SG_ERR_SHAPE;
    if (sorted_pairs ? (int64_t)x_rows * K >= ((int64_t)1 << 31) : x_rows != rows) return SG_ERR_SHAPE;
    if (K % 16 != 0) return SG_ERR_ALIGN;
    if (rows == 0 || N == 0) return SG_OK;
    if ((!y_f32 && !y_bf16) || !expert_offsets) return SG_ERR_NULL;
    if (K > 0 && (!W_codes || !W_scales || (x_rows > 0 && (!x_codes || !x_scales)))) return SG_ERR_NULL;
    if (!aligned(x_codes, 16) || !aligned(W_codes, 16) || !aligned(x_scales, 4) ||
        !aligned(W_scales, 4) || !aligned(expert_offsets, 4) || !aligned(sorted_pairs, 4) ||
        !aligned(y_f32, 16) || !aligned(y_bf16, 16))
        return SG_ERR_ALIGN;
    const sg::Fp8BlockPlan plan = sg::fp8_grouped_plan(rows, E, N, K, y_f32 != nullptr);
    sg::Fp8Product a{x_codes, x_scales, W_codes, W_scales, rows, N, K, x_rows, y_f32, y_bf16, nullptr};
    a.offsets = expert_offsets, a.E = E, a.pairs = sorted_pairs, a.topk = topk;
    return product(plan, a, nullptr, static_cast<hipStream_t>(stream));
}

size_t skinny_moe_fp8_step_workspace(int32_t T, int32_t topk, int32_t E, int32_t H, int32_t F) {
    StepLayout L;
    return step_layout(T, topk, E, H, F, &L) ? L.total : 0;
}

sg_status skinny_moe_fp8_step(const sg_moe_fp8_step* a, void* workspace, size_t workspace_bytes,
                              void* stream) {
    if (!a) return SG_ERR_NULL;
    StepLayout L;
    if (!step_layout(a->T, a->topk, a->E, a->H, a->F, &L))
        return a->H > 0 && a->F > 0 && (a->H % 16 != 0 || a->F % 16 != 0) ? SG_ERR_ALIGN
                                                                          : SG_ERR_SHAPE;
    const int32_t T = a->T, topk = a->topk, E = a->E, H = a->H, F = a->F, P = T * topk;
    if (T == 0) return SG_OK;
    // every check of the calls below, made here before the first launch
    if (!a->x || !a->topk_ids || !a->topk_weights || !a->W_gate_up || !a->gate_up_scales ||
        !a->W_down || !a->down_scales || !a->out)
        return SG_ERR_NULL;
    if (!aligned(a->x, 16) || !aligned(a->r, 16) || !aligned(a->out, 16) ||
        !aligned(a->W_gate_up, 16) || !aligned(a->W_down, 16) || !aligned(a->topk_ids, 4) ||
        !aligned(a->topk_weights, 4) || !aligned(a->gate_up_scales, 4) || !aligned(a->down_scales, 4))
        return SG_ERR_ALIGN;
    if (!workspace || workspace_bytes < L.total) return SG_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SG_ERR_ALIGN;

    char* base = static_cast<char*>(workspace);
    uint8_t* q = reinterpret_cast<uint8_t*>(base + L.q);
    float* sq = reinterpret_cast<float*>(base + L.sq);
    int32_t* offsets = reinterpret_cast<int32_t*>(base + L.offsets);
    int32_t* sorted = reinterpret_cast<int32_t*>(base + L.sorted);
    int32_t* positions = reinterpret_cast<int32_t*>(base + L.positions);
    float* u = reinterpret_cast<float*>(base + L.u);
    uint8_t* p = reinterpret_cast<uint8_t*>(base + L.p);
    float* sp = reinterpret_cast<float*>(base + L.sp);
    float* y = reinterpret_cast<float*>(base + L.y);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    sg_status st;
    if ((st = sort(T, topk, E, a->topk_ids, offsets, sorted, positions, base + L.sort, hs)) != SG_OK)
        return st;
    if ((st = quant(T, H, a->x, false, false, q, sq, hs)) != SG_OK) return st;
    sg::Fp8Product up{q, sq, a->W_gate_up, a->gate_up_scales, P, 2 * F, H, T, u, nullptr, nullptr};
    up.offsets = offsets, up.E = E, up.pairs = sorted, up.topk = topk;
    if (L.gated) up.N = F, up.y_f32 = nullptr, up.codes = p, up.scales = sp;
    if ((st = product(L.up, up, nullptr, hs)) != SG_OK) return st;
    if (!L.gated && (st = quant(P, F, u, true, true, p, sp, hs)) != SG_OK) return st;
    // The rows of y stay fp32 up to the weighted sum: rounded to bf16 they put as much error
    // into out as its own rounding does, and all of out where experts cancel.  (Product
    // and sum of 2003 tokens, 48 experts: 446 us, with bf16 rows 370.)
    sg::Fp8Product down{p, sp, a->W_down, a->down_scales, P, H, F, P, y, nullptr, nullptr};
    down.offsets = offsets, down.E = E;
    if ((st = product(L.down, down, nullptr, hs)) != SG_OK) return st;
    (void)hipGetLastError();
    return done(sg::launch_moe_combine(y, T, topk, (int64_t)H * 4, true, false, positions, a->topk_weights,
                                       a->r, a->out, hs),
                SG_KERNEL_MOE_ROWS, 1, "moe_combine", T, topk, H);
}

}  // extern "C"
