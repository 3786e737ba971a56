// int8_api.cpp -- the C ABI of the 8-bit integer operators (declared in
// include/skinny_gemm.h): argument checks, launches and launch counts, and the
// gated MLP step composed of them.  As for every other entry point, what the
// host can see is refused before anything is launched, and an accepted call
// only enqueues kernels on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "launch.h"
#include "plan_internal.h"
#include "skinny_gemm.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Squares below the normal range keep few bits; next to a normal eps that is at
// most 2^-150 / 2^-126, one rounding, next to a smaller one it would show.
bool eps_ok(float eps) { return eps >= std::numeric_limits<float>::min() && std::isfinite(eps); }

bool gemm_sizes_ok(int32_t M, int32_t N, int32_t K) {
    return M >= 0 && M <= SG_INT8_MAX_M && N >= 0 && N <= (1 << 20) && K >= 0 && K <= SG_INT8_MAX_K;
}

bool rows_ok(int32_t M, int32_t K) {
    return M >= 0 && M <= SG_INT8_MAX_M && K >= 1 && K <= SG_ROW_MAX_K;
}

// Byte offsets of the MLP step's intermediates in its workspace.
struct MlpLayout {
    size_t q, sq, u, p, sp, gemm, total;
    sg::Int8Plan up, down;  // the two products
    bool gated;             // the gated product is taken in the first one's epilogue
};

bool mlp_layout(int32_t M, int32_t H, int32_t F, MlpLayout* L) {
    if (M < 0 || M > SG_INT8_MAX_M || H < 16 || H > SG_ROW_MAX_K || F < 16 || F > SG_ROW_MAX_K ||
        H % 16 != 0 || F % 16 != 0)
        return false;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const size_t m = (size_t)M;
    L->q = take(m * H);
    L->sq = take(m * 4);
    // the projections' outputs, or (gated in the epilogue) the gated product alone
    L->up = sg::int8_plan(M > 0 ? M : 1, 2 * F, H);
    L->down = sg::int8_plan(M > 0 ? M : 1, H, F);
    L->gated = sg::int8_gated_ok(L->up);
    L->u = take(m * F * (L->gated ? 4 : 8));
    L->p = take(m * F);
    L->sp = take(m * 4);
    const size_t a = L->up.workspace, b = L->down.workspace;
    L->gemm = take(M == 0 ? 0 : a > b ? a : b);
    L->total = at;
    return true;
}

// The launches of one checked product, counted and logged.
sg_status product(const sg::Int8Plan& p, int32_t M, int32_t N, int32_t K, const int8_t* xq,
                  const float* xs, const int8_t* wq, const float* ws, const sg_bf16* r, float* y_f32,
                  sg_bf16* y_bf16, void* workspace, hipStream_t stream) {
    (void)hipGetLastError();
    const sg::Int8Epilogue ep{xs, ws, y_f32, y_bf16, r};
    if (sg::launch_gemm_int8(p, M, N, K, xq, wq, ep, workspace, stream) != hipSuccess)
        return SG_ERR_HIP;
    for (int i = 0; i < p.launches(); ++i) sg::count_launch(SG_KERNEL_INT8);
    if (p.workspace > 0) sg::count_launch(SG_KERNEL_REDUCE);
    if (sg::launch_log_enabled())
        std::fprintf(stderr, "[skinny_gemm] int8 M=%d N=%d K=%d launches=%d%s%s\n", M, N, K,
                     p.launches(), p.workspace > 0 ? " +reduce pass" : "", r ? " residual" : "");
    return SG_OK;
}

}  // namespace

extern "C" {

sg_status skinny_rmsnorm(int32_t M, int32_t K, const sg_bf16* x, const sg_bf16* r,
                         const sg_bf16* g, float eps, sg_bf16* h, sg_bf16* y_bf16, int8_t* codes,
                         float* scales, void* stream) {
    if (!rows_ok(M, K) || !eps_ok(eps)) return SG_ERR_SHAPE;
    if (K % 8 != 0) return SG_ERR_ALIGN;
    if (M == 0) return SG_OK;
    if (!x || !g || (!y_bf16 && !codes) || (codes != nullptr) != (scales != nullptr))
        return SG_ERR_NULL;
    if (!aligned16(x) || !aligned16(r) || !aligned16(g) || !aligned16(h) || !aligned16(y_bf16) ||
        !aligned16(codes) || !aligned4(scales))
        return SG_ERR_ALIGN;
    (void)hipGetLastError();
    if (sg::launch_rmsnorm(M, K, x, r, g, eps, h, y_bf16, codes, scales,
                           static_cast<hipStream_t>(stream)) != hipSuccess)
        return SG_ERR_HIP;
    sg::count_launch(SG_KERNEL_RMSNORM);
    if (sg::launch_log_enabled())
        std::fprintf(stderr, "[skinny_gemm] rmsnorm M=%d K=%d%s%s%s\n", M, K,
                     r ? " residual" : "", y_bf16 ? " bf16" : "", codes ? " int8" : "");
    return SG_OK;
}

sg_status skinny_quant_int8(int32_t M, int32_t K, const sg_bf16* x_bf16, const float* x_f32,
                            int32_t gated, int8_t* codes, float* scales, void* stream) {
    if (!rows_ok(M, K) || (gated != 0 && gated != 1)) return SG_ERR_SHAPE;
    if (K % 8 != 0) return SG_ERR_ALIGN;
    if (M == 0) return SG_OK;
    if ((x_bf16 != nullptr) == (x_f32 != nullptr) || !codes || !scales) return SG_ERR_NULL;
    if (!aligned16(x_bf16) || !aligned16(x_f32) || !aligned16(codes) || !aligned4(scales))
        return SG_ERR_ALIGN;
    (void)hipGetLastError();
    const void* x = x_f32 ? static_cast<const void*>(x_f32) : x_bf16;
    if (sg::launch_quant_int8(M, K, x, x_f32 != nullptr, gated != 0, codes, scales,
                              static_cast<hipStream_t>(stream)) != hipSuccess)
        return SG_ERR_HIP;
    sg::count_launch(SG_KERNEL_QUANT_INT8);
    if (sg::launch_log_enabled())
        std::fprintf(stderr, "[skinny_gemm] quant_int8 M=%d K=%d %s%s\n", M, K,
                     x_f32 ? "fp32" : "bf16", gated ? " gated" : "");
    return SG_OK;
}

size_t skinny_gemm_int8_workspace(int32_t M, int32_t N, int32_t K) {
    if (!gemm_sizes_ok(M, N, K) || K % 16 != 0 || M == 0 || N == 0) return 0;
    return sg::int8_plan(M, N, K).workspace;
}

sg_status skinny_gemm_int8(int32_t M, int32_t N, int32_t K, const int8_t* x_codes,
                           const float* x_scales, const int8_t* W_codes, const float* W_scales,
                           const sg_bf16* r, float* y_f32, sg_bf16* y_bf16, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (!gemm_sizes_ok(M, N, K)) return SG_ERR_SHAPE;
    if (K % 16 != 0) return SG_ERR_ALIGN;
    if (M == 0 || N == 0) return SG_OK;
    if ((!y_f32 && !y_bf16) || !x_scales || !W_scales) return SG_ERR_NULL;
    if (K > 0 && (!x_codes || !W_codes)) return SG_ERR_NULL;
    if (!aligned16(x_codes) || !aligned16(W_codes) || !aligned4(x_scales) || !aligned4(W_scales) ||
        !aligned16(r) || !aligned16(y_f32) || !aligned16(y_bf16))
        return SG_ERR_ALIGN;
    const sg::Int8Plan plan = sg::int8_plan(M, N, K);
    if (plan.workspace > 0) {
        if (!workspace || workspace_bytes < plan.workspace) return SG_ERR_WORKSPACE;
        if (!aligned16(workspace)) return SG_ERR_ALIGN;
    }
    return product(plan, M, N, K, x_codes, x_scales, W_codes, W_scales, r, y_f32, y_bf16, workspace,
                   static_cast<hipStream_t>(stream));
}

size_t skinny_mlp_int8_step_workspace(int32_t M, int32_t H, int32_t F) {
    MlpLayout L;
    return mlp_layout(M, H, F, &L) ? L.total : 0;
}

sg_status skinny_mlp_int8_step(const sg_mlp_int8_step* a, void* workspace, size_t workspace_bytes,
                               void* stream) {
    if (!a) return SG_ERR_NULL;
    MlpLayout L;
    if (!mlp_layout(a->M, a->H, a->F, &L))
        return a->H > 0 && a->F > 0 && (a->H % 16 != 0 || a->F % 16 != 0) ? SG_ERR_ALIGN
                                                                          : SG_ERR_SHAPE;
    if (!eps_ok(a->eps)) return SG_ERR_SHAPE;
    if (a->M == 0) return SG_OK;
    // every check of the calls below, made here before the first launch
    if (!a->x || !a->g || !a->W_gate_up || !a->gate_up_scales || !a->W_down || !a->down_scales ||
        !a->out)
        return SG_ERR_NULL;
    if (!aligned16(a->x) || !aligned16(a->r) || !aligned16(a->g) || !aligned16(a->W_gate_up) ||
        !aligned16(a->W_down) || !aligned16(a->out) || !aligned4(a->gate_up_scales) ||
        !aligned4(a->down_scales))
        return SG_ERR_ALIGN;
    if (!workspace || workspace_bytes < L.total) return SG_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SG_ERR_ALIGN;

    char* base = static_cast<char*>(workspace);
    int8_t* q = reinterpret_cast<int8_t*>(base + L.q);
    float* sq = reinterpret_cast<float*>(base + L.sq);
    float* u = reinterpret_cast<float*>(base + L.u);
    int8_t* p = reinterpret_cast<int8_t*>(base + L.p);
    float* sp = reinterpret_cast<float*>(base + L.sp);
    void* gw = base + L.gemm;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    sg_status st;
    // out holds h between the norm and the down projection, which adds to it
    if ((st = skinny_rmsnorm(a->M, a->H, a->x, a->r, a->g, a->eps, a->out, nullptr, q, sq,
                             stream)) != SG_OK)
        return st;
    if (L.gated) {
        // long prompts: the gated product leaves the projection's epilogue, u is [M, F]
        const sg::Int8Epilogue ep{sq, a->gate_up_scales, u, nullptr, nullptr};
        if (sg::launch_gated_int8(L.up, a->M, a->F, a->H, q, a->W_gate_up, ep, hs) != hipSuccess)
            return SG_ERR_HIP;
        for (int i = 0; i < L.up.launches(); ++i) sg::count_launch(SG_KERNEL_INT8);
        if (sg::launch_log_enabled())
            std::fprintf(stderr, "[skinny_gemm] int8 gated M=%d F=%d H=%d launches=%d\n", a->M, a->F,
                         a->H, L.up.launches());
    } else if ((st = product(L.up, a->M, 2 * a->F, a->H, q, sq, a->W_gate_up, a->gate_up_scales,
                             nullptr, u, nullptr, gw, hs)) != SG_OK) {
        return st;
    }
    if ((st = skinny_quant_int8(a->M, a->F, nullptr, u, L.gated ? 0 : 1, p, sp, stream)) != SG_OK)
        return st;
    return product(L.down, a->M, a->H, a->F, p, sp, a->W_down, a->down_scales, a->out, nullptr,
                   a->out, gw, hs);
}

}  // extern "C"
