// fp8_block_checks.cpp -- drives the host code of the block-scaled FP8 operators and
// of the rows by expert (argument checks, the product's choice of kernel, the step's
// layout) under AddressSanitizer on a host without a GPU.  Every call made here
// returns before any launch.  Exit status 0 when every status and size is what the
// header promises.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "skinny_gemm.h"

namespace {

int failures = 0;

void expect(bool ok, const char* what, int line) {
    if (!ok) {
        std::fprintf(stderr, "fp8_block_checks: line %d: %s\n", line, what);
        ++failures;
    }
}
#define EXPECT(c) expect((c), #c, __LINE__)

// Fake device addresses: never dereferenced, every call below returns first.
template <class T>
T* fake(uintptr_t a) {
    return reinterpret_cast<T*>(a);
}

void sizes() {
    uint8_t* q = fake<uint8_t>(4096);
    float* s = fake<float>(4096);
    const int32_t Ms[] = {0, 1, 16, 17, 33, 64, 300, 2049, 65536, SG_INT8_MAX_M};
    const int32_t Ns[] = {0, 1, 17, 1000, 8192, 36864, 1 << 20};
    const int32_t Ks[] = {0, 16, 528, 1040, 7168, 18432, SG_FP8_MAX_K};
    for (int32_t M : Ms)
        for (int32_t N : Ns)
            for (int32_t K : Ks)
                for (int32_t f32 : {0, 1}) {
                    const size_t w = skinny_gemm_fp8_block_workspace(M, N, K, f32);
                    EXPECT(w <= ((size_t)1 << 30) && w % 16 == 0);
                    if (M <= 32 || N == 0 || K < 1024) EXPECT(w == 0);
                    if (w > 0)  // a missing or short workspace is refused
                        EXPECT(skinny_gemm_fp8_block(M, N, K, q, s, q, s, nullptr, f32 ? s : nullptr,
                                                     f32 ? nullptr : fake<sg_bf16>(4096), fake<void>(4096),
                                                     w - 1, nullptr) == SG_ERR_WORKSPACE);
                }
    for (int32_t E : {1, 48, 384, SG_MOE_MAX_EXPERTS})
        for (int32_t topk : {1, 8, SG_MOE_MAX_TOPK}) {
            size_t sort = 0, step = 0;
            for (int32_t T = 1; (int64_t)T * topk <= SG_MOE_MAX_PAIRS; T = T * 3 + 1) {
                const size_t w = skinny_moe_sort_workspace(T, topk, E);
                EXPECT(w >= sort);  // one for the most tokens serves fewer
                sort = w;
                if (w > 0)
                    EXPECT(skinny_moe_sort(T, topk, E, fake<int32_t>(4096), fake<int32_t>(4096), nullptr,
                                           fake<int32_t>(4096), fake<void>(4096), w - 1,
                                           nullptr) == SG_ERR_WORKSPACE);
                const size_t v = skinny_moe_fp8_step_workspace(T, topk, E, 272, 144);
                EXPECT(v > (size_t)T * topk * 144 && v >= w);
                step = v;
            }
            EXPECT(step > 0);
            EXPECT(skinny_moe_sort_workspace(SG_MOE_MAX_PAIRS, topk + 1, E) == 0);
        }
}

void refusals() {
    uint8_t* q = fake<uint8_t>(4096);
    float* s = fake<float>(4096);
    int32_t* i = fake<int32_t>(4096);
    sg_bf16* b = fake<sg_bf16>(4096);
    EXPECT(skinny_quant_fp8(4, 36, b, nullptr, 0, q, s, nullptr) == SG_ERR_ALIGN);
    EXPECT(skinny_quant_fp8(4, 32, b, s, 0, q, s, nullptr) == SG_ERR_NULL);
    EXPECT(skinny_quant_fp8(INT32_MIN, INT32_MAX, b, nullptr, 1, q, s, nullptr) == SG_ERR_SHAPE);
    EXPECT(skinny_gemm_fp8_block(4, 8, 24, q, s, q, s, b, s, b, nullptr, 0, nullptr) == SG_ERR_ALIGN);
    EXPECT(skinny_gemm_fp8_block(INT32_MIN, 8, 32, q, s, q, s, b, s, b, nullptr, 0, nullptr) == SG_ERR_SHAPE);
    EXPECT(skinny_gemm_fp8_block(4, 8, 32, q, s, q, s, b, nullptr, nullptr, nullptr, 0, nullptr) ==
           SG_ERR_NULL);
    EXPECT(skinny_gemm_fp8_block(0, 8, 32, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                 nullptr, 0, nullptr) == SG_OK);
    EXPECT(skinny_moe_sort(INT32_MAX, SG_MOE_MAX_TOPK, 4, i, i, i, i, nullptr, 0, nullptr) == SG_ERR_SHAPE);
    EXPECT(skinny_moe_sort(4, 0, 4, i, i, i, i, nullptr, 0, nullptr) == SG_ERR_SHAPE);
    EXPECT(skinny_moe_sort(4, 2, 4, nullptr, i, i, i, nullptr, 0, nullptr) == SG_ERR_NULL);
    EXPECT(skinny_moe_gather(4, 2, 12, b, 0, i, b, nullptr) == SG_ERR_ALIGN);
    EXPECT(skinny_moe_gather(0, 2, 16, nullptr, 0, nullptr, nullptr, nullptr) == SG_OK);
    EXPECT(skinny_moe_combine(4, 2, 16, b, 2, i, s, b, b, nullptr) == SG_ERR_SHAPE);
    EXPECT(skinny_moe_combine_grad(4, 2, 16, b, b, 0, i, nullptr, b, s, nullptr) == SG_ERR_NULL);
    EXPECT(grouped_skinny_gemm_fp8(4, 4, 2, 16, 24, q, s, q, s, i, nullptr, 1, s, nullptr, nullptr) ==
           SG_ERR_ALIGN);
    EXPECT(grouped_skinny_gemm_fp8(4, 5, 2, 16, 32, q, s, q, s, i, nullptr, 1, s, nullptr, nullptr) ==
           SG_ERR_SHAPE);
    EXPECT(grouped_skinny_gemm_fp8(SG_MOE_MAX_PAIRS, SG_MOE_MAX_PAIRS, 2, 16, SG_FP8_MAX_K, q, s, q, s, i, i,
                                   1, s, nullptr, nullptr) == SG_ERR_SHAPE);
    sg_moe_fp8_step step;
    std::memset(&step, 0, sizeof step);
    EXPECT(skinny_moe_fp8_step(nullptr, nullptr, 0, nullptr) == SG_ERR_NULL);
    EXPECT(skinny_moe_fp8_step(&step, nullptr, 0, nullptr) == SG_ERR_SHAPE);
    step.topk = 2, step.E = 4, step.H = 32, step.F = 48;
    EXPECT(skinny_moe_fp8_step(&step, nullptr, 0, nullptr) == SG_OK);  // no tokens
    step.T = 3;
    EXPECT(skinny_moe_fp8_step(&step, nullptr, 0, nullptr) == SG_ERR_NULL);
    step.x = b, step.topk_ids = i, step.topk_weights = s, step.W_gate_up = q, step.gate_up_scales = s;
    step.W_down = q, step.down_scales = s, step.out = b;
    EXPECT(skinny_moe_fp8_step(&step, fake<void>(4096), skinny_moe_fp8_step_workspace(3, 2, 4, 32, 48) - 1,
                               nullptr) == SG_ERR_WORKSPACE);
    step.F = 56;
    EXPECT(skinny_moe_fp8_step(&step, fake<void>(4096), 1 << 20, nullptr) == SG_ERR_ALIGN);
    uint64_t launches[SG_NUM_COUNTERS];
    skinny_gemm_get_counters(launches);
    for (uint64_t n : launches) EXPECT(n == 0);
}

}  // namespace

int main() {
    sizes();
    refusals();
    if (failures) return 1;
    std::printf("fp8_block_checks: ok\n");
    return 0;
}
