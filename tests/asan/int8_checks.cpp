// int8_checks.cpp -- drives the host code of the 8-bit integer operators
// (argument checks, the product's choice of kernel, the MLP step's layout)
// under AddressSanitizer on a host without a GPU.  Every call made here
// returns before any launch.  Exit status 0 when every status and size is what
// the header promises.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "skinny_gemm.h"

namespace {

int failures = 0;

void expect(bool ok, const char* what, int line) {
    if (!ok) {
        std::fprintf(stderr, "int8_checks: line %d: %s\n", line, what);
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
    const int32_t Ms[] = {0, 1, 7, 16, 33, 64, 65, 300, 4097, SG_INT8_MAX_M};
    const int32_t Ns[] = {0, 1, 16, 17, 1000, 4096, 8192, 36864, 1 << 20};
    const int32_t Ks[] = {0, 16, 64, 1040, 7168, 18432, 65536, SG_INT8_MAX_K};
    for (int32_t M : Ms)
        for (int32_t N : Ns)
            for (int32_t K : Ks) {
                const size_t w = skinny_gemm_int8_workspace(M, N, K);
                EXPECT(w <= ((size_t)1 << 30) && w % 16 == 0);
                EXPECT(w == skinny_gemm_int8_workspace(M, N, K));
                if (M == 0 || N == 0 || K < 1024) EXPECT(w == 0);
                if (w > 0)  // a missing or short workspace is refused
                    EXPECT(skinny_gemm_int8(M, N, K, fake<int8_t>(4096), fake<float>(4096),
                                            fake<int8_t>(4096), fake<float>(4096), nullptr,
                                            fake<float>(4096), nullptr, fake<void>(4096), w - 1,
                                            nullptr) == SG_ERR_WORKSPACE);
            }
    for (int32_t M : Ms)
        for (int32_t H : {16, 272, 7168, SG_ROW_MAX_K})
            for (int32_t F : {16, 528, 18432, SG_ROW_MAX_K})
                EXPECT(skinny_mlp_int8_step_workspace(M, H, F) >= (size_t)M * (H + 5 * (size_t)F));
}

void refusals() {
    int8_t* q = fake<int8_t>(4096);
    float* s = fake<float>(4096);
    sg_bf16* b = fake<sg_bf16>(4096);
    EXPECT(skinny_gemm_int8(4, 8, 24, q, s, q, s, b, s, b, nullptr, 0, nullptr) == SG_ERR_ALIGN);
    EXPECT(skinny_gemm_int8(4, 8, SG_INT8_MAX_K + 16, q, s, q, s, b, s, b, nullptr, 0, nullptr) ==
           SG_ERR_SHAPE);
    EXPECT(skinny_gemm_int8(INT32_MIN, INT32_MIN, INT32_MIN, q, s, q, s, b, s, b, nullptr, 0,
                            nullptr) == SG_ERR_SHAPE);
    EXPECT(skinny_gemm_int8(4, 8, 32, q, s, q, s, b, nullptr, nullptr, nullptr, 0, nullptr) ==
           SG_ERR_NULL);
    EXPECT(skinny_gemm_int8(0, 8, 32, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                            nullptr, 0, nullptr) == SG_OK);
    EXPECT(skinny_rmsnorm(4, 32, b, b, b, std::numeric_limits<float>::quiet_NaN(), b, b, q, s,
                          nullptr) == SG_ERR_SHAPE);
    EXPECT(skinny_rmsnorm(4, INT32_MAX, b, b, b, 1e-6f, b, b, q, s, nullptr) == SG_ERR_SHAPE);
    EXPECT(skinny_rmsnorm(4, 32, b, b, b, 1e-6f, b, nullptr, nullptr, nullptr, nullptr) == SG_ERR_NULL);
    EXPECT(skinny_quant_int8(4, 32, b, s, 0, q, s, nullptr) == SG_ERR_NULL);
    EXPECT(skinny_quant_int8(4, 36, b, nullptr, 0, q, s, nullptr) == SG_ERR_ALIGN);
    EXPECT(skinny_quant_int8(INT32_MAX, 32, b, nullptr, 0, q, s, nullptr) == SG_ERR_SHAPE);
    sg_mlp_int8_step step;
    std::memset(&step, 0, sizeof step);
    EXPECT(skinny_mlp_int8_step(nullptr, nullptr, 0, nullptr) == SG_ERR_NULL);
    EXPECT(skinny_mlp_int8_step(&step, nullptr, 0, nullptr) == SG_ERR_SHAPE);
    step.H = 32, step.F = 48, step.eps = 1e-6f;
    EXPECT(skinny_mlp_int8_step(&step, nullptr, 0, nullptr) == SG_OK);  // no rows
    step.M = 3;
    EXPECT(skinny_mlp_int8_step(&step, nullptr, 0, nullptr) == SG_ERR_NULL);
    step.x = b, step.g = b, step.W_gate_up = q, step.gate_up_scales = s, step.W_down = q;
    step.down_scales = s, step.out = b;
    EXPECT(skinny_mlp_int8_step(&step, fake<void>(4096),
                                skinny_mlp_int8_step_workspace(3, 32, 48) - 1, nullptr) ==
           SG_ERR_WORKSPACE);
    step.F = 56;
    EXPECT(skinny_mlp_int8_step(&step, fake<void>(4096), 1 << 20, nullptr) == SG_ERR_ALIGN);
    uint64_t launches[SG_NUM_COUNTERS];
    skinny_gemm_get_counters(launches);
    for (uint64_t n : launches) EXPECT(n == 0);
}

}  // namespace

int main() {
    sizes();
    refusals();
    if (failures) return 1;
    std::printf("int8_checks: ok\n");
    return 0;
}
