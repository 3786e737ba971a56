// lds_limit_checks.cpp -- launches whose LDS depends on the sizes (skinny_moe_sort, and the
// chunk kernels of skinny_gemm and skinny_gemm_fp8) on a host without a GPU: the runtime's
// calls that set a kernel's dynamic LDS limit and launch it are replaced by records.  A
// limit is a property of the kernel, shared by every thread that launches it, so no call
// may set it below what another call's launch takes.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <map>

#include "skinny_gemm.h"

namespace {
std::map<const void*, int> least, most;  // limit set least, launched with most
int launches = 0;
}  // namespace

extern "C" hipError_t hipFuncSetAttribute(const void* f, hipFuncAttribute, int value) {
    if (!least.count(f) || value < least[f]) least[f] = value;
    return hipSuccess;
}

extern "C" hipError_t hipLaunchKernel(const void* f, dim3, dim3, void**, size_t lds, hipStream_t) {
    if (!most.count(f) || (int)lds > most[f]) most[f] = (int)lds;
    ++launches;
    return hipSuccess;
}

// the launch configuration on its way from the call to the kernel's host stub
namespace {
dim3 grid_of, block_of;
size_t lds_of = 0;
}  // namespace

extern "C" hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t) {
    grid_of = grid, block_of = block, lds_of = lds;
    return hipSuccess;
}

extern "C" hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
    *grid = grid_of, *block = block_of, *lds = lds_of, *stream = nullptr;
    return hipSuccess;
}

extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }

int main() {
    int32_t* p = reinterpret_cast<int32_t*>((uintptr_t)4096);  // never dereferenced
    for (int32_t E : {4096, 48, 1024, 1025, 1, 4096, 384})
        for (int32_t T : {1, 64, 65, 512, 513, 8192, 8193, 100000, 1 << 19}) {
            const sg_status st = skinny_moe_sort(T, 8, E, p, p, p, p, p, (size_t)1 << 40, nullptr);
            if (st != SG_OK) {
                std::fprintf(stderr, "T %d E %d: status %d\n", T, E, st);
                return 1;
            }
        }
    // the chunk kernels: bf16 rows by bf16 and by block-scaled FP8 weights
    sg_bf16* b = reinterpret_cast<sg_bf16*>((uintptr_t)4096);
    float* y = reinterpret_cast<float*>((uintptr_t)4096);
    for (int32_t M : {64, 9, 12, 17, 33, 48, 64})
        for (int32_t N : {512, 4096, 8192, 36864})
            for (int32_t K : {256, 1024, 2048, 4096, 7168, 8192, 16384}) {
                sg_plan plan;
                if (skinny_gemm_plan(M, N, K, &plan) != SG_OK ||
                    skinny_gemm(&plan, b, b, y, nullptr, p, (size_t)1 << 40, nullptr) != SG_OK ||
                    skinny_gemm_fp8(M, N, K, b, reinterpret_cast<uint8_t*>(b), y, nullptr, y, nullptr, p,
                                    (size_t)1 << 40, nullptr) != SG_OK) {
                    std::fprintf(stderr, "%d x %d x %d is refused\n", M, N, K);
                    return 1;
                }
            }
    int bad = 0;
    for (const auto& k : most)
        if (k.second > 0 && (!least.count(k.first) || least[k.first] < k.second)) {
            std::fprintf(stderr, "a kernel launched with %d bytes of LDS has its limit set to %d by another call\n",
                         k.second, least.count(k.first) ? least[k.first] : -1);
            ++bad;
        }
    if (launches < 100) std::fprintf(stderr, "%d launches\n", launches);
    if (bad || launches < 100) return 1;
    std::printf("lds_limit_checks: ok\n");
    return 0;
}
