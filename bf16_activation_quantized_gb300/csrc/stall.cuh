// stall.cuh -- for a test's build of one translation unit: the producers of every other
// pair of CTAs stop issuing copies from stage `at` on, so that the waits behind them run out.
#pragma once

#include <cuda_runtime.h>

namespace w4a16 {
namespace {

#ifdef W4A16_TEST_STALL
__device__ int g_stall_at = -1;
__device__ __forceinline__ bool stalled(int stage) {
    return g_stall_at >= 0 && stage >= g_stall_at && blockIdx.x / 2 % 2 == 1;
}
#else
__device__ __forceinline__ bool stalled(int) { return false; }
#endif

}  // namespace
}  // namespace w4a16

#ifdef W4A16_TEST_STALL
#define W4A16_STALL_ENTRY(name)                                                      \
    extern "C" int name(int at) {                                                    \
        return int(cudaMemcpyToSymbol(w4a16::g_stall_at, &at, sizeof at));           \
    }
#else
#define W4A16_STALL_ENTRY(name)
#endif
