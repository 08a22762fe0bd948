// pa_long.cuh -- packed fp32 arithmetic and small helpers that the two
// tensor-core attention kernels share: the plain one (pa_long.cu: causal steps
// and the cascade prefix pass) and the windowed one (pa_long_window.cu).
#pragma once

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kLongWarps = 12;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescaleThreshold = 8.0f;

// The lowest n bits set, n clamped to 0 .. 64.
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return warp_mbar_wait(bar, parity, abort);
}

// The three-input maximum.  (The softmax warps are bound by instruction issue, so each score
// costs half an FMA, half an add, half a conversion, half a maximum and one exponential.)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

}  // namespace

}  // namespace pa
