// Rows of logits: keys that order their values with ties, and reductions over a wave.
#pragma once
#include <math.h>

#include "kda_device.h"

namespace kda {

// Keys order like (value descending, token ascending) when compared as larger first.  No key of a
// token is 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t key_of(float x, int token) {
    return ((uint64_t)ordered(x + 0.f) << 32) | (0xFFFFFFFFu - (uint32_t)token);
}
// NaN counts as -inf (the maximum's result is its other operand); -0 becomes +0 where a key is made
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY); }

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int off) {
    const uint32_t lo = __shfl_xor((uint32_t)x, off, 64), hi = __shfl_xor((uint32_t)(x >> 32), off, 64);
    return ((uint64_t)hi << 32) | lo;
}

// x of lane ^ 1, ^ 2, then mirrored in 8 and in 16 lanes, then of lane ^ 16 and ^ 32: six steps after
// which a maximum or minimum covers the wave
template <int LEVEL>
__device__ __forceinline__ float other_lane(float x) {
    if constexpr (LEVEL < 4) {
        constexpr int ctrl = LEVEL == 0 ? 0xB1 : LEVEL == 1 ? 0x4E : LEVEL == 2 ? 0x141 : 0x140;
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, 0xF, 0xF, true));
    } else {
        return __shfl_xor(x, LEVEL == 4 ? 16 : 32, 64);
    }
}
template <int LEVEL>
__device__ __forceinline__ float max_min_step(float x, int shift) {
    const float y = other_lane<LEVEL>(x);
    return LEVEL < shift ? fmaxf(x, y) : fminf(x, y);
}

}  // namespace kda
