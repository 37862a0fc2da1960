// The activations of the expert products' epilogue, and their slopes.
#pragma once

#include <hip/hip_runtime.h>

#include "ops.hpp"

namespace moe {

// By the hardware's exponential and reciprocal (1 ulp each): off by at most (|h| + 4) 2^-23 of itself
// while the exponential is finite; below h = -88 it is 0 (the reciprocal of a value above 2^126 is none).
__device__ __forceinline__ float sigmoid(float h) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(h * -1.44269504f));
}
// The distribution function of the normal distribution.
__device__ __forceinline__ float normal_cdf(float h) { return 0.5f * erfcf(h * -0.70710678f); }

__device__ __forceinline__ float activate(int act, float h) {
    if (act == ACT_RELU) return h > 0.0f ? h : 0.0f;
    if (act == ACT_GELU) return h * normal_cdf(h);
    if (act == ACT_SILU) return h * sigmoid(h);
    return h;
}
__device__ __forceinline__ float slope(int act, float h) {
    if (act == ACT_RELU) return h > 0.0f ? 1.0f : 0.0f;
    if (act == ACT_GELU) return normal_cdf(h) + h * 0.39894228f * __builtin_amdgcn_exp2f(h * h * -0.72134752f);
    if (act == ACT_SILU) {
        const float s = sigmoid(h);
        return s * (1.0f + h * (1.0f - s));
    }
    return 1.0f;
}

}  // namespace moe
