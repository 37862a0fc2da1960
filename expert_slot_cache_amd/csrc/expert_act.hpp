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
// The distribution function of the normal distribution.  Its tail Phi(-|h|) is e(h) t P(t) with
// e(h) = exp(-h^2 / 2) and t = 1 / (1 + |h| / 4): what is left of the tail over e is a smooth function of
// t that is 0 at t = 0, and P is the polynomial of degree 9 whose largest relative error is least (4.8e-8 with
// the fp32 coefficients below; fitted to erfcx in fp64 by reweighted least squares).  Off by less than
// (16 + h^2) 2^-24 of itself, h^2 for the rounding of the exponent, with an ulp each of the exponential and the
// reciprocal.  erfcf took three times as long: 32768 x 4096 gradients
// in bf16 246 us, 170 with this (relu 163).
struct Normal {
    float e, cdf;
    __device__ __forceinline__ explicit Normal(float h) {
        const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(h), 0.25f, 1.0f));
        e = __builtin_amdgcn_exp2f(h * h * -0.72134752f);
        float q = 0.01978236995637417f;
        q = fmaf(q, t, -0.08087875694036484f);
        q = fmaf(q, t, 0.0955994576215744f);
        q = fmaf(q, t, -0.031719598919153214f);
        q = fmaf(q, t, 0.06370015442371368f);
        q = fmaf(q, t, 0.058974843472242355f);
        q = fmaf(q, t, 0.08160316199064255f);
        q = fmaf(q, t, 0.09346634894609451f);
        q = fmaf(q, t, 0.09973642975091934f);
        q = fmaf(q, t, 0.0997355654835701f);
        const float tail = e * (q * t);
        cdf = h < 0.0f ? tail : 1.0f - tail;
    }
};

// A NaN stays one through every activation and slope.
__device__ __forceinline__ float activate(int act, float h) {
    if (act == ACT_RELU) return h <= 0.0f ? 0.0f : h;
    if (act == ACT_GELU) return h * Normal(h).cdf;
    if (act == ACT_SILU) return h * sigmoid(h);
    return h;
}
__device__ __forceinline__ float slope(int act, float h) {
    if (act == ACT_RELU) return h > 0.0f ? 1.0f : h <= 0.0f ? 0.0f : h;
    if (act == ACT_GELU) {
        const Normal v(h);
        return fmaf(h * 0.39894228f, v.e, v.cdf);
    }
    if (act == ACT_SILU) {
        const float s = sigmoid(h);
        return s * (1.0f + h * (1.0f - s));
    }
    return 1.0f;
}

}  // namespace moe
