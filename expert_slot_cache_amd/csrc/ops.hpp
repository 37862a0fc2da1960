// Launchers of the operators around the experts (router, sorted rows, e4m3 products);
// C++ linkage, used by ops.cpp only, which checks every argument first.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

namespace moe {

constexpr int kBlock = 128;   // values of a row (and rows of a matrix) that share one scale

// ---- route.hip ----
hipError_t launch_route(int atype, const void* logits, int64_t stride, int T, int E, int K, bool renorm, int32_t* ids,
                        float* w, hipStream_t s);
hipError_t launch_route_backward(int atype, const void* logits, int64_t stride, const int32_t* ids, const float* w,
                                 const float* dw, int T, int E, int K, bool renorm, void* dlogits, int64_t dstride,
                                 hipStream_t s);

// ---- rows.hip ----
// Bytes of the block counts that sorting T*K pairs needs (0: one launch does it all).
size_t sort_workspace(int T, int K, int E);
hipError_t launch_sort(int atype, const void* x, int64_t stride, const int32_t* ids, int T, int K, int E, int H,
                       bool f8, void* sorted, float* scales, int32_t* offsets, int32_t* rows, void* workspace,
                       hipStream_t s);
hipError_t launch_combine(int atype, const void* ys, const int32_t* rows, const float* w, const void* resid, int T,
                          int K, int H, void* out, hipStream_t s);
hipError_t launch_combine_backward(int atype, const void* dout, const void* ys, const int32_t* rows, const float* w,
                                   int T, int K, int H, void* dys, float* dw, hipStream_t s);

// ---- scaled.hip ----
struct ProductArgs {
    const uint8_t* x;         // [M][K] e4m3
    const float* xs;          // [M][KB]
    const uint8_t* w;         // [G][N][K] e4m3
    const float* ws;          // [G][NB][KB]
    const int32_t* offsets;   // [G+1] or null (G = 1: every row)
    void* out;                // [M][N] fp32 / bf16, or [M][N/2] e4m3
    float* os;                // [M][N/256] (SwiGLU) or null
    int M, G, N, K;
};
enum { OUT_F32 = 0, OUT_BF16 = 1, OUT_SWIGLU = 2 };
hipError_t launch_scaled_product(const ProductArgs& a, int out, hipStream_t s);

}  // namespace moe
