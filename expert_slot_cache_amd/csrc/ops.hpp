// Launchers of the operators around the experts (routers, sorted rows, products);
// C++ linkage, used by ops.cpp only, which checks every argument first.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "kernels.hpp"

namespace moe {

constexpr int kBlock = 128;   // values of a row (and rows of a matrix) that share one scale

// ---- route.hip ----
hipError_t launch_route(int atype, const void* logits, int64_t stride, int T, int E, int K, bool renorm, int32_t* ids,
                        float* w, hipStream_t s);
hipError_t launch_route_backward(int atype, const void* logits, int64_t stride, const int32_t* ids, const float* w,
                                 const float* dw, int T, int E, int K, bool renorm, void* dlogits, int64_t dstride,
                                 hipStream_t s);

// ---- route_groups.hip ----
constexpr int kMaxGroups = 64;   // a wave's lanes
struct RouteGroups {
    int E, K;
    int n_groups, kept, group_top;
    bool sigmoid, renorm;
    float scale;
};
hipError_t launch_route_groups(int atype, const void* logits, int64_t stride, const float* bias, int T,
                               const RouteGroups& r, int32_t* ids, float* w, hipStream_t s);
hipError_t launch_route_groups_backward(int atype, const void* logits, int64_t stride, const int32_t* ids, const float* w,
                                        const float* dw, int T, const RouteGroups& r, void* dlogits, int64_t dstride,
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

// f of two formats as constants (the second is fp32 or the first).
template <class F>
hipError_t by_types(int at, int ot, F f) {
    typedef std::integral_constant<int, A_F32> F32;
    typedef std::integral_constant<int, A_BF16> BF16;
    if (at == A_F32) return f(F32{}, F32{});
    return ot == A_F32 ? f(BF16{}, F32{}) : f(BF16{}, BF16{});
}

// ---- expert.hip ----
enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3, ACT_SWIGLU = 4 };
struct ExpertArgs {
    const void* x;            // [M][K]
    const void* w;            // [G][N][K]
    const float* bias;        // [G][N] or null
    const void* resid;        // [M][N or N/2] or null
    const int32_t* offsets;   // [G+1] or null (G = 1: every row)
    void* out;                // [M][N or N/2]
    void* pre;                // [M][N] or null
    int M, G, N, K, act;
};
hipError_t launch_expert_product(int atype, int out_atype, const ExpertArgs& a, hipStream_t s);

// ---- activation.hip ----
// Bytes of the partial sums of a bias' gradient.
size_t activation_workspace(int M, int G, int N);
struct ActivationArgs {
    const void* dout;         // [M][N or N/2]
    const void* pre;          // [M][N] or null (ACT_NONE)
    const int32_t* offsets;
    void* dpre;               // [M][N] or null
    float* dbias;             // [G][N] or null
    float* partial;
    int M, G, N, act;
};
hipError_t launch_activation_backward(int atype, int out_atype, const ActivationArgs& a, hipStream_t s);

// ---- expert_backward.hip ----
// Bytes of the partial sums of the matrices' gradients (0: none are needed).
size_t expert_backward_workspace(int M, int G, int N, int K);
struct ExpertGradArgs {
    const void* dpre;         // [M][N]
    const void* x;            // [M][K], for dw
    const void* w;            // [G][N][K], for dx
    const int32_t* offsets;
    void* dx;                 // [M][K] or null
    void* dw;                 // [G][N][K] or null
    float* partial;
    int M, G, N, K;
};
hipError_t launch_expert_backward(int atype, int dw_atype, const ExpertGradArgs& a, hipStream_t s);

}  // namespace moe
