// C entry points of the operators around the experts: argument checks, then one launcher.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "kernels.hpp"
#include "moe_pool.h"
#include "ops.hpp"

namespace moe {
void set_last_error(const char* msg);   // moe_pool.cpp
}

namespace {

// A launch has fewer than 2^32 lanes: 256 for each token, or 512 for 2^15 elements of a product
// and the short last tiles of its groups.
constexpr int64_t kMaxPairs = (int64_t)1 << 24;
constexpr int32_t kMaxTokens = (1 << 24) - 1;
constexpr int64_t kMaxElements = (int64_t)1 << 36;
constexpr int32_t kMaxHidden = 1 << 17;

moe_status_t fail(moe_status_t code, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    moe::set_last_error(msg);
    return code;
}

moe_status_t launched(hipError_t e, const char* what) {
    return e == hipSuccess ? MOE_OK : fail(MOE_EHIP, "%s launch failed: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A null pointer, or one that is not aligned to its elements.
bool bad(const void* p, size_t elem) { return !p || !aligned(p, elem); }

size_t act_size(int32_t atype) { return atype == MOE_A_F32 ? 4 : 2; }

#define CHECK(cond, ...) \
    do { \
        if (!(cond)) return fail(MOE_EINVAL, __VA_ARGS__); \
    } while (0)

// The sizes every operator on (token, expert) pairs shares.
moe_status_t check_pairs(int32_t atype, int32_t T, int32_t K) {
    CHECK(atype == MOE_A_F32 || atype == MOE_A_BF16, "atype %d invalid", atype);
    CHECK(T >= 0 && T <= kMaxTokens, "n_tokens %d outside [0,%d]", T, kMaxTokens);
    CHECK(K >= 1 && K <= moe::kMaxTopK, "top_k %d outside [1,%d]", K, moe::kMaxTopK);
    CHECK((int64_t)T * K <= kMaxPairs, "n_tokens * top_k above %lld", (long long)kMaxPairs);
    return MOE_OK;
}

moe_status_t check_route(int32_t atype, int64_t stride, int32_t T, int32_t E, int32_t K, int32_t norm) {
    if (const moe_status_t st = check_pairs(atype, T, K)) return st;
    CHECK(E >= 1 && E <= moe::kMaxExperts, "n_experts %d outside [1,%d]", E, moe::kMaxExperts);
    CHECK(K <= E, "top_k %d above n_experts %d", K, E);
    CHECK(norm == MOE_ROUTE_SOFTMAX || norm == MOE_ROUTE_RENORM, "norm %d invalid", norm);
    CHECK(stride >= E && stride <= ((int64_t)1 << 32), "row stride %lld invalid for %d experts", (long long)stride, E);
    return MOE_OK;
}

moe_status_t check_hidden(int32_t H) {
    CHECK(H >= 1 && H <= kMaxHidden, "hidden %d outside [1,%d]", H, kMaxHidden);
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_route(int32_t atype, const void* logits_dev, int64_t logits_stride, int32_t n_tokens,
                       int32_t n_experts, int32_t top_k, int32_t norm, int32_t* topk_ids_dev, float* topk_w_dev,
                       void* stream) {
    if (const moe_status_t st = check_route(atype, logits_stride, n_tokens, n_experts, top_k, norm)) return st;
    if (n_tokens == 0) return MOE_OK;
    CHECK(!bad(logits_dev, act_size(atype)) && !bad(topk_ids_dev, 4) && !bad(topk_w_dev, 4), "null or misaligned buffer");
    return launched(moe::launch_route(atype, logits_dev, logits_stride, n_tokens, n_experts, top_k,
                                      norm == MOE_ROUTE_RENORM, topk_ids_dev, topk_w_dev,
                                      static_cast<hipStream_t>(stream)),
                    "route");
}

moe_status_t moe_route_backward(int32_t atype, const void* logits_dev, int64_t logits_stride,
                                const int32_t* topk_ids_dev, const float* topk_w_dev, const float* d_topk_w_dev,
                                int32_t n_tokens, int32_t n_experts, int32_t top_k, int32_t norm, void* d_logits_dev,
                                int64_t d_logits_stride, void* stream) {
    if (const moe_status_t st = check_route(atype, d_logits_stride, n_tokens, n_experts, top_k, norm)) return st;
    const size_t es = act_size(atype);
    if (norm == MOE_ROUTE_SOFTMAX) {
        if (const moe_status_t st = check_route(atype, logits_stride, n_tokens, n_experts, top_k, norm)) return st;
        CHECK(n_tokens == 0 || !bad(logits_dev, es), "null or misaligned buffer");
    }
    if (n_tokens == 0) return MOE_OK;
    CHECK(!bad(topk_ids_dev, 4) && !bad(topk_w_dev, 4) && !bad(d_topk_w_dev, 4) && !bad(d_logits_dev, es),
          "null or misaligned buffer");
    return launched(moe::launch_route_backward(atype, logits_dev, logits_stride, topk_ids_dev, topk_w_dev, d_topk_w_dev,
                                               n_tokens, n_experts, top_k, norm == MOE_ROUTE_RENORM, d_logits_dev,
                                               d_logits_stride, static_cast<hipStream_t>(stream)),
                    "route_backward");
}

size_t moe_sort_workspace_bytes(int32_t n_tokens, int32_t top_k, int32_t n_experts) {
    if (check_pairs(MOE_A_F32, n_tokens, top_k) || n_experts < 1 || n_experts > moe::kMaxExperts) return 0;
    return moe::sort_workspace(n_tokens, top_k, n_experts);
}

moe_status_t moe_sort_tokens(int32_t atype, const void* x_dev, int64_t x_stride, const int32_t* topk_ids_dev,
                             int32_t n_tokens, int32_t top_k, int32_t n_experts, int32_t hidden, int32_t to_fp8,
                             void* sorted_dev, float* scales_dev, int32_t* offsets_dev, int32_t* rows_dev,
                             void* workspace_dev, size_t workspace_bytes, void* stream) {
    if (const moe_status_t st = check_pairs(atype, n_tokens, top_k)) return st;
    CHECK(n_experts >= 1 && n_experts <= moe::kMaxExperts, "n_experts %d outside [1,%d]", n_experts, moe::kMaxExperts);
    CHECK(to_fp8 == 0 || to_fp8 == 1, "to_fp8 %d invalid", to_fp8);
    CHECK(!bad(offsets_dev, 4), "null or misaligned buffer");
    if (x_dev) {
        if (const moe_status_t st = check_hidden(hidden)) return st;
        CHECK(x_stride >= hidden && x_stride <= ((int64_t)1 << 32), "row stride %lld invalid for hidden %d",
              (long long)x_stride, hidden);
        CHECK(!to_fp8 || hidden % 16 == 0, "hidden %d: e4m3 rows need a multiple of 16", hidden);
    }
    if (n_tokens > 0) {
        CHECK(!bad(topk_ids_dev, 4) && !bad(rows_dev, 4), "null or misaligned buffer");
        if (x_dev) {
            CHECK(aligned(x_dev, act_size(atype)) && !bad(sorted_dev, to_fp8 ? 16 : act_size(atype)),
                  "null or misaligned buffer");
            CHECK(!to_fp8 || !bad(scales_dev, 4), "null or misaligned scales");
        }
    }
    const size_t need = moe::sort_workspace(n_tokens, top_k, n_experts);
    CHECK(need == 0 || (!bad(workspace_dev, 4) && workspace_bytes >= need), "this sort needs %zu bytes of workspace", need);
    return launched(moe::launch_sort(atype, n_tokens ? x_dev : nullptr, x_stride, topk_ids_dev, n_tokens, top_k,
                                     n_experts, x_dev ? hidden : 0, to_fp8 != 0, sorted_dev, scales_dev, offsets_dev, rows_dev,
                                     workspace_dev, static_cast<hipStream_t>(stream)),
                    "sort");
}

moe_status_t moe_combine_rows(int32_t atype, const void* ys_dev, const int32_t* rows_dev, const float* topk_w_dev,
                              const void* resid_dev, int32_t n_tokens, int32_t top_k, int32_t hidden, void* out_dev,
                              void* stream) {
    if (const moe_status_t st = check_pairs(atype, n_tokens, top_k)) return st;
    if (const moe_status_t st = check_hidden(hidden)) return st;
    if (n_tokens == 0) return MOE_OK;
    const size_t es = act_size(atype);
    CHECK(!bad(ys_dev, es) && !bad(rows_dev, 4) && aligned(topk_w_dev, 4) && aligned(resid_dev, es) && !bad(out_dev, es),
          "null or misaligned buffer");
    return launched(moe::launch_combine(atype, ys_dev, rows_dev, topk_w_dev, resid_dev, n_tokens, top_k, hidden,
                                        out_dev, static_cast<hipStream_t>(stream)),
                    "combine");
}

moe_status_t moe_combine_rows_backward(int32_t atype, const void* d_out_dev, const void* ys_dev,
                                       const int32_t* rows_dev, const float* topk_w_dev, int32_t n_tokens,
                                       int32_t top_k, int32_t hidden, void* d_ys_dev, float* d_topk_w_dev,
                                       void* stream) {
    if (const moe_status_t st = check_pairs(atype, n_tokens, top_k)) return st;
    if (const moe_status_t st = check_hidden(hidden)) return st;
    if (n_tokens == 0) return MOE_OK;
    const size_t es = act_size(atype);
    CHECK(!bad(d_out_dev, es) && !bad(ys_dev, es) && !bad(rows_dev, 4) && !bad(topk_w_dev, 4) && !bad(d_ys_dev, es) &&
              !bad(d_topk_w_dev, 4),
          "null or misaligned buffer");
    return launched(moe::launch_combine_backward(atype, d_out_dev, ys_dev, rows_dev, topk_w_dev, n_tokens, top_k,
                                                 hidden, d_ys_dev, d_topk_w_dev, static_cast<hipStream_t>(stream)),
                    "combine_backward");
}

moe_status_t moe_scaled_product(const void* x_dev, const float* x_scales_dev, const void* w_dev,
                                const float* w_scales_dev, const int32_t* offsets_dev, int32_t n_rows,
                                int32_t n_groups, int32_t n_cols, int32_t depth, int32_t epilogue, void* out_dev,
                                float* out_scales_dev, void* stream) {
    CHECK(n_rows >= 0 && n_rows <= kMaxPairs, "n_rows %d outside [0,%lld]", n_rows, (long long)kMaxPairs);
    CHECK(n_groups >= 1 && n_groups <= moe::kMaxExperts, "n_groups %d outside [1,%d]", n_groups, moe::kMaxExperts);
    CHECK(n_groups == 1 || offsets_dev, "%d groups need offsets", n_groups);
    CHECK(aligned(offsets_dev, 4), "misaligned offsets");
    CHECK(n_cols >= 1 && n_cols <= 2 * kMaxHidden, "n_cols %d outside [1,%d]", n_cols, 2 * kMaxHidden);
    CHECK((int64_t)n_rows * n_cols <= kMaxElements, "n_rows * n_cols above %lld", (long long)kMaxElements);
    CHECK(depth >= 16 && depth <= kMaxHidden && depth % 16 == 0, "depth %d: multiples of 16 up to %d", depth, kMaxHidden);
    CHECK(epilogue >= MOE_PRODUCT_F32 && epilogue <= MOE_PRODUCT_SWIGLU, "epilogue %d invalid", epilogue);
    const bool swiglu = epilogue == MOE_PRODUCT_SWIGLU;
    CHECK(!swiglu || n_cols % 256 == 0, "n_cols %d: the SwiGLU epilogue needs a multiple of 256", n_cols);
    if (n_rows == 0) return MOE_OK;
    CHECK(!bad(x_dev, 16) && !bad(w_dev, 16) && !bad(x_scales_dev, 4) && !bad(w_scales_dev, 4) &&
              !bad(out_dev, swiglu ? 16 : epilogue == MOE_PRODUCT_F32 ? 4 : 2) && (!swiglu || !bad(out_scales_dev, 4)),
          "null or misaligned buffer (x and w: 16 bytes)");
    moe::ProductArgs a{};
    a.x = static_cast<const uint8_t*>(x_dev);
    a.xs = x_scales_dev;
    a.w = static_cast<const uint8_t*>(w_dev);
    a.ws = w_scales_dev;
    a.offsets = offsets_dev;
    a.out = out_dev;
    a.os = swiglu ? out_scales_dev : nullptr;
    a.M = n_rows;
    a.G = n_groups;
    a.N = n_cols;
    a.K = depth;
    return launched(moe::launch_scaled_product(a, epilogue, static_cast<hipStream_t>(stream)), "scaled_product");
}

}  // extern "C"
