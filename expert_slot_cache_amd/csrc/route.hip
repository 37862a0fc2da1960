// The router's top-k and its gradient.
//
//   p   = softmax(l)                         over the E logits of a token
//   ids = the K largest logits, largest first, equal ones in ascending id order
//   w   = p[ids], or (renormalised) exp(l[ids]) / sum of exp(l[ids])
// and, with s = sum_k w_k dw_k and g_e the sum of dw over the k that chose e,
//   dl_e = p_e (g_e - s)                     or  sum over those k of w_k (dw_k - s).
// "Running 125B MoE on Two 32 GB Cards", section 4.2: on a tie of two logits the lower
// id wins.
//
// A wave takes a token.  Lane i holds the logits i*V .. i*V + V-1 as unsigned keys in
// float order, so the lowest lane and the lowest register of equal keys is the lowest id.
// A round of the selection is one wave-wide maximum (six DPP steps, no LDS), a ballot of
// the lanes that hold it and a removal in the first of them.  Softmax sums are fp32.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"
#include "ops_dev.hpp"

namespace moe {
namespace {

constexpr int kTokensPerBlock = 4;   // waves per workgroup

// Float order as unsigned order, every real key > 0 (0 marks a key that is absent or
// taken).  NaN counts as -inf, and both zeros are equal.
__device__ __forceinline__ uint32_t key_of(float l) {
    if (!(l == l)) l = -__builtin_inff();
    const uint32_t b = l == 0.0f ? 0u : __float_as_uint(l);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}
// exp(l - m) for l <= m, with the limits at infinite logits: equal ones count 1 each.
// A row of -inf alone (m = -inf) has no softmax: every term is 0.
__device__ __forceinline__ float term(float l, float m) {
    if (m == -__builtin_inff()) return 0.0f;
    return l == m ? 1.0f : expf(l - m);
}

// A token's logits: V consecutive ones per lane, as keys; 0 past the end.  `wide` (host:
// base and stride allow it and E is a multiple of V): 16-byte loads.
template <int AT, int V>
__device__ __forceinline__ void load_keys(const void* logits, size_t row, int E, int lane, bool wide, uint32_t key[V]) {
    constexpr int PER = AT == A_F32 ? 4 : 8;
    const int e0 = lane * V;
    if constexpr (V >= PER) {
        if (wide) {
            const char* p = static_cast<const char*>(logits) + (row + e0) * (AT == A_F32 ? 4 : 2);
            uint4 q[V / PER];
            if (e0 < E) {
#pragma unroll
                for (int c = 0; c < V / PER; ++c) q[c] = reinterpret_cast<const uint4*>(p)[c];
            }
#pragma unroll
            for (int c = 0; c < V / PER; ++c) {
                const uint32_t u[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const float l = AT == A_F32 ? __uint_as_float(u[i & 3]) : widen_bf16((uint16_t)(u[i >> 1] >> (16 * (i & 1))));
                    key[c * PER + i] = e0 < E ? key_of(l) : 0u;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = e0 + j < E ? key_of(load_one<AT>(logits, row + e0 + j)) : 0u;
}

template <int AT, int V, bool RENORM>
__global__ __launch_bounds__(64 * kTokensPerBlock) void k_route(const void* __restrict__ logits, int64_t stride, int T,
        int E, int K, bool wide, int32_t* __restrict__ ids, float* __restrict__ w) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kTokensPerBlock + (threadIdx.x >> 6);
    if (t >= T) return;
    uint32_t key[V];
    load_keys<AT, V>(logits, (size_t)t * (size_t)stride, E, lane, wide, key);
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) best = key[j] > best ? key[j] : best;
    uint32_t top = wave_max_u32(best);
    const float m = logit_of(top);
    float sum = 0.0f;
    if constexpr (!RENORM) {
#pragma unroll
        for (int j = 0; j < V; ++j) sum += key[j] ? term(logit_of(key[j]), m) : 0.0f;
        sum = wave_sum(sum);
    }
    int my_id = 0;
    uint32_t my_key = 0;
    for (int k = 0; k < K; ++k) {
        if (k) top = wave_max_u32(best);
        const int first = __builtin_ctzll(__ballot(best == top));   // some lane holds top
        // the first lane's lowest register with that key, removed
        int at = V;
        uint32_t next = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool hit = key[j] == top && at == V;
            if (hit) at = j;
            const uint32_t rest = hit ? 0u : key[j];
            next = rest > next ? rest : next;
            if (lane == first) key[j] = rest;
        }
        if (lane == first) best = next;
        const int id = first * V + __builtin_amdgcn_readlane(at, first);
        if (lane == k) {
            my_id = id;
            my_key = top;
        }
    }
    float mine = lane < K ? term(logit_of(my_key), m) : 0.0f;
    if constexpr (RENORM) sum = wave_sum(mine);
    if (lane < K) {
        const size_t o = (size_t)t * K + lane;
        ids[o] = my_id;
        w[o] = sum > 0.0f ? mine / sum : 0.0f;
    }
}

template <int AT, int V, bool RENORM>
__global__ __launch_bounds__(64 * kTokensPerBlock) void k_route_backward(const void* __restrict__ logits, int64_t stride,
        const int32_t* __restrict__ ids, const float* __restrict__ w, const float* __restrict__ dw, int T, int E, int K,
        bool wide, bool wide_out, void* __restrict__ dl, int64_t dstride) {
    extern __shared__ float lds[];
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kTokensPerBlock + (threadIdx.x >> 6);
    if (t >= T) return;
    // g[e]: what the chosen experts add, one row of 64 V floats per wave
    float* g = lds + (threadIdx.x >> 6) * (64 * V);
    int id = -1;
    float wk = 0.0f, dk = 0.0f;
    if (lane < K) {
        const size_t o = (size_t)t * K + lane;
        id = ids[o];
        wk = w[o];
        dk = dw[o];
        if ((unsigned)id >= (unsigned)E) id = -1;
    }
    const float s = wave_sum(id >= 0 ? wk * dk : 0.0f);
    const float mine = RENORM ? wk * (dk - s) : dk;
    // an id chosen twice gets the sum over its k, in k order, from each of them alike
    float total = 0.0f;
    for (int k = 0; k < K; ++k) {
        const int other = __builtin_amdgcn_readlane(id, k);
        const float c = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(mine), k));
        total += other == id ? c : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) g[j * 64 + lane] = 0.0f;
    __builtin_amdgcn_wave_barrier();   // LDS operations of one wave complete in order
    if (id >= 0) g[id] = total;
    __builtin_amdgcn_wave_barrier();
    float d[V];
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = g[lane * V + j];
    if constexpr (!RENORM) {
        uint32_t key[V];
        load_keys<AT, V>(logits, (size_t)t * (size_t)stride, E, lane, wide, key);
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) best = key[j] > best ? key[j] : best;
        const float m = logit_of(wave_max_u32(best));
        float p[V], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            p[j] = key[j] ? term(logit_of(key[j]), m) : 0.0f;
            sum += p[j];
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = p[j] > 0.0f ? p[j] * inv * (d[j] - s) : 0.0f;
    }
    const size_t row = (size_t)t * (size_t)dstride;
    const int e0 = lane * V;
    constexpr int PER = AT == A_F32 ? 4 : 8;
    if constexpr (V >= PER) {
        if (wide_out) {
            if (e0 < E) {
                char* p = static_cast<char*>(dl) + (row + e0) * (AT == A_F32 ? 4 : 2);
#pragma unroll
                for (int c = 0; c < V / PER; ++c) {
                    uint32_t u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (AT == A_F32) u[i] = __float_as_uint(d[c * 4 + i]);
                        else u[i] = round_bf16(d[c * 8 + 2 * i]) | (uint32_t)round_bf16(d[c * 8 + 2 * i + 1]) << 16;
                    }
                    reinterpret_cast<uint4*>(p)[c] = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (e0 + j < E) store_one<AT>(dl, row + e0 + j, d[j]);
}

// 16-byte accesses: every lane's V values start on 16 bytes and lie inside the row.
bool is_wide(const void* p, int64_t stride, int esize, int V, int E) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * esize % 16 == 0 && V * esize % 16 == 0 && E % V == 0;
}

template <class F>
hipError_t by_width(int E, F f) {
    if (E <= 64) return f(std::integral_constant<int, 1>{});
    if (E <= 128) return f(std::integral_constant<int, 2>{});
    if (E <= 256) return f(std::integral_constant<int, 4>{});
    if (E <= 512) return f(std::integral_constant<int, 8>{});
    if (E <= 1024) return f(std::integral_constant<int, 16>{});
    if (E <= 2048) return f(std::integral_constant<int, 32>{});
    return f(std::integral_constant<int, 64>{});
}

template <int AT, bool RENORM>
hipError_t route(const void* logits, int64_t stride, int T, int E, int K, int32_t* ids, float* w, hipStream_t s) {
    return by_width(E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((k_route<AT, V, RENORM>), dim3((T + kTokensPerBlock - 1) / kTokensPerBlock),
                           dim3(64 * kTokensPerBlock), 0, s, logits, stride, T, E, K,
                           is_wide(logits, stride, AT == A_F32 ? 4 : 2, V, E), ids, w);
        return hipGetLastError();
    });
}

template <int AT, bool RENORM>
hipError_t route_backward(const void* logits, int64_t stride, const int32_t* ids, const float* w, const float* dw, int T,
                          int E, int K, void* dl, int64_t dstride, hipStream_t s) {
    return by_width(E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        constexpr int es = AT == A_F32 ? 4 : 2;
        hipLaunchKernelGGL((k_route_backward<AT, V, RENORM>), dim3((T + kTokensPerBlock - 1) / kTokensPerBlock),
                           dim3(64 * kTokensPerBlock), kTokensPerBlock * 64 * V * sizeof(float), s, logits, stride, ids,
                           w, dw, T, E, K, is_wide(logits, stride, es, V, E), is_wide(dl, dstride, es, V, E), dl, dstride);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_route(int atype, const void* logits, int64_t stride, int T, int E, int K, bool renorm, int32_t* ids,
                        float* w, hipStream_t s) {
    if (atype == A_F32)
        return renorm ? route<A_F32, true>(logits, stride, T, E, K, ids, w, s) : route<A_F32, false>(logits, stride, T, E, K, ids, w, s);
    return renorm ? route<A_BF16, true>(logits, stride, T, E, K, ids, w, s) : route<A_BF16, false>(logits, stride, T, E, K, ids, w, s);
}

hipError_t launch_route_backward(int atype, const void* logits, int64_t stride, const int32_t* ids, const float* w,
                                 const float* dw, int T, int E, int K, bool renorm, void* dl, int64_t dstride,
                                 hipStream_t s) {
    if (atype == A_F32)
        return renorm ? route_backward<A_F32, true>(logits, stride, ids, w, dw, T, E, K, dl, dstride, s)
                      : route_backward<A_F32, false>(logits, stride, ids, w, dw, T, E, K, dl, dstride, s);
    return renorm ? route_backward<A_BF16, true>(logits, stride, ids, w, dw, T, E, K, dl, dstride, s)
                  : route_backward<A_BF16, false>(logits, stride, ids, w, dw, T, E, K, dl, dstride, s);
}

}  // namespace moe
