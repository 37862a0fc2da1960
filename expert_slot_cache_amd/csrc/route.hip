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
// Sixteen lanes (a DPP row) take a token up to 512 experts, a wave above that.  Lane i of them
// holds the logits i*V .. i*V + V-1 as unsigned keys in float order, so that of equal keys the
// lowest lane's lowest one is the lowest id (a bf16 logit's key holds the id as well, and no two
// are equal).  The keys are put in order by eights; a round of the selection is the maximum of
// the eights' heads over the lanes (DPP, no LDS), which the first lane that holds it takes out of
// the first of its eights that does.  Softmax sums are fp32.  A large call is bound by the
// instructions issued: 16384 tokens of 512 experts, top-10, take 17.0 us in fp32 (33.5 MB read)
// and 12.5 us in bf16; one token per wave and a search through its registers took 22 us in
// fp32, exchanges of neighbours throughout, which keep equal keys in place, 17.9 and 16.8 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"
#include "route_dev.hpp"

namespace moe {
namespace {

template <int AT, int L, int V, bool RENORM>
__global__ __launch_bounds__(64 * kTokensPerBlock) void k_route(const void* __restrict__ logits, int64_t stride, int T,
        int E, int K, int32_t* __restrict__ ids, float* __restrict__ w) {
    constexpr int PER = 64 / L;                        // tokens of a wave
    __shared__ uint2 found[kTokensPerBlock][PER][kMaxTopK];   // (id, key) in order
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = lane / L, l = lane % L;            // the wave's token, and the lane in it
    const int t = (blockIdx.x * kTokensPerBlock + wave) * PER + sub;
    const bool here = t < T;                           // the wave's other lanes go through the motions,
    const int n = here ? E : 0;                        // with no logits
    float logit[V], sum = 0.0f;
    load_logits<AT, V>(logits, (size_t)(here ? t : 0) * (size_t)stride, n, l, logit);
    const float m = softmax_sum<L, V>(logit, !RENORM, &sum);
    constexpr bool NAMES = AT == A_F32;
    Eights<V, NAMES> keys;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = l * V + j;                       // absent keys: none equal
        if constexpr (NAMES) keys.key[j] = e < n ? key_of(logit[j]) : (uint32_t)j;
        else keys.key[j] = e < n ? key_of(logit[j], e) : (uint32_t)j;
    }
    keys.order();
    const uint64_t below = L == 64 ? 0 : ((1ull << lane) - 1) & (0xffffull << (lane & 48));   // of this token's
    for (int k = 0; k < K; ++k) {
        const uint32_t best = keys.best(), top = lanes_max<L>(best);
        bool mine = best == top;
        if constexpr (NAMES) {
            const uint64_t holds = __ballot(mine);
            if constexpr (L == 64) mine = lane == __builtin_ctzll(holds);   // some lane holds top
            else mine = mine && (holds & below) == 0;
        }
        const int at = keys.take(top, mine);
        if (mine) found[wave][sub][k] = make_uint2(NAMES ? (uint32_t)(l * V + at) : 0xffff - (top & 0xffff), top);
    }
    __builtin_amdgcn_wave_barrier();                   // LDS operations of one wave complete in order
    const uint2* f = found[wave][sub];
    float mine[kMaxTopK / L];
    if constexpr (RENORM) sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxTopK / L; ++i) {
        const int k = l + i * L;
        mine[i] = k < K ? term(NAMES ? logit_of(f[k].y) : logit_of_id(f[k].y), m) : 0.0f;
        if constexpr (RENORM) sum += mine[i];
    }
    if constexpr (RENORM) sum = lanes_sum<L>(sum);
#pragma unroll
    for (int i = 0; i < kMaxTopK / L; ++i) {
        const int k = l + i * L;
        if (!here || k >= K) continue;
        const size_t o = (size_t)t * K + k;
        ids[o] = (int32_t)f[k].x;
        w[o] = sum > 0.0f ? mine[i] / sum : 0.0f;
    }
}

template <int AT, int V, bool RENORM>
__global__ __launch_bounds__(64 * kTokensPerBlock) void k_route_backward(const void* __restrict__ logits, int64_t stride,
        const int32_t* __restrict__ ids, const float* __restrict__ w, const float* __restrict__ dw, int T, int E, int K,
        void* __restrict__ dl, int64_t dstride) {
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
        float l[V], sum = 0.0f;
        load_logits<AT, V>(logits, (size_t)t * (size_t)stride, E, lane, l);
        const float m = softmax_sum<64, V>(l, true, &sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float p = term(l[j], m);
            d[j] = p > 0.0f ? p * inv * (d[j] - s) : 0.0f;
        }
    }
    const size_t row = (size_t)t * (size_t)dstride;
    const int e0 = lane * V;
    constexpr int N = Piece<AT>::N;
    if constexpr (V >= N) {
#pragma unroll
        for (int c = 0; c < V; c += N) {
            Piece<AT> p;
#pragma unroll
            for (int j = 0; j < N; ++j) p.v[j] = d[c + j];
            const int left = E - e0 - c;
            if (left >= N) p.template store<true, false>(dl, (int64_t)(row + e0 + c), N);
            else p.template store<false, false>(dl, (int64_t)(row + e0 + c), left);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < E) store_one<AT>(dl, row + e0 + j, d[j]);
    }
}

template <int AT, bool RENORM>
hipError_t route(const void* logits, int64_t stride, int T, int E, int K, int32_t* ids, float* w, hipStream_t s) {
    auto run = [&](auto lanes, auto v) {
        constexpr int L = decltype(lanes)::value, V = decltype(v)::value;
        constexpr int tokens = kTokensPerBlock * 64 / L;
        hipLaunchKernelGGL((k_route<AT, L, V, RENORM>), dim3((T + tokens - 1) / tokens), dim3(64 * kTokensPerBlock), 0, s,
                           logits, stride, T, E, K, ids, w);
        return hipGetLastError();
    };
    if (E > 512) return by_width<16>(64, E, [&](auto v) { return run(std::integral_constant<int, 64>{}, v); });
    return by_width<1>(16, E, [&](auto v) {
        if constexpr (decltype(v)::value <= 32) return run(std::integral_constant<int, 16>{}, v);
        else return hipErrorInvalidValue;              // more than 512
    });
}

template <int AT, bool RENORM>
hipError_t route_backward(const void* logits, int64_t stride, const int32_t* ids, const float* w, const float* dw, int T,
                          int E, int K, void* dl, int64_t dstride, hipStream_t s) {
    return by_width<1>(64, E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((k_route_backward<AT, V, RENORM>), dim3((T + kTokensPerBlock - 1) / kTokensPerBlock),
                           dim3(64 * kTokensPerBlock), kTokensPerBlock * 64 * V * sizeof(float), s, logits, stride, ids,
                           w, dw, T, E, K, dl, dstride);
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
