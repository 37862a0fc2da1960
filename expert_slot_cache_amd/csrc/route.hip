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
#include "ops_dev.hpp"

namespace moe {
namespace {

constexpr int kTokensPerBlock = 4;   // waves per workgroup

// Float order as unsigned order, every real key > 0x7f0000 (less marks one that is absent or taken).
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}
// A bf16 logit's key has its lower half to spare: the id, the lowest largest.  No two are equal.
__device__ __forceinline__ uint32_t key_of(float l, int id) { return (key_of(l) & 0xffff0000u) | (uint32_t)(0xffff - id); }
__device__ __forceinline__ float logit_of_id(uint32_t k) { return logit_of(k & 0x80000000u ? k & 0xffff0000u : k | 0xffffu); }
// exp(l - m) for l <= m: the difference first, so that rows of any size keep in range (a whole
// row of the type's lowest value is a uniform one), then 2^(d log2 e), within |d| 2^-23 of the
// value.  With m infinite: equal logits count 1 each, the limit at +inf, and a row of -inf alone
// has no softmax, every term is 0.
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float finite_term(float l, float m) { return __builtin_amdgcn_exp2f((l - m) * kLog2e); }
__device__ __forceinline__ float term(float l, float m) {
    if (fabsf(m) < __builtin_inff()) return finite_term(l, m);
    return m > 0.0f && l == m ? 1.0f : 0.0f;
}

// The largest value over the L lanes of a token (16: a DPP row, or the wave), in all of them.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (L == 64) return wave_max_u32(v);
    auto turn = [&](auto ctrl) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xf, 0xf, false);
        v = o > v ? o : v;
    };
    turn(std::integral_constant<int, 0x128>{});   // row_ror:8, 4, 2, 1
    turn(std::integral_constant<int, 0x124>{});
    turn(std::integral_constant<int, 0x122>{});
    turn(std::integral_constant<int, 0x121>{});
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (L == 64) return wave_sum(v);
    auto turn = [&](auto ctrl) {
        v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    turn(std::integral_constant<int, 0x128>{});
    turn(std::integral_constant<int, 0x124>{});
    turn(std::integral_constant<int, 0x122>{});
    turn(std::integral_constant<int, 0x121>{});
    return v;
}

// A lane's V keys in eights, each in descending order, and (NAMES) the places its keys had.
template <int V, bool NAMES>
struct Eights {
    static constexpr int W = V < 8 ? V : 8, N = V / W;
    uint32_t key[V];
    uint32_t names[NAMES ? N : 1];   // four bits per key
    template <class F>
    static __device__ __forceinline__ void exchange(uint32_t* k, uint32_t* name, int i, int j, F falls) {
        // values, not elements: a choice between two elements becomes an address
        const uint32_t a = k[i], b = k[j];
        if constexpr (NAMES) {
            const uint32_t an = name[i], bn = name[j];
            const bool swap = falls(a, an, b, bn);
            name[i] = swap ? bn : an;
            name[j] = swap ? an : bn;
            k[i] = swap ? b : a;
            k[j] = swap ? a : b;
        } else {
            k[i] = max(a, b);
            k[j] = min(a, b);
        }
    }
    // By Batcher's merge exchange: 19 for eight keys; of four or two those whose sides exist.  That
    // may turn equal keys round: where a wave has some, exchanges of neighbours put them right.
    __device__ __forceinline__ void order() {
        constexpr int net[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                    {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
        uint32_t name[V];
        bool equal = false;
#pragma unroll
        for (int j = 0; j < V; ++j) name[j] = j % W;
#pragma unroll
        for (int g = 0; g < N; ++g) {
#pragma unroll
            for (int i = 0; i < 19; ++i)
                if (net[i][1] < W)
                    exchange(key + g * W, name + g * W, net[i][0], net[i][1],
                             [](uint32_t a, uint32_t, uint32_t b, uint32_t) { return a < b; });
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) equal |= key[g * W + j] == key[g * W + j + 1];
        }
        if constexpr (NAMES) {
            if (__any(equal))
#pragma unroll
                for (int g = 0; g < N; ++g)
#pragma unroll
                    for (int r = 0; r < W; ++r)
#pragma unroll
                        for (int j = r & 1; j + 1 < W; j += 2)
                            exchange(key + g * W, name + g * W, j, j + 1, [](uint32_t a, uint32_t an, uint32_t b, uint32_t bn) {
                                return a == b && an > bn;
                            });
#pragma unroll
            for (int g = 0; g < N; ++g) {
                names[g] = 0;
#pragma unroll
                for (int j = 0; j < W; ++j) names[g] |= name[g * W + j] << (4 * j);
            }
        }
    }
    __device__ __forceinline__ uint32_t best() const {
        uint32_t b = key[0];
#pragma unroll
        for (int g = 1; g < N; ++g) b = max(b, key[g * W]);
        return b;
    }
    // Where `mine`: takes `top` out of the first of the eights that it heads; (NAMES) its place.
    __device__ __forceinline__ int take(uint32_t top, bool mine) {
        int at = 0;
#pragma unroll
        for (int g = 0; g < N; ++g) {
            const bool hit = mine && key[g * W] == top;
            if constexpr (NAMES) {
                mine = mine && !hit;
                at = hit ? g * W + (int)(names[g] & 15) : at;
                names[g] = hit ? names[g] >> 4 : names[g];
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const uint32_t next = j + 1 < W ? key[g * W + j + 1] : 0u;
                key[g * W + j] = hit ? next : key[g * W + j];
            }
        }
        return at;
    }
};

// A token's logits: V consecutive ones per lane; NaN counts as -inf (fmaxf drops it), both zeros
// are equal (-0 + 0 = 0), and past the end there are -inf.
template <int AT, int V>
__device__ __forceinline__ void load_logits(const void* logits, size_t row, int E, int lane, float l[V]) {
    constexpr int N = Piece<AT>::N;
    const int e0 = lane * V;
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = -__builtin_inff();
    auto piece = [&](int c) {                              // a lane comes back to its lines: not `once`
        Piece<AT> p;
        p.template load<true>(logits, (int64_t)(row + e0 + c), N, false);
#pragma unroll
        for (int j = 0; j < N; ++j) l[c + j] = p.v[j];
    };
    if (V >= N && E % V == 0) {                            // no lane has a part of its share: no choice per piece
        if (e0 < E)
#pragma unroll
            for (int c = 0; c + N <= V; c += N) piece(c);
    } else if (V >= N) {
#pragma unroll
        for (int c = 0; c + N <= V; c += N) {
            if (e0 + c + N <= E) piece(c);
            else if (e0 + c < E)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (e0 + c + j < E) l[c + j] = load_one<AT>(logits, row + e0 + c + j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < E) l[j] = load_one<AT>(logits, row + e0 + j);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = fmaxf(l[j], -__builtin_inff()) + 0.0f;
}

// The largest logit of a token's L lanes, and, with `all`, the sum of the terms.
template <int L, int V>
__device__ __forceinline__ float softmax_sum(const float l[V], bool all, float* sum) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) best = max(best, key_of(l[j]));
    const float m = logit_of(lanes_max<L>(best));
    if (all) {
        float s = 0.0f;
        if (__all(fabsf(m) < __builtin_inff())) {      // the same terms, without their special cases
#pragma unroll
            for (int j = 0; j < V; ++j) s += finite_term(l[j], m);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) s += term(l[j], m);
        }
        *sum = lanes_sum<L>(s);
    }
    return m;
}

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

// The least of V, 2V, .. 64 keys per lane that `lanes` lanes hold E keys with.
template <int V, class F>
hipError_t by_width(int lanes, int E, F f) {
    if constexpr (V < 64)
        if (E > lanes * V) return by_width<2 * V>(lanes, E, f);
    return f(std::integral_constant<int, V>{});
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
