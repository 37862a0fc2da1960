// Device helpers of the routers: logits as ordered keys, and the selection of the largest.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops_dev.hpp"

namespace moe {

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

template <int L>
__device__ __forceinline__ uint32_t lanes_or(uint32_t v) {
    if constexpr (L == 64) return wave_reduce_u32(v, [](uint32_t a, uint32_t b) { return a | b; });
    auto turn = [&](auto ctrl) { v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xf, 0xf, false); };
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

// The least of V, 2V, .. 64 keys per lane that `lanes` lanes hold E keys with.
template <int V, class F>
hipError_t by_width(int lanes, int E, F f) {
    if constexpr (V < 64)
        if (E > lanes * V) return by_width<2 * V>(lanes, E, f);
    return f(std::integral_constant<int, V>{});
}

}  // namespace moe
