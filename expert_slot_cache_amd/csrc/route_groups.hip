// A router whose choice has a bias for balance and is kept to the best groups of experts, and its
// gradient.
//
//   s_e = softmax(l)_e, or 1 / (1 + exp(-l_e))                  the scores
//   c_e = s_e + b_e                                             what is chosen by
//   G_g = the sum of the one or two largest c of group g        the groups are runs of E / n_groups experts
//   ids = the K largest c of the experts of the kept groups' largest G
//   w   = scale s[ids], or (renormalised) scale s[ids] / sum of s[ids]
// and, with S = sum_k w_k dw_k and g_e the sum of dw over the k that chose e,
//   softmax:               dl_e = p_e (scale g_e - S)
//   softmax, renormalised: dl_e = the sum over the k of e of w_k (dw_k - S / scale)
//   sigmoid:               ... of w_k (1 - s_k) dw_k, renormalised w_k (1 - s_k) (dw_k - S / scale):
// w_k / scale stands for the score's share, so that no sum has to be taken again.
//
// Choices are compared as in 64 bits, for two experts whose scores differ in the tenth digit are
// no tie.  They are taken in fp32, with a bound of what that may be off, and put in order as in
// the plain router (sixteen lanes a token up to 512 experts, a wave above that); where two
// neighbours in that order, or the last group kept and the first left out, lie nearer to each
// other than the bound, the wave takes that token once more in fp64.  Without a bias the logits
// themselves are the order, which needs no bound.
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "route_dev.hpp"

namespace moe {
namespace {

// A score with its largest common factor taken out, exp(min(l, 0) - shift) / (1 + exp(-|l|)):
// with shift = 0 the sigmoid, with the least of 0 and the largest of some logits a term of their
// ratios that stays in range whatever their size.
__device__ __forceinline__ float sigmoid_term(float l, float shift) {
    const float below = fminf(l, 0.0f);
    const float top = below == shift ? 1.0f : __builtin_amdgcn_exp2f((below - shift) * kLog2e);
    return top * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-fabsf(l) * kLog2e));
}

// The order of doubles as unsigned numbers above 0.
__device__ __forceinline__ uint64_t key64_of(double c) {
    const uint64_t b = __builtin_bit_cast(uint64_t, c);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ uint64_t shfl64(uint64_t v, int mask) {
    return (uint64_t)(uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), mask) << 32 | (uint32_t)__shfl_xor((int)(uint32_t)v, mask);
}
__device__ __forceinline__ double shfl64(double v, int mask) {
    return __builtin_bit_cast(double, shfl64(__builtin_bit_cast(uint64_t, v), mask));
}

// A token by a whole wave in fp64: its K experts into ids, in order.  VS: experts of a lane,
// 64 apart.
template <int AT, int VS>
__device__ __forceinline__ void choose_exactly(const void* __restrict__ logits, size_t row, const float* __restrict__ bias,
                                            const RouteGroups& r, uint2* found) {
    const int lane = threadIdx.x & 63;
    const double low = -(double)__builtin_inff();
    float l[VS];
    double c[VS];
    float m = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < VS; ++j) {
        const int e = j * 64 + lane;
        l[j] = e < r.E ? fmaxf(load_one<AT>(logits, row + e), -__builtin_inff()) : -__builtin_inff();
        m = fmaxf(m, l[j]);
    }
    double sum = 1.0;
    if (!r.sigmoid) {
#pragma unroll
        for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
        sum = 0.0;
    }
#pragma unroll
    for (int j = 0; j < VS; ++j) {
        if (r.sigmoid) c[j] = 1.0 / (1.0 + exp(-(double)l[j]));
        else if (fabsf(m) < __builtin_inff()) c[j] = exp((double)l[j] - (double)m);
        else c[j] = m > 0.0f && l[j] == m ? 1.0 : 0.0;
        if (!r.sigmoid) sum += c[j];
    }
    if (!r.sigmoid) {
#pragma unroll
        for (int d = 32; d; d >>= 1) sum += shfl64(sum, d);
        if (sum == 0.0) sum = 1.0;
    }
    uint64_t key[VS];                                      // 0: no choice
#pragma unroll
    for (int j = 0; j < VS; ++j) {
        const int e = j * 64 + lane;
        c[j] /= sum;
        // without a bias the order is the logits'
        double by = bias ? c[j] + (e < r.E ? (double)bias[e] : 0.0) : (double)l[j];
        if (!(by == by) || l[j] == -__builtin_inff()) by = low;
        if (bias) c[j] = by;
        else if (by == low) c[j] = low;
        key[j] = e < r.E ? key64_of(by + 0.0) : 0;
    }
    if (r.kept < r.n_groups) {
        const int size = r.E / r.n_groups;
        double score = low;
        for (int g = 0; g < r.n_groups; ++g) {
            double one = low, two = low;
#pragma unroll
            for (int j = 0; j < VS; ++j) {
                const int e = j * 64 + lane - g * size;
                if (e < 0 || e >= size) continue;
                two = fmax(two, fmin(one, c[j]));
                one = fmax(one, c[j]);
            }
#pragma unroll
            for (int d = 32; d; d >>= 1) {
                const double o1 = shfl64(one, d), o2 = shfl64(two, d);
                two = fmax(fmin(one, o1), fmax(two, o2));
                one = fmax(one, o1);
            }
            if (lane == g) score = r.group_top > 1 && two > low ? one + two : one;
        }
        int rank = 0;
        for (int g = 0; g < r.n_groups; ++g) {
            const uint64_t b = __builtin_bit_cast(uint64_t, score);
            const double o = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), g) << 32 |
                                                            (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, g));
            rank += o > score || (o == score && g < lane);
        }
        const uint64_t kept = __ballot(lane < r.n_groups && rank < r.kept);
#pragma unroll
        for (int j = 0; j < VS; ++j) {
            const int e = j * 64 + lane;
            if (e < r.E && !((kept >> (e / size)) & 1)) key[j] = 0;
        }
    }
    for (int k = 0; k < r.K; ++k) {
        uint64_t top = 0;
        int at = 0;
#pragma unroll
        for (int j = 0; j < VS; ++j)
            if (key[j] > top) {
                top = key[j];
                at = j * 64 + lane;
            }
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            const uint64_t o = shfl64(top, d);
            const int oat = __shfl_xor(at, d);
            if (o > top || (o == top && oat < at)) {
                top = o;
                at = oat;
            }
        }
#pragma unroll
        for (int j = 0; j < VS; ++j)
            if (j * 64 + lane == at) key[j] = 0;
        if (lane == 0) found[k].x = (uint32_t)at;
    }
}

template <int AT, int L, int V>
__global__ __launch_bounds__(64 * kTokensPerBlock) void k_route_groups(const void* __restrict__ logits, int64_t stride,
        const float* __restrict__ bias, int T, RouteGroups r, int32_t* __restrict__ ids, float* __restrict__ w) {
    constexpr int PER = 64 / L;                        // tokens of a wave
    __shared__ uint2 found[kTokensPerBlock][PER][kMaxTopK + 1];   // (id, key) in order
    __shared__ float shared_g[kTokensPerBlock][PER][kMaxGroups];
    extern __shared__ float shared_c[];                // [waves][PER][L * V], where groups are left out
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = lane / L, i = lane % L;            // the wave's token, and the lane in it
    const int t = (blockIdx.x * kTokensPerBlock + wave) * PER + sub;
    const bool here = t < T;
    const int n = here ? r.E : 0;
    const size_t row = (size_t)(here ? t : 0) * (size_t)stride;
    const float low = -__builtin_inff();
    float c[V], m = 0.0f, sum = 1.0f;
    load_logits<AT, V>(logits, row, n, i, c);
    if (!r.sigmoid) m = softmax_sum<L, V>(c, true, &sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    // What a choice may be off in fp32, twice.  Sigmoid: the exponential moves it by at most
    // s (1 - s) (1 + |l|) 2^-23, the sum and the reciprocal by 1.5 * 2^-23.  Softmax: a term is off
    // by (|d| + 1) 2^-23 of itself and the sum by (V + 4) 2^-24, of at most the largest p (inv).
    const float off = r.sigmoid ? 0x1p-21f : inv * (V + 16) * 0x1p-23f;
    const bool by_group = r.kept < r.n_groups;
    auto score_of = [&](float l) { return r.sigmoid ? sigmoid_term(l, 0.0f) : term(l, m) * inv; };
    if (bias)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = i * V + j;
            const float b = e < n ? bias[e] : 0.0f;
            const float s = score_of(c[j]) + b;
            c[j] = c[j] == low ? low : fmaxf(s, low) + 0.0f;    // NaN counts as -inf
        }
    bool unsure = false;
    uint64_t kept = ~0ull;
    int g = 0, at = 0;                                 // of the lane's first expert
    const int size = r.E / r.n_groups;
    if (by_group) {
        float* cs = shared_c + (wave * PER + sub) * (L * V);
        float* gs = shared_g[wave][sub];
#pragma unroll
        for (int j = 0; j < V; ++j) cs[i * V + j] = c[j];
        __builtin_amdgcn_wave_barrier();               // LDS operations of one wave complete in order
        // a group's score by one lane, the lanes of a token starting at different banks
        for (int q = i; q < r.n_groups; q += L) {
            float one = low, two = low;
            int o = i < size ? i : i % size;
            for (int j = 0; j < size; ++j) {
                const float v = cs[q * size + o];
                two = fmaxf(two, fminf(one, v));
                one = fmaxf(one, v);
                o = o + 1 == size ? 0 : o + 1;
            }
            if (r.group_top > 1 && two > low) one = bias ? one + two : score_of(one) + score_of(two);
            else if (r.group_top > 1 && !bias && one > low) one = score_of(one);
            gs[q] = one;
        }
        __builtin_amdgcn_wave_barrier();
        float least = __builtin_inff(), most = low;    // of the kept, of the others
        uint32_t lo = 0, hi = 0;
        for (int q = i; q < r.n_groups; q += L) {
            const float v = gs[q];
            int rank = 0;
            for (int o = 0; o < r.n_groups; ++o) {
                const float u = gs[o];
                rank += u > v || (u == v && o < q);
            }
            if (rank < r.kept) {
                least = fminf(least, v);
                if (q < 32) lo |= 1u << q;
                else hi |= 1u << (q - 32);
            } else {
                most = fmaxf(most, v);
            }
        }
#pragma unroll
        for (int d = 1; d < L; d <<= 1) {
            least = fminf(least, __shfl_xor(least, d));
            most = fmaxf(most, __shfl_xor(most, d));
            lo |= (uint32_t)__shfl_xor((int)lo, d);
            hi |= (uint32_t)__shfl_xor((int)hi, d);
        }
        kept = (uint64_t)hi << 32 | lo;
        // infinite scores that are alike are so in fp64 too (their difference is NaN)
        if (bias || r.group_top > 1) unsure = least - most <= 2.0f * off + (fabsf(least) + fabsf(most)) * 0x1p-22f;
        g = i * V / size;
        at = i * V - g * size;
    }
    Eights<V, true> keys;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = i * V + j;                       // absent keys: none equal
        const bool can = e < n && (!by_group || ((kept >> g) & 1));
        keys.key[j] = can ? key_of(c[j]) : (uint32_t)j;
        if (by_group && ++at == size) {
            at = 0;
            ++g;
        }
    }
    keys.order();
    uint2* f = found[wave][sub];
    const uint64_t below = L == 64 ? 0 : ((1ull << lane) - 1) & (0xffffull << (lane & 48));   // of this token's
    const int rounds = bias ? r.K + 1 : r.K;           // and the first that is not chosen
    for (int k = 0; k < rounds; ++k) {
        const uint32_t best = keys.best(), top = lanes_max<L>(best);
        bool mine = best == top;
        const uint64_t holds = __ballot(mine);
        if constexpr (L == 64) mine = lane == __builtin_ctzll(holds);
        else mine = mine && (holds & below) == 0;
        const int place = keys.take(top, mine);
        if (mine) f[k] = make_uint2((uint32_t)(i * V + place), top);
    }
    __builtin_amdgcn_wave_barrier();
    if (bias) {
        for (int k = i; k < r.K && here; k += L) {
            const uint2 a = f[k], b = f[k + 1];
            if (b.y <= 0x7f0000u) continue;            // nothing is left
            const float x = logit_of(a.y), y = logit_of(b.y);
            if (!(x - y <= off + (fabsf(x) + fabsf(y)) * 0x1p-23f)) continue;
            // two chosen ones with the same logit and bias are a tie in fp64 too
            unsure = unsure || k + 1 == r.K || bias[a.x] != bias[b.x] ||
                     load_one<AT>(logits, row + a.x) != load_one<AT>(logits, row + b.x);
        }
    }
    uint64_t again = __ballot(unsure && here);
    while (again) {
        const int who = __builtin_ctzll(again), token = who / L;
        again &= L == 64 ? 0 : ~(0xffffull << (16 * token));
        const int tt = (blockIdx.x * kTokensPerBlock + wave) * PER + token;
        choose_exactly<AT, (L * V + 63) / 64>(logits, (size_t)tt * (size_t)stride, bias, r, found[wave][token]);
    }
    __builtin_amdgcn_wave_barrier();
    float l[kMaxTopK / L], big = low;
#pragma unroll
    for (int q = 0; q < kMaxTopK / L; ++q) {
        const int k = i + q * L;
        l[q] = here && k < r.K ? fmaxf(load_one<AT>(logits, row + f[k].x), low) : low;
        big = fmaxf(big, l[q]);
    }
    big = logit_of(lanes_max<L>(key_of(big)));
    const float top = r.renorm ? big : m;              // softmax: the terms' largest
    const float shift = r.renorm ? fminf(big, 0.0f) : 0.0f;
    float all = 0.0f;
#pragma unroll
    for (int q = 0; q < kMaxTopK / L; ++q) {
        l[q] = r.sigmoid ? (l[q] == low ? 0.0f : sigmoid_term(l[q], shift)) : term(l[q], top);
        all += l[q];
    }
    if (r.renorm) all = lanes_sum<L>(all);
    else all = sum;
#pragma unroll
    for (int q = 0; q < kMaxTopK / L; ++q) {
        const int k = i + q * L;
        if (!here || k >= r.K) continue;
        const size_t o = (size_t)t * r.K + k;
        ids[o] = (int32_t)f[k].x;
        w[o] = all > 0.0f ? r.scale * (l[q] / all) : 0.0f;
    }
}

template <int AT, int V>
__global__ __launch_bounds__(64 * kTokensPerBlock) void k_route_groups_backward(const void* __restrict__ logits,
        int64_t stride, const int32_t* __restrict__ ids, const float* __restrict__ w, const float* __restrict__ dw, int T,
        RouteGroups r, void* __restrict__ dl, int64_t dstride) {
    extern __shared__ float lds[];
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kTokensPerBlock + (threadIdx.x >> 6);
    if (t >= T) return;
    const bool dense = !r.sigmoid && !r.renorm;        // every logit has a gradient
    float* g = lds + (threadIdx.x >> 6) * (64 * V);    // what the chosen experts add
    const size_t from = (size_t)t * (size_t)stride;
    int id = -1;
    float wk = 0.0f, dk = 0.0f;
    if (lane < r.K) {
        const size_t o = (size_t)t * r.K + lane;
        id = ids[o];
        wk = w[o];
        dk = dw[o];
        if ((unsigned)id >= (unsigned)r.E) id = -1;
    }
    const float s = wave_sum(id >= 0 ? wk * dk : 0.0f);
    float mine = dense ? r.scale * dk : wk * (r.renorm ? dk - s / r.scale : dk);
    if (r.sigmoid && id >= 0) {                        // 1 - s = the sigmoid of -l; a masked logit's weight is 0
        const float l = load_one<AT>(logits, from + id);
        mine = l > -__builtin_inff() ? mine * sigmoid_term(-l, 0.0f) : 0.0f;
    }
    // an id chosen twice gets the sum over its k, in k order, from each of them alike
    float total = 0.0f;
    for (int k = 0; k < r.K; ++k) {
        const int other = __builtin_amdgcn_readlane(id, k);
        const float c = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(mine), k));
        total += other == id ? c : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) g[j * 64 + lane] = 0.0f;
    __builtin_amdgcn_wave_barrier();                   // LDS operations of one wave complete in order
    if (id >= 0) g[id] = total;
    __builtin_amdgcn_wave_barrier();
    float d[V];
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = g[lane * V + j];
    if (dense) {
        float l[V], sum = 0.0f;
        load_logits<AT, V>(logits, from, r.E, lane, l);
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
            const int left = r.E - e0 - c;
            if (left >= N) p.template store<true, false>(dl, (int64_t)(row + e0 + c), N);
            else p.template store<false, false>(dl, (int64_t)(row + e0 + c), left);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < r.E) store_one<AT>(dl, row + e0 + j, d[j]);
    }
}

template <int AT>
hipError_t route_groups(const void* logits, int64_t stride, const float* bias, int T, const RouteGroups& r, int32_t* ids,
                        float* w, hipStream_t s) {
    auto run = [&](auto lanes, auto v) {
        constexpr int L = decltype(lanes)::value, V = decltype(v)::value;
        constexpr int tokens = kTokensPerBlock * 64 / L;
        const size_t lds = r.kept < r.n_groups ? (size_t)tokens * L * V * sizeof(float) : 0;
        hipLaunchKernelGGL((k_route_groups<AT, L, V>), dim3((T + tokens - 1) / tokens), dim3(64 * kTokensPerBlock), lds, s,
                           logits, stride, bias, T, r, ids, w);
        return hipGetLastError();
    };
    if (r.E > 512) return by_width<16>(64, r.E, [&](auto v) { return run(std::integral_constant<int, 64>{}, v); });
    return by_width<1>(16, r.E, [&](auto v) {
        if constexpr (decltype(v)::value <= 32) return run(std::integral_constant<int, 16>{}, v);
        else return hipErrorInvalidValue;              // more than 512
    });
}

template <int AT>
hipError_t route_groups_backward(const void* logits, int64_t stride, const int32_t* ids, const float* w, const float* dw,
                                 int T, const RouteGroups& r, void* dl, int64_t dstride, hipStream_t s) {
    return by_width<1>(64, r.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((k_route_groups_backward<AT, V>), dim3((T + kTokensPerBlock - 1) / kTokensPerBlock),
                           dim3(64 * kTokensPerBlock), kTokensPerBlock * 64 * V * sizeof(float), s, logits, stride, ids,
                           w, dw, T, r, dl, dstride);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_route_groups(int atype, const void* logits, int64_t stride, const float* bias, int T,
                               const RouteGroups& r, int32_t* ids, float* w, hipStream_t s) {
    if (atype == A_F32) return route_groups<A_F32>(logits, stride, bias, T, r, ids, w, s);
    return route_groups<A_BF16>(logits, stride, bias, T, r, ids, w, s);
}

hipError_t launch_route_groups_backward(int atype, const void* logits, int64_t stride, const int32_t* ids, const float* w,
                                        const float* dw, int T, const RouteGroups& r, void* dl, int64_t dstride,
                                        hipStream_t s) {
    if (atype == A_F32) return route_groups_backward<A_F32>(logits, stride, ids, w, dw, T, r, dl, dstride, s);
    return route_groups_backward<A_BF16>(logits, stride, ids, w, dw, T, r, dl, dstride, s);
}

}  // namespace moe
