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
// the plain router (sixteen lanes a token up to 512 experts, a wave above that).  Where two neighbours
// among the first K + 1 lie nearer to each other than the bound, the wave takes these K + 1 once more in
// fp64; where the last group kept and the first left out do, or the last expert chosen and the second
// one not, all of the token's.  Without a bias the logits
// themselves are the order, which needs no bound.
//
// A group's sum is taken from the largest two of each run of eight (of fewer below 65 experts)
// where every such run lies in one group, else from its experts one by one.  16384 tokens of 512
// experts, top-10 in fp32, sigmoid, take 17 us without bias and groups, 22 with the 4 best of 8 groups,
// 30 with a bias: about one token in a thousand is taken again, and the call waits for the last (36 us
// where each of them was with all of its experts).  Where choices are equal, most tokens are: bf16 logits
// with one bias for all take 50 us, and logits that are all the same 94, with groups 117.  Masked experts
// cost nothing: next to one the order is in no doubt (28 to 34 us with all but 10 to 20 masked).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ops.hpp"
#include "route_dev.hpp"
#include "route_doubt.hpp"

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

// The sigmoid where exponentials that run over do no harm.
__device__ __forceinline__ float sigmoid_of(float l) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-l * kLog2e));
}

// The order of doubles as unsigned numbers above 0.
__device__ __forceinline__ uint64_t key64_of(double c) {
    const uint64_t b = __builtin_bit_cast(uint64_t, c);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        v += __builtin_bit_cast(double, (uint64_t)(uint32_t)__shfl_xor((int)(uint32_t)(b >> 32), d) << 32 |
                                            (uint32_t)__shfl_xor((int)(uint32_t)b, d));
    }
    return v;
}

// A token by a whole wave in fp64: its K experts into `found`, in order.  cs: 8 E bytes in LDS, the
// logits and biases, then the choices, then their order.  Few tokens come here, and every token's wave
// has the registers and the code that this takes: loops over LDS, loads requested four at a time.
template <int AT>
__device__ __forceinline__ void choose_exactly(const void* __restrict__ logits, size_t row, const float* __restrict__ bias,
                                               const RouteGroups& r, uint64_t* cs, uint2* found) {
    const int lane = threadIdx.x & 63;
    const double low = -(double)__builtin_inff();
    auto logit = [&](int e) { return fmaxf(load_one<AT>(logits, row + e), -__builtin_inff()); };
    auto put = [&](int e, double c) { cs[e] = __builtin_bit_cast(uint64_t, c); };
    auto at_of = [&](int e) { return __builtin_bit_cast(double, cs[e]); };
    float m = -__builtin_inff();
#pragma unroll 4
    for (int e = lane; e < r.E; e += 64) {
        const float l = logit(e), b = bias ? bias[e] : 0.0f;
        m = fmaxf(m, l);
        cs[e] = (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(l);
    }
    m = logit_of(wave_max_u32(key_of(m)));
    double sum = 0.0;
    for (int pass = r.sigmoid ? 1 : 0; pass < 2; ++pass) {  // softmax: the sum first
#pragma unroll 1
        for (int e = lane; e < r.E; e += 64) {
            const float l = __uint_as_float((uint32_t)cs[e]), b = __uint_as_float((uint32_t)(cs[e] >> 32));
            // of equal infinities the difference is 0
            const double t = exp(r.sigmoid ? -(double)l : l == m ? 0.0 : (double)l - (double)m);
            if (pass == 0) {
                sum += t;
            } else {
                const double c = (r.sigmoid ? 1.0 : t) / (r.sigmoid ? 1.0 + t : sum) + (double)b;
                put(e, c == c && l > -__builtin_inff() ? c + 0.0 : low);
            }
        }
        if (pass == 0) sum = wave_sum64(sum);
    }
    __builtin_amdgcn_wave_barrier();
    uint64_t kept = ~0ull;
    int size = r.E;
    if (r.kept < r.n_groups) {
        size = r.E / r.n_groups;
        double one = low, two = low;
        if (lane < r.n_groups) {
            int o = lane % size;                           // the lanes start at different banks
#pragma unroll 4
            for (int j = 0; j < size; ++j) {
                const double v = at_of(lane * size + o);
                two = fmax(two, fmin(one, v));
                one = fmax(one, v);
                o = o + 1 == size ? 0 : o + 1;
            }
        }
        const double score = r.group_top > 1 && two > low ? one + two : one;
        int rank = 0;
        for (int g = 0; g < r.n_groups; ++g) {
            const uint64_t b = __builtin_bit_cast(uint64_t, score);
            const double o = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), g) << 32 |
                                                            (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, g));
            rank += o > score || (o == score && g < lane);
        }
        kept = __ballot(lane < r.n_groups && rank < r.kept);
    }
#pragma unroll 1
    for (int e = lane; e < r.E; e += 64) {
        // without a bias the order is the logits'
        const double by = bias ? at_of(e) : (double)logit(e) + 0.0;
        cs[e] = (kept >> (e / size)) & 1 ? key64_of(by) : 0;   // 0: no choice
    }
    for (int k = 0; k < r.K; ++k) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll 4
        for (int e = lane; e < r.E; e += 64) {
            const uint64_t v = cs[e];
            at = v > best ? e : at;
            best = v > best ? v : best;
        }
        // the largest over the wave, its upper half first; of equal ones the lowest expert
        const uint32_t hi = wave_max_u32((uint32_t)(best >> 32));
        const uint32_t lo = wave_max_u32((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        const bool top = best == ((uint64_t)hi << 32 | lo);
        at = (int)(0xffffu - wave_max_u32(top ? 0xffffu - (uint32_t)at : 0u));
        if (lane == 0) {
            found[k].x = (uint32_t)at;
            cs[at] = 0;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// The K experts of a token among the first K + 1 of its order (K + 1 <= 64), by their choices in fp64, one
// a lane.  m: the largest logit.
template <int AT>
__device__ __forceinline__ void order_exactly(const void* __restrict__ logits, size_t row, const float* __restrict__ bias,
                                              const RouteGroups& r, float m, uint2* found) {
    const int lane = threadIdx.x & 63, n = r.K + 1;
    auto logit = [&](int e) { return fmaxf(load_one<AT>(logits, row + e), -__builtin_inff()); };
    double sum = 0.0;
    if (!r.sigmoid) {
#pragma unroll 4
        for (int e = lane; e < r.E; e += 64) {
            const float l = logit(e);
            sum += exp(l == m ? 0.0 : (double)l - (double)m);
        }
        sum = wave_sum64(sum);
    }
    const uint2 mine = found[min(lane, n - 1)];
    const float l = mine.y > 0x7f0000u ? logit((int)mine.x) : 0.0f;      // else none is left
    const float b = mine.y > 0x7f0000u ? bias[mine.x] : 0.0f;
    const double t = exp(r.sigmoid ? -(double)l : l == m ? 0.0 : (double)l - (double)m);
    const double c = (r.sigmoid ? 1.0 : t) / (r.sigmoid ? 1.0 + t : sum) + (double)b;
    const uint64_t key = mine.y > 0x7f0000u ? key64_of(c == c && l > -__builtin_inff() ? c + 0.0 : -(double)__builtin_inff()) : 0;
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), i) << 32 |
                           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, i);
        rank += o > key || (o == key && (uint32_t)__builtin_amdgcn_readlane((int)mine.x, i) < mine.x);
    }
    __builtin_amdgcn_wave_barrier();
    if (lane < n) found[rank].x = mine.x;
    __builtin_amdgcn_wave_barrier();
}

// Bytes of a wave's choices: fp32 for each of its tokens, or two for each eight, or fp64 for one token
// (not wanted where the logits are the order and no group is left out).
template <int L, int V>
constexpr int group_bytes = std::max(std::max(64 * V * 4, 64 * Eights<V, true>::N * 8), L * V * 8);

template <int AT, int L, int V>
__global__ __launch_bounds__(64 * kTokensPerBlock) void k_route_groups(const void* __restrict__ logits, int64_t stride,
        const float* __restrict__ bias, int T, RouteGroups r, int32_t* __restrict__ ids, float* __restrict__ w) {
    constexpr int PER = 64 / L;                        // tokens of a wave
    __shared__ uint2 found[kTokensPerBlock][PER][kMaxTopK + 2];   // (id, key) in order
    extern __shared__ __align__(16) char shared_c[];   // group_bytes<L, V> a wave
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
    const uint64_t below = L == 64 ? 0 : ((1ull << lane) - 1) & (0xffffull << (lane & 48));   // of this token's
    auto soft = [&](float l) { return __builtin_amdgcn_exp2f((l == m ? 0.0f : l - m) * kLog2e) * inv; };
    auto score_of = [&](float l) { return r.sigmoid ? sigmoid_term(l, 0.0f) : soft(l); };   // l > -inf
    if (bias) {
        float b[V];
        load_logits<A_F32, V>(bias, 0, n, i, b);           // a bias of NaN, too, is -inf
        auto choice = [&](int j, float s) { c[j] = c[j] == low ? low : fmaxf(s + b[j], low) + 0.0f; };
        if (r.sigmoid) {
#pragma unroll
            for (int j = 0; j < V; ++j) choice(j, sigmoid_of(c[j]));
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) choice(j, soft(c[j]));
        }
    }
    Eights<V, true> keys;
    constexpr int W = Eights<V, true>::W, N = Eights<V, true>::N;
    char* mine_c = shared_c + wave * group_bytes<L, V>;
    bool unsure = false;
    uint64_t kept = ~0ull;
    int g = 0, at = 0, end = -1;
    if (by_group) {
        const int size = r.E / r.n_groups, each = (r.n_groups + L - 1) / L;   // a lane's groups: i * each ..
        // where every eight lies in one group, a group's largest two are among its eights' first two
        const bool eights = size % W == 0;
        const int parts = eights ? size / W : size;        // of a group, in LDS
        if (eights) {
            float2* to = reinterpret_cast<float2*>(mine_c) + sub * (L * N) + i * N;
#pragma unroll
            for (int q = 0; q < N; ++q) {
                float one = c[q * W], two = low;
#pragma unroll
                for (int j = 1; j < W; ++j) {
                    two = fmaxf(two, fminf(one, c[q * W + j]));
                    one = fmaxf(one, c[q * W + j]);
                }
                to[q] = make_float2(one, two);
            }
        } else {
            float* to = reinterpret_cast<float*>(mine_c) + sub * (L * V) + i * V;
#pragma unroll
            for (int j = 0; j < V; ++j) to[j] = c[j];
        }
        __builtin_amdgcn_wave_barrier();                   // LDS operations of one wave complete in order
        constexpr int GROUPS = kMaxGroups / L;             // of a lane
        uint32_t gk[GROUPS];
        GroupSum sums[GROUPS];
#pragma unroll
        for (int a = 0; a < GROUPS; ++a) {
            gk[a] = 0;
            sums[a] = {low, 0.0f};
            const int q = i * each + a;
            if (a >= each || q >= r.n_groups) continue;
            float one = low, two = low;
            int o = q % parts;                             // the lanes start at different banks
#pragma unroll 4
            for (int j = 0; j < parts; ++j) {
                float2 v;
                if (eights) v = reinterpret_cast<const float2*>(mine_c)[sub * (L * N) + q * parts + o];
                else v = make_float2(reinterpret_cast<const float*>(mine_c)[sub * (L * V) + q * parts + o], low);
                two = fmaxf(fmaxf(two, v.y), fminf(one, v.x));
                one = fmaxf(one, v.x);
                o = o + 1 == parts ? 0 : o + 1;
            }
            if (r.group_top > 1 && !bias) {                // these are logits
                one = one > low ? score_of(one) : low;
                two = two > low ? score_of(two) : low;
            }
            sums[a] = group_sum(one, two, r.group_top > 1, off);
            gk[a] = key_of(sums[a].value);
        }
        // the kept groups, one after another
        uint32_t lo = 0, hi = 0;
        for (int k = 0; k < r.kept; ++k) {
            uint32_t best = 0;
#pragma unroll
            for (int a = 0; a < GROUPS; ++a) best = max(best, gk[a]);
            const uint32_t top = lanes_max<L>(best);
            const uint64_t holds = __ballot(best == top);
            bool mine = best == top;
            if constexpr (L == 64) mine = lane == __builtin_ctzll(holds);
            else mine = mine && (holds & below) == 0;
#pragma unroll
            for (int a = 0; a < GROUPS; ++a)
                if (mine && gk[a] == top) {
                    const int q = i * each + a;
                    if (q < 32) lo |= 1u << q;
                    else hi |= 1u << (q - 32);
                    gk[a] = 0;
                    mine = false;
                }
        }
        // Is the least that any kept one may be above the most that any other may?  (Of largest logits
        // nothing is off.)  Where all that are left out are groups of masked experts, those kept are the first.
        if (bias || r.group_top > 1) {
            float least = __builtin_inff(), most = low;
#pragma unroll
            for (int a = 0; a < GROUPS; ++a) {
                const int q = i * each + a;
                const bool is_kept = ((q < 32 ? lo >> q : hi >> (q - 32)) & 1) != 0;
                if (a >= each || q >= r.n_groups) continue;
                if (is_kept) least = fminf(least, sums[a].value - sums[a].off);
                else most = fmaxf(most, sums[a].value + sums[a].off);
            }
            least = -logit_of(lanes_max<L>(key_of(-least)));
            most = logit_of(lanes_max<L>(key_of(most)));
            unsure = most > low && !(least > most);
        }
        lo = lanes_or<L>(lo);
        hi = lanes_or<L>(hi);
        kept = (uint64_t)hi << 32 | lo;
        g = i * V / size;                                  // of the lane's first expert
        at = i * V - g * size;
        end = size;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const bool can = i * V + j < n && ((kept >> g) & 1);
        keys.key[j] = can ? key_of(c[j]) : (uint32_t)j;    // the others: none equal
        if (++at == end) {
            at = 0;
            ++g;
        }
    }
    keys.order();
    uint2* f = found[wave][sub];
    const int rounds = bias ? r.K + 2 : r.K;           // and the first two that are not chosen
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
    bool swapped = false;                              // two of the first K + 1 may have to change places
    if (bias) {
        auto near = [&](const uint2& a, const uint2& b) {
            return b.y > 0x7f0000u && near_choices(logit_of(a.y), logit_of(b.y), off);   // else none is left
        };
        for (int k = i; k < r.K && here; k += L) {
            const uint2 a = f[k], b = f[k + 1];
            if (!near(a, b)) continue;
            // two chosen ones with the same logit and bias are a tie in fp64 too
            if (k + 1 < r.K && bias[a.x] == bias[b.x] && load_one<AT>(logits, row + a.x) == load_one<AT>(logits, row + b.x)) continue;
            swapped = true;
            unsure = unsure || r.K == kMaxTopK || (k + 1 == r.K && near(a, f[k + 2]));
        }
    }
    uint64_t again = __ballot(unsure && here), swaps = __ballot(swapped && here);
    while (again | swaps) {
        const int token = __builtin_ctzll(again | swaps) / L;
        const uint64_t its = L == 64 ? ~0ull : 0xffffull << (16 * token);
        const size_t from = (size_t)((blockIdx.x * kTokensPerBlock + wave) * PER + token) * (size_t)stride;
        if (again & its) choose_exactly<AT>(logits, from, bias, r, reinterpret_cast<uint64_t*>(mine_c), found[wave][token]);
        else order_exactly<AT>(logits, from, bias, r, __shfl(m, token * L), found[wave][token]);
        again &= ~its;
        swaps &= ~its;
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
        const size_t lds = bias || r.kept < r.n_groups ? (size_t)kTokensPerBlock * group_bytes<L, V> : 0;
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
