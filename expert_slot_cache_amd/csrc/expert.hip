// The products of sorted rows with their expert's matrix in the activation format, and their
// gradients.  For the rows r of group g (offsets[g] <= r < offsets[g+1]):
//
//   h = x[r] w[g]^T + bias[g],  out = act(h) + resid[r]          (pre = h)
//   d_pre = d_out act'(pre),    d_bias[g] = sum_r d_pre[r]
//   d_x[r] = d_pre[r] w[g],     d_w[g] = sum_r d_pre[r] x[r]^T
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"
#include "ops_dev.hpp"
#include "works.hpp"

namespace moe {
namespace {

__device__ __forceinline__ float sigmoid(float h) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(h * -1.44269504f));
}
// The distribution function of the normal distribution.
__device__ __forceinline__ float normal_cdf(float h) { return 0.5f * erfcf(h * -0.70710678f); }

__device__ __forceinline__ float activate(int act, float h) {
    if (act == ACT_RELU) return h > 0.0f ? h : 0.0f;
    if (act == ACT_GELU) return h * normal_cdf(h);
    if (act == ACT_SILU) return h * sigmoid(h);
    return h;
}
__device__ __forceinline__ float slope(int act, float h) {
    if (act == ACT_RELU) return h > 0.0f ? 1.0f : 0.0f;
    if (act == ACT_GELU) return normal_cdf(h) + h * 0.39894228f * __builtin_amdgcn_exp2f(h * h * -0.72134752f);
    if (act == ACT_SILU) {
        const float s = sigmoid(h);
        return s * (1.0f + h * (1.0f - s));
    }
    return 1.0f;
}

enum { FORWARD, ROWS, MATRICES };

// A workgroup computes 64 x 64 outputs, a thread 4 x 4 of them, 16 apart: i of the rows (or, of a
// matrix' gradient, of its rows), j of the columns.
template <int MODE, int AT, int OT>
__global__ __launch_bounds__(256) void k_simple(const void* __restrict__ a, const void* __restrict__ b, ExpertArgs p,
                                                int nblocks) {
    __shared__ float as[16][65], bs[16][65];
    const int tid = threadIdx.x, ti = tid >> 4, tj = tid & 15;
    const int M = p.M, N = p.N, K = p.K;
    int group, row0, rows, nb, r0 = 0, depth;              // depth: what is summed over
    if (MODE == MATRICES) {
        group = blockIdx.z;
        row0 = blockIdx.y * 64;
        rows = min(64, N - row0);
        nb = blockIdx.x;
        int hi = M;
        if (p.offsets) {
            r0 = min(max(p.offsets[group], 0), M);
            hi = min(max(p.offsets[group + 1], r0), M);
        }
        depth = hi - r0;
    } else {
        const Works<64> works(p.offsets, p.G, M, nblocks);
        if ((int)blockIdx.x >= works.total) return;
        const Work tl = works.at(blockIdx.x);
        group = tl.group, row0 = tl.row0, rows = tl.rows, nb = tl.nb;
        depth = MODE == FORWARD ? K : N;
    }
    const bool gated = MODE == FORWARD && p.act == ACT_SWIGLU;
    const int half = N / 2, cols = MODE == FORWARD ? (gated ? half : N) : K;
    const size_t wg = (size_t)group * N * K;
    auto column = [&](int c) {                             // of the tile's column c: where it is, or -1
        if (gated) {
            const int n = nb * 32 + (c & 31);
            return n < half ? n + (c >> 5) * half : -1;
        }
        return nb * 64 + c < cols ? nb * 64 + c : -1;
    };
    float acc[4][4] = {};
    for (int k0 = 0; k0 < depth; k0 += 16) {
        for (int e = tid; e < 1024; e += 256) {
            const int k = MODE == MATRICES ? e >> 6 : e & 15, i = MODE == MATRICES ? e & 63 : e >> 4;
            float v = 0.0f;
            if (i < rows && k0 + k < depth) {
                if (MODE == FORWARD) v = load_one<AT>(a, (size_t)(row0 + i) * K + k0 + k);
                else if (MODE == ROWS) v = load_one<AT>(a, (size_t)(row0 + i) * N + k0 + k);
                else v = load_one<AT>(a, (size_t)(r0 + k0 + k) * N + row0 + i);
            }
            as[k][i] = v;
            const int kb = MODE == FORWARD ? e & 15 : e >> 6, j = MODE == FORWARD ? e >> 4 : e & 63;
            const int n = column(j);
            v = 0.0f;
            if (n >= 0 && k0 + kb < depth) {
                if (MODE == FORWARD) v = load_one<AT>(b, wg + (size_t)n * K + k0 + kb);
                else if (MODE == ROWS) v = load_one<AT>(b, wg + (size_t)(k0 + kb) * K + n);
                else v = load_one<AT>(b, (size_t)(r0 + k0 + kb) * K + n);
            }
            bs[kb][j] = v;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k) {
            float av[4], bv[4];
            for (int q = 0; q < 4; ++q) av[q] = as[k][ti + 16 * q], bv[q] = bs[k][tj + 16 * q];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += av[i] * bv[j];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (ti + 16 * i >= rows) continue;
        const size_t r = row0 + ti + 16 * i;
        if (MODE != FORWARD) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = column(tj + 16 * j);
                if (n >= 0) store_one<OT>(p.out, (MODE == MATRICES ? wg : 0) + r * K + n, acc[i][j]);
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = column(tj + 16 * j);
            if (n < 0) continue;
            if (p.bias) acc[i][j] += p.bias[(size_t)group * N + n];
            if (p.pre) store_one<AT>(p.pre, r * N + n, acc[i][j]);
            if (gated) continue;
            const float v = activate(p.act, acc[i][j]);
            store_one<OT>(p.out, r * N + n, v + (p.resid ? load_one<OT>(p.resid, r * N + n) : 0.0f));
        }
        if (gated)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int n = column(tj + 16 * j);
                if (n < 0) continue;
                const float v = acc[i][j] * sigmoid(acc[i][j]) * acc[i][j + 2];
                store_one<OT>(p.out, r * half + n, v + (p.resid ? load_one<OT>(p.resid, r * half + n) : 0.0f));
            }
    }
}

// ---- the gradient before the activation ------------------------------------------------------

constexpr int kActRows = 64;   // rows of a partial sum

// A thread takes a column of up to 64 rows of a group; their sum goes to the place of the tile,
// which no other has: row0 / 64 + group rises by one at least from a tile to the next.
template <int AT, int OT>
__global__ __launch_bounds__(256) void k_activation_backward(ActivationArgs p, int nblocks) {
    const Works<kActRows> works(p.offsets, p.G, p.M, nblocks);
    if ((int)blockIdx.x >= works.total) return;
    const Work tl = works.at(blockIdx.x);
    const bool gated = p.act == ACT_SWIGLU;
    const int half = p.N / 2, n = tl.nb * 256 + threadIdx.x;
    if (n >= (gated ? half : p.N)) return;
    float sum = 0.0f, up_sum = 0.0f;
    for (int i = 0; i < tl.rows; ++i) {
        const size_t r = tl.row0 + i;
        if (gated) {
            const float d = load_one<OT>(p.dout, r * half + n);
            const float g = load_one<AT>(p.pre, r * p.N + n), u = load_one<AT>(p.pre, r * p.N + half + n);
            const float dg = d * u * slope(ACT_SILU, g), du = d * g * sigmoid(g);
            sum += dg;
            up_sum += du;
            if (p.dpre) {
                store_one<AT>(p.dpre, r * p.N + n, dg);
                store_one<AT>(p.dpre, r * p.N + half + n, du);
            }
        } else {
            float d = load_one<OT>(p.dout, r * p.N + n);
            if (p.act != ACT_NONE) d *= slope(p.act, load_one<AT>(p.pre, r * p.N + n));
            sum += d;
            if (p.dpre) store_one<AT>(p.dpre, r * p.N + n, d);
        }
    }
    if (p.dbias) {
        float* to = p.partial + (size_t)(tl.row0 / kActRows + tl.group) * p.N + n;
        to[0] = sum;
        if (gated) to[half] = up_sum;
    }
}

__global__ __launch_bounds__(256) void k_bias_sums(ActivationArgs p) {
    const int n = blockIdx.x * 256 + threadIdx.x, g = blockIdx.y;
    if (n >= p.N) return;
    int lo = 0, hi = p.M;
    if (p.offsets) {
        // as the works bound them: falling offsets count as the largest before them
        for (int i = 0; i <= g; ++i) lo = min(max(p.offsets[i], lo), p.M);
        hi = min(max(p.offsets[g + 1], lo), p.M);
    }
    const int tiles = (hi - lo + kActRows - 1) / kActRows;
    const float* from = p.partial + (size_t)(lo / kActRows + g) * p.N + n;
    float sum = 0.0f;
    for (int i = 0; i < tiles; ++i) sum += from[(size_t)i * p.N];
    p.dbias[(size_t)g * p.N + n] = sum;
}

// Tiles of 64 rows that M rows of G groups can have.
int64_t most(int64_t M, int64_t G, bool offsets) { return offsets ? M / 64 + (G < M ? G : M) : (M + 63) / 64; }

template <int MODE, int AT, int OT>
hipError_t simple(const void* a, const void* b, const ExpertArgs& p, hipStream_t s) {
    const int cols = MODE != FORWARD ? p.K : p.act == ACT_SWIGLU ? p.N : (p.N + 63) / 64 * 64;
    const int nblocks = (cols + 63) / 64;
    if (MODE == MATRICES) {
        hipLaunchKernelGGL((k_simple<MODE, AT, OT>), dim3(nblocks, (p.N + 63) / 64, p.G), dim3(256), 0, s, a, b, p, nblocks);
    } else {
        hipLaunchKernelGGL((k_simple<MODE, AT, OT>), dim3((unsigned)(nblocks * most(p.M, p.G, p.offsets))), dim3(256), 0, s, a,
                           b, p, nblocks);
    }
    return hipGetLastError();
}

// f of the two formats as constants (the second is fp32 or the first).
template <class F>
hipError_t by_types(int at, int ot, F f) {
    typedef std::integral_constant<int, A_F32> F32;
    typedef std::integral_constant<int, A_BF16> BF16;
    if (at == A_F32) return f(F32{}, F32{});
    return ot == A_F32 ? f(BF16{}, F32{}) : f(BF16{}, BF16{});
}

}  // namespace

hipError_t launch_expert_product(int atype, int out_atype, const ExpertArgs& a, hipStream_t s) {
    return by_types(atype, out_atype, [&](auto at, auto ot) {
        return simple<FORWARD, decltype(at)::value, decltype(ot)::value>(a.x, a.w, a, s);
    });
}

size_t activation_workspace(int M, int G, int N) { return (size_t)(M / kActRows + G) * N * sizeof(float); }

hipError_t launch_activation_backward(int atype, int out_atype, const ActivationArgs& a, hipStream_t s) {
    return by_types(atype, out_atype, [&](auto at, auto ot) {
        const int nblocks = ((a.act == ACT_SWIGLU ? a.N / 2 : a.N) + 255) / 256;
        if (a.M > 0) {
            hipLaunchKernelGGL((k_activation_backward<decltype(at)::value, decltype(ot)::value>),
                               dim3((unsigned)(nblocks * most(a.M, a.G, a.offsets))), dim3(256), 0, s, a, nblocks);
            if (const hipError_t e = hipGetLastError()) return e;
        }
        if (a.dbias) hipLaunchKernelGGL(k_bias_sums, dim3((a.N + 255) / 256, a.G), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

size_t expert_backward_workspace(int atype, int M, int G, int N, int K) { return 0; }

hipError_t launch_expert_backward(int atype, int dw_atype, const ExpertGradArgs& g, hipStream_t s) {
    ExpertArgs a{};
    a.offsets = g.offsets;
    a.M = g.M, a.G = g.G, a.N = g.N, a.K = g.K;
    if (g.dx && g.M > 0) {
        a.out = g.dx;
        const hipError_t e = atype == A_F32 ? simple<ROWS, A_F32, A_F32>(g.dpre, g.w, a, s)
                                            : simple<ROWS, A_BF16, A_BF16>(g.dpre, g.w, a, s);
        if (e) return e;
    }
    if (!g.dw) return hipSuccess;
    a.out = g.dw;
    return by_types(atype, dw_atype, [&](auto at, auto ot) {
        return simple<MATRICES, decltype(at)::value, decltype(ot)::value>(g.dpre, g.x, a, s);
    });
}

}  // namespace moe
