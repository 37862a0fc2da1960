// Back through the product of sorted rows with their group's matrix: for the rows r of group g
//
//   d_x[r] = d_pre[r] w[g],     d_w[g] = sum_r d_pre[r]^T x[r]
#include <hip/hip_runtime.h>

#include "expert_core.hpp"
#include "ops.hpp"
#include "product_tile.hpp"
#include "works.hpp"

namespace moe {
namespace {

// d_x: as the forward product, the matrix read across its rows.
template <class C, int AT>
__global__ __launch_bounds__(64 * C::WAVES) void k_expert_rows(ExpertGradArgs p, int nblocks) {
    constexpr int F = C::F, FA = C::FA, FB = C::FB, ES = AT == A_F32 ? 4 : 2;
    __shared__ __align__(1024) char lds[kCoreLds<C>];
    const Works<C::PB> works(p.offsets, p.G, p.M, nblocks);
    const int per = (works.total + 7) >> 3;                // as in the forward product
    const int jx = workgroup() >> 3;
    const int wk = (workgroup() & 7) * per + jx;
    if (jx >= per || wk >= works.total) return;
    const Work tl = works.at(wk);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wa = wave % C::WA, wb = wave / C::WA;
    const int N = p.N, K = p.K, k0 = tl.nb * C::PA;
    const Operand a{static_cast<const char*>(p.w) + ((size_t)tl.group * N * K + k0) * ES, (uint32_t)K * ES, (K - k0) * ES, N};
    const Operand b{static_cast<const char*>(p.dpre) + (size_t)tl.row0 * N * ES, (uint32_t)N * ES, tl.rows, N * ES};
    Sums<F> acc[FA][FB];
    const bool live = wb * F * FB < tl.rows;
    core<C, AT, true, false, false>(lds, a, a, b, live, acc);
    const int c0 = k0 + wa * FA * F, r0 = tl.row0 + wb * FB * F;
    each_run<C, false>(lds, acc, tl.rows - wb * FB * F, [&](int r, int c, float* v, float*) {
        if (c0 + c < K) store8<AT>(p.dx, (size_t)(r0 + r) * K + c0 + c, c0 + c + 8 <= K, v);
    });
}

// d_w: both operands across their rows, the rows of a group (of split `s` of them) the summed dimension.
template <class C, int AT>
__global__ __launch_bounds__(64 * C::WAVES) void k_expert_matrices(ExpertGradArgs p, int dw_at, int kblocks, int tiles, int splits) {
    constexpr int F = C::F, FA = C::FA, FB = C::FB, ES = AT == A_F32 ? 4 : 2;
    constexpr int DEPTH = C::RB / ES;
    __shared__ __align__(1024) char lds[kCoreLds<C>];
    // Groups differ in rows, and a tile's time with them: every XCD (workgroup b runs on XCD b % 8) takes a
    // share of each group, its column blocks of x where there are eight.  One run of groups to each XCD
    // took 331 us where this takes 273 (64 groups of 256 rows, 2048 x 2048).
    const int wk = workgroup(), split = wk / tiles % splits, group = wk / tiles / splits;
    if (group >= p.G) return;
    const int nb = wk % tiles / kblocks, kb = wk % tiles % kblocks;
    int lo = 0, hi = p.M;
    if (p.offsets) {
        lo = min(max(p.offsets[group], 0), p.M);
        hi = min(max(p.offsets[group + 1], lo), p.M);
    }
    if (splits > 1) {                                      // whole stages to each
        const int each = ((hi - lo + DEPTH - 1) / DEPTH + splits - 1) / splits * DEPTH;
        lo = min(lo + split * each, hi);
        hi = min(lo + each, hi);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wa = wave % C::WA, wb = wave / C::WA;
    const int N = p.N, K = p.K, k0 = kb * C::PA, n0 = nb * C::PB;
    const Operand a{static_cast<const char*>(p.x) + ((size_t)lo * K + k0) * ES, (uint32_t)K * ES, (K - k0) * ES, hi - lo};
    const Operand b{static_cast<const char*>(p.dpre) + ((size_t)lo * N + n0) * ES, (uint32_t)N * ES, (N - n0) * ES, hi - lo};
    Sums<F> acc[FA][FB];
    const bool live = n0 + wb * F * FB < N;
    core<C, AT, true, true, false>(lds, a, a, b, live, acc);
    const size_t to = (splits > 1 ? (size_t)split * p.G + group : (size_t)group) * N * K;
    const int c0 = k0 + wa * FA * F, r0 = n0 + wb * FB * F;
    each_run<C, false>(lds, acc, N - r0, [&](int r, int c, float* v, float*) {
        if (c0 + c >= K) return;
        const size_t at = to + (size_t)(r0 + r) * K + c0 + c;
        const bool whole = c0 + c + 8 <= K;
        if (splits > 1) store8<A_F32>(p.partial, at, whole, v);
        else store8_as<AT>(dw_at, p.dw, at, whole, v);
    });
}

// The sums of the splits, in their order.
__global__ __launch_bounds__(256) void k_join(const float* __restrict__ partial, void* __restrict__ dw, int dw_at, size_t n,
                                              int splits) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(partial + i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(partial + (size_t)s * n + i);
    if (dw_at == A_F32) {
        *reinterpret_cast<f32x4_t*>(static_cast<float*>(dw) + i) = v;
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dw) + i) =
            make_uint2(round_bf16(v[0]) | (uint32_t)round_bf16(v[1]) << 16, round_bf16(v[2]) | (uint32_t)round_bf16(v[3]) << 16);
    }
}

template <class C, int AT>
hipError_t rows(const ExpertGradArgs& p, hipStream_t s) {
    const int nblocks = (p.K + C::PA - 1) / C::PA;
    const int64_t grid = (nblocks * most_tiles(p.M, p.G, p.offsets, C::PB) + 7) / 8 * 8;
    hipLaunchKernelGGL((k_expert_rows<C, AT>), blocks_of(grid, C::WAVES), dim3(64 * C::WAVES), 0, s, p, nblocks);
    return hipGetLastError();
}

template <int AT>
hipError_t rows(const ExpertGradArgs& p, hipStream_t s) {
    return expert_tile<false>(std::integral_constant<bool, AT == A_BF16>{}, p.M, p.G, p.K, p.offsets,
                              [&](auto tile) { return rows<decltype(tile), AT>(p, s); });
}

template <int AT>
hipError_t matrices(const ExpertGradArgs& p, int dw_at, hipStream_t s) {
    return matrix_tile(p.M, p.G, p.N, p.K, [&](auto tile, int splits) {
        typedef decltype(tile) C;
        const int kblocks = (p.K + C::PA - 1) / C::PA, tiles = kblocks * ((p.N + C::PB - 1) / C::PB);
        const int64_t grid = (int64_t)tiles * splits * p.G;
        hipLaunchKernelGGL((k_expert_matrices<C, AT>), blocks_of(grid, C::WAVES), dim3(64 * C::WAVES), 0, s, p, dw_at, kblocks, tiles,
                           splits);
        if (splits > 1) {
            if (const hipError_t e = hipGetLastError()) return e;
            const size_t n = (size_t)p.G * p.N * p.K;
            hipLaunchKernelGGL(k_join, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, s, p.partial, p.dw, dw_at, n, splits);
        }
        return hipGetLastError();
    });
}

}  // namespace

size_t expert_backward_workspace(int M, int G, int N, int K) {
    const int splits = matrix_tile(M, G, N, K, [](auto, int n) { return n; });
    return splits > 1 ? (size_t)splits * G * N * K * sizeof(float) : 0;
}

hipError_t launch_expert_backward(int atype, int dw_atype, const ExpertGradArgs& p, hipStream_t s) {
    if (p.dx && p.M > 0) {
        const hipError_t e = atype == A_F32 ? rows<A_F32>(p, s) : rows<A_BF16>(p, s);
        if (e) return e;
    }
    if (!p.dw) return hipSuccess;
    return atype == A_F32 ? matrices<A_F32>(p, dw_atype, s) : matrices<A_BF16>(p, dw_atype, s);
}

}  // namespace moe
