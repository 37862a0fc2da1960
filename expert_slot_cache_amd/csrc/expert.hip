// The product of sorted rows with their group's matrix in the activation format, with bias,
// activation and residual in the epilogue.  For the rows r of group g (offsets[g] <= r < offsets[g+1]):
//
//   h = x[r] w[g]^T + bias[g],  out = act(h) + resid[r]          (pre = h)
#include <hip/hip_runtime.h>

#include "expert_act.hpp"
#include "expert_core.hpp"
#include "product_tile.hpp"
#include "works.hpp"

namespace moe {
namespace {

template <class C, int AT, bool GATED>
__global__ __launch_bounds__(64 * C::WAVES) void k_expert(ExpertArgs p, int out_at, int nblocks) {
    constexpr int F = C::F, FA = C::FA, FB = C::FB, ES = AT == A_F32 ? 4 : 2;
    constexpr int COLS = GATED ? C::PA / 2 : C::PA, HF = GATED ? FA / 2 : FA;
    __shared__ __align__(1024) char lds[kCoreLds<C>];
    const Works<C::PB> works(p.offsets, p.G, p.M, nblocks);
    // workgroup b runs on XCD b % 8: each XCD takes one contiguous run of the work
    const int per = (works.total + 7) >> 3;
    const int jx = workgroup() >> 3;
    const int wk = (workgroup() & 7) * per + jx;
    if (jx >= per || wk >= works.total) return;
    const Work tl = works.at(wk);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wa = wave % C::WA, wb = wave / C::WA;
    const int N = p.N, K = p.K, width = GATED ? N / 2 : N, n0 = tl.nb * COLS;
    const uint32_t pitch = (uint32_t)K * ES;
    const char* w = static_cast<const char*>(p.w) + ((size_t)tl.group * N + n0) * pitch;
    const Operand a{w, pitch, min(COLS, width - n0), (int)pitch};
    const Operand up{w + (size_t)(GATED ? width : 0) * pitch, pitch, a.rows, a.depth};
    const Operand b{static_cast<const char*>(p.x) + (size_t)tl.row0 * pitch, pitch, tl.rows, (int)pitch};
    const int c0 = n0 + wa * HF * F, r0 = tl.row0 + wb * FB * F;     // of the wave's part
    const int lanes_c = c0 + (int)(threadIdx.x & 63) % (HF * F / 8) * 8;
    const bool here = lanes_c < width, whole = lanes_c + 8 <= width;
    float bias[8], up_bias[8];                             // requested ahead of the tile's copies
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float* from = p.bias + (size_t)tl.group * N + lanes_c + i;
        const bool there = p.bias && lanes_c + i < width;
        bias[i] = there ? from[0] : 0.0f;
        up_bias[i] = GATED && there ? from[width] : 0.0f;
    }
    Sums<F> acc[FA][FB];
    const bool live = wb * F * FB < tl.rows;
    core<C, AT, false, false, GATED>(lds, a, up, b, live, acc);

    each_run<C, GATED>(lds, acc, tl.rows - wb * FB * F, [&](int r, int c, float* v, float* up) {
        if (!here) return;
        const size_t row = r0 + r, n = c0 + c;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += bias[i];
        if (p.pre) store8<AT>(p.pre, row * N + n, whole, v);
        if constexpr (GATED) {
#pragma unroll
            for (int i = 0; i < 8; ++i) up[i] += up_bias[i];
            if (p.pre) store8<AT>(p.pre, row * N + width + n, whole, up);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid(v[i]) * up[i];
        } else if (p.act != ACT_NONE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = activate(p.act, v[i]);
        }
        const size_t at = row * width + n;
        if (p.resid) {
            float more[8];
            if (AT == A_F32 || out_at == A_F32) load8<A_F32>(p.resid, at, whole, more);
            else load8<A_BF16>(p.resid, at, whole, more);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += more[i];
        }
        store8_as<AT>(out_at, p.out, at, whole, v);
    });
}

template <class C, int AT, bool GATED>
hipError_t expert(const ExpertArgs& p, int out_at, hipStream_t s) {
    constexpr int COLS = GATED ? C::PA / 2 : C::PA;
    const int nblocks = ((GATED ? p.N / 2 : p.N) + COLS - 1) / COLS;
    const int64_t grid = (nblocks * most_tiles(p.M, p.G, p.offsets, C::PB) + 7) / 8 * 8;
    hipLaunchKernelGGL((k_expert<C, AT, GATED>), blocks_of(grid, C::WAVES), dim3(64 * C::WAVES), 0, s, p, out_at, nblocks);
    return hipGetLastError();
}

template <int AT, bool GATED>
hipError_t expert(const ExpertArgs& p, int out_at, hipStream_t s) {
    return expert_tile<GATED>(std::integral_constant<bool, AT == A_BF16>{}, p.M, p.G, p.N, p.offsets, [&](auto tile) { return expert<decltype(tile), AT, GATED>(p, out_at, s); });
}

}  // namespace

hipError_t launch_expert_product(int atype, int out_atype, const ExpertArgs& p, hipStream_t s) {
    const bool gated = p.act == ACT_SWIGLU;
    if (atype == A_F32) return gated ? expert<A_F32, true>(p, out_atype, s) : expert<A_F32, false>(p, out_atype, s);
    return gated ? expert<A_BF16, true>(p, out_atype, s) : expert<A_BF16, false>(p, out_atype, s);
}

}  // namespace moe
