// Back through the epilogue of an expert product: for the rows r of group g
//
//   d_pre[r] = d_out[r] act'(pre[r]),   d_bias[g] = sum_r d_pre[r]
#include <hip/hip_runtime.h>

#include "expert_act.hpp"
#include "ops_dev.hpp"
#include "works.hpp"

namespace moe {
namespace {

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

}  // namespace

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

}  // namespace moe
