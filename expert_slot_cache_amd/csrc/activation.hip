// Back through the epilogue of an expert product: for the rows r of group g
//
//   d_pre[r] = d_out[r] act'(pre[r]),   d_bias[g] = sum_r d_pre[r]
//
// Memory binds it: every value is read once and written once, 16 bytes a lane (8 columns in bf16,
// two pieces in fp32).  A workgroup takes 256 columns of up to 64 rows of a group, 32 lanes to a row,
// so that a thread has eight rows to itself, whose loads are requested four at a time, and a small
// call still gives many CUs work: 333 x 1000 in fp32, GELU, takes 12.0 us (one thread to a
// column's 64 rows: 31.7).  32768 rows, SwiGLU of 4096 columns, bf16, with the bias' gradient (671 MB): 140 us.  The
// bias' sums are fp32 in a tile (a thread's eight rows, then the eight threads of a column) and fp64 over the
// tiles of a group, in a second launch, each in a fixed order.
#include <hip/hip_runtime.h>

#include "expert_act.hpp"
#include "expert_core.hpp"
#include "ops.hpp"
#include "product_tile.hpp"
#include "works.hpp"

namespace moe {
namespace {

constexpr int kActCols = 256;                              // of a workgroup
constexpr int kLanes = kActCols / 8, kSlices = 256 / kLanes;

// Rows of a workgroup: 64, or 16 where those would be too few workgroups to hide a load's latency.
// Measured (us, 16 / 64 rows, GELU in fp32 without the bias' gradient): 333 x 1000, 8.1 / 9.1; 2048 x 2048
// (256 workgroups of 64), 8.3 / 11.1; with it 4096 x 2048 (512), 21.3 / 21.2, and 16384 rows of 64 groups,
// SwiGLU of 2048 columns in bf16, 36.3 / 35.3.
int act_rows(int64_t M, int64_t G, int64_t N) {
    return (N + kActCols - 1) / kActCols * most_tiles(M, G, G > 1, 64) < 512 ? 16 : 64;
}

// The sums of a tile go to the place of its rows, which no other tile has: row0 / rows + group rises
// by one at least from a tile to the next.
__device__ __forceinline__ size_t place(int row0, int group, int rows) { return (size_t)(row0 / rows + group); }

template <int AT, int OT, int ACT, int ROWS>
__global__ __launch_bounds__(256) void k_activation_backward(ActivationArgs p, int nblocks) {
    constexpr bool GATED = ACT == ACT_SWIGLU;
    __shared__ float sums[kSlices][kActCols * (GATED ? 2 : 1)];
    const Works<ROWS> works(p.offsets, p.G, p.M, nblocks);
    if ((int)blockIdx.x >= works.total) return;
    const Work tl = works.at(blockIdx.x);
    const int width = GATED ? p.N / 2 : p.N, n0 = tl.nb * kActCols;
    const int lane = threadIdx.x % kLanes, slice = threadIdx.x / kLanes, n = n0 + lane * 8;
    const bool whole = n + 8 <= width;
    float sum[8] = {}, up_sum[8] = {};
    if (n < width) {
        constexpr int BATCH = ROWS < 32 ? ROWS / kSlices : 4;                           // rows requested at a time: d_pre may lie in pre or d_out
#pragma unroll 1
        for (int i0 = slice; i0 < tl.rows; i0 += BATCH * kSlices) {
            float d[BATCH][8], h[BATCH][8], u[GATED ? BATCH : 1][8];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const size_t r = tl.row0 + min(i0 + k * kSlices, tl.rows - 1);
                load8<OT>(p.dout, r * width + n, whole, d[k]);
                if (GATED || ACT != ACT_NONE) load8<AT>(p.pre, r * p.N + n, whole, h[k]);
                if constexpr (GATED) load8<AT>(p.pre, r * p.N + width + n, whole, u[k]);
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (i0 + k * kSlices >= tl.rows) break;
                const size_t r = tl.row0 + i0 + k * kSlices;
                if constexpr (GATED) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float s = sigmoid(h[k][j]), g = h[k][j] * s;
                        const float du = d[k][j] * g;
                        d[k][j] = d[k][j] * u[k][j] * (s * (1.0f + h[k][j] * (1.0f - s)));
                        u[k][j] = du;
                        up_sum[j] += du;
                    }
                    if (p.dpre) store8<AT>(p.dpre, r * p.N + width + n, whole, u[k]);
                } else if constexpr (ACT != ACT_NONE) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[k][j] *= slope(ACT, h[k][j]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += d[k][j];
                if (p.dpre) store8<AT>(p.dpre, r * p.N + n, whole, d[k]);
            }
        }
    }
    if (!p.dbias) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sums[slice][lane * 8 + j] = sum[j];
        if constexpr (GATED) sums[slice][kActCols + lane * 8 + j] = up_sum[j];
    }
    __syncthreads();
    float* to = p.partial + place(tl.row0, tl.group, ROWS) * p.N;
    for (int c = threadIdx.x; c < kActCols * (GATED ? 2 : 1); c += 256) {
        const int col = c % kActCols;
        if (n0 + col >= width) continue;
        float v = 0.0f;
#pragma unroll
        for (int s = 0; s < kSlices; ++s) v += sums[s][c];
        to[(c >= kActCols ? width : 0) + n0 + col] = v;
    }
}

// The sums of a group's tiles: 32 columns by eight slices of the tiles.  In fp64, for a slice of 2^24 rows is a
// chain of 32768 additions.  Its loads bound it, sixteen at a time: both launches of 2^22 rows of 16 columns
// in fp32 take 577 us (eight at a time, fp64: 729, fp32: 703).
__global__ __launch_bounds__(256) void k_bias_sums(ActivationArgs p, int rows) {
    __shared__ double sums[8][32];
    const int g = blockIdx.y, lane = threadIdx.x & 31, slice = threadIdx.x >> 5, n = blockIdx.x * 32 + lane;
    int lo = 0, hi = p.M;
    if (p.offsets) {
        lo = min(max(p.offsets[g], 0), p.M);
        hi = min(max(p.offsets[g + 1], lo), p.M);
    }
    const int tiles = (hi - lo + rows - 1) / rows;
    double v = 0.0;
    if (n < p.N) {
        const float* from = p.partial + place(lo, g, rows) * p.N + n;
#pragma unroll 16
        for (int i = slice; i < tiles; i += 8) v += from[(size_t)i * p.N];
    }
    sums[slice][lane] = v;
    __syncthreads();
    if (slice || n >= p.N) return;
#pragma unroll
    for (int s = 1; s < 8; ++s) v += sums[s][lane];
    p.dbias[(size_t)g * p.N + n] = (float)v;
}

}  // namespace

size_t activation_workspace(int M, int G, int N) { return (size_t)(M / act_rows(M, G, N) + G) * N * sizeof(float); }

hipError_t launch_activation_backward(int atype, int out_atype, const ActivationArgs& a, hipStream_t s) {
    const int rows = act_rows(a.M, a.G, a.N);
    const int nblocks = ((a.act == ACT_SWIGLU ? a.N / 2 : a.N) + kActCols - 1) / kActCols;
    const int64_t grid = nblocks * most_tiles(a.M, a.G, a.offsets, rows);   // 2^36 values: below 2^24 of them
    auto run = [&](auto at, auto ot, auto act) {
        constexpr int AT = decltype(at)::value, OT = decltype(ot)::value, ACT = decltype(act)::value;
        if (rows == 16)
            hipLaunchKernelGGL((k_activation_backward<AT, OT, ACT, 16>), dim3((unsigned)grid), dim3(256), 0, s, a, nblocks);
        else
            hipLaunchKernelGGL((k_activation_backward<AT, OT, ACT, 64>), dim3((unsigned)grid), dim3(256), 0, s, a, nblocks);
        return hipGetLastError();
    };
    if (grid > 0) {
        const hipError_t e = by_types(atype, out_atype, [&](auto at, auto ot) {
            switch (a.act) {
            case ACT_RELU: return run(at, ot, std::integral_constant<int, ACT_RELU>{});
            case ACT_GELU: return run(at, ot, std::integral_constant<int, ACT_GELU>{});
            case ACT_SILU: return run(at, ot, std::integral_constant<int, ACT_SILU>{});
            case ACT_SWIGLU: return run(at, ot, std::integral_constant<int, ACT_SWIGLU>{});
            default: return run(at, ot, std::integral_constant<int, ACT_NONE>{});
            }
        });
        if (e) return e;
    }
    if (a.dbias) hipLaunchKernelGGL(k_bias_sums, dim3((a.N + 31) / 32, a.G), dim3(256), 0, s, a, rows);
    return hipGetLastError();
}

}  // namespace moe
