// The product of sorted rows with their expert's matrix in 8-bit floating point (e4m3),
// one scale for each 128 values of a row and each 128 x 128 values of a matrix:
//
//   out[r][n] = sum_b xs[r][b] ws[g][n/128][b] (sum_{k in block b} x[r][k] w[g][n][k])
//
// for the rows r of group g (offsets[g] <= r < offsets[g+1]).  The matrix rows are the MFMA's
// A operand, the tokens its B operand, so an accumulator register holds one token per lane
// and a token's scale is one value per lane; a block of 128 is summed from zero and one fp32
// FMA per element adds it with its scale.  Both operands load a lane's 32 bytes of a block
// the same way (16 at 16 (lane/16) and 16 at 64 + 16 (lane/16)): a sum over k does not depend
// on the order of k as long as both agree on it.
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "ops_dev.hpp"

namespace moe {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Eight e4m3 codes as bf16 (exact: three mantissa bits).
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi) {
    const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8_t{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// One block of 128, 32 codes per lane of each operand, summed from zero by the bf16 matrix
// instruction: the products are exact in fp32 and so, nearly, is their sum (within 2^-20 of
// the largest).
struct Wide {
    bf16x8_t v[4];
};
__device__ __forceinline__ Wide widen_block(const uint4 a[2]) {
    return {{widen8(a[0].x, a[0].y), widen8(a[0].z, a[0].w), widen8(a[1].x, a[1].y), widen8(a[1].z, a[1].w)}};
}
__device__ __forceinline__ f32x4_t mfma_block(const Wide& a, const Wide& b) {
    f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
}

// Row tile number `tile` of all groups' tiles of TM rows, in group order: its group, first
// row and rows (0: there is no such tile).  Every wave finds it for itself: a lane counts
// the tiles of its run of groups, a prefix over the lanes picks the run.  Offsets outside
// [0, M] or falling ones (they are device data) count as empty groups, so that no row
// outside the buffers is ever touched.
struct Tile {
    int group, row0, rows;
};
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ offsets, int G, int M, int TM, int tile) {
    if (!offsets) {
        const int row0 = tile * TM;
        return {0, row0, row0 < M ? min(TM, M - row0) : 0};
    }
    const int lane = threadIdx.x & 63;
    const int per = (G + 63) >> 6;
    const int g0 = min(lane * per, G), g1 = min(g0 + per, G);
    int own = 0;
    int lo = min(max(offsets[g0], 0), M);
    for (int g = g0; g < g1; ++g) {
        const int hi = min(max(offsets[g + 1], lo), M);
        own += (hi - lo + TM - 1) / TM;
        lo = hi;
    }
    int incl = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    const uint64_t past = __ballot(incl > tile);
    if (!past) return {0, 0, 0};
    const int who = __builtin_ctzll(past);
    int found_g = 0, found_row = 0, found_n = 0;
    if (lane == who) {
        int left = tile - (incl - own);
        lo = min(max(offsets[g0], 0), M);
        for (int g = g0; g < g1; ++g) {
            const int hi = min(max(offsets[g + 1], lo), M);
            const int n = (hi - lo + TM - 1) / TM;
            if (left < n) {
                found_g = g;
                found_row = lo + left * TM;
                found_n = min(TM, hi - found_row);
                break;
            }
            left -= n;
            lo = hi;
        }
    }
    return {__builtin_amdgcn_readlane(found_g, who), __builtin_amdgcn_readlane(found_row, who),
            __builtin_amdgcn_readlane(found_n, who)};
}

__device__ __forceinline__ float silu_mul(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

// Few rows per group: the matrix streams from memory straight into MFMA operands.
// A workgroup takes MT tiles of 16 rows of one group and 16 NT WN matrix rows; its WN x KS
// waves split the matrix rows and the blocks of k (wave ks takes blocks ks, ks + KS, ...),
// and the KS partial sums meet in LDS, in order.  SwiGLU: WN = 8, NT = 2, a wave's two tiles
// being 16 gate rows and the 16 up rows of the same columns, so that a workgroup holds all
// 128 columns that share a scale.
template <int NT, int MT, int WN, int KS, int OUT>
__global__ __launch_bounds__(64 * WN * KS) void k_product_stream(ProductArgs a, int nblocks, int kb_n) {
    constexpr int U = NT * MT >= 4 ? 2 : 4;           // blocks of k requested at a time
    constexpr int COLS = OUT == OUT_SWIGLU ? 16 * WN : 16 * NT * WN;   // columns written
    constexpr int PAD = 4;                            // floats: column runs start on other banks
    __shared__ float red[KS][NT][MT][WN][16][16 + PAD];
    const int nb = blockIdx.x % nblocks, tile = blockIdx.x / nblocks;
    const Tile tl = find_tile(a.offsets, a.G, a.M, 16 * MT, tile);
    if (!tl.rows) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % WN, ks = wave / WN;
    const int q = lane >> 4, l16 = lane & 15;
    const int K = a.K;
    const int n_half = a.N / 2;
    const uint8_t* wg = a.w + (size_t)tl.group * a.N * K;
    const float* sg = a.ws + (size_t)tl.group * ((a.N + kBlock - 1) / kBlock) * kb_n;
    const uint8_t* wp[NT];
    const float* sp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        int n0 = OUT == OUT_SWIGLU ? t * n_half + nb * COLS + wn * 16 : nb * COLS + (wn * NT + t) * 16;
        n0 = min(n0, a.N - 1);
        sp[t] = sg + (size_t)(n0 / kBlock) * kb_n;
        wp[t] = wg + (size_t)min(n0 + l16, a.N - 1) * K;
    }
    const uint8_t* xp[MT];
    const float* xsp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const size_t r = tl.row0 + min(m * 16 + l16, tl.rows - 1);   // rows past the end: never stored
        xp[m] = a.x + r * K;
        xsp[m] = a.xs + r * kb_n;
    }
    f32x4_t acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const uint4 none = make_uint4(0, 0, 0, 0);
    for (int kb0 = ks; kb0 < kb_n; kb0 += KS * U) {
        uint4 wv[U][NT][2], xv[U][MT][2];
        float ss[U][NT], xs[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * KS;
            const int k = kb * kBlock + q * 16;
            const bool in0 = k < K, in1 = k + 64 < K;   // K is a multiple of 16
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                wv[u][t][0] = in0 ? *reinterpret_cast<const uint4*>(wp[t] + k) : none;
                wv[u][t][1] = in1 ? *reinterpret_cast<const uint4*>(wp[t] + k + 64) : none;
                ss[u][t] = kb < kb_n ? sp[t][kb] : 0.0f;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                xv[u][m][0] = in0 ? *reinterpret_cast<const uint4*>(xp[m] + k) : none;
                xv[u][m][1] = in1 ? *reinterpret_cast<const uint4*>(xp[m] + k + 64) : none;
                xs[u][m] = kb < kb_n ? xsp[m][kb] : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (kb0 + u * KS < kb_n) {
                Wide xw[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) xw[m] = widen_block(xv[u][m]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const Wide ww = widen_block(wv[u][t]);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const f32x4_t part = mfma_block(ww, xw[m]);
                        const float s = ss[u][t] * xs[u][m];
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[t][m][i] += s * part[i];
                    }
                }
            }
    }
    // accumulator element i: matrix row 4 (lane/16) + i of the tile, token lane % 16
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            *reinterpret_cast<f32x4_t*>(&red[ks][t][m][wn][l16][4 * q]) = acc[t][m];
    __syncthreads();
    if constexpr (OUT == OUT_SWIGLU) {
        // 32 lanes a row, 4 columns each
        for (int it = threadIdx.x; it < MT * 16 * 32; it += 64 * WN * KS) {
            const int c4 = it & 31, r = it >> 5;
            const int m = r >> 4, l = r & 15, wc = c4 >> 2, c = (c4 & 3) * 4;
            float v[4], big = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float g = 0.0f, u = 0.0f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    g += red[s][0][m][wc][l][c + i];
                    u += red[s][NT - 1][m][wc][l][c + i];
                }
                v[i] = silu_mul(g, u);
                const float mag = fabsf(v[i]);
                if (mag < __builtin_inff()) big = fmaxf(big, mag);
                else v[i] = __builtin_nanf("");
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) big = fmaxf(big, __shfl_xor(big, d));
            if (r < tl.rows) {
                const float scale = f8_scale(big), inv = f8_inverse(scale);
                const size_t row = tl.row0 + r;
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + row * n_half + nb * COLS + c4 * 4) =
                    f8_pack(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                if (c4 == 0) a.os[row * (n_half / kBlock) + nb] = scale;
            }
        }
    } else {
        for (int it = threadIdx.x; it < MT * 16 * COLS; it += 64 * WN * KS) {
            const int c = it % COLS, r = it / COLS;
            const int n = nb * COLS + c;
            if (r >= tl.rows || n >= a.N) continue;
            const int wc = c / (16 * NT), t = (c / 16) % NT;
            float v = 0.0f;
#pragma unroll
            for (int s = 0; s < KS; ++s) v += red[s][t][r >> 4][wc][r & 15][c & 15];
            store_one<OUT == OUT_F32 ? A_F32 : A_BF16>(a.out, (size_t)(tl.row0 + r) * a.N + n, v);
        }
    }
}

// Tiles of TM rows that the groups can have: each group's last one may be short.
int64_t most_tiles(const ProductArgs& a, int TM) {
    const int64_t full = ((int64_t)a.M + TM - 1) / TM;
    if (!a.offsets) return full;
    return (int64_t)a.M / TM + (a.G < a.M ? a.G : a.M);
}

template <int NT, int MT, int WN, int KS, int OUT>
hipError_t stream(const ProductArgs& a, hipStream_t s) {
    constexpr int COLS = OUT == OUT_SWIGLU ? 16 * WN : 16 * NT * WN;
    const int cols = OUT == OUT_SWIGLU ? a.N / 2 : a.N;
    const int nblocks = (cols + COLS - 1) / COLS, kb_n = (a.K + kBlock - 1) / kBlock;
    const int64_t grid = nblocks * most_tiles(a, 16 * MT);
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_product_stream<NT, MT, WN, KS, OUT>), dim3((unsigned)grid), dim3(64 * WN * KS), 0, s, a,
                       nblocks, kb_n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled_product(const ProductArgs& a, int out, hipStream_t s) {
    if (out == OUT_SWIGLU) return stream<2, 1, 8, 2, OUT_SWIGLU>(a, s);
    if (out == OUT_BF16) return stream<1, 1, 1, 4, OUT_BF16>(a, s);
    return stream<1, 1, 1, 4, OUT_F32>(a, s);
}

}  // namespace moe
