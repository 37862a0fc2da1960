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

// The row tiles of all groups, TM rows each, in group order.  Every wave counts them for
// itself: a lane takes a run of groups, a prefix over the lanes orders the runs.  Offsets
// outside [0, M] or falling ones (they are device data) count as empty groups, so that no
// row outside the buffers is ever touched.
struct Tile {
    int group, row0, rows;
};
template <int TM>
struct Tiles {
    const int32_t* offsets;
    int M, g0, g1, lo0, hi0, own, incl, total;   // lo0, hi0: the rows of group g0
    __device__ __forceinline__ Tiles(const int32_t* __restrict__ off, int G, int M_) : offsets(off), M(M_) {
        if (!off) {
            total = (M + TM - 1) / TM;
            return;
        }
        const int lane = threadIdx.x & 63;
        const int per = (G + 63) >> 6;
        g0 = min(lane * per, G);
        g1 = min(g0 + per, G);
        lo0 = bound(off[g0], 0);
        hi0 = g0 < g1 ? bound(off[g0 + 1], lo0) : lo0;
        own = (hi0 - lo0 + TM - 1) / TM;
        int lo = hi0;
        for (int g = g0 + 1; g < g1; ++g) {
            const int hi = bound(off[g + 1], lo);
            own += (hi - lo + TM - 1) / TM;
            lo = hi;
        }
        incl = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
        total = __builtin_amdgcn_readlane(incl, 63);
    }
    __device__ __forceinline__ int bound(int v, int lo) const { return min(max(v, lo), M); }
    // Tile number `tile`, 0 <= tile < total.
    __device__ __forceinline__ Tile at(int tile) const {
        if (!offsets) return {0, tile * TM, min(TM, M - tile * TM)};
        const int who = __builtin_ctzll(__ballot(incl > tile));
        int group = 0, row0 = 0, rows = 0;
        if ((int)(threadIdx.x & 63) == who) {
            int left = tile - (incl - own);
            int lo = lo0;
            for (int g = g0; g < g1; ++g) {
                const int hi = g == g0 ? hi0 : bound(offsets[g + 1], lo);
                const int n = (hi - lo + TM - 1) / TM;
                if (left < n) {
                    group = g;
                    row0 = lo + left * TM;
                    rows = min(TM, hi - row0);
                    break;
                }
                left -= n;
                lo = hi;
            }
        }
        return {__builtin_amdgcn_readlane(group, who), __builtin_amdgcn_readlane(row0, who),
                __builtin_amdgcn_readlane(rows, who)};
    }
};

__device__ __forceinline__ float silu_mul(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

// ---- the kernel ------------------------------------------------------------------------------
//
// A workgroup takes TW matrix rows x TT rows of one group.  A stage is one block of 128: 128
// bytes of each matrix row and token row, copied from memory straight into LDS (16 bytes a
// lane, no registers), and the block's scales; S stages form a ring, filled S - 1 stages
// ahead, with one barrier per stage.  In LDS a row is eight 16-byte chunks, chunk c at place
// c ^ (row % 8), so that the rows a fragment reads at one chunk lie in different banks; the
// copy places lane i's 16 bytes at 16 i, so a lane picks its source chunk accordingly.
//
// The waves form WW x WT; each computes 16 FA matrix rows x 16 FB token rows.  The matrix
// rows of a wave are dealt to its FA fragments four at a time, so that the fragments'
// accumulators of one lane are consecutive columns of the output.
//
// The bf16 and e4m3 outputs use the fp8 matrix instruction (twice the bf16 rate).  It aligns
// each eight products (k .. k+7) to the largest of them and keeps 13 bits below its leading
// one (measured), so a block's sum is off by less than 2^-10 of the sum over the eights of
// their largest product, typically 2^-16 of the result: far below the 2^-8 of a bf16 output.
// An fp32 output takes the bf16 instruction on the widened codes instead.
typedef __attribute__((address_space(3))) char lds_char;

__device__ __forceinline__ f32x4_t mfma_codes(const uint4 a[2], const uint4 b[2]) {
    const i32x8_t av = {(int)a[0].x, (int)a[0].y, (int)a[0].z, (int)a[0].w, (int)a[1].x, (int)a[1].y, (int)a[1].z, (int)a[1].w};
    const i32x8_t bv = {(int)b[0].x, (int)b[0].y, (int)b[0].z, (int)b[0].w, (int)b[1].x, (int)b[1].y, (int)b[1].z, (int)b[1].w};
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, zero, 0, 0, 0, 0, 0, 0);
}

// 16 (or 4) bytes per lane from memory to LDS: lane i's go to lds + 16 i (4 i).  The compiler
// does not count these loads: the kernel waits for them itself, before its barrier.  M0 holds
// the LDS address; the compiler keeps nothing there (it sets it right before its own uses).
__device__ __forceinline__ void copy16(uint32_t lds, uint32_t voff, const uint8_t* base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t lds, const uint8_t* p) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t lds, const float* p) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory");
}
// All but this wave's newest N copies have landed and its LDS reads are done, and so for
// every wave of the workgroup.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __align__(16) const uint8_t k_zeros[16] = {};   // what lies past the end of a row

template <int TW_, int TT_, int WAVES_, int S_>
struct Shape {
    static constexpr int TW = TW_, TT = TT_, WAVES = WAVES_, S = S_;
    static constexpr int WT = TT > 64 ? TT / 64 : 1;       // waves along tokens,
    static constexpr int WW = WAVES / WT;                  // along matrix rows
    static constexpr int FA = TW / WW / 16, FB = TT / WT / 16;   // fragments of a wave
    static constexpr int NA = TW / 8 / WAVES;              // a wave's copies of 8 matrix rows,
    static constexpr int NB = TT / 8 / WAVES;              // of 8 token rows (0: not every wave has one)
    static constexpr int XWAVES = TT / 8;                  // waves with one, where NB is 0
    static constexpr int SWAVES = (TT + 2 + 63) / 64;      // the last waves copy the scales, 64 each
    static constexpr int SCALES = (TW + TT) * 128;         // their place in a stage: TT, then the matrix'
    static constexpr int STAGE = SCALES + SWAVES * 256;
    static constexpr int LDS = S * STAGE;
    static_assert(FA >= 1 && FB >= 1 && NA >= 1 && (NB > 0 || XWAVES + SWAVES <= WAVES) && SWAVES <= WAVES, "");
};

template <class C, int OUT>
__global__ __launch_bounds__(64 * C::WAVES) void k_product(ProductArgs a, int nblocks, int kb_n) {
    constexpr bool GATED = OUT == OUT_SWIGLU;
    constexpr int FA = C::FA, FB = C::FB, NA = C::NA, NB = C::NB, TT = C::TT, WAVES = C::WAVES;
    constexpr int HF = GATED ? FA / 2 : FA;               // fragments of one half
    constexpr int CF = HF < 4 ? HF : 4;                   // fragments that share runs of columns
    constexpr int COLS = GATED ? C::TW / 2 : C::TW;       // columns written
    static_assert(!GATED || (C::TW == 256 && HF >= 1), "a scale's 128 columns in one workgroup");
    __shared__ __align__(1024) char lds[C::LDS];
    const Tiles<TT> tiles(a.offsets, a.G, a.M);
    // workgroup b runs on XCD b % 8: each XCD takes one contiguous run of the (tile, column
    // block) list, column block fastest, so that what shares rows or matrices shares an L2
    const int nwork = tiles.total * nblocks;
    const int per = (nwork + 7) >> 3;
    const int jx = (int)(blockIdx.x >> 3);
    const int wk = (int)(blockIdx.x & 7) * per + jx;
    if (jx >= per || wk >= nwork) return;
    const int nb = wk % nblocks;
    const Tile tl = tiles.at(wk / nblocks);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ww = wave % C::WW, wt = wave / C::WW;
    const int q = lane >> 4, l16 = lane & 15;
    const int K = a.K, n_half = a.N / 2;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
    const uint8_t* wg = a.w + (size_t)tl.group * a.N * K;
    const float* sg = a.ws + (size_t)tl.group * ((a.N + kBlock - 1) / kBlock) * kb_n;

    // this wave's copies: LDS rows (wave + WAVES i) * 8 + lane / 8
    const int l8 = lane >> 3, chunk = ((lane & 7) ^ l8) * 16;
    constexpr int NB1 = NB > 0 ? NB : 1;
    uint32_t aoff[NA], boff[NB1];
    const uint8_t* abase[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int row = (wave + WAVES * i) * 8;           // of this copy's first LDS row
        const int sec = row / (16 * FA), j = (row / 16) % FA, r = (row % 16) + l8;
        const int half = GATED ? j / HF : 0, jj = GATED ? j % HF : j;
        const int col = sec * 16 * HF + (jj / CF) * 16 * CF + (r >> 2) * 4 * CF + (jj % CF) * 4 + (r & 3);
        const int n0 = half * n_half + nb * COLS;
        abase[i] = wg + (size_t)n0 * K;
        aoff[i] = (uint32_t)min(col, a.N - 1 - n0) * (uint32_t)K + chunk;   // rows past the end: never stored
    }
    const bool has_x = NB > 0 || wave < C::XWAVES;
    const uint8_t* bbase = a.x + (size_t)tl.row0 * K;
#pragma unroll
    for (int i = 0; i < NB1; ++i)
        boff[i] = (uint32_t)min((wave + WAVES * i) * 8 + l8, tl.rows - 1) * (uint32_t)K + chunk;
    // the scales: slot i < TT holds token i's, the slots behind them those of the matrix' blocks
    // of 128 rows: gate and up, or the one or two of these TW rows
    const bool has_s = wave >= WAVES - C::SWAVES;
    const int slot = (wave - (WAVES - C::SWAVES)) * 64 + lane;
    const int nb_last = (a.N + kBlock - 1) / kBlock - 1;
    const int first = GATED ? nb : nb * COLS / kBlock;
    const int second = GATED ? n_half / kBlock + nb : min(first + 1, nb_last);
    const float* sp = slot < TT ? a.xs + (size_t)(tl.row0 + min(max(slot, 0), tl.rows - 1)) * kb_n
                                : sg + (size_t)(slot == TT + 1 ? second : first) * kb_n;
    const int copies = NA + (NB > 0 ? NB : has_x ? 1 : 0) + (has_s ? 1 : 0);   // of this wave, a stage
    const bool tail = K % kBlock != 0;

    auto fill = [&](int kb, int stage) {
        const uint32_t at = lds0 + stage * C::STAGE;
        const size_t k0 = (size_t)kb * kBlock;
        if (tail && kb == kb_n - 1) {
            const bool in = (int)k0 + chunk < K;
#pragma unroll
            for (int i = 0; i < NA; ++i) copy16(at + (wave + WAVES * i) * 1024, in ? abase[i] + aoff[i] + k0 : k_zeros);
            if (has_x)
#pragma unroll
                for (int i = 0; i < NB1; ++i)
                    copy16(at + C::TW * 128 + (wave + WAVES * i) * 1024, in ? bbase + boff[i] + k0 : k_zeros);
        } else {
#pragma unroll
            for (int i = 0; i < NA; ++i) copy16(at + (wave + WAVES * i) * 1024, aoff[i], abase[i] + k0);
            if (has_x)
#pragma unroll
                for (int i = 0; i < NB1; ++i) copy16(at + C::TW * 128 + (wave + WAVES * i) * 1024, boff[i], bbase + k0);
        }
        if (has_s) copy4(at + C::SCALES + (wave - (WAVES - C::SWAVES)) * 256, sp + kb);
    };

    f32x4_t acc[FA][FB];
#pragma unroll
    for (int j = 0; j < FA; ++j)
#pragma unroll
        for (int m = 0; m < FB; ++m) acc[j][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const bool idle = wt * 16 * FB >= tl.rows;             // no token of this wave: it only copies
    const int place = (q ^ (l16 & 7)) * 16;                // chunk q of a row; chunk q + 4 is at place ^ 64
    auto compute = [&](const char* st) {
        const float* sc = reinterpret_cast<const float*>(st + C::SCALES);
        const char* A = st + (ww * 16 * FA + l16) * 128;
        const char* B = st + C::TW * 128 + (wt * 16 * FB + l16) * 128;
        uint4 b[FB][2], av[2][2];
        float xs[FB];
        f32x4_t part[2][FB];
        auto fragment = [&](uint4 v[2], const char* p) {
            v[0] = *reinterpret_cast<const uint4*>(p + place);
            v[1] = *reinterpret_cast<const uint4*>(p + (place ^ 64));
        };
#pragma unroll
        for (int m = 0; m < FB; ++m) {
            fragment(b[m], B + m * 2048);
            xs[m] = sc[wt * 16 * FB + m * 16 + l16];
        }
        fragment(av[0], A);
        const float w0 = sc[TT], w1 = sc[TT + 1];
        auto scale = [&](int j) { return GATED ? (j < HF ? w0 : w1) : (ww * 16 * FA + j * 16) < kBlock ? w0 : w1; };
        auto add = [&](int j, int m) {
            const float s = scale(j) * xs[m];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][m][i] += s * part[j & 1][m][i];
        };
        Wide bw[OUT == OUT_F32 ? FB : 1];
        if constexpr (OUT == OUT_F32)
#pragma unroll
            for (int m = 0; m < FB; ++m) bw[m] = widen_block(b[m]);
        // the sums of fragment j - 1 are added between the products of fragment j
#pragma unroll
        for (int j = 0; j < FA; ++j) {
            if (j + 1 < FA) fragment(av[(j + 1) & 1], A + (j + 1) * 2048);
            if constexpr (OUT == OUT_F32) {
                const Wide aw = widen_block(av[j & 1]);
#pragma unroll
                for (int m = 0; m < FB; ++m) {
                    part[j & 1][m] = mfma_block(aw, bw[m]);
                    if (j > 0) add(j - 1, m);
                }
            } else {
#pragma unroll
                for (int m = 0; m < FB; ++m) {
                    part[j & 1][m] = mfma_codes(av[j & 1], b[m]);
                    if (j > 0) add(j - 1, m);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < FB; ++m) add(FA - 1, m);
    };
    // stage kb: wait for this wave's copies of it (those of the S - 2 stages behind it stay in
    // flight), then for every wave's; all have then left stage kb - 1, whose place is refilled
#pragma unroll
    for (int i = 0; i < C::S - 1; ++i)
        if (i < kb_n) fill(i, i);
    constexpr int BASE = NA + NB;                          // a wave copies BASE, or one or two more
    int stage = 0, ahead = C::S - 1;
    for (int kb = 0; kb < kb_n; ++kb) {
        if (C::S == 2 || kb + C::S - 2 >= kb_n) wait_and_meet<0>();
        else if (copies == BASE) wait_and_meet<(C::S - 2) * BASE>();
        else wait_and_meet<(C::S - 2) * (BASE + 1)>();
        if (kb + C::S - 1 < kb_n) fill(kb + C::S - 1, ahead);
        if (!idle) compute(lds + stage * C::STAGE);
        stage = stage + 1 == C::S ? 0 : stage + 1;
        ahead = ahead + 1 == C::S ? 0 : ahead + 1;
    }

    if constexpr (GATED) {
        // a lane holds 4 HF consecutive columns of a token, the lanes q = 0..3 and the WW waves
        // the 128 that share a scale
        constexpr int V = 4 * HF;
        float* big = reinterpret_cast<float*>(lds);        // [TT][WW], after the last stage
        __syncthreads();
#pragma unroll
        for (int m = 0; m < FB; ++m) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < HF; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = silu_mul(acc[j][m][i], acc[j + HF][m][i]);
                    const float mag = fabsf(v);
                    if (mag < __builtin_inff()) top = fmaxf(top, mag);
                    else v = __builtin_nanf("");
                    acc[j][m][i] = v;
                }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            if (q == 0) big[(wt * 16 * FB + m * 16 + l16) * C::WW + ww] = top;
        }
        __syncthreads();
        uint8_t* out = static_cast<uint8_t*>(a.out);
#pragma unroll
        for (int m = 0; m < FB; ++m) {
            const int r = wt * 16 * FB + m * 16 + l16;
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < C::WW; ++i) top = fmaxf(top, big[r * C::WW + i]);
            if (r >= tl.rows) continue;
            const float scale = f8_scale(top), inv = f8_inverse(scale);
            uint32_t u[HF];
#pragma unroll
            for (int j = 0; j < HF; ++j)
                u[j] = f8_pack(acc[j][m][0] * inv, acc[j][m][1] * inv, acc[j][m][2] * inv, acc[j][m][3] * inv);
            const size_t row = tl.row0 + r;
            uint32_t* o = reinterpret_cast<uint32_t*>(out + row * n_half + nb * COLS + ww * 16 * HF + q * V);
            if constexpr (HF == 4) *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
            else if constexpr (HF == 2) *reinterpret_cast<uint2*>(o) = make_uint2(u[0], u[1]);
            else *o = u[0];
            if (ww == 0 && q == 0) a.os[row * (n_half / kBlock) + nb] = scale;
        }
    } else {
        constexpr int es = OUT == OUT_F32 ? 4 : 2;
        const bool wide = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && (size_t)a.N * es % 16 == 0;
#pragma unroll
        for (int m = 0; m < FB; ++m) {
            const int r = wt * 16 * FB + m * 16 + l16;
            if (r >= tl.rows) continue;
            const size_t row = (size_t)(tl.row0 + r) * a.N;
#pragma unroll
            for (int jc = 0; jc < FA / CF; ++jc) {
                const int n = nb * COLS + ww * 16 * FA + jc * 16 * CF + q * 4 * CF;
                if (wide && n + 4 * CF <= a.N) {
                    if constexpr (OUT == OUT_F32) {
#pragma unroll
                        for (int j = 0; j < CF; ++j)
                            *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + row + n + 4 * j) = acc[jc * CF + j][m];
                    } else {
                        uint32_t u[2 * CF];
#pragma unroll
                        for (int j = 0; j < CF; ++j) {
                            const f32x4_t v = acc[jc * CF + j][m];
                            u[2 * j] = round_bf16(v[0]) | (uint32_t)round_bf16(v[1]) << 16;
                            u[2 * j + 1] = round_bf16(v[2]) | (uint32_t)round_bf16(v[3]) << 16;
                        }
                        if constexpr (CF == 1) {
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row + n) = make_uint2(u[0], u[1]);
                        } else {
#pragma unroll
                            for (int j = 0; j < CF / 2; ++j)
                                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row + n + 8 * j) =
                                    make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < CF; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (n + 4 * j + i < a.N)
                                store_one<OUT == OUT_F32 ? A_F32 : A_BF16>(a.out, row + n + 4 * j + i, acc[jc * CF + j][m][i]);
                }
            }
        }
    }
}

// Tiles of TM rows that the groups can have: each group's last one may be short.
int64_t most_tiles(const ProductArgs& a, int TM) {
    const int64_t full = ((int64_t)a.M + TM - 1) / TM;
    if (!a.offsets) return full;
    return (int64_t)a.M / TM + (a.G < a.M ? a.G : a.M);
}

template <class C, int OUT>
hipError_t product(const ProductArgs& a, hipStream_t s) {
    constexpr int COLS = OUT == OUT_SWIGLU ? C::TW / 2 : C::TW;
    const int cols = OUT == OUT_SWIGLU ? a.N / 2 : a.N;
    const int nblocks = (cols + COLS - 1) / COLS, kb_n = (a.K + kBlock - 1) / kBlock;
    const int64_t grid = (nblocks * most_tiles(a, C::TT) + 7) / 8 * 8;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_product<C, OUT>), dim3((unsigned)grid), dim3(64 * C::WAVES), 0, s, a, nblocks, kb_n);
    return hipGetLastError();
}

template <int OUT>
hipError_t by_rows(const ProductArgs& a, hipStream_t s) {
    const int64_t avg = a.M / a.G;
    if constexpr (OUT != OUT_F32)
        if (avg >= 128) return product<Shape<256, 256, 8, 2>, OUT>(a, s);
    if (avg >= 64) return product<Shape<256, 128, 8, 3>, OUT>(a, s);
    if (avg >= 16) return product<Shape<256, 64, 8, 3>, OUT>(a, s);
    if constexpr (OUT == OUT_SWIGLU) return product<Shape<256, 16, 8, 4>, OUT>(a, s);
    else if ((int64_t)(a.N / 128) * (a.G < a.M ? a.G : a.M) >= 512) return product<Shape<128, 16, 4, 4>, OUT>(a, s);
    else return product<Shape<64, 16, 4, 7>, OUT>(a, s);
}

}  // namespace

hipError_t launch_scaled_product(const ProductArgs& a, int out, hipStream_t s) {
    if (out == OUT_SWIGLU) return by_rows<OUT_SWIGLU>(a, s);
    if (out == OUT_BF16) return by_rows<OUT_BF16>(a, s);
    return by_rows<OUT_F32>(a, s);
}

}  // namespace moe
