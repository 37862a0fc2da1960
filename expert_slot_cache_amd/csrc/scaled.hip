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

#include <type_traits>

#include "ops.hpp"
#include "ops_dev.hpp"
#include "product_tile.hpp"
#include "works.hpp"

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
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
// instruction: the products are exact and added in fp32 (measured off by at most 2^-21 of the sum
// of their magnitudes; 128 additions of two half steps would be 2^-16).  The fp8 instruction, at twice the rate, is no choice: it aligns each eight
// products (k .. k+7) to the largest of them and drops what lies 13 bits below its leading one
// (measured), so where large products cancel nothing that is left of the sum need be right.
// What that costs where the matrix rate binds: 32768 rows of 64 groups, N = K = 4096, take 1150
// us, 685 with it; 512 rows of 97 groups, 4096 x 1536, where memory binds, 110 against 107.
struct Wide {
    bf16x8_t v[4];
};
__device__ __forceinline__ Wide widen_block(const i32x8_t& a) {
    return {{widen8(a[0], a[1]), widen8(a[2], a[3]), widen8(a[4], a[5]), widen8(a[6], a[7])}};
}
__device__ __forceinline__ f32x4_t mfma_block(const Wide& a, const Wide& b) {
    f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
}

// silu(gate) * up with the hardware's exponential and reciprocal (1 ulp each): within about
// (4 + |gate|) 2^-24 of the value, far below the half step 2^-4 of the e4m3 code it becomes, while
// the exponential and the reciprocal are normal numbers; below gate = -87.3 the latter is none, and
// below -88.7 the result is 0, as the quotient in fp32 is.  The exact quotient and exponential
// took as long as three stages of a tile.
__device__ __forceinline__ float silu_mul(float gate, float up) {
    return gate * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gate * -1.44269504f)) * up;
}

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

typedef __attribute__((address_space(3))) char lds_char;

// 16 (or 4) bytes per lane from memory to LDS: lane i's go to lds + 16 i (4 i).  The compiler
// does not count these loads: the kernel waits for them itself, before its barrier.  The LDS
// address is an operand in M0, which the compiler so knows to be taken; one wait state lies between
// the two.  A base is a sum made by scalar instructions: a load has to wait for no result of theirs.
__device__ __forceinline__ void copy16(uint32_t lds, uint32_t voff, const uint8_t* base) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(lds), "v"(voff), "s"(base) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t lds, const float* p) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t lds, const float* p) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off" ::"{m0}"(lds), "v"(p) : "memory");
}
// All but this wave's newest N copies have landed and its LDS reads are done, and so for
// every wave of the workgroup.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <class T>
struct Shape {
    static constexpr int TW = T::TW, TT = T::TT, WAVES = T::WAVES, S = T::S;
    static constexpr int WT = TT > 64 ? TT / 64 : 1;       // waves along tokens,
    static constexpr int WW = WAVES / WT;                  // along matrix rows
    static constexpr int FA = TW / WW / 16, FB = TT / WT / 16;   // fragments of a wave
    static constexpr int AR = FA > 1 ? 2 : 1;              // matrix fragments in registers
    static constexpr int NA = TW / 8 / WAVES;              // a wave's copies of 8 matrix rows,
    static constexpr int NB = TT / 8 / WAVES;              // of 8 token rows (0: not every wave has one)
    static constexpr int XWAVES = TT / 8;                  // waves with one, where NB is 0
    static constexpr int SWAVES = (TT + 2 + 63) / 64;      // the last waves copy the scales, 64 each
    static constexpr int STAGE = (TW + TT) * 128;
    static constexpr int SCALES = S * STAGE;               // their place: TT, then the matrix', per block
    static constexpr int FOURS = S <= 5 ? 2 : 4;           // or four blocks at a time (see fill)
    static constexpr int LDS = SCALES + SWAVES * 64 * 4 * (4 * FOURS > S ? 4 * FOURS : S);
    static_assert(FA >= 1 && FB >= 1 && NA >= 1 && (NB > 0 || XWAVES <= WAVES) && SWAVES <= WAVES, "");
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
    const Works<TT> works(a.offsets, a.G, a.M, nblocks);
    // workgroup b runs on XCD b % 8: each XCD takes one contiguous run of the work
    const int per = (works.total + 7) >> 3;
    const int jx = (int)(blockIdx.x >> 3);
    const int wk = (int)(blockIdx.x & 7) * per + jx;
    if (jx >= per || wk >= works.total) return;
    const Work tl = works.at(wk);
    const int nb = tl.nb;
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
    // A token's scale lies in a line of memory of its own, so four blocks' scales are copied at
    // once where rows of scales start on 16 bytes (one block's cost as much as a third of its
    // codes); FOURS such groups are kept, so that none is overwritten while S - 1 stages ahead
    // of its last use.
    const bool fours = TT >= 64 && kb_n % 4 == 0 && (reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws)) % 16 == 0;
    // In a last, shorter block the chunks past the end of a row are copied from its last 16
    // bytes (`over` back from where they would be) and cleared in LDS once they have landed.
    const int tail = K % kBlock;
    const uint32_t over = tail && chunk >= tail ? chunk - (tail - 16) : 0;

    auto fill = [&](int kb, int stage) {
        const uint32_t at = lds0 + stage * C::STAGE;
        const size_t k0 = (size_t)kb * kBlock;
        const uint32_t back = kb == kb_n - 1 ? over : 0;
#pragma unroll
        for (int i = 0; i < NA; ++i) copy16(at + (wave + WAVES * i) * 1024, aoff[i] - back, abase[i] + k0);
        if (has_x)
#pragma unroll
            for (int i = 0; i < NB1; ++i) copy16(at + C::TW * 128 + (wave + WAVES * i) * 1024, boff[i] - back, bbase + k0);
        if (has_s) {
            const int sw = wave - (WAVES - C::SWAVES);
            if (!fours) copy4(lds0 + C::SCALES + (stage * C::SWAVES + sw) * 256, sp + kb);
            else if (kb % 4 == 0) copy16(lds0 + C::SCALES + (kb / 4 % C::FOURS * C::SWAVES + sw) * 1024, sp + kb);
        }
    };

    constexpr int BASE = NA + NB;                          // a wave's copies of rows, a stage; or one more
    // Waits until all but the newest N stages of this wave's copies of rows have landed, and
    // meets.  The scales' copies are not counted: a wave that made some waits for a little more.
    auto landed = [&](auto stages) {
        constexpr int N = decltype(stages)::value;
        if (NB > 0 || !has_x) wait_and_meet<N * BASE>();
        else wait_and_meet<N * (BASE + 1)>();
    };
    auto clear = [&](int stage) {                          // the last block's chunks past the end
        __syncthreads();
        for (int i = tid; i < (C::TW + TT) * 8; i += 64 * WAVES) {
            const int r = i >> 3, c = i & 7;
            if (c * 16 >= tail) *reinterpret_cast<i32x4_t*>(lds + stage * C::STAGE + r * 128 + ((c ^ (r & 7)) * 16)) = i32x4_t{0, 0, 0, 0};
        }
        __syncthreads();
    };
    // In the middle of stage kb, once a wave has read all that it needs of it: wait until this
    // wave's copies of stage kb + 1 have landed (those of the S - 2 stages behind it stay in
    // flight, but at the end of the row, where there are fewer), then for every wave's; the
    // place of stage kb is refilled.
    auto meet = [&](int kb, int stage, int next) {
        if (kb + 1 >= kb_n) return;
        if (kb + C::S - 1 < kb_n) landed(std::integral_constant<int, C::S - 2>{});
        else wait_and_meet<0>();
        if (kb + C::S < kb_n) fill(kb + C::S, stage);
        if (tail && kb + 2 == kb_n) clear(next);
    };
#pragma unroll
    for (int i = 0; i < C::S; ++i)
        if (i < kb_n) fill(i, i);
    if (kb_n >= C::S) landed(std::integral_constant<int, C::S - 1>{});
    else wait_and_meet<0>();
    if (tail && kb_n == 1) clear(0);

    f32x4_t acc[FA][FB];
#pragma unroll
    for (int j = 0; j < FA; ++j)
#pragma unroll
        for (int m = 0; m < FB; ++m) acc[j][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (wt * 16 * FB >= tl.rows) {                         // no token for this wave: it only copies
        for (int kb = 0, stage = 0; kb < kb_n; ++kb) {
            const int next = stage + 1 == C::S ? 0 : stage + 1;
            meet(kb, stage, next);
            stage = next;
        }
        if constexpr (GATED) {                             // and meets the others where they share maxima
            __syncthreads();
            __syncthreads();
        }
        return;
    }

    constexpr int AR = C::AR, P = FA * FB < 3 ? FA * FB : 3;   // P: sums on their way to acc
    const int place = (q ^ (l16 & 7)) * 16;                // chunk q of a row; chunk q + 4 is at place ^ 64
    const int a0 = (ww * 16 * FA + l16) * 128 + place, b0 = C::TW * 128 + (wt * 16 * FB + l16) * 128 + place;
    auto fragment = [&](i32x8_t& v, const char* at, int to) {
        const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(at + to);
        const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(at + (to ^ 64));
        v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    i32x8_t b[FB], av[AR];
    fragment(av[0], lds, a0);
#pragma unroll
    for (int m = 0; m < FB; ++m) fragment(b[m], lds, b0 + m * 2048);
    int stage = 0;
    for (int kb = 0; kb < kb_n; ++kb) {
        // Product i (of fragments i / FB and i % FB), the adds of product i - 2, and the reads
        // that the products to come need, those of the next stage among them, in this order:
        // the compiler's own moves the reads next to their uses and the adds behind all products.
        const int next = stage + 1 == C::S ? 0 : stage + 1;
        const char* st = lds + stage * C::STAGE;
        const char* nx = lds + next * C::STAGE;
        const float* sc = reinterpret_cast<const float*>(lds + C::SCALES) +
                          (fours ? kb / 4 % C::FOURS * C::SWAVES * 256 + kb % 4 : stage * C::SWAVES * 64);
        const int each = fours ? 4 : 1;
        float xs[FB];
#pragma unroll
        for (int m = 0; m < FB; ++m) xs[m] = sc[(wt * 16 * FB + m * 16 + l16) * each];
        const float w0 = sc[TT * each], w1 = sc[(TT + 1) * each];
        f32x4_t part[P];
        Wide bw[FB], aw;
        auto add = [&](int i) {
            const int j = i / FB, m = i % FB;
            const float ws = GATED ? (j < HF ? w0 : w1) : (ww * 16 * FA + j * 16) < kBlock ? w0 : w1;
            const float s = ws * xs[m];
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[j][m][k] += s * part[i % P][k];
            asm volatile("" : "+v"(acc[j][m]));            // here, not sunk behind the meeting
        };
#pragma unroll
        for (int j = 0; j < FA; ++j) {
            if (AR > 1 && j + 1 < FA) fragment(av[(j + 1) % AR], st, a0 + (j + 1) * 2048);
            if (j == FA - 1) meet(kb, stage, next);
            if (AR > 1 && j + 1 == FA) fragment(av[(j + 1) % AR], nx, a0);
            aw = widen_block(av[j % AR]);
#pragma unroll
            for (int m = 0; m < FB; ++m) {
                const int i = j * FB + m;
                if (j == 0) bw[m] = widen_block(b[m]);
                part[i % P] = mfma_block(aw, bw[m]);
                if (j + 1 == FA) fragment(b[m], nx, b0 + m * 2048);
                if (i >= P - 1) add(i - (P - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (AR == 1) fragment(av[0], nx, a0);
#pragma unroll
        for (int i = FA * FB - P + 1; i < FA * FB; ++i) add(i);
        stage = next;
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

template <class C, int OUT>
hipError_t product(const ProductArgs& a, hipStream_t s) {
    constexpr int COLS = OUT == OUT_SWIGLU ? C::TW / 2 : C::TW;
    const int cols = OUT == OUT_SWIGLU ? a.N / 2 : a.N;
    const int nblocks = (cols + COLS - 1) / COLS, kb_n = (a.K + kBlock - 1) / kBlock;
    const int64_t grid = (nblocks * most_tiles(a.M, a.G, a.offsets, C::TT) + 7) / 8 * 8;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_product<C, OUT>), dim3((unsigned)grid), dim3(64 * C::WAVES), 0, s, a, nblocks, kb_n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled_product(const ProductArgs& a, int out, hipStream_t s) {
    auto run = [&](auto o) {
        constexpr int OUT = decltype(o)::value;
        return product_tile<OUT == OUT_SWIGLU>(a.M, a.G, a.N, a.offsets, [&](auto tile) {
            return product<Shape<decltype(tile)>, OUT>(a, s);
        });
    };
    if (out == OUT_SWIGLU) return run(std::integral_constant<int, OUT_SWIGLU>{});
    if (out == OUT_BF16) return run(std::integral_constant<int, OUT_BF16>{});
    return run(std::integral_constant<int, OUT_F32>{});
}

}  // namespace moe
