// Tiles of a product on the matrix instruction, for bf16 and fp32 operands that lie in memory with
// the summed dimension along their rows or across them.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops_dev.hpp"
#include "product_tile.hpp"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

// 16 bytes per lane from memory to LDS: lane i's from base + off go to lds + 16 i, zeros where off lies
// past the buffer's end.  The compiler does not count these loads: the kernel waits for them itself,
// before its barrier.  The LDS address is an operand in M0, which the compiler so knows to be taken.
__device__ __forceinline__ void copy_bounded(uint32_t lds, uint32_t off, i32x4_t buffer) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(lds), "v"(off), "s"(buffer) : "memory");
}
__device__ __forceinline__ i32x4_t buffer_of(const char* base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return {__builtin_amdgcn_readfirstlane((int)(uint32_t)p), __builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xffffu)),
            __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
constexpr uint32_t kPastEnd = 0x80000000u;   // no buffer here is as long

// All but this wave's newest N copies have landed and its LDS reads are done, and so for
// every wave of the workgroup.
template <int N>
__device__ __forceinline__ void core_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One operand of a tile.  Along: `rows` rows from base on, `pitch` bytes apart, each `depth` bytes of
// the summed dimension.  Across: the summed dimension counts the rows, `depth` of them, of `rows`
// bytes each.  In LDS an along row is RB bytes, its 16-byte chunks exchanged so that the rows a
// fragment reads at one chunk lie in different banks; an across row is P elements, its 64-byte
// pieces exchanged so that the four rows that a transposing read takes do.
struct Operand {
    const char* base;
    uint32_t pitch;
    int rows, depth;
};

template <class C, int AT, bool ACROSS, int P>
struct Side {
    static constexpr int ES = AT == A_F32 ? 4 : 2, F = C::F, RB = C::RB;
    static constexpr int DEPTH = RB / ES;                  // a stage's, in elements
    static constexpr int PITCH = ACROSS ? P * ES : RB;     // of a row in LDS
    static constexpr int STEP = 64 / F * (16 / ES);        // of the summed dimension, an instruction (fp32: four)
    static constexpr int KK = DEPTH / STEP;
    static __device__ __forceinline__ int turn(int row) {  // what a row's chunks are exchanged by
        if (ACROSS) return AT == A_F32 ? 0 : P >= 128 ? row & 3 : P == 64 ? (row >> 1) & 1 : 0;
        return RB == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
    }
    // What lane `lane` of copy number c takes: offset from the stage's base.
    static __device__ __forceinline__ uint32_t source(int c, int lane, uint32_t pitch) {
        constexpr int PER = PITCH / 16;                    // chunks of an LDS row
        if constexpr (ACROSS) {
            const int at = c * 64 + lane, row = at / PER, chunk = at % PER;
            return row * pitch + ((chunk / 4 ^ turn(row)) * 4 + chunk % 4) * 16;
        } else {
            const int row = lane / PER;                    // and 1024 / RB rows a copy, added by the caller
            return (lane % PER ^ turn(c * C::ROWS + row)) * 16;
        }
    }
};

// A wave's fragments of one side, FR of them from element `first` of the tile on.
template <class C, int AT, bool ACROSS, int P, int FR>
struct Fragments {
    typedef Side<C, AT, ACROSS, P> S;
    static constexpr int F = C::F, KK = S::KK;
    typedef typename std::conditional<AT == A_F32, f32x4_t, bf16x8_t>::type Value;
    uint32_t at[ACROSS ? (AT == A_F32 ? 1 : FR) : KK];
    __device__ __forceinline__ Fragments(int first, int lane) {
        const int part = lane / F, l = lane % F;           // of the summed dimension; of the tile
        if constexpr (!ACROSS) {
            const int row = first + l;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) at[kk] = row * C::RB + ((kk * (64 / F) + part) ^ S::turn(row)) * 16;
        } else if constexpr (AT == A_F32) {
            at[0] = 4 * part * S::PITCH + (first + l) * 4;
        } else {
            const int i = lane & 15, row = 8 * part + (i >> 2);
#pragma unroll
            for (int f = 0; f < FR; ++f) {
                const int byte = (first + f * F + (F == 32 ? lane & 16 : 0) + 4 * (i & 3)) * 2;
                at[f] = row * S::PITCH + ((byte / 64) ^ S::turn(row)) * 64 + byte % 64;
            }
        }
    }
    __device__ __forceinline__ Value read(const char* lds, int f, int kk) const {
        if constexpr (!ACROSS) {
            return *reinterpret_cast<const Value*>(lds + at[kk] + f * F * C::RB);
        } else if constexpr (AT == A_F32) {
            Value v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float*>(lds + at[0] + (kk * S::STEP + i) * S::PITCH + f * F * 4);
            return v;
        } else {
            typedef __attribute__((address_space(3))) bf16x4_t lds_b4;
            const auto* p = (const __attribute__((address_space(3))) char*)(lds + at[f] + kk * S::STEP * S::PITCH);
            const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_b4*)p);
            const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_b4*)(p + 4 * S::PITCH));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

template <int F>
using Sums = typename std::conditional<F == 32, f32x16_t, f32x4_t>::type;

template <int F>
__device__ __forceinline__ Sums<F> multiply(bf16x8_t a, bf16x8_t b, Sums<F> c) {
    if constexpr (F == 32) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// Sixteen bytes of a row are four steps of the fp32 instruction: a sum over k does not depend on the
// order of k as long as both operands agree on it.
template <int F>
__device__ __forceinline__ Sums<F> multiply(f32x4_t a, f32x4_t b, Sums<F> c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F == 32) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
        else c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    }
    return c;
}

// A tile's sums.  GATED: the A side's fragments are dealt to two operands, a wave's first half from
// `a`, its second from `up`.  The sums of a wave with live = false are not taken.
template <class C, int AT, bool TA, bool TB, bool GATED>
__device__ __forceinline__ void core(char* lds, const Operand& a, const Operand& up, const Operand& b, bool live,
                                     Sums<C::F> (&acc)[C::FA][C::FB]) {
    typedef Side<C, AT, TA, C::PA> SA;
    typedef Side<C, AT, TB, C::PB> SB;
    constexpr int F = C::F, FA = C::FA, FB = C::FB, NA = C::NA, NB = C::NB, WAVES = C::WAVES, KK = SA::KK, S = C::S;
    constexpr int ES = SA::ES, DEPTH = SA::DEPTH;
    static_assert(!GATED || (!TA && FA % 2 == 0), "");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wa = wave % C::WA, wb = wave / C::WA;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
    const int depth = TA ? a.depth : a.depth / ES;
    const int stages = (depth + DEPTH - 1) / DEPTH;
    const int tail = (depth - (stages - 1) * DEPTH) * ES;  // bytes of a row in the last stage
    constexpr int NB1 = NB > 0 ? NB : 1;
    const bool has_b = NB > 0 || wave < C::CB;
    uint32_t aoff[NA], boff[NB1];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int c = wave + WAVES * i;
        aoff[i] = SA::source(c, lane, a.pitch);
        if constexpr (!TA) {
            int row = c * C::ROWS;                         // of this copy's first LDS row
            if constexpr (GATED) {
                const int sec = row / (F * FA), j = row / F % FA, r = row % F;
                row = sec * (F * FA / 2) + j % (FA / 2) * F + r;
            }
            aoff[i] += (row + lane / (C::RB / 16)) * a.pitch;
        }
    }
#pragma unroll
    for (int i = 0; i < NB1; ++i) {
        const int c = wave + WAVES * i;
        boff[i] = SB::source(c, lane, b.pitch);
        if constexpr (!TB) boff[i] += (c * C::ROWS + lane / (C::RB / 16)) * b.pitch;
    }
    // In the last, shorter stage an along row's chunks past its end are zeros; across, the rows are.  A
    // stage behind the last is all zeros: nothing is read for it, and it keeps the count of copies.
    auto bytes = [&](const Operand& o, bool across, int st) -> uint32_t {
        if (st >= stages) return 0;
        if (across) return (uint32_t)(min(DEPTH, o.depth - st * DEPTH) - 1) * o.pitch + o.rows;
        return (uint32_t)o.rows * o.pitch - st * C::RB;
    };
    auto buffer = [&](const Operand& o, bool across, int st) {
        return buffer_of(o.base + (across ? (size_t)st * DEPTH * o.pitch : (size_t)st * C::RB), bytes(o, across, st));
    };
    auto past = [&](int c) {                               // this lane's chunk of an along row lies past the end
        const int row = c * C::ROWS + lane / (C::RB / 16);
        return ((lane % (C::RB / 16)) ^ Side<C, AT, false, C::PA>::turn(row)) * 16 >= tail;
    };
    i32x4_t ba, bu, bb;
    uint32_t to;
    bool last;
    auto refill = [&](int st, int stage) {                 // stage st goes to place `stage`:
        ba = buffer(a, TA, st);
        if constexpr (GATED) bu = buffer(up, false, st);
        bb = buffer(b, TB, st);
        to = lds0 + stage * C::STAGE;
        last = st == stages - 1;
    };
    auto copy = [&](int i) {                               // its copy number i of this wave
        const bool of_a = i < NA;
        const int c = wave + WAVES * (of_a ? i : i - NA);
        if (!of_a && !has_b) return;
        uint32_t off = of_a ? aoff[i] : boff[i - NA];
        if (!(of_a ? TA : TB) && last && past(c)) off = kPastEnd;
        if (!of_a) copy_bounded(to + C::PA * C::RB + c * 1024, off, bb);
        else if (GATED && c * C::ROWS / F % FA >= FA / 2) copy_bounded(to + c * 1024, off, bu);
        else copy_bounded(to + c * 1024, off, ba);
    };
    constexpr int COPIES = NA + NB1;
    // Waits until all but the newest N stages of this wave's copies have landed, and meets.
    auto landed = [&](auto n) {
        constexpr int N = decltype(n)::value;
        if (NB > 0 || !has_b) core_meet<N * (NA + NB)>();
        else core_meet<N * (NA + 1)>();
    };
#pragma unroll
    for (int j = 0; j < FA; ++j)
#pragma unroll
        for (int m = 0; m < FB; ++m)
#pragma unroll
            for (int i = 0; i < F * F / 64; ++i) acc[j][m][i] = 0.0f;
    if (stages == 0) return;
    for (int i = 0; i < S; ++i) {
        refill(i, i);
#pragma unroll
        for (int c = 0; c < COPIES; ++c) copy(c);
    }
    landed(std::integral_constant<int, S - 1>{});
    if (!live) {                                           // it only copies
        for (int st = 0, stage = 0; st < stages; ++st) {
            landed(std::integral_constant<int, S - 2>{});
            refill(st + S, stage);
#pragma unroll
            for (int c = 0; c < COPIES; ++c) copy(c);
            stage = stage + 1 == S ? 0 : stage + 1;
        }
        core_meet<0>();
        return;
    }
    const Fragments<C, AT, TA, C::PA, FA> fa(wa * F * FA, lane);
    const Fragments<C, AT, TB, C::PB, FB> fb(wb * F * FB, lane);
    typename Fragments<C, AT, TA, C::PA, FA>::Value av[2][FA], bv[2][FB];
    auto read = [&](int set, const char* st, int kk, int i) {          // fragment i of those of step kk
        if (i < FB) bv[set][i] = fb.read(st + C::PA * C::RB, i, kk);
        else av[set][i - FB] = fa.read(st, i - FB, kk);
    };
    constexpr int READS = FA + FB, PRODUCTS = FA * FB;
#pragma unroll
    for (int i = 0; i < READS; ++i) read(0, lds, 0, i);
    static_assert(KK % 2 == 0, "two sets of fragments in turn");
    int stage = 0;
    for (int st = 0; st < stages; ++st) {
        const int next = stage + 1 == S ? 0 : stage + 1;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            // Before a stage's last step a wave has read all that it needs of it: wait for the next
            // stage, everyone's, and fill this one's place again.  Between the products, in this order,
            // the reads for the next step and the copies: the compiler's own order puts them first.
            const bool turn = kk + 1 == KK;
            if (turn) {
                landed(std::integral_constant<int, S - 2>{});
                refill(st + S, stage);
            }
            const char* from = lds + (turn ? next : stage) * C::STAGE;
#pragma unroll
            for (int i = 0; i < PRODUCTS; ++i) {
                const int j = i / FB, m = i % FB;
                acc[j][m] = multiply<F>(av[kk & 1][j], bv[kk & 1][m], acc[j][m]);
#pragma unroll
                for (int k = i * READS / PRODUCTS; k < (i + 1) * READS / PRODUCTS; ++k) read((kk + 1) & 1, from, turn ? 0 : kk + 1, k);
                if (turn)
#pragma unroll
                    for (int k = i * COPIES / PRODUCTS; k < (i + 1) * COPIES / PRODUCTS; ++k) copy(k);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        stage = next;
    }
    core_meet<0>();                                        // the copies of zeros, too, before the ring is used again
}

// Bytes that a wave's sums take on their way out.
template <class C>
constexpr int kOutPitch = C::FA * C::F + 4;               // floats of a row: rows apart by 16 bytes more than a multiple of 128
template <class C>
constexpr int kOutBytes = C::WAVES * C::F * kOutPitch<C> * 4;
template <class C>
constexpr int kCoreLds = C::LDS > kOutBytes<C> ? C::LDS : kOutBytes<C>;   // of a workgroup

// The sums leave through LDS, F rows of a wave at a time, so that a lane has eight consecutive columns
// of a row and the lanes side by side the next ones: f(row, column, v, up) for all rows below `rows`,
// both counted within the wave's part; the column is the lane's own throughout.  GATED: v is the gate,
// up the other half's.  Every wave of the workgroup comes here; one without rows does nothing.
template <class C, bool GATED, class Fn>
__device__ __forceinline__ void each_run(char* lds, const Sums<C::F> (&acc)[C::FA][C::FB], int rows, Fn f) {
    constexpr int F = C::F, PITCH = kOutPitch<C>, WIDTH = GATED ? C::FA * F / 2 : C::FA * F;
    constexpr int LANES = WIDTH / 8, STEP = 64 / LANES;    // lanes of a row, rows at a time
    __syncthreads();                                       // the ring is no longer read
    const int lane = threadIdx.x & 63;
    float* mine = reinterpret_cast<float*>(lds) + (threadIdx.x >> 6) * (F * PITCH);
    float* to = mine + (lane & (F - 1)) * PITCH + 4 * (lane / F);
    const int col = lane % LANES * 8;
#pragma unroll
    for (int m = 0; m < C::FB; ++m) {
        if (m * F >= rows) break;
        __builtin_amdgcn_wave_barrier();                   // LDS operations of one wave complete in order
#pragma unroll
        for (int j = 0; j < C::FA; ++j)
#pragma unroll
            for (int q = 0; q < F * F / 256; ++q) {
                f32x4_t v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = acc[j][m][4 * q + i];
                *reinterpret_cast<f32x4_t*>(to + j * F + 8 * q) = v;
            }
        __builtin_amdgcn_wave_barrier();
        const int end = min(F, rows - m * F);
#pragma unroll 1
        for (int r = lane / LANES; r < end; r += STEP) {
            float v[8], up[GATED ? 8 : 1];
            const float* from = mine + r * PITCH + col;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = from[i];
            if constexpr (GATED)
#pragma unroll
                for (int i = 0; i < 8; ++i) up[i] = from[WIDTH + i];
            f(m * F + r, col, v, up);
        }
    }
}

// Eight consecutive values of a row, the second four only where they lie in it.
template <int AT>
__device__ __forceinline__ void load8(const void* p, size_t i, bool whole, float v[8]) {
    if constexpr (AT == A_F32) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i);
        const f32x4_t b = whole ? *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i + 4) : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = a[j], v[j + 4] = b[j];
    } else {                                               // rows of whole eights
        const u32x4_t a = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = widen_bf16((uint16_t)(a[j >> 1] >> (16 * (j & 1))));
    }
}
template <int AT>
__device__ __forceinline__ void store8(void* p, size_t i, bool whole, const float v[8]) {
    if constexpr (AT == A_F32) {
        *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i) = f32x4_t{v[0], v[1], v[2], v[3]};
        if (whole) *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
        u32x4_t u;
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = round_bf16(v[2 * j]) | (uint32_t)round_bf16(v[2 * j + 1]) << 16;
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i) = u;
    }
}
// In the format `at`, which is fp32 or AT.
template <int AT>
__device__ __forceinline__ void store8_as(int at, void* p, size_t i, bool whole, const float v[8]) {
    if (AT == A_F32 || at == A_F32) store8<A_F32>(p, i, whole, v);
    else store8<A_BF16>(p, i, whole, v);
}

}  // namespace moe
