// Device helpers shared by the operators around the experts.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

#include "kernels.hpp"

namespace moe {

// A value per lane combined over the wave by four row shifts and two row broadcasts
// (DPP, no LDS); every lane gets the result, which lane 63 holds.  `old` is the
// operation's neutral value, taken where a shift has no source lane.
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce_u32(uint32_t v, Op op) {
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));   // row_shr:1
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));   // row_shr:2
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));   // row_shr:4
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));   // row_shr:8
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));   // row_bcast:15
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));   // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    return wave_reduce_u32(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_sum(float v) {
    return __uint_as_float(wave_reduce_u32(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// The lanes below this one that are set in m.
__device__ __forceinline__ int lanes_below(uint64_t m) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

__device__ __forceinline__ float widen_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
// The nearest bf16 (ties to even); a NaN stays a NaN.
__device__ __forceinline__ uint16_t round_bf16(float f) {
    const __bf16 b = (__bf16)f;
    return __builtin_bit_cast(uint16_t, b);
}
template <int AT>
__device__ __forceinline__ float load_one(const void* p, size_t i) {
    if constexpr (AT == A_F32) return static_cast<const float*>(p)[i];
    else return widen_bf16(static_cast<const uint16_t*>(p)[i]);
}
template <int AT>
__device__ __forceinline__ void store_one(void* p, size_t i, float v) {
    if constexpr (AT == A_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = round_bf16(v);
}

// Sixteen bytes at a time wherever an element may start: rows of any length and stride move in
// whole 16-byte pieces but for the last, shorter one (global accesses need no more alignment
// than their elements').  `once`: past the caches' retention.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <int AT>
struct Bits;
template <>
struct Bits<A_F32> {
    typedef uint32_t one;
    typedef uint32_t four __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Bits<A_BF16> {
    typedef uint16_t one;
    typedef uint32_t four __attribute__((ext_vector_type(4), aligned(2)));
};
template <int AT>
__device__ __forceinline__ u32x4_t load16(const void* p, bool once) {
    const auto* q = static_cast<const typename Bits<AT>::four*>(p);
    return once ? __builtin_nontemporal_load(q) : *q;
}
template <int AT, bool ONCE>
__device__ __forceinline__ void store16(void* p, u32x4_t v) {
    auto* q = static_cast<typename Bits<AT>::four*>(p);
    if constexpr (ONCE) __builtin_nontemporal_store(v, q);
    else *q = v;
}

// Sixteen bytes of a row as fp32 values.  FULL: all of them lie in the row; otherwise `left` do.
template <int AT>
struct Piece {
    static constexpr int ES = AT == A_F32 ? 4 : 2, N = 16 / ES;
    float v[N];
    template <bool FULL>
    __device__ __forceinline__ void load(const void* p, int64_t i, int left, bool once) {   // i: element index
        if constexpr (FULL) {
            const u32x4_t q = load16<AT>(static_cast<const char*>(p) + i * ES, once);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if constexpr (AT == A_F32) v[j] = __uint_as_float(q[j]);
                else v[j] = widen_bf16((uint16_t)(q[j >> 1] >> (16 * (j & 1))));
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = j < left ? load_one<AT>(p, (size_t)i + j) : 0.0f;
        }
    }
    template <bool FULL, bool ONCE>
    __device__ __forceinline__ void store(void* p, int64_t i, int left) const {
        if constexpr (FULL) {
            u32x4_t q;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (AT == A_F32) q[j] = __float_as_uint(v[j]);
                else q[j] = round_bf16(v[2 * j]) | (uint32_t)round_bf16(v[2 * j + 1]) << 16;
            }
            store16<AT, ONCE>(static_cast<char*>(p) + i * ES, q);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < left) store_one<AT>(p, (size_t)i + j, v[j]);
        }
    }
};

// The e4m3 scale of a block whose largest finite magnitude is `big`: the smallest power
// of two that brings it to 448 = 1.75 * 2^8 or less, 1 for a block of zeros.  A power of
// two divides exactly, so the only rounding is the one to e4m3 (half a step at most:
// 2^-4 of the value), and a user's own arithmetic finds the same codes.
__device__ __forceinline__ float f8_scale(float big) {
    if (big == 0.0f) return 1.0f;
    const uint32_t b = __float_as_uint(big);
    // biased exponent of the scale; a subnormal or tiny block keeps 2^-126
    int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < 1 ? 1 : e;
    return __uint_as_float((uint32_t)e << 23);
}
// 1 / scale, exactly: scale = 2^(e - 127) with 1 <= e <= 247.
__device__ __forceinline__ float f8_inverse(float scale) {
    return __uint_as_float((254u << 23) - __float_as_uint(scale));
}
// Four values, already scaled, as e4m3 codes (ties to even).  Infinities become NaN codes,
// as NaN does: e4m3 has no infinity.
__device__ __forceinline__ uint32_t f8_pack(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    return (uint32_t)r;
}

}  // namespace moe
