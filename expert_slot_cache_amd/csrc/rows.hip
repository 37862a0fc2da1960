// Tokens sorted by expert and back, and the gradient.
//
//   rows[t][k]    = place of pair (t, k) among the pairs with an id in [0, E), sorted by
//                   id and, within an id, in (t, k) order; -1 for any other id
//   offsets[e]    = rows of the experts before e; offsets[E] = rows in all
//   sorted[rows[t][k]] = x[t], or its e4m3 codes with a power-of-two scale per 128 values
//   out[t]        = resid[t] + sum_k w[t][k] ys[rows[t][k]]     (k in order, fp32)
//   d_ys[rows[t][k]] = w[t][k] d_out[t],   d_w[t][k] = <d_out[t], ys[rows[t][k]]>
//
// The sort is a counting sort without atomics on positions, so it is stable and gives the
// same places every time: a wave ranks its 64 pairs by matching ids over ballots (one per
// bit of an id), waves and workgroups take their turn through prefix sums of the counts.
// Everything else moves rows: a token is read once for all of its K copies.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "ops.hpp"
#include "ops_dev.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRounds = 4;                         // pairs per lane and pass of a workgroup
constexpr int kPass = kThreads * kRounds;          // pairs a workgroup ranks at a time
constexpr int kMaxBlocks = 256;                    // workgroups of the two-launch sort
// Pairs up to which every workgroup of the one launch sorts them all for itself.
constexpr int kOneLaunch = 2 * kPass;
constexpr int kSorters = 512;                      // workgroups of that launch: two per CU hold

// Pairs per workgroup of the two-launch sort (whole passes, at most kMaxBlocks workgroups).
__host__ __device__ inline int64_t sort_chunk(int64_t P) {
    const int64_t passes = (P + kPass - 1) / kPass;
    return (passes + kMaxBlocks - 1) / kMaxBlocks * kPass;
}

// Dynamic LDS: base[E] int32, then cnt[kWaves][E] uint16.
size_t sort_lds(int E) { return (size_t)E * 4 + (size_t)kWaves * E * 2; }

// Rows that are read once are loaded past the caches' retention.  Whether they are also stored that
// way goes by the call and the kernel that reads them next, timed together (us, cached / past):
//  sorted copies, then their combine, of 2048 bf16: 8 a token 64 MiB 39 / 45, 109 MiB 63 / 67, 128 MiB
//    82 / 77, 256 MiB 153 / 142; 1 a token 96 MiB 104 / 107, 128 MiB 144 / 136: past from 120 MiB on.
//    (The sort alone: past from 16 MiB on.)
//  sorted e4m3 rows of 4096, then their product with 512 columns: 8 a token 4 MiB 40.2 / 39.4, 24 MiB
//    75.3 / 74.4, 128 MiB 215 / 216; 1 a token 16 MiB 63.0 / 64.2; alone 8 a token 16.8 / 14.7 at 24
//    MiB, 44 / 36 at 128: always past.
//  the sum of rows of 2048, then an addition to it: 8 a token, rows of 128 MiB 51.2 / 51.7; 2 a token,
//    of 64 MiB 44 / 46; 1 a token 68 / 72; alone 44.3 / 42.3, 32.6 / 31.8, 47.5 / 45.9: never past.
//  its gradient, then the rows' combine: 8 a token 75 MiB 53.7 / 55.8, 187 MiB 130 / 138, 256 MiB
//    190.5 / 190, 512 MiB 356 / 344: past what the last cache holds, 256 MiB.
constexpr int64_t kCopiesPast = (int64_t)120 << 20;
constexpr int64_t kGradientPast = (int64_t)256 << 20;

// Exclusive prefix sums of v[0 .. E) in place, by the whole workgroup; returns the sum.
__device__ int block_scan(int32_t* v, int E) {
    __shared__ int wave_total[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (E + kThreads - 1) / kThreads;
    const int e0 = min(tid * per, E), e1 = min(e0 + per, E);
    int own = 0;
    for (int e = e0; e < e1; ++e) own += v[e];
    int incl = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    int at = incl - own, all = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        at += i < wave ? wave_total[i] : 0;
        all += wave_total[i];
    }
    for (int e = e0; e < e1; ++e) {
        const int c = v[e];
        v[e] = at;
        at += c;
    }
    __syncthreads();
    return all;
}

// One pass of ranking: the workgroup's pairs p0 .. p0 + kPass, wave by wave, 64 at a time.
// id[r] (-1: not a pair of any expert), then rank[r] (the pair's place among this wave's of
// its expert so far); cnt[wave][e] ends as the wave's count.  No barrier inside.
__device__ __forceinline__ void load_pass(const int32_t* __restrict__ ids, int64_t p0, int64_t end, int E, int id[kRounds]) {
    const int64_t first = p0 + (int64_t)(threadIdx.x >> 6) * (kRounds * 64) + (threadIdx.x & 63);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int64_t p = first + r * 64;
        const int v = p < end ? ids[p] : -1;
        id[r] = (unsigned)v < (unsigned)E ? v : -1;
    }
}
__device__ __forceinline__ void rank_pass(int E, int bits, uint16_t* cnt, const int id[kRounds], int rank[kRounds]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint16_t* mine = cnt + wave * E;
    for (int e = lane; e < E; e += 64) mine[e] = 0;
    __builtin_amdgcn_wave_barrier();   // LDS operations of one wave complete in order
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        uint64_t same = __ballot(id[r] >= 0);
        rank[r] = 0;
        if (same == 0) continue;                           // few pairs: most rounds have none
        for (int b = 0; b < bits; ++b) {
            const bool one = (id[r] >> b) & 1;
            const uint64_t m = __ballot(one);
            same &= one ? m : ~m;
        }
        if (id[r] >= 0) {
            const int before = lanes_below(same);
            const int sofar = mine[id[r]];
            rank[r] = sofar + before;
            __builtin_amdgcn_wave_barrier();
            if (before == 0) mine[id[r]] = (uint16_t)(sofar + __popcll(same));
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Counts of the pairs p0 .. end by expert in h[E] (zeroed here; a barrier follows), `id` holding
// the first pass of them already.
__device__ __forceinline__ void count_pairs(const int32_t* __restrict__ ids, int64_t p0, int64_t end, int E, int32_t* h,
                                            const int id[kRounds]) {
    for (int e = threadIdx.x; e < E; e += kThreads) h[e] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        if (id[r] >= 0) atomicAdd(&h[id[r]], 1);           // counts: the order does not matter
    for (int64_t p = p0 + kPass + threadIdx.x; p < end; p += kThreads) {
        const int v = ids[p];
        if ((unsigned)v < (unsigned)E) atomicAdd(&h[v], 1);
    }
    __syncthreads();
}
// The pairs p0 .. end in their order: put(p, the pair's row), base[e] being the next row of e and
// `id` the first pass of them.
template <class F>
__device__ __forceinline__ void place_pairs(const int32_t* __restrict__ ids, int64_t p0, int64_t end, int E, int bits,
                                            int32_t* base, uint16_t* cnt, int id[kRounds], F put) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t q0 = p0; q0 < end; q0 += kPass) {
        int rank[kRounds];
        if (q0 > p0) load_pass(ids, q0, end, E, id);
        rank_pass(E, bits, cnt, id, rank);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int64_t p = q0 + wave * (kRounds * 64) + r * 64 + lane;
            if (p >= end) continue;
            int v = -1;
            if (id[r] >= 0) {
                v = base[id[r]] + rank[r];
                for (int i = 0; i < wave; ++i) v += cnt[i * E + id[r]];
            }
            put(p, v);
        }
        __syncthreads();
        if (q0 + kPass >= end) break;
        for (int e = threadIdx.x; e < E; e += kThreads) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) sum += cnt[i * E + e];
            base[e] += sum;
        }
        __syncthreads();
    }
}

// ---- a token's row to its K places -----------------------------------------------------
// bx lanes side by side, of all the workgroups that share the row, walk it from piece c on;
// rows: the token's K places.
template <int AT, bool STREAM>
__device__ __forceinline__ void copy_row(const void* x, int64_t row, int H, const int32_t* rows, int K, void* out, int c,
                                         int bx) {
    using V = Piece<AT>;
    typedef typename Bits<AT>::one One;
    const One* src = static_cast<const One*>(x) + row;
    One* dst = static_cast<One*>(out);
    for (; c * V::N < H; c += bx) {
        const int e = c * V::N;
        if (e + V::N <= H) {
            const u32x4_t q = load16<AT>(src + e, true);
            for (int k = 0; k < K; ++k)
                if (rows[k] >= 0) store16<AT, STREAM>(dst + ((int64_t)rows[k] * H + e), q);
        } else {
            for (int i = e; i < H; ++i)
                for (int k = 0; k < K; ++k)
                    if (rows[k] >= 0) dst[(int64_t)rows[k] * H + i] = src[i];
        }
    }
}

// e4m3: a lane takes 16 values, eight lanes side by side a block of 128 (bx is a multiple
// of 8, H of 16; a last block may be shorter).
template <int AT, bool STREAM>
__device__ __forceinline__ void round_row(const void* x, int64_t row, int H, const int32_t* rows, int K, uint8_t* out,
                                          float* scales, int c, int bx) {
    using V = Piece<AT>;
    const int n = H / 16, nb = (H + kBlock - 1) / kBlock;
    const int steps = (n - c / 8 * 8 + bx - 1) / bx;   // eight lanes take part in each step's exchange
    for (int s = 0; s < steps; ++s, c += bx) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        if (c < n) {
#pragma unroll
            for (int i = 0; i < 16 / V::N; ++i) {
                V p;
                p.template load<true>(x, row + (int64_t)c * 16 + i * V::N, V::N, true);
#pragma unroll
                for (int j = 0; j < V::N; ++j) v[i * V::N + j] = p.v[j];
            }
        }
        float big = 0.0f;   // of the finite values: a NaN or an infinity poisons its own code alone
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float a = fabsf(v[i]);
            if (a < __builtin_inff()) big = fmaxf(big, a);
            else v[i] = __builtin_nanf("");
        }
        big = fmaxf(big, __shfl_xor(big, 1));
        big = fmaxf(big, __shfl_xor(big, 2));
        big = fmaxf(big, __shfl_xor(big, 4));
        if (c >= n) continue;
        const float scale = f8_scale(big), inv = f8_inverse(scale);
        u32x4_t q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = f8_pack(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
        for (int k = 0; k < K; ++k) {
            const int64_t r = rows[k];
            if (r < 0) continue;
            store16<A_F32, STREAM>(out + r * H + (int64_t)c * 16, q);   // on 16 bytes
            if ((c & 7) == 0) scales[r * nb + (c >> 3)] = scale;
        }
    }
}

struct Spread {
    const void* x;
    int64_t stride;
    int T, K, H, bx;
    void* out;
    float* scales;
};

template <int AT, bool F8, bool STREAM>
__device__ __forceinline__ void spread_token(const Spread& a, int64_t t, const int32_t* rows, int c) {
    if constexpr (F8) round_row<AT, STREAM>(a.x, t * a.stride, a.H, rows, a.K, static_cast<uint8_t*>(a.out), a.scales, c, a.bx * gridDim.y);
    else copy_row<AT, STREAM>(a.x, t * a.stride, a.H, rows, a.K, a.out, c, a.bx * gridDim.y);
}

// At most kOneLaunch pairs: every workgroup sorts them all (a few microseconds, less than two
// more launches and the waits for them), the first writes rows and offsets, and each spreads its
// own tokens from the places it found.  No more than kSorters workgroups, so that all run at
// once and none sorts after another has.  64 experts, against 2048 pairs and a token more in
// three launches (us): 256 x 8 rows of 4096 to e4m3 11.3 / 12.7, 2048 x 1 of 1024 10.4 / 11.0, of
// 4096 15.6 / 14.3; 256 x 8 of 16384, fp32, 33.9 / 34.9; 4096 experts, of 4096: 20.7 / 27.8.
template <int AT, bool F8, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_sort_one(Spread a, const int32_t* __restrict__ ids, int E, int bits,
        int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
    extern __shared__ int32_t lds[];
    __shared__ int32_t place[kOneLaunch];
    int32_t* base = lds;
    const int P = a.T * a.K;
    const bool writes = blockIdx.x == 0 && blockIdx.y == 0;
    int id[kRounds];
    load_pass(ids, 0, P, E, id);
    count_pairs(ids, 0, P, E, base, id);
    const int all = block_scan(base, E);
    if (writes) {
        for (int e = threadIdx.x; e < E; e += kThreads) offsets[e] = base[e];
        if (threadIdx.x == 0) offsets[E] = all;
    }
    place_pairs(ids, 0, P, E, bits, base, reinterpret_cast<uint16_t*>(lds + E), id, [&](int64_t p, int v) {
        place[p] = v;
        if (writes) rows[p] = v;
    });
    if (!a.x) return;
    const int by = kThreads / a.bx;
    for (int t = blockIdx.x * by + threadIdx.x / a.bx; t < a.T; t += gridDim.x * by)
        spread_token<AT, F8, STREAM>(a, t, place + t * a.K, blockIdx.y * a.bx + (threadIdx.x & (a.bx - 1)));
}

// More pairs: counts per workgroup, then places, then the rows (a launch each).  Every workgroup
// of the second sums the counts of all (at most 256 x E of them): few where E is, but with 4096
// experts that is most of the time.  Places alone, us, at 64 / 512 / 4096 experts: 2^15 pairs 8.4 /
// 10.8 / 31.8, 2^18 16 / 27 / 150, 2^22 70 / 88 / 253, 2^24 256 / 314 / 610.
__global__ __launch_bounds__(kThreads) void k_sort_count(const int32_t* __restrict__ ids, int64_t P, int64_t chunk, int E,
        int32_t* __restrict__ counts) {
    extern __shared__ int32_t lds[];
    const int64_t p0 = blockIdx.x * chunk;
    const int64_t end = p0 + chunk < P ? p0 + chunk : P;
    int id[kRounds];
    load_pass(ids, p0, end, E, id);
    count_pairs(ids, p0, end, E, lds, id);
    for (int e = threadIdx.x; e < E; e += kThreads) counts[(int64_t)blockIdx.x * E + e] = lds[e];
}

__global__ __launch_bounds__(kThreads) void k_sort_place(const int32_t* __restrict__ ids, int64_t P, int64_t chunk, int E,
        int bits, const int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
    extern __shared__ int32_t lds[];
    int32_t* base = lds;
    uint16_t* cnt = reinterpret_cast<uint16_t*>(lds + E);
    int32_t* before = reinterpret_cast<int32_t*>(cnt);   // [E], until cnt is used
    const int nb = gridDim.x, b = blockIdx.x;
    const int64_t p0 = b * chunk, end = p0 + chunk < P ? p0 + chunk : P;
    int id[kRounds];
    load_pass(ids, p0, end, E, id);
    for (int e = threadIdx.x; e < E; e += kThreads) {   // of all workgroups, and of those before this one
        int sum = 0, mine = 0;
        for (int i = 0; i < nb; i += 16) {
            int c[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) c[k] = counts[(int64_t)min(i + k, nb - 1) * E + e];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                sum += i + k < nb ? c[k] : 0;
                mine += i + k < b ? c[k] : 0;
            }
        }
        base[e] = sum;
        before[e] = mine;
    }
    __syncthreads();
    const int all = block_scan(base, E);
    for (int e = threadIdx.x; e < E; e += kThreads) {
        const int first = base[e];
        if (b == 0) offsets[e] = first;
        base[e] = first + before[e];                    // this workgroup's first row of e
    }
    if (b == 0 && threadIdx.x == 0) offsets[E] = all;
    __syncthreads();
    place_pairs(ids, p0, end, E, bits, base, cnt, id, [&](int64_t p, int v) { rows[p] = v; });
}

template <int AT, bool F8, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_spread(Spread a, const int32_t* __restrict__ rows) {
    const int by = kThreads / a.bx;
    int64_t t = (int64_t)blockIdx.x * by + threadIdx.x / a.bx;
    if (a.bx >= 64) t = __builtin_amdgcn_readfirstlane((int)t);   // one token per wave: its places are scalars
    if (t < a.T) spread_token<AT, F8, STREAM>(a, t, rows + t * a.K, blockIdx.y * a.bx + (threadIdx.x & (a.bx - 1)));
}

// ---- back: the weighted sum -------------------------------------------------------------
template <int AT>
__global__ __launch_bounds__(kThreads) void k_combine_rows(const void* __restrict__ ys, const int32_t* __restrict__ rows,
        const float* __restrict__ w, const void* __restrict__ resid, int T, int K, int H, int bx,
        void* __restrict__ out) {
    using V = Piece<AT>;
    constexpr int KU = 8;   // rows in flight per lane
    const int by = kThreads / bx;
    int t = blockIdx.x * by + threadIdx.x / bx;
    if (bx >= 64) t = __builtin_amdgcn_readfirstlane(t);
    const int c = (blockIdx.y * bx + (threadIdx.x & (bx - 1))) * V::N;
    if (t >= T || c >= H) return;
    const unsigned P = (unsigned)T * (unsigned)K;
    auto piece = [&](auto whole) {
        constexpr bool FULL = decltype(whole)::value;
        const int left = H - c;
        V acc;
#pragma unroll
        for (int i = 0; i < V::N; ++i) acc.v[i] = 0.0f;
        for (int k0 = 0; k0 < K; k0 += KU) {
            V y[KU];
            bool on[KU];
            float wk[KU];
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                const int k = k0 + j;
                const int r = k < K ? rows[(int64_t)t * K + k] : -1;
                on[j] = (unsigned)r < P;   // any other place: a pair that went to no expert
                wk[j] = on[j] && w ? w[(int64_t)t * K + k] : 1.0f;
                if (on[j]) y[j].template load<FULL>(ys, (int64_t)r * H + c, left, true);
            }
#pragma unroll
            for (int j = 0; j < KU; ++j)
                if (on[j])
#pragma unroll
                    for (int i = 0; i < V::N; ++i) acc.v[i] += wk[j] * y[j].v[i];
        }
        if (resid) {
            V r;
            r.template load<FULL>(resid, (int64_t)t * H + c, left, true);
#pragma unroll
            for (int i = 0; i < V::N; ++i) acc.v[i] += r.v[i];
        }
        acc.template store<FULL, false>(out, (int64_t)t * H + c, left);
    };
    if (c + V::N <= H) piece(std::true_type{});
    else piece(std::false_type{});
}

// W waves take a token and up to eight of its pairs (grid.y walks the groups of pairs): d_out[t]
// is read once for them, each pair's dot product stays in a register per lane and is summed
// over the lanes, then the waves, at the end, in a fixed order.  How many waves: combine_backward.
template <int AT, bool STREAM, int W>
__global__ __launch_bounds__(W > kWaves ? 64 * W : kThreads) void k_combine_rows_backward(const void* __restrict__ dout,
        const void* __restrict__ ys, const int32_t* __restrict__ rows, const float* __restrict__ w, int T, int K, int per,
        int H, void* __restrict__ dys, float* __restrict__ dw) {
    using V = Piece<AT>;
    constexpr int KU = 8;
    constexpr int TOKENS = W > kWaves ? 1 : kWaves / W;   // of a workgroup
    __shared__ float sums[W > 1 ? W : 1][KU];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x * TOKENS + wave / W, part = wave % W;
    if (t >= T) return;                                 // W > 1: one token a workgroup, which has one
    const int k0 = blockIdx.y * per, n = min(per, K - k0);
    const unsigned P = (unsigned)T * (unsigned)K;
    int64_t at[KU];
    float wk[KU], dot[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
        const int64_t p = (int64_t)t * K + k0 + j;
        const int r = j < n ? rows[p] : -1;
        at[j] = (unsigned)r < P ? (int64_t)r * H : -1;
        wk[j] = at[j] >= 0 ? w[p] : 0.0f;
        dot[j] = 0.0f;
    }
    for (int c = (part * 64 + lane) * V::N; c < H; c += W * 64 * V::N) {
        auto piece = [&](auto whole) {
            constexpr bool FULL = decltype(whole)::value;
            const int left = H - c;
            V d, y[KU];
            d.template load<FULL>(dout, (int64_t)t * H + c, left, false);
#pragma unroll
            for (int j = 0; j < KU; ++j)
                if (at[j] >= 0) y[j].template load<FULL>(ys, at[j] + c, left, true);
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                if (at[j] < 0) continue;
                V o;
#pragma unroll
                for (int i = 0; i < V::N; ++i) {
                    dot[j] += y[j].v[i] * d.v[i];
                    o.v[i] = wk[j] * d.v[i];
                }
                o.template store<FULL, STREAM>(dys, at[j] + c, left);
            }
        };
        if (c + V::N <= H) piece(std::true_type{});
        else piece(std::false_type{});
    }
#pragma unroll
    for (int j = 0; j < KU; ++j) {
        if (j >= n) break;
        const float sum = wave_sum(dot[j]);
        if (lane != 0) continue;
        if constexpr (W == 1) dw[(int64_t)t * K + k0 + j] = sum;
        else sums[part][j] = sum;
    }
    if constexpr (W > 1) {
        __syncthreads();
        if ((int)threadIdx.x < n) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) sum += sums[i][threadIdx.x];
            dw[(int64_t)t * K + k0 + threadIdx.x] = sum;
        }
    }
}

int bits_of(int E) {
    int b = 0;
    while ((1 << b) < E) ++b;
    return b;
}
// Lanes that share a row of n pieces: a power of two in [lo, 256].
int lanes_for(int n, int lo) {
    int bx = lo;
    while (bx < n && bx < kThreads) bx *= 2;
    return bx;
}

template <int AT, bool F8, bool STREAM>
hipError_t sort(const Spread& a0, const int32_t* ids, int E, int32_t* offsets, int32_t* rows, int32_t* counts,
                hipStream_t s) {
    Spread a = a0;
    const int pieces = F8 ? a.H / 16 : (a.H + Piece<AT>::N - 1) / Piece<AT>::N;
    a.bx = lanes_for(pieces, 8);
    const int64_t P = (int64_t)a.T * a.K;
    const int bits = bits_of(E);
    const int by = kThreads / a.bx;
    const int tokens_grid = (a.T + by - 1) / by;
    // few tokens: a row's pieces go over several workgroups
    const int columns = tokens_grid < 512 ? (pieces + a.bx - 1) / a.bx : 1;
    if (P <= kOneLaunch) {
        const int across = std::min(columns, std::max(kSorters / std::max(tokens_grid, 1), 1));
        const dim3 grid = a.x ? dim3(std::min(tokens_grid, kSorters), across) : dim3(1);
        hipLaunchKernelGGL((k_sort_one<AT, F8, STREAM>), grid, dim3(kThreads), sort_lds(E), s, a, ids, E, bits, offsets, rows);
        return hipGetLastError();
    }
    const dim3 grid(tokens_grid, columns);
    const int64_t chunk = sort_chunk(P);
    const int nb = (int)((P + chunk - 1) / chunk);
    hipLaunchKernelGGL(k_sort_count, dim3(nb), dim3(kThreads), (size_t)E * 4, s, ids, P, chunk, E, counts);
    hipLaunchKernelGGL(k_sort_place, dim3(nb), dim3(kThreads), sort_lds(E), s, ids, P, chunk, E, bits, counts, offsets,
                       rows);
    if (!a.x) return hipGetLastError();
    hipLaunchKernelGGL((k_spread<AT, F8, STREAM>), grid, dim3(kThreads), 0, s, a, rows);
    return hipGetLastError();
}

template <int AT>
hipError_t combine(const void* ys, const int32_t* rows, const float* w, const void* resid, int T, int K, int H,
                   void* out, hipStream_t s) {
    const int n = (H + Piece<AT>::N - 1) / Piece<AT>::N;
    const int bx = lanes_for(n, 8), by = kThreads / bx;
    hipLaunchKernelGGL((k_combine_rows<AT>), dim3((T + by - 1) / by, (n + bx - 1) / bx), dim3(kThreads), 0, s, ys,
                       rows, w, resid, T, K, H, bx, out);
    return hipGetLastError();
}

template <int AT, bool STREAM>
hipError_t combine_backward(const void* dout, const void* ys, const int32_t* rows, const float* w, int T, int K, int H,
                            void* dys, float* dw, hipStream_t s) {
    const int groups = (K + 7) / 8, per = (K + groups - 1) / groups;
    auto run = [&](auto waves) {
        constexpr int W = decltype(waves)::value, tokens = W > kWaves ? 1 : kWaves / W;
        hipLaunchKernelGGL((k_combine_rows_backward<AT, STREAM, W>), dim3((T + tokens - 1) / tokens, groups),
                           dim3(W > kWaves ? 64 * W : kThreads), 0, s, dout, ys, rows, w, T, K, per, H, dys, dw);
        return hipGetLastError();
    };
    // Several waves walk a row where one a token would leave CUs without one, or where a token's rows
    // are long in all and fill most of the steps that four waves take together.  bf16, us with 1 / 4
    // / 16: 250 x 8 x 4096 43 / 17 / 13, 500 x 8 x 4096 45 / 20 / 22; 1000 x 8 x 1024 17.2 / 13.0,
    // 1500 x 8 x 1024 19.6 / 21.8; 6000 x 8 x 2048 (a whole step) 110 / 90, 6000 x 8 x 2560 (1.25 of
    // two) 124 / 128, 6000 x 8 x 3000 (1.46 of two) 160 / 139; 10000 x 1 x 4096 (512 pieces) 53.7 / 57.3,
    // 10000 x 4 x 2048 (1024) 82.3 / 81.3, 10000 x 4 x 4096 (2048) 166 / 140.
    const int64_t waves = (int64_t)T * groups;
    const int pieces = (H + Piece<AT>::N - 1) / Piece<AT>::N, steps = (pieces + 255) / 256;
    if (waves < 256 && pieces > 256) return run(std::integral_constant<int, 16>{});
    if (pieces > 64 && (waves < 1280 || (3 * pieces >= 2 * 256 * steps && per * pieces > 1024)))
        return run(std::integral_constant<int, 4>{});
    return run(std::integral_constant<int, 1>{});
}

}  // namespace

size_t sort_workspace(int T, int K, int E) {
    const int64_t P = (int64_t)T * K;
    if (P <= kOneLaunch) return 0;
    const int64_t chunk = sort_chunk(P);
    return (size_t)((P + chunk - 1) / chunk) * (size_t)E * sizeof(int32_t);
}

hipError_t launch_sort(int atype, const void* x, int64_t stride, const int32_t* ids, int T, int K, int E, int H,
                       bool f8, void* sorted, float* scales, int32_t* offsets, int32_t* rows, void* workspace,
                       hipStream_t s) {
    const Spread a{x, stride, T, K, H, 0, sorted, scales};
    int32_t* counts = static_cast<int32_t*>(workspace);
    auto run = [&](auto at) {
        constexpr int AT = decltype(at)::value;
        if (f8) return sort<AT, true, true>(a, ids, E, offsets, rows, counts, s);
        const bool stream = (int64_t)T * K * H * (AT == A_F32 ? 4 : 2) > kCopiesPast;
        return stream ? sort<AT, false, true>(a, ids, E, offsets, rows, counts, s)
                      : sort<AT, false, false>(a, ids, E, offsets, rows, counts, s);
    };
    return atype == A_F32 ? run(std::integral_constant<int, A_F32>{}) : run(std::integral_constant<int, A_BF16>{});
}

hipError_t launch_combine(int atype, const void* ys, const int32_t* rows, const float* w, const void* resid, int T,
                          int K, int H, void* out, hipStream_t s) {
    if (atype == A_F32) return combine<A_F32>(ys, rows, w, resid, T, K, H, out, s);
    return combine<A_BF16>(ys, rows, w, resid, T, K, H, out, s);
}

hipError_t launch_combine_backward(int atype, const void* dout, const void* ys, const int32_t* rows, const float* w,
                                   int T, int K, int H, void* dys, float* dw, hipStream_t s) {
    const bool stream = (int64_t)T * K * H * (atype == A_F32 ? 4 : 2) > kGradientPast;
    if (atype == A_F32)
        return stream ? combine_backward<A_F32, true>(dout, ys, rows, w, T, K, H, dys, dw, s)
                      : combine_backward<A_F32, false>(dout, ys, rows, w, T, K, H, dys, dw, s);
    return stream ? combine_backward<A_BF16, true>(dout, ys, rows, w, T, K, H, dys, dw, s)
                  : combine_backward<A_BF16, false>(dout, ys, rows, w, T, K, H, dys, dw, s);
}

}  // namespace moe
