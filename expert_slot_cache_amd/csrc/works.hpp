// The work of a product of sorted rows: which rows of which group a workgroup takes.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

#include "product_tile.hpp"

namespace moe {

// A launch of that many workgroups, and this one's number in it.
inline dim3 blocks_of(int64_t workgroups, int waves) {
    const Grid g = grid_of(workgroups, waves);
    return dim3((unsigned)g.columns, (unsigned)g.rows);
}
__device__ __forceinline__ int workgroup() { return (int)(blockIdx.x + blockIdx.y * gridDim.x); }

// The work: the row tiles of all groups, TM rows each, times the column blocks of the matrix.
// Every wave counts the tiles for itself: a lane takes a run of groups, a prefix over the lanes
// orders the runs.  Offsets outside [0, M] or falling ones (they are device data) are
// brought into [0, M], so that no row outside the buffers is ever touched.
//
// A group's work is listed up to four tiles at a time: those tiles of one column block, then
// of the next.  Workgroups that run side by side on an XCD then read few different matrix and
// token rows, and its L2 passes most requests on only once.
struct Work {
    int group, row0, rows, nb;
};
template <int TM>
struct Works {
    static constexpr int SIDE = 4;
    const int32_t* offsets;
    int M, nblocks, total;
    int g0, g1, lo0, own, incl;        // of this lane: its groups, the first one's row, tiles, prefix of tiles
    __device__ __forceinline__ Works(const int32_t* __restrict__ off, int G, int M_, int nblocks_)
        : offsets(off), M(M_), nblocks(nblocks_) {
        if (!off) {
            total = (M + TM - 1) / TM * nblocks;
            return;
        }
        const int lane = threadIdx.x & 63;
        const int per = (G + 63) >> 6;
        g0 = min(lane * per, G);
        g1 = min(g0 + per, G);
        lo0 = bound(off[g0], 0);
        own = 0;
        int lo = lo0;
        walk(lo, [&](int, int, int n) {
            own += n;
            return false;
        });
        incl = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
        total = __builtin_amdgcn_readlane(incl, 63) * nblocks;
    }
    __device__ __forceinline__ int bound(int v, int lo) const { return min(max(v, lo), M); }
    // f(group, the row behind its last, its tiles) over this lane's groups, until f says so; `lo` follows.
    // Eight offsets are requested at a time.
    template <class F>
    __device__ __forceinline__ void walk(int& lo, F f) const {
        for (int g = g0; g < g1; g += 8) {
            int end[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) end[k] = offsets[min(g + 1 + k, g1)];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (g + k >= g1) return;
                const int hi = bound(end[k], lo);
                if (f(g + k, hi, (hi - lo + TM - 1) / TM)) return;
                lo = hi;
            }
        }
    }
    // Number i, 0 <= i < total.
    __device__ __forceinline__ Work at(int i) const {
        int group = 0, lo = 0, hi = M;
        if (offsets) {
            const int tile = i / nblocks;              // counting tiles alone: which group's
            const int who = __builtin_ctzll(__ballot(incl > tile));
            int first = incl - own;                    // the first tile of the lane's group g
            if ((int)(threadIdx.x & 63) == who) {
                lo = lo0;
                walk(lo, [&](int g, int end, int n) {
                    group = g;
                    hi = end;
                    if (tile < first + n) return true;
                    first += n;
                    return false;
                });
            }
            group = __builtin_amdgcn_readlane(group, who);
            lo = __builtin_amdgcn_readlane(lo, who);
            hi = __builtin_amdgcn_readlane(hi, who);
            i -= __builtin_amdgcn_readlane(first, who) * nblocks;
        }
        const int n = (hi - lo + TM - 1) / TM;         // the group's tiles
        const int side = i / (SIDE * nblocks) * SIDE, wide = min(SIDE, n - side);
        i -= side * nblocks;
        const int row0 = lo + (side + i % wide) * TM;
        return {group, row0, min(TM, hi - row0), i / wide};
    }
};

}  // namespace moe
