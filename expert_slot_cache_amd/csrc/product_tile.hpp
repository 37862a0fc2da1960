// The tile that a product takes, by its sizes alone (host only, no GPU).
#pragma once

#include <cstdint>

namespace moe {

// TW matrix rows x TT rows of one group by WAVES waves, S stages in the ring.
template <int TW_, int TT_, int WAVES_, int S_>
struct Tile {
    static constexpr int TW = TW_, TT = TT_, WAVES = WAVES_, S = S_;
};

// Tiles of TM rows that M rows of G groups can have: each group's last one may be short.
inline int64_t most_tiles(int64_t M, int64_t G, bool offsets, int TM) {
    if (!offsets) return (M + TM - 1) / TM;
    return M / TM + (G < M ? G : M);
}

// f of the tile, by the rows that a group has on average and by the workgroups that a tile gives
// (256 CUs).  The largest one wins whose tiles the groups fill and which still gives nearly
// every CU a workgroup.  Measured (us; both sides of each border; N 4096 and 64 groups where
// nothing else is said; SwiGLU: both products of an expert, hidden 2048 and inter 1024):
//   256 x 128 / 128 x 64    32768 rows, K 4096: 1162 / 1462;  4096 rows, K 2048: 164 / 167
//   128 x 64 / 128 x 16     1024 rows, K 2048: 114 / 110, 512 rows: 104 / 90;
//                           32 rows of 25 groups, K 1024: 17.1 / 13.2
//   128 x 64 / 64 x 32      one group: 2048 x 2048, K 4096: 50 / 78;  1024 x 1024, K 4096: 32 / 24;
//                           333 x 1000, K 1040: 12.7 / 8.3
//   64 x 32 / 32 x 16       one group, N 2048, K 2048: 128 rows 11.0 / 10.9, 64 rows 10.5 / 9.2
//   SwiGLU 256 x 128 / 64   16384 rows: 305 / 337;  4096 rows: 145 / 154;  2048 rows: 118 / 122
//   SwiGLU 256 x 64 / 32    1024 rows: 96 / 98;  one group: 2000 rows 43 / 51, 1000 rows 36 / 30
//   SwiGLU 256 x 32 / 16    512 rows: 79 / 85;  256 rows: 72 / 70;  64 rows: 54 / 51
template <bool SWIGLU, class F>
auto product_tile(int64_t M, int64_t G, int64_t N, bool offsets, F f) {
    const int64_t avg = M / G;
    auto fills = [&](int TW, int TT, int64_t least) { return (N + TW - 1) / TW * most_tiles(M, G, offsets, TT) >= least; };
    constexpr int64_t kMost = 192;
    if (avg >= 32 && fills(256, 128, kMost)) return f(Tile<256, 128, 8, 3>{});
    if constexpr (SWIGLU) {
        if (avg >= 16 && fills(256, 64, kMost)) return f(Tile<256, 64, 8, 3>{});
        if (avg >= 6 && fills(256, 32, kMost)) return f(Tile<256, 32, 8, 4>{});
        return f(Tile<256, 16, 8, 4>{});
    } else {
        if (avg >= 16 && fills(128, 64, kMost)) return f(Tile<128, 64, 4, 3>{});
        if (avg < 16 && fills(128, 16, kMost)) return f(Tile<128, 16, 4, 4>{});
        if (fills(64, 32, 128)) return f(Tile<64, 32, 4, 5>{});
        return f(Tile<32, 16, 2, 8>{});
    }
}

// ---- products in the activation format ----
//
// A workgroup of WA x WB waves computes PA columns x PB rows of the output, in fragments of F x F
// (the columns are the instruction's A operand, so that four accumulators of a lane are consecutive
// columns).  A stage of the ring holds RB bytes of the summed dimension of each of them; S stages.
template <int PA_, int PB_, int WA_, int WB_, int F_, int RB_, int S_>
struct CoreTile {
    static constexpr int PA = PA_, PB = PB_, WA = WA_, WB = WB_, F = F_, RB = RB_, S = S_;
    static constexpr int WAVES = WA * WB, FA = PA / WA / F, FB = PB / WB / F;
    static constexpr int ROWS = 1024 / RB;                // rows of a copy (1024 bytes, 16 a lane)
    static constexpr int CA = PA * RB / 1024, CB = PB * RB / 1024;   // copies of a stage,
    static constexpr int NA = CA / WAVES, NB = CB / WAVES;           // a wave's (NB 0: the first CB waves have one)
    static constexpr int STAGE = (PA + PB) * RB, LDS = S * STAGE;
    static_assert(FA >= 1 && FB >= 1 && NA >= 1 && NA * WAVES == CA && (NB > 0 ? NB * WAVES == CB : CB < WAVES), "");
    static_assert(S >= 2 && LDS <= 160 * 1024 && (RB == 128 || (RB == 64 && F == 32)), "");
};

template <class F>
auto expert_tile(int64_t M, int64_t G, int64_t N, bool offsets, F f) {
    const int64_t avg = M / G;
    auto fills = [&](int PA, int PB, int64_t least) { return (N + PA - 1) / PA * most_tiles(M, G, offsets, PB) >= least; };
    constexpr int64_t kMost = 192;
    if (avg >= 64 && fills(256, 256, kMost)) return f(CoreTile<256, 256, 2, 4, 32, 64, 4>{});
    if (avg >= 32 && fills(128, 128, kMost)) return f(CoreTile<128, 128, 2, 2, 32, 128, 3>{});
    if (avg < 16 && fills(128, 16, kMost)) return f(CoreTile<128, 16, 4, 1, 16, 128, 4>{});
    if (avg >= 16 && fills(64, 64, 128)) return f(CoreTile<64, 64, 1, 2, 32, 128, 4>{});
    return f(CoreTile<32, 16, 1, 1, 16, 128, 8>{});
}

// f of the tile of a matrix' gradient, and the parts that its rows are split into.
template <class F>
auto matrix_tile(int64_t M, int64_t G, int64_t N, int64_t K, F f) {
    auto splits = [&](int PA, int PB) {
        const int64_t tiles = G * ((K + PA - 1) / PA) * ((N + PB - 1) / PB);
        int64_t n = (384 + tiles - 1) / tiles;
        const int64_t most = M / G / 512;
        if (n > most) n = most;
        return (int)(n > 1 ? n : 1);
    };
    if (N >= 192 && K >= 192 && G * ((K + 255) / 256) * ((N + 255) / 256) >= 192)
        return f(CoreTile<256, 256, 2, 4, 32, 64, 4>{}, 1);
    return f(CoreTile<128, 64, 2, 2, 32, 128, 4>{}, splits(128, 64));
}

}  // namespace moe
