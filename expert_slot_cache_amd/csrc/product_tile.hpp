// The tile that a product takes, by its sizes alone (host only, no GPU).
#pragma once

#include <cstdint>
#include <type_traits>

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

// One dimension of a launch has fewer than 2^32 lanes.  More workgroups lie in rows of at most 2^22, of a
// multiple of 8, so that a workgroup's number, x + y columns, tells its XCD as x alone does; up to 7 of a
// row have nothing to do.
struct Grid {
    int64_t columns, rows;
};
inline Grid grid_of(int64_t workgroups, int waves) {
    if (workgroups * 64 * waves < (int64_t)1 << 32) return {workgroups, 1};
    const int64_t most = 1 << 22, rows = (workgroups + most - 1) / most;
    return {((workgroups + rows - 1) / rows + 7) / 8 * 8, rows};
}

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

// f of the tile of a product in the activation format, by the rows that a group has on average and by
// the workgroups that a tile gives (256 CUs), N the columns of its output.  The largest one wins whose
// tiles the groups fill and which still gives nearly every CU a workgroup.  Measured (us, bf16; both
// sides of each border; 64 groups, 2048 x 2048 where nothing else is said):
//   256 x 256 / 256 x 128   512 rows a group, 4096 x 4096: 1214 / 1280;  256 rows: 241 / 220;
//                           one group, 4096 x 4096: 4096 rows 113 / 150, 2048 rows (128 tiles) 93 / 65
//   256 x 128 / 128 x 64    256 rows a group: 220 / 262;  128: 169 / 168;  64: 142 / 130;
//                           one group, 2048 rows (128 tiles): 28.7 / 25.6
//   128 x 64 / 64 x 64      64 rows a group: 129 / 136;  32: 120 / 117;
//                           one group: 1024 rows 17.0 / 18.1, 512 rows (128 tiles) 15.6 / 12.9
//   64 x 64 / 64 x 32       32 rows a group: 117 / 112, back to the rows 113 / 120;  16: 108 / 96;
//                           one group: 512 rows 12.9 / 14.1;  333 x 1000, depth 1040 (96 tiles): 8.2 / 7.0
//   64 x 32 / 32 x 32       one group: 4096 x 4096, one row (64 tiles) 17.4 / 11.2;  64 rows (64 tiles) 8.7 / 7.8;
//                           333 x 1000 (176 tiles): 7.0 / 8.0
//   fp32, 128 x 64 / 64 x 64   8 groups of 1024 rows, 4096 x 2048: 1188 / 1074;  of 512, 2048 x 2048: 321 / 290;
//                           with the 64 x 64 of SwiGLU: 1075 / 1215 and 324 / 357
//   fp32, 64 x 64 / 64 x 32    8 groups of 512 rows: 290 / 298;  64 of 16 rows, 1024 x 1024: 91 / 64
//   fp32, 64 x 32 / 32 x 32    333 x 1000 (176 tiles): 15.1 / 13.8;  64 rows (64 tiles): 24.3 / 15.0;
//                           64 groups of 16 rows, 1024 x 1024: 64 / 58, back to the rows 58 / 64;  of 8 rows,
//                           1024 x 2048: 97 / 93, 96 / 99;  of 2 rows: 80 / 77, 74 / 79 (one rule for both ways)
// (fp32's products take sixteen times as long: larger tiles gain nothing).  SwiGLU's small
// tiles have two waves instead of four: a wave's fragments are gate and up.  Where bf16 is the
// constant std::false_type, f is asked for no tile that fp32 does not take.
template <bool SWIGLU, class Bf16, class F>
auto expert_tile(Bf16 bf16, int64_t M, int64_t G, int64_t N, bool offsets, F f) {
    constexpr bool kAny = !std::is_same<Bf16, std::false_type>::value;
    const int64_t avg = M / G;
    auto fills = [&](int PA, int PB, int64_t least) { return (N + PA - 1) / PA * most_tiles(M, G, offsets, PB) >= least; };
    constexpr int64_t kMost = 192;
    if constexpr (kAny) {
        if (bf16 && avg >= 384 && fills(256, 256, kMost)) return f(CoreTile<256, 256, 2, 4, 32, 128, 2>{});
        if (bf16 && avg >= 128 && fills(256, 128, kMost)) return f(CoreTile<256, 128, 4, 2, 32, 128, 3>{});
    }
    if constexpr (kAny || SWIGLU)
        if ((bf16 ? avg >= 48 : SWIGLU && avg >= 768) && fills(128, 64, kMost)) return f(CoreTile<128, 64, 2, 2, 32, 128, 3>{});
    if (avg >= 32 && fills(64, 64, kMost)) return f(CoreTile<64, 64, SWIGLU ? 1 : 2, 2, 32, 128, SWIGLU ? 4 : 3>{});
    if (fills(64, 32, bf16 ? 128 : 256)) return f(CoreTile<64, 32, 2, 2, 16, 128, 4>{});
    return f(CoreTile<32, 32, SWIGLU ? 1 : 2, 2, 16, 128, 6>{});
}

// f of the tile of a matrix' gradient, N x K for each group, and of the parts that a group's rows are
// split into where the tiles are too few for 256 CUs.  Measured as above, in bf16:
//   256 x 256 / 256 x 128   64 groups: 512 rows each 427 / 433, 256 rows 333 / 331, 8 rows 145 / 130;
//                           one group of 8192 rows, 4096 x 4096: 211 / 241
//   256 x 128 / 128 x 128   64 groups of 256 rows: 331 / 368;  one of 8192 rows (128 / 256 tiles): 103 / 83
//   128 x 128 / 128 x 64    one group of 2048 rows, 1024 x 1024 (64 / 128 tiles): 23 / 16
//   parts 1, 2, 4, 8, 16    one group, 64 x 2048 (16 tiles): 16384 rows 86, -, -, 20.0, 20.9;  4096 rows
//                           25, 16, 14.2, 14.2, -;  1024 rows 9.8, -, 12.9;  2048 rows, 1024 x 1024: 15.7, 18.3;
//                           64 x 2048 again: 4095 rows 25, 17, 13.1, 13.1;  3000 rows 19.5, 14.3, 12.4;
//                           2048 rows 14.7, 12.3, 12.5;  1500 rows 11.8, 11.4;  1024 rows 10.8, 12.7
// A part keeps 2048 rows, so a call of few columns between 1500 and 8191 rows takes up to 12 us more than with
// four parts.  fp32 takes the same tiles and parts, and would gain from smaller and from more of them:
//   256 x 128 / 128 x 128   64 groups: 256 rows each, 2048 x 2048: 1122 / 1088;  512 rows, 1024 x 2048: 1258 / 1138
//   128 x 128 / 128 x 64    one group of 8192 rows, 2048 x 2048: 527 / 491
//   parts 1, 2, 4, 8        64 x 2048: 16384 rows 529, 270, 142, 78;  4096 rows 135, 73, 41, 27;  2048 rows 71, 40, 24, 18
template <class F>
auto matrix_tile(int64_t M, int64_t G, int64_t N, int64_t K, F f) {
    const int64_t avg = M / G;
    auto tiles = [&](int PA, int PB) { return G * ((K + PA - 1) / PA) * ((N + PB - 1) / PB); };
    constexpr int64_t kMost = 192;
    if (avg >= 384 && tiles(256, 256) >= kMost) return f(CoreTile<256, 256, 2, 4, 32, 64, 4>{}, 1);
    if (tiles(256, 128) >= kMost) return f(CoreTile<256, 128, 4, 2, 32, 64, 3>{}, 1);
    if (tiles(128, 128) >= kMost) return f(CoreTile<128, 128, 2, 2, 32, 64, 3>{}, 1);
    const int64_t few = 256 / tiles(128, 64), rows = avg / 2048, n = few < rows ? few : rows;
    return f(CoreTile<128, 64, 2, 2, 32, 128, 3>{}, (int)(n < 1 ? 1 : n > 16 ? 16 : n));
}

}  // namespace moe
