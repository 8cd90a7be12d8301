// Which kernel an E4M3 product takes (f8.hip). Pure host C++, so that tests can
// ask for the form of a shape.
//
// A form costs its rounds of 256 workgroups times a round's time per block of K,
// in 10 ns on MI355X (beside some 4 us a call): few rows by their row groups
// with the weights streaming, tiles with the chip full. Few rows are taken
// where they cost no more than the cheapest tile, else the largest tile that
// costs no more than that, or than the weights' bytes take at 5.5 TB/s: where
// those bound the call the larger tiles stream them better (37 tokens, 2 of 8
// experts of 14336 x 4096: wide 113 us, half 119; 512 tokens, 8 of 128 of 1536 x
// 2048: wide 87, quarter 96). M x N x K by few rows and by quarter tiles, weights
// in cache: 64 x 4096 x 4096 9.2 and 9.7 us, 16 x 8192 x 8192 13.9 and 14.2, 1 x
// 14336 x 4096 16.5 and 11.7, 32 x 14336 x 4096 20.1 and 12.4 (weights from HBM:
// 24.9 and 16.1). By quarter, half and small tiles: 256 x 4096 x 4096 11.4, 15.9
// and 18.3 us, 512 x 4096 x 4096 19.7, 17.1 and 21.5, 1001 x 4096 x 4096 35.8,
// 26.6 and 21.7. By small, wide and large ones: 1001 x 4096 x 4096 21, 28 and 46
// us, 2048 x 14336 x 4096 163, 149 and 129.
#pragma once

#include <limits.h>

namespace q4v {

enum F8Form { kF8Rows, kF8Quarter, kF8Half, kF8Small, kF8Wide, kF8Large };

// Columns, rows and round of the tiles, kF8Quarter first.
struct F8Tile {
    int bn, bm, round;
};
constexpr F8Tile kF8Tiles[5] = {{64, 64, 25}, {128, 64, 40}, {128, 128, 70}, {256, 128, 110}, {256, 256, 190}};
constexpr int kF8RowsRound[5] = {0, 11, 12, 14, 19};   // by row groups

// rg: row groups of the few-row form.
struct F8Choice {
    F8Form form;
    int rg;
};

// Cost of the few-row form: `passes` times N / 16 workgroups of rg row groups.
inline long long f8_rows_cost(long long passes, int N, int rg)
{
    return (passes * (((long long)N + 15) / 16) + 255) / 256 * kF8RowsRound[rg];
}

// Over tiles_m(bm) row tiles of bm rows in all, of `groups` weight matrices;
// rows: the cost of the few-row form.
template <class TilesM>
inline F8Form f8_choose(long long groups, long long rows, int N, TilesM tiles_m)
{
    long long cost[5], least = LLONG_MAX;
    for (int i = 0; i < 5; ++i) {
        const F8Tile t = kF8Tiles[i];
        cost[i] = (tiles_m(t.bm) * (((long long)N + t.bn - 1) / t.bn) + 255) / 256 * t.round;
        least = cost[i] < least ? cost[i] : least;
    }
    if (rows <= least)
        return kF8Rows;
    const long long bytes = groups * N / 430, limit = least > bytes ? least : bytes;
    int i = 4;
    while (cost[i] > limit)
        --i;
    return (F8Form)(kF8Quarter + i);
}

inline F8Choice f8_form(int M, int N)
{
    // Row groups of the few-row form: the fewest at the least cost, so that few
    // weight rows spread over more workgroups (64 x 1024 x 4096: 7.3 us by one
    // pass of four row groups, 5.2 by four of one; 128 x 256 x 7168: 11.4 us in
    // quarter tiles, 5.0 so).
    int rg = 0;
    long long rows = LLONG_MAX;
    for (int i = 1; i <= 4; ++i) {
        const long long passes = (M + 16LL * i - 1) / (16 * i), c = f8_rows_cost(passes, N, i);
        if (passes <= 65535 && c < rows)
            rg = i, rows = c;
    }
    return {f8_choose(1, rows, N, [&](int bm) { return ((long long)M + bm - 1) / bm; }), rg};
}

// Over G groups of M rows in all. The host knows the mean size only. Few rows:
// with room for groups of twice the mean (longer ones take several passes).
// Tiles: a group ends within one, half filled on average.
inline F8Choice f8_form_grouped(int G, int M, int N)
{
    const long long hit = G < M ? G : M, mean = (M + hit - 1) / hit;
    const int rg = mean <= 8 ? 1 : mean <= 16 ? 2 : mean <= 32 ? 4 : 0;
    const long long rows = rg ? f8_rows_cost(hit, N, rg) : LLONG_MAX;
    return {f8_choose(hit, rows, N, [&](int bm) { const long long t = M / bm + hit / 2; return t > hit ? t : hit; }), rg};
}

}  // namespace q4v
