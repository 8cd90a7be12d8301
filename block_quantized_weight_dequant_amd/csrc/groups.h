// Ragged groups of rows, as the grouped products take them: positions
// [offsets[e], offsets[e + 1]) of the sorted list belong to group e, position p
// stands for row order[p] (p itself without an order), and row r multiplies
// activation row r / share.
//
// offsets and order are device data that the host never sees, so they are
// clamped where they are read: a bound outside [previous bound, M] is pulled
// into it, and a row outside [0, M) is skipped. Groups may even overlap (bounds
// that fall): their tiles are counted without overflow, and those that pass
// the tiles of a workspace are left out. Wrong contents give wrong rows, never
// an access outside the arrays.
#pragma once

#include "device_common.h"
#include "validate.h"

namespace q4k {

struct Groups {
    const int *offsets;   // [G + 1]
    const int *order;     // [M], or null
    int G, M, share;
    int tiles;            // row tiles of the workspace (which holds no others), if there is one
};

// Rows of group e: positions lo .. hi - 1.
__device__ __forceinline__ void group_bounds(const Groups &gr, int e, int &lo, int &hi)
{
    lo = min(max(gr.offsets[e], 0), gr.M);
    hi = min(max(gr.offsets[e + 1], lo), gr.M);
}

// Row of position p, or -1 when the list names none.
__device__ __forceinline__ int group_row(const Groups &gr, int p)
{
    const int r = gr.order ? gr.order[p] : p;
    return (unsigned)r < (unsigned)gr.M ? r : -1;
}

struct GroupTile {
    int e;        // group, or -1 past the last tile
    int lo, hi;   // its positions
    int mt, nt;   // row tile and column tile within the group
    int before;   // row tiles of the groups before it
};

// Tile t of the grid that covers the groups one after another, each with
// ceil(rows / bm) x tiles_n tiles, row tiles fastest (the tiles that follow
// each other share the group's weight columns). Every wavefront finds it for
// itself: lane l takes group base + l, and a prefix sum over the lanes says
// which group holds t. 64 groups take one load, one six-step scan and one
// ballot.
__device__ __forceinline__ GroupTile find_group_tile(const Groups &gr, int t, int bm, int tiles_n)
{
    const int lane = threadIdx.x & 63;
    int run = 0;
    for (int base = 0; base < gr.G; base += 64) {
        int lo = 0, hi = 0;
        if (base + lane < gr.G)
            group_bounds(gr, base + lane, lo, hi);
        // A group of a grid has at most 2^24 tiles (M <= 2^30 rows of one column
        // tile in tiles of 64; with more columns y, and before it this card's
        // memory, ends sooner). The cut keeps the sums of overlapping groups
        // from overflowing.
        const int tiles = (int)min((long long)((hi - lo + bm - 1) / bm) * tiles_n, 1LL << 24);
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(sum, d);
            if (lane >= d)
                sum += v;
        }
        const uint64_t past = __ballot((unsigned)run + (unsigned)sum > (unsigned)t);
        if (past) {
            const int l = __builtin_ctzll(past);
            GroupTile g;
            g.e = base + l;
            g.lo = __builtin_amdgcn_readlane(lo, l);
            g.hi = __builtin_amdgcn_readlane(hi, l);
            const int first = run + __builtin_amdgcn_readlane(sum - tiles, l);
            const int tm = (g.hi - g.lo + bm - 1) / bm, in = t - first;
            g.nt = in / tm;
            g.mt = in - g.nt * tm;
            g.before = first / tiles_n;
            return g;
        }
        run = (int)min((unsigned)run + (unsigned)__builtin_amdgcn_readlane(sum, 63), 1u << 30);
    }
    return {-1, 0, 0, 0, 0, 0};
}

// Workgroups go to the eight XCDs in turn: tile index of workgroup L such that
// each XCD takes runs of eight consecutive tiles (which share weight columns
// in its L2) without the total being known.
__device__ __forceinline__ int xcd_runs(int L) { return (L & ~63) | ((L & 7) << 3) | ((L >> 3) & 7); }

// Grid that covers every tile of at most M rows in G groups, whole runs; at most
// kMaxGroupTiles of them can be told apart.
constexpr long long kMaxGroupTiles = 1LL << 30;
inline long long group_grid(long long G, long long M, long long bm, long long tiles_n)
{
    return (q4v::group_row_tiles(G, M, bm) * tiles_n + 63) / 64 * 64;
}

}  // namespace q4k
