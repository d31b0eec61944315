// deal.hpp -- how the work of the grouped products is dealt to workgroups:
// whole-number arithmetic without memory, the same on the device and on the
// host, so that a host program can check it for any number of workgroups.
#pragma once

#include <stdint.h>

namespace gc {

// Sums of tiles stop here.  Offsets that fall, which no grouping has, can make
// the groups' tiles more than an int counts (512 groups of 2^27 rows each);
// the sums then stand still, and the tiles past them are left out.
constexpr int MOST_TILES = 1 << 30;
__host__ __device__ __forceinline__ int add_tiles(int a, int b)
{
    const uint32_t s = (uint32_t)a + (uint32_t)b;
    return s < (uint32_t)MOST_TILES ? (int)s : MOST_TILES;
}

// Tiles of few rows: the K quads (4 steps of 32) of all tiles form one line,
// which `pieces` workgroups take in equal pieces: piece w is [bound(w),
// bound(w+1)).  A bound that would leave less than `least` quads of a tile on
// one side moves to the tile's edge.
struct Line {
    int64_t quads;             // tiles * per_tile
    int per_tile, pieces, least;
    // `smallest` quads are worth a piece of a tile; a tile of fewer is a piece
    // itself (never cut, and as many pieces as there are tiles).
    __host__ __device__ __forceinline__ Line(int tiles, int quads_of_tile, int smallest, int most_pieces)
    {
        per_tile = quads_of_tile;
        quads = (int64_t)tiles * per_tile;
        least = smallest < per_tile ? smallest : per_tile;
        const int64_t n = quads / least;
        pieces = n < 1 ? 1 : n < most_pieces ? (int)n : most_pieces;
    }
    __host__ __device__ __forceinline__ int64_t bound(int w) const
    {
        int64_t b = quads * w / pieces;
        const int r = (int)(b % per_tile);
        if (r < least)
            b -= r;
        else if (per_tile - r < least)
            b += per_tile - r;
        return b;
    }
    // the piece that holds quad q (the last with bound <= q)
    __host__ __device__ __forceinline__ int piece_of(int64_t q) const
    {
        const int64_t guess = q * pieces / quads;
        int w = guess < pieces ? (int)guess : pieces - 1;
        while (w + 1 < pieces && bound(w + 1) <= q)
            ++w;
        while (w > 0 && bound(w) > q)
            --w;
        return w;
    }
};

// Sums over pieces of K: so many pieces that `workgroups` have about one of
// `tiles` tiles each, 1 to 16, none shorter than 8 of the `steps` K-steps, and
// the `plane` bytes of each piece's sums within `room`.
__host__ __device__ __forceinline__ int sum_pieces(int64_t workgroups, int64_t tiles, int steps, int64_t plane,
                                                   int64_t room)
{
    int64_t n = (workgroups + tiles / 2) / tiles;
    n = n < steps / 8 ? n : steps / 8;
    n = n < room / plane ? n : room / plane;
    n = n < 16 ? n : 16;
    return n < 1 ? 1 : (int)n;
}

// lora_add's second half: its kernel and how much of it a workgroup walks.
constexpr int EX_THREADS = 256, EX_WAVES = 4, EX_COLS = 64 * EX_WAVES;
constexpr int XR_COLS = 512, XR_ROWS = 128;              // columns, and most rows, of a workgroup

// Workgroups of expand_kernel that a CU holds at once (their blocks of up fill
// its LDS), for `steps` steps of 32 that cover r.
__host__ __device__ constexpr int expand_resident(int steps) { return steps == 1 ? 3 : steps <= 3 ? 2 : 1; }

struct ExpandPlan {
    bool rows;                 // expand_rows_kernel, else expand_kernel
    int steps, span, spans;    // see ExpandArgs
    int64_t grid;
};
__host__ __device__ __forceinline__ ExpandPlan expand_plan(int64_t M, int64_t N, int64_t E, int r, int64_t cus)
{
    auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
    ExpandPlan pl = {};
    pl.steps = (r + 31) / 32;
    pl.rows = (M + E - 1) / E >= 32;
    if (pl.rows) {
        // Rows per workgroup: the fewest (of 16 to 128) with which all
        // workgroups have a place at once, two per CU (one for r > 64).
        pl.spans = (int)((N + XR_COLS - 1) / XR_COLS);
        const int64_t places = cus * (pl.steps <= 2 ? 2 : 1);
        auto units = [&](int64_t rows) { return least(M, (M + rows - 1) / rows + E) * pl.spans; };
        pl.span = 16;
        while (pl.span < XR_ROWS && units(pl.span) > places)
            pl.span += 16;
        pl.grid = least(units(pl.span), places);
        return pl;
    }
    // Spans of columns: about as many workgroups as have a place at once.  (The
    // row tiles counted here are more than there will be.)
    const int64_t places = cus * expand_resident(pl.steps);
    const int64_t tiles_n = (N + EX_COLS - 1) / EX_COLS;
    const int64_t tiles_m = least(M, (M + 15) / 16 + E);
    const int64_t some = places * 5 / 4 / tiles_m, want = least(tiles_n, some < 1 ? 1 : some);
    pl.span = (int)((tiles_n + want - 1) / want);
    pl.spans = (int)((tiles_n + pl.span - 1) / pl.span);
    pl.grid = least(tiles_m * pl.spans, cus * 8);
    return pl;
}

// Tiles of many rows: unit t of queue x, in hands of `hand` units.
constexpr int TK_QUEUES = 8;
__host__ __device__ __forceinline__ int queue_unit(int x, int t, int hand)
{
    return (t / hand * TK_QUEUES + x) * hand + t % hand;
}

// The units of workgroup b of G where there are no tickets to draw: workgroups
// x, x + 8, ... share queue x in turn; where there are fewer workgroups than
// queues, each takes several queues whole.
struct Share {
    int queue, next, step, skip;
    __host__ __device__ __forceinline__ Share(int b, int G)
        : queue(b % TK_QUEUES), next(b / TK_QUEUES), step((G - b % TK_QUEUES + TK_QUEUES - 1) / TK_QUEUES),
          skip(G < TK_QUEUES ? G : TK_QUEUES)
    {
    }
    // The next unit below `units`, or -1.
    __host__ __device__ __forceinline__ int draw(int hand, int units)
    {
        for (; queue < TK_QUEUES; queue += skip, next = 0) {
            const int u = queue_unit(queue, next, hand);
            next += step;
            if (u < units)
                return u;
        }
        return -1;
    }
};

}  // namespace gc
