// grouped.hip -- host side of the C ABI declared in include/gemm_coll_grouped.h:
// argument validation, choice of the kernel instance, launches.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

#include "combine.hpp"
#include "gemm_coll_grouped.h"
#include "grouped.hpp"
#include "grouped_tile.hpp"
#include "host.hpp"
#include "lora.hpp"
#include "route.hpp"

static_assert(GC_GROUPS_MAX == gc::RT_GROUPS && GC_GROUPS_MAX == gc::GR_GROUPS, "groups");
static_assert(GC_TOPK_MAX == gc::RT_TOP, "k");
static_assert(GC_SCORE_SOFTMAX == gc::SCORE_SOFTMAX && GC_SCORE_SIGMOID == gc::SCORE_SIGMOID, "scores");

namespace {

using namespace gc::host;

// Lanes per token and experts per lane: rows of 16 lanes up to 256 experts,
// whole waves beyond.
int route_lanes(int E) { return E <= 256 ? 16 : 64; }
int route_values(int E)
{
    int v = 1;
    while (v * route_lanes(E) < E)
        v *= 2;
    return v;
}

template <bool BF16, bool ONE>
void launch_route(const gc::RouteArgs &a, int blocks, hipStream_t st)
{
    const dim3 g(blocks), b(gc::RT_THREADS);
    if (route_lanes(a.E) == 64) {
        if (route_values(a.E) == 8)
            hipLaunchKernelGGL((gc::route_kernel<64, 8, BF16, ONE>), g, b, 0, st, a);
        else
            hipLaunchKernelGGL((gc::route_kernel<64, 16, BF16, ONE>), g, b, 0, st, a);
        return;
    }
    switch (route_values(a.E)) {
    case 1: hipLaunchKernelGGL((gc::route_kernel<16, 1, BF16, ONE>), g, b, 0, st, a); break;
    case 2: hipLaunchKernelGGL((gc::route_kernel<16, 2, BF16, ONE>), g, b, 0, st, a); break;
    case 4: hipLaunchKernelGGL((gc::route_kernel<16, 4, BF16, ONE>), g, b, 0, st, a); break;
    case 8: hipLaunchKernelGGL((gc::route_kernel<16, 8, BF16, ONE>), g, b, 0, st, a); break;
    default: hipLaunchKernelGGL((gc::route_kernel<16, 16, BF16, ONE>), g, b, 0, st, a); break;
    }
}

// Routing (with logits) and grouping of a.T * a.k items.
int route_and_group(gc::RouteArgs &a, bool route, bool bf16, void *workspace, uint64_t bytes,
                    hipStream_t st)
{
    // One workgroup for everything: up to two tokens for each row of lanes, and
    // more where there is no workspace for more workgroups.
    const int64_t items = (int64_t)a.T * a.k;
    const int at_once = gc::RT_THREADS / route_lanes(a.E);
    if (items <= gc::ROUTE_ONE_ITEMS && (!route || a.T <= 2 * at_once || (a.offsets && !workspace))) {
        if (!route)
            hipLaunchKernelGGL((gc::route_kernel<16, 0, false, true>), dim3(1), dim3(gc::RT_THREADS), 0, st, a);
        else if (bf16)
            launch_route<true, true>(a, 1, st);
        else
            launch_route<false, true>(a, 1, st);
        return launched();
    }
    // Blocks of consecutive tokens: as many as a workgroup routes at a time, or
    // about 512 items to group; at most RT_BLOCKS (more only where a block
    // would pass RT_ITEMS).
    const int64_t few = route ? std::min(at_once, std::max(1, 512 / a.k)) : std::max(1, 512 / a.k);
    const int64_t per = std::min<int64_t>(
        gc::RT_ITEMS / a.k, std::max<int64_t>(few, (a.T + gc::RT_BLOCKS - 1) / gc::RT_BLOCKS));
    const int blocks = (int)((a.T + per - 1) / per);
    a.block_tokens = (int)per;
    a.cstride = (a.E + 7) / 8 * 8;
    if (a.offsets) {
        if (!good16(workspace) || bytes < (uint64_t)(kCountBytes + (int64_t)blocks * a.cstride * 2))
            return GC_EINVAL;
        a.counts = (uint16_t *)((char *)workspace + kCountBytes);
    }
    if (!route)
        hipLaunchKernelGGL((gc::route_kernel<16, 0, false, false>), dim3(blocks), dim3(gc::RT_THREADS), 0, st, a);
    else if (bf16)
        launch_route<true, false>(a, blocks, st);
    else
        launch_route<false, false>(a, blocks, st);
    if (a.offsets)
        hipLaunchKernelGGL(gc::place_kernel, dim3(blocks), dim3(gc::RT_THREADS), 0, st, a);
    return launched();
}

template <int NB, int RB, int D, int EPI>
void launch_stream(gc::GroupedArgs &a, int cus, hipStream_t st)
{
    const int64_t f = EPI == gc::EPI_GLU ? a.N / 2 : a.N, bn = EPI == gc::EPI_GLU ? 8 * NB : 16 * NB;
    a.tiles_n = (int)((f + bn - 1) / bn);
    const int grid = workers(cus);
    a.part_slots = 2 * grid;
    // A piece of fewer than 4 quads (16 K-steps) costs more to hand over than
    // it saves; without a workspace no tile is cut at all.
    const int kt = (a.K + gc::BK - 1) / gc::BK;
    a.min_quads = a.part ? 4 : std::max(1, (kt + 3) / 4);
    hipLaunchKernelGGL((gc::stream_kernel<NB, RB, D, EPI>), dim3(grid), dim3(gc::ST_THREADS), 0, st, a);
}

template <int EPI>
void launch_stream_rows(gc::GroupedArgs &a, int blocks, int cus, hipStream_t st)
{
    switch (blocks) {
    case 1: launch_stream<8, 1, 4, EPI>(a, cus, st); break;
    case 2: launch_stream<8, 2, 3, EPI>(a, cus, st); break;
    default: launch_stream<8, 4, 3, EPI>(a, cus, st); break;
    }
}

// Middle sums of the adapters: tiles of 16, 32 or 64 rows, K cut into pieces
// (sum_pieces).  (M = 4096, K = 7168, r = 64, 8 adapters: 4 pieces 20 us, 3 pieces
// 24, 7 pieces with smaller rings 27.)
template <int NB, int RB, int D>
void launch_sums_rows(gc::GroupedArgs &a, int cus, hipStream_t st)
{
    const int bm = 16 * RB, kt = (a.K + gc::BK - 1) / gc::BK;
    const int64_t most = std::min<int64_t>(a.S, (int64_t)(a.S + bm - 1) / bm + a.E);
    const int64_t about = std::min<int64_t>(a.S, (int64_t)a.S / bm + (RB == 4 ? (a.E + 1) / 2 : a.E));
    a.tiles_n = 1;
    a.splits = gc::sum_pieces(cus, about, kt, (int64_t)a.S * a.N * 4, kSumBytes);
    const int grid = (int)std::min<int64_t>(most * a.splits, 4 * cus);
    hipLaunchKernelGGL((gc::stream_kernel<NB, RB, D, gc::EPI_SUMS>), dim3(grid), dim3(gc::ST_THREADS), 0, st, a);
}

template <int NB>
void launch_sums(gc::GroupedArgs &a, int64_t rows_per_group, int cus, hipStream_t st)
{
    if (rows_per_group <= 16)
        launch_sums_rows<NB, 1, 4>(a, cus, st);
    else if (rows_per_group <= 32)
        launch_sums_rows<NB, 2, NB == 8 ? 3 : 4>(a, cus, st);
    else
        launch_sums_rows<NB, 4, NB == 8 ? 3 : 4>(a, cus, st);
}

// How a grouped product is run.
struct GroupedPlan {
    bool tiles;      // tile_kernel, else stream_kernel
    int splits;      // tile_kernel: pieces of K
    int blocks;      // stream_kernel: blocks of 16 rows in a tile
};

// The cheapest by three estimates in us, fitted to all of them measured at 391
// sizes (K 264 to 7168, N 264 to 7168, 1 to 64 groups of 1 to 3900 rows, equal
// and skewed).  Their rates are constants of the fit, with every group that
// could have a row counted as read, and not the bandwidths that are reached:
// skewed groups leave some empty (with 48 of 64 groups of K 7168, N 1792 in
// use, 4.9 TB/s).
//   stream   reads the weights at 6 TB/s, and again for every further tile of
//            rows at 11, or at 21 where the L2s hold them; twice as much (half
//            for PLAIN) where its row pieces are not whole lines of 128 bytes;
//            each 16 rows of a tile take its CU 0.037 us a K-step, and 19
//            K-steps more to begin and end; and 2.5 us
//   tiles    rounds of tiles (one at least) of 0.36 us a K-step, 0.55 with 256
//            rows, 0.72 with 256 rows on every CU, and 1.1 K-steps more; the
//            weights at 6.2 TB/s at best; and 18 us
//   split    in 2, 3, 4, 6 or 8 pieces: their rounds the same, 25 us, and the
//            sums written and read at 4 TB/s; where the sums have room
// At the sizes of the fit the choice is 1.1 % slower than the best of all on
// average, 34 % at worst.  At 204 random sizes outside it, estimates without a
// tile's beginning and end and with the step of a full chip took 1.6 % longer
// on average, between 0.78 and 1.75 times as long.
// us measured, stream / tiles / best split: K 7168, N 1792, 64 groups of 16
// rows with GLU 283 / 276 / 295; 8 groups of 8 rows 37 / 90 / 42, of 64 rows
// 43 / 96 / 47, of 192 rows 116 / 117 / 70, of 256 rows 153 / 128 / 88 (the
// choice is three pieces, 94), of 1024 rows 453 / 180 / -.  Groups are taken as
// equally large, as many as there are rows at most, and all S rows as present;
// a stream tile has room for twice the average rows, for real groups are not
// equal.
GroupedPlan plan_grouped(int64_t S, int64_t K, int64_t N, int64_t F, int E, bool glu, bool workspace, int cus)
{
    GroupedPlan pl = {};
    const int64_t used = std::min<int64_t>(E, S), rows = (S + used - 1) / used;
    const int kt = (int)((K + gc::BK - 1) / gc::BK);
    const double w = (double)used * K * N * 2e-6;                       // MB of weights
    pl.blocks = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    const double lines = (N % 64 != 0 || F % 64 != 0) ? (glu ? 2.0 : 1.5) : 1.0;
    const int64_t passes = (rows + 16 * pl.blocks - 1) / (16 * pl.blocks), strip = glu ? 64 : 128;
    const double work = (double)used * passes * pl.blocks * ((F + strip - 1) / strip) * (kt + 19) / cus;
    const double t_stream = 2.5 + w * lines * (1 / 6.0 + (double)(passes - 1) / (w > 32 ? 11.0 : 21.0)) + 0.037 * work;
    const int64_t bn = glu ? gc::BN / 2 : gc::BN, tiles_n = (F + bn - 1) / bn;
    const double tiles = (double)used * std::max(1.0, (double)rows / 256 + 0.5) * tiles_n;
    auto rounds = [&](double units, int steps) {
        const double busy = std::min(1.0, units / cus), height = (double)std::min<int64_t>(rows, 256);
        return std::max(1.0, units / cus) * (steps + 1.1) * (0.36 + 0.097 * busy + height * (0.00074 + 0.00027 * busy));
    };
    pl.splits = 1;
    double best = 18 + std::max(rounds(tiles, kt), w / 6.2);
    for (int q = 2; workspace && q <= 8 && kt / q >= 16 && q * S * N * 4 <= kSumBytes;
         q += q < 4 ? 1 : 2) {
        const double t = 25 + std::max(rounds(q * tiles, (kt + q - 1) / q), w / 6.2) +
                         (double)q * S * N * 8e-6 / 4.0;
        if (t < best) {
            best = t;
            pl.splits = q;
        }
    }
    pl.tiles = best < t_stream;
    return pl;
}

template <bool GLU>
void launch_tiles(gc::GroupedArgs &a, int splits, int cus, hipStream_t st)
{
    const int f = GLU ? a.N / 2 : a.N, bn = GLU ? gc::BN / 2 : gc::BN;
    a.tiles_n = (f + bn - 1) / bn;
    a.splits = splits;
    if (splits == 1) {
        hipLaunchKernelGGL((gc::tile_kernel<GLU, false>), dim3(cus), dim3(gc::NT), 0, st, a);
        return;
    }
    a.sums = a.part;
    hipLaunchKernelGGL((gc::tile_kernel<GLU, true>), dim3(cus), dim3(gc::NT), 0, st, a);
    const int64_t vecs = (int64_t)a.S * f / 8;
    const int grid = (int)std::min<int64_t>((vecs + gc::FINISH_THREADS - 1) / gc::FINISH_THREADS, 8 * cus);
    hipLaunchKernelGGL((gc::finish_kernel<GLU>), dim3(grid), dim3(gc::FINISH_THREADS), 0, st, a);
}

void launch_expand(gc::ExpandArgs &a, int cus, hipStream_t st)
{
    const gc::ExpandPlan pl = gc::expand_plan(a.M, a.N, a.E, a.r, cus);
    const dim3 g((unsigned)pl.grid), b(gc::EX_THREADS);
    a.span = pl.span;
    a.spans = pl.spans;
    if (pl.rows) {
        switch (pl.steps) {
        case 1: hipLaunchKernelGGL((gc::expand_rows_kernel<1>), g, b, 0, st, a); break;
        case 2: hipLaunchKernelGGL((gc::expand_rows_kernel<2>), g, b, 0, st, a); break;
        case 3: hipLaunchKernelGGL((gc::expand_rows_kernel<3>), g, b, 0, st, a); break;
        default: hipLaunchKernelGGL((gc::expand_rows_kernel<4>), g, b, 0, st, a); break;
        }
        return;
    }
    switch (pl.steps) {
    case 1: hipLaunchKernelGGL((gc::expand_kernel<1>), g, b, 0, st, a); break;
    case 2: hipLaunchKernelGGL((gc::expand_kernel<2>), g, b, 0, st, a); break;
    case 3: hipLaunchKernelGGL((gc::expand_kernel<3>), g, b, 0, st, a); break;
    default: hipLaunchKernelGGL((gc::expand_kernel<4>), g, b, 0, st, a); break;
    }
}

}  // namespace

extern "C" {

int64_t gemm_coll_grouped_workspace_bytes(void)
{
    int cus = 0;
    const int err = cu_count(cus);
    return err ? err : base_bytes(cus);
}

int64_t gemm_coll_lora_workspace_bytes(int64_t M, int r)
{
    if (M < 0 || r < 0)
        return GC_EINVAL;
    int cus = 0;
    const int err = cu_count(cus);
    return err ? err : std::max(base_bytes(cus), kCountBytes + M * r * 4);
}

int gemm_coll_moe_route(const void *logits, int logits_type, int64_t stride, int64_t T, int E, int k,
                        int score, const float *bias, int renormalize, float scale, int32_t *ids,
                        float *weights, int32_t *offsets, int32_t *rows, int32_t *slots,
                        void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (T < 0 || E < 1 || E > GC_GROUPS_MAX || k < 1 || k > GC_TOPK_MAX || stride < E)
        return GC_EINVAL;
    if ((logits_type != GC_F32 && logits_type != GC_BF16) ||
        (score != GC_SCORE_SOFTMAX && score != GC_SCORE_SIGMOID))
        return GC_EINVAL;
    const bool group = offsets || rows || slots;
    if (group && (!good4(offsets) || (T > 0 && (!good4(rows) || !good4(slots)))))
        return GC_EINVAL;
    if (T > ((int64_t)1 << 24) / k)
        return GC_ENOTSUP;
    const uintptr_t elem = logits_type == GC_BF16 ? 2 : 4;
    if (T > 0 && (!logits || !aligned(logits, elem) || !good4(ids) || !good4(weights)))
        return GC_EINVAL;
    if (bias && !aligned(bias, 4))
        return GC_EINVAL;
    if (T == 0 && !group)
        return GC_OK;
    const int v = route_values(E);
    gc::RouteArgs a = {};
    a.logits = logits;
    a.stride = stride;
    a.bias = bias;
    a.T = (int)T;
    a.E = E;
    a.k = k;
    a.per_row = k;
    a.score = score;
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.rows = rows;
    a.slots = slots;
    a.vec = E % v == 0 && stride % v == 0 && aligned(logits, std::min<uintptr_t>(16, v * elem));
    return route_and_group(a, true, logits_type == GC_BF16, workspace, workspace_bytes, (hipStream_t)stream);
}

int gemm_coll_group_rows(const int32_t *ids, int64_t T, int k, int groups, int32_t *offsets,
                         int32_t *rows, int32_t *slots, void *workspace, uint64_t workspace_bytes,
                         void *stream)
{
    if (T < 0 || k < 1 || groups < 1 || groups > GC_GROUPS_MAX || !good4(offsets))
        return GC_EINVAL;
    if (T > ((int64_t)1 << 24) / k)
        return GC_ENOTSUP;
    if (T > 0 && (!good4(ids) || !good4(rows) || !good4(slots)))
        return GC_EINVAL;
    // (Blocks are of items, not of rows, which may be longer than a block.)
    gc::RouteArgs a = {};
    a.T = (int)T * k;
    a.E = groups;
    a.k = 1;
    a.per_row = k;
    a.ids = const_cast<int32_t *>(ids);      // (only read: no routing)
    a.offsets = offsets;
    a.rows = rows;
    a.slots = slots;
    return route_and_group(a, false, false, workspace, workspace_bytes, (hipStream_t)stream);
}

int gemm_coll_grouped_gemm(const gc_bf16 *X, int64_t T, const gc_bf16 *W, const int32_t *offsets,
                           const int32_t *rows, int64_t S, int64_t K, int64_t N, int E, int act,
                           gc_bf16 *out, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (T < 0 || S < 0 || K < 0 || N < 0 || E < 1 || E > GC_GROUPS_MAX)
        return GC_EINVAL;
    if (act != GC_ACT_NONE && act != GC_ACT_SILU_GLU)
        return GC_EINVAL;
    if (K % 8 != 0 || N % (act == GC_ACT_SILU_GLU ? 16 : 8) != 0 || (!rows && T < S))
        return GC_EINVAL;
    if (T > INT32_MAX || S > INT32_MAX / 2 || K > INT32_MAX || N > kMaxCols)
        return GC_ENOTSUP;
    if (!fits(T, K) || !fits(K, N) || !fits(S, N))
        return GC_ENOTSUP;
    if (S == 0 || N == 0)
        return GC_OK;
    if (!good4(offsets) || (rows && !aligned(rows, 4)) || !good16(out))
        return GC_EINVAL;
    if (K > 0 && ((T > 0 && !good16(X)) || !good16(W)))
        return GC_EINVAL;
    int cus = 0;
    if (int err = cu_count(cus))
        return err;
    gc::GroupedArgs a = {};
    if (workspace) {
        if (!good16(workspace) || workspace_bytes < (uint64_t)base_bytes(cus))
            return GC_EINVAL;
        a.count = (uint32_t *)workspace;
        a.part = (float *)((char *)workspace + kCountBytes);
    }
    a.X = X;
    a.W = W;
    a.offsets = offsets;
    a.rows = rows;
    a.out = out;
    a.T = (int)T;
    a.S = (int)S;
    a.K = (int)K;
    a.N = (int)N;
    a.E = E;
    const bool glu = act == GC_ACT_SILU_GLU;
    const hipStream_t st = (hipStream_t)stream;
    const GroupedPlan pl = plan_grouped(S, K, N, glu ? N / 2 : N, E, glu, workspace != nullptr, cus);
    if (pl.tiles && glu)
        launch_tiles<true>(a, pl.splits, cus, st);
    else if (pl.tiles)
        launch_tiles<false>(a, pl.splits, cus, st);
    else if (glu)
        launch_stream_rows<gc::EPI_GLU>(a, pl.blocks, cus, st);
    else
        launch_stream_rows<gc::EPI_PLAIN>(a, pl.blocks, cus, st);
    return launched();
}

int gemm_coll_grouped_plan(int64_t S, int64_t K, int64_t N, int E, int act, int with_workspace, int cus,
                           gc_grouped_plan *plan)
{
    if (!plan || S < 0 || K < 0 || N < 0 || E < 1 || E > GC_GROUPS_MAX || cus < 1 || cus > 4096 ||
        (act != GC_ACT_NONE && act != GC_ACT_SILU_GLU) || K % 8 != 0 ||
        N % (act == GC_ACT_SILU_GLU ? 16 : 8) != 0)
        return GC_EINVAL;
    if (S > INT32_MAX / 2 || K > INT32_MAX || N > kMaxCols || !fits(K, N) || !fits(S, N))
        return GC_ENOTSUP;
    *plan = {0, 1, 0};
    if (S == 0 || N == 0)
        return GC_OK;
    const GroupedPlan pl = plan_grouped(S, K, N, act == GC_ACT_SILU_GLU ? N / 2 : N, E, act == GC_ACT_SILU_GLU,
                                        with_workspace != 0, cus);
    plan->tiles = pl.tiles;
    plan->splits = pl.tiles ? pl.splits : 1;
    plan->block_rows = pl.tiles ? 0 : 16 * pl.blocks;
    return GC_OK;
}

int gemm_coll_moe_combine(const gc_bf16 *Y, int64_t S, const int32_t *slots, const float *weights,
                          int64_t T, int k, int64_t N, const gc_bf16 *partials, int npeers,
                          int64_t peer_stride, gc_bf16 *out, void *stream)
{
    if (S < 0 || T < 0 || N < 0 || k < 1 || k > GC_TOPK_MAX || npeers < 0 || npeers > 15 || N % 8 != 0)
        return GC_EINVAL;
    if (S > INT32_MAX || T > INT32_MAX || N > INT32_MAX)
        return GC_ENOTSUP;
    if (T == 0 || N == 0)
        return GC_OK;
    if (!good4(slots) || !good4(weights) || !good16(out) || (S > 0 && !good16(Y)))
        return GC_EINVAL;
    if (npeers > 0 && (!good16(partials) || peer_stride % 8 != 0 || (npeers > 1 && peer_stride < T * N)))
        return GC_EINVAL;
    gc::CombineArgs a = {};
    a.Y = Y;
    a.slots = slots;
    a.weights = weights;
    a.partials = partials;
    a.peer_stride = peer_stride;
    a.out = out;
    a.T = (int)T;
    a.S = (int)S;
    a.N = (int)N;
    a.k = k;
    a.npeers = npeers;
    a.col_groups = (int)((N / 8 + 63) / 64);
    a.items = T * a.col_groups;
    // (a launch counts its threads in 32 bits)
    const int64_t blocks =
        std::min<int64_t>((a.items + gc::CB_WAVES - 1) / gc::CB_WAVES, UINT32_MAX / gc::CB_THREADS);
    hipLaunchKernelGGL(gc::combine_kernel, dim3((unsigned)blocks), dim3(gc::CB_THREADS), 0,
                       (hipStream_t)stream, a);
    return launched();
}

int gemm_coll_lora_add(const gc_bf16 *base, const gc_bf16 *X, const gc_bf16 *down, const gc_bf16 *up,
                       const float *scale, const int32_t *offsets, const int32_t *rows, int64_t M,
                       int64_t K, int64_t N, int r, int G, gc_bf16 *out, void *workspace,
                       uint64_t workspace_bytes, void *stream)
{
    if (M < 0 || K < 0 || N < 0 || r < 8 || r > 128 || G < 1 || G >= GC_GROUPS_MAX)
        return GC_EINVAL;
    if (K % 8 != 0 || N % 8 != 0 || r % 8 != 0)
        return GC_EINVAL;
    if (M > INT32_MAX / 2 || K > INT32_MAX || N > kMaxCols)
        return GC_ENOTSUP;
    if (!fits(M, K) || !fits(M, N) || !fits(M, r) || !fits(K, r) || !fits(r, N))
        return GC_ENOTSUP;
    if (M == 0 || N == 0)
        return GC_OK;
    if (!good16(base) || !good16(out) || !good16(up) || !good4(scale) || !good4(offsets) || !good4(rows))
        return GC_EINVAL;
    if (K > 0 && (!good16(X) || !good16(down)))
        return GC_EINVAL;
    int cus = 0;
    if (int err = cu_count(cus))
        return err;
    if (!good16(workspace) || workspace_bytes < (uint64_t)std::max(base_bytes(cus), kCountBytes + M * r * 4))
        return GC_EINVAL;
    const hipStream_t st = (hipStream_t)stream;
    gc::GroupedArgs a = {};
    a.X = X;
    a.W = down;
    a.offsets = offsets;
    a.rows = rows;
    a.sums = (float *)((char *)workspace + kCountBytes);
    a.T = (int)M;
    a.S = (int)M;
    a.K = (int)K;
    a.N = r;
    a.E = G;
    const int64_t avg = (M + G - 1) / G;
    if (r <= 16)
        launch_sums<1>(a, avg, cus, st);
    else if (r <= 32)
        launch_sums<2>(a, avg, cus, st);
    else if (r <= 64)
        launch_sums<4>(a, avg, cus, st);
    else
        launch_sums<8>(a, avg, cus, st);
    gc::ExpandArgs x = {};
    x.base = base;
    x.out = out;
    x.sums = a.sums;
    x.scale = scale;
    x.splits = a.splits;
    x.up = up;
    x.offsets = offsets;
    x.rows = rows;
    x.M = (int)M;
    x.N = (int)N;
    x.r = r;
    x.E = G;
    x.copy = out != base;
    launch_expand(x, cus, st);
    return launched();
}

}  // extern "C"
