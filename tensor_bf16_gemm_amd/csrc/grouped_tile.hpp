// grouped_tile.hpp -- gfx950 device code of the grouped products with many
// rows per group, where the matrix cores and the LDS bound them (see
// grouped.hpp for what is computed and for few rows).
//
// A workgroup of eight waves (2 along rows, 4 along columns) takes a tile of
// up to 256 positions of one group by 256 columns (for GLU 128 gate and the
// same 128 up columns, so that a lane holds both).  K advances 32 per step
// through four LDS stages filled by direct loads three steps ahead; the two
// waves of a SIMD alternate, one reading fragments and asking for loads
// while the other multiplies (the schedule of gc_kernel.hpp).  Gathered rows
// cost nothing: every lane of a load has an address of its own.
//
// Tile heights of 32, 64, .. 256 share one launch: a group's last tile is as
// tall as its rows need.  A step moves 32 KB of fragments of W and 8 KB per 32
// rows through the LDS besides the loads' 16 KB + 2 KB per 32 rows, so a
// 32-row tile costs about half of a 256-row one, not an eighth.
//
// The tiles of a group are numbered by bands of GROUP_M row tiles, columns
// next, rows of the band last: the tiles in flight on one XCD share rows of X
// and columns of W in its L2.  Groups are taken from the largest to the
// smallest, so that short tiles come last, and the line of tiles is dealt in
// hands of two tiles per CU of an XCD to eight queues, one for each, from
// which its workgroups draw tickets (from the next where theirs is empty).
// (32768 rows in 64 groups, 4 rounds of tiles: 826 to 860 us by machine; in
// turn on one machine 811, against 845 in the order of the groups, and 936
// with all short tiles last, which read W twice.)
//
// Fewer tiles than CUs: K is cut into p.splits equal pieces, each unit (piece,
// tile) leaves its fp32 sums in the workspace, and finish_kernel, a launch of
// its own at the bandwidth of the whole chip, adds them in the order of K and
// applies the end.  (8 groups of 256 rows, K 7168, N 1792: 88 us in four
// pieces, 128 whole.)
//
// What bounds it: the fragments' LDS traffic and the power limit, as in
// gc_kernel (one group of 8192 rows, N 8192, K 7168: 1.40 PFLOP/s, a library
// product of that size 1.36); with ragged groups also the last round of tiles
// and the rows the tiles are padded with (32768 rows over 64 groups, K 7168,
// N 1792 with GLU: MFMA busy 53 % of the cycles, CUs busy 83 %), with K = 896
// the stores (65536 rows, N 7168, 891 us: on a machine where it took 860, 717
// were left without them).
#pragma once

#include "grouped.hpp"

namespace gc {

constexpr int TK_GROUP_M = 6, TK_HAND = 64;
// Counters of a launch, zero between launches: one ticket per queue (64 bytes
// apart), and the workgroups that are through.
constexpr int TK_TICKET_STRIDE = 16, TK_DONE = TK_QUEUES * TK_TICKET_STRIDE;

struct TileAt {
    int e, lo, hi, m0, nt;
    int piece, k_begin, steps;     // piece of K: `steps` steps from step k_begin on
};

// One tile of 32*FMT positions.  SUMS: its fp32 sums go to p.sums.
template <int FMT, bool GLU, bool SUMS>
__device__ __forceinline__ void run_tile(const GroupedArgs &p, uint32_t lds0, const TileAt &at, int wave,
                                         int lane)
{
    constexpr int WMt = 16 * FMT, BMt = 2 * WMt;
    const int wm = wave >> 2, wn = wave & 3;
    const int fi = lane & 15, fg = lane >> 4;
    const int F = GLU ? p.N / 2 : p.N;
    const uint32_t N2 = (uint32_t)p.N * 2u;
    const int KT = at.steps;
    const u32x4_t rW = make_rsrc4(p.W + (size_t)at.e * p.K * p.N, (uint32_t)p.K * N2);
    const u32x4_t rX = make_rsrc4(p.X, (uint32_t)p.T * (uint32_t)p.K * 2u);

    // Loads, as in gc_kernel: instruction j of a wave fills rows 16 * (2 *
    // wave + j) + lane / 4 of the A stage and rows 4 * wave + 2 * j + lane / 32
    // of the B stage, with the stored chunks swizzled there.
    const int a_c = (lane & 3) ^ ((lane >> 3) & 3);
    uint32_t a_off[2], b_off[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = 16 * (2 * wave + j) + (lane >> 2), m = at.m0 + r;
        int src = -1;
        if (r < BMt && m >= at.lo && m < at.hi)
            src = p.rows ? p.rows[m] : m;
        a_off[j] = (unsigned)src < (unsigned)p.T
                       ? ((uint32_t)src * (uint32_t)p.K + (uint32_t)(8 * a_c)) * 2u
                       : OOB;
        const int k = 4 * wave + 2 * j + (lane >> 5);
        const int fk = (k & 3) | (((k >> 3) & 1) << 2);
        const int slot = lane & 31;
        const int c = 16 * ((slot >> 1) ^ fk) + 8 * (slot & 1);     // column in the tile
        int n;
        if (GLU) {
            const int h = at.nt * (BN / 2) + (c & (BN / 2 - 1));
            n = h >= F ? -1 : c < BN / 2 ? h : F + h;
        } else {
            n = at.nt * BN + c < p.N ? at.nt * BN + c : -1;
        }
        b_off[j] = n >= 0 ? ((uint32_t)k * (uint32_t)p.N + (uint32_t)n) * 2u : OOB;
    }
    auto stage = [&](int s) { return lds0 + (uint32_t)(s * (A_BYTES + B_BYTES)); };
    // Loads of step kt; past the K loop the same number of empty ones.  (An
    // offset of OOB plus a step's advance, below 2^31, is still out of range.)
    auto load = [&](int kt, uint32_t st) {
        const int k0 = (at.k_begin + kt) * BK;
        const bool live = kt < KT;
        const uint32_t ka = (uint32_t)k0 * 2u, kb = (uint32_t)k0 * N2;
        const uint32_t la = st + (uint32_t)(2 * wave * 1024);
        const uint32_t lb = st + (uint32_t)(A_BYTES + 4 * wave * 512);
        if (live && k0 + BK <= p.K) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                dma16(rX, la + j * 1024, a_off[j] + ka);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                dma16(rW, lb + j * 1024, b_off[j] + kb);
        } else {
            // (rows of W past K lie past its buffer)
            const bool on = live && k0 + 8 * a_c < p.K;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                dma16(rX, la + j * 1024, on ? a_off[j] + ka : OOB);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                dma16(rW, lb + j * 1024, live && k0 < p.K ? b_off[j] + kb : OOB);
        }
    };
    const uint32_t a_frag = (uint32_t)(wm * WMt * 64 + fi * 64 + ((fg ^ ((fi >> 1) & 3)) << 4));
    const int fB = (fi >> 2) | ((fg & 1) << 2);
    uint32_t b_frag[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        // column block of the wave: for GLU blocks 0, 1 gate and 2, 3 up
        const int q = GLU ? 8 * (j >> 1) + 2 * wn + (j & 1) : 4 * wn + j;
        b_frag[j] = (uint32_t)(A_BYTES + (8 * fg + (fi >> 2)) * 512 + 8 * (fi & 3) + (q >> 3) * 256 +
                               (((q & 7) ^ fB) * 32));
    }
    f32x4_t acc[FMT][FN];
#pragma unroll
    for (int i = 0; i < FMT; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

    load(0, stage(0));
    load(1, stage(1));
    load(2, stage(2));
    const bool lag = wave >= 4;
    wait_vmcnt<2 * DMA_PER_STEP>();
    if (lag)
        barrier_only();
    auto step = [&](auto uc, int kt) {
        constexpr int u = decltype(uc)::value;
        const uint32_t cs = opaque(stage(u)), ns = stage((u + 3) & 3);
        barrier_only();
        bf16x8_t fa[FN], fb[FMT];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            bf16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                (lds_bf16x4_t *)lds_ptr<bf16x4_t>(cs + b_frag[j]));
            bf16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                (lds_bf16x4_t *)lds_ptr<bf16x4_t>(cs + b_frag[j] + 4 * 512));
            fa[j] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        }
#pragma unroll
        for (int i = 0; i < FMT; ++i)
            fb[i] = *lds_ptr<bf16x8_t>(cs + a_frag + i * 1024);
        load(kt + 3, ns);
        wait_vmcnt<2 * DMA_PER_STEP>();       // the wave's loads of step kt + 1 have landed
        wait_lgkmcnt0();
        barrier_only();
#pragma unroll
        for (int i = 0; i < FMT; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[j], fb[i], acc[i][j], 0, 0, 0);
    };
    int kt = 0;
    for (; kt + 4 <= KT; kt += 4) {
        step(std::integral_constant<int, 0>{}, kt);
        step(std::integral_constant<int, 1>{}, kt + 1);
        step(std::integral_constant<int, 2>{}, kt + 2);
        step(std::integral_constant<int, 3>{}, kt + 3);
    }
    if (kt < KT)
        step(std::integral_constant<int, 0>{}, kt);
    if (kt + 1 < KT)
        step(std::integral_constant<int, 1>{}, kt + 1);
    if (kt + 2 < KT)
        step(std::integral_constant<int, 2>{}, kt + 2);
    if (!lag)
        barrier_only();

    if constexpr (SUMS) {
        // 4 columns of a row per lane and block
        const int ln = opaque_v(lane);
        const int fi2 = ln & 15, fg2 = ln >> 4;
#pragma unroll
        for (int i = 0; i < FMT; ++i) {
            const int m = at.m0 + wm * WMt + 16 * i + fi2;
            float *row = p.sums + ((size_t)at.piece * p.S + m) * p.N;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int h = GLU ? at.nt * (BN / 2) + 32 * wn + 16 * (j & 1) + 4 * fg2
                                  : at.nt * BN + 64 * wn + 16 * j + 4 * fg2;
                if (m < at.hi && h < F)
                    *(f32x4_t *)(row + (GLU && j >= 2 ? F + h : h)) = acc[i][j];
            }
        }
        return;
    }

    // ---- epilogue: 16-byte stores of 8 columns per lane ----
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.out, (uint32_t)p.S * (uint32_t)F * 2u);
    const int ln = opaque_v(lane);
    const int fi2 = ln & 15, fg2 = ln >> 4;
    const int p8 = 8 * (fg2 >> 1) + 16 * (fg2 & 1);
#pragma unroll
    for (int i = 0; i < FMT; ++i) {
        const int m = at.m0 + wm * WMt + 16 * i + fi2;
        const bool row = m < at.hi;
        if constexpr (GLU) {
            const int n = at.nt * (BN / 2) + 32 * wn + p8;
            const u32x4_t pk = pack_pair(silu_mul(acc[i][0], acc[i][2]), silu_mul(acc[i][1], acc[i][3]));
            store16(ro, row && n < F ? ((uint32_t)m * (uint32_t)F + (uint32_t)n) * 2u : OOB, pk);
        } else {
#pragma unroll
            for (int h = 0; h < FN / 2; ++h) {
                const int n = at.nt * BN + 64 * wn + 32 * h + p8;
                store16(ro, row && n < F ? ((uint32_t)m * (uint32_t)F + (uint32_t)n) * 2u : OOB,
                        pack_pair(acc[i][2 * h], acc[i][2 * h + 1]));
            }
        }
    }
}

template <bool GLU, bool SUMS>
__global__ __launch_bounds__(NT, 2) void tile_kernel(GroupedArgs p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t stages[STAGES * (A_BYTES + B_BYTES)];
    __shared__ int first[GR_GROUPS + 1];                 // by rank of size
    __shared__ int2 range[GR_GROUPS];
    __shared__ int16_t order[GR_GROUPS];                 // the group of each rank
    __shared__ int wsum[WAVES];
    __shared__ int s_next;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = gridDim.x;
    for (int e = tid; e < p.E; e += NT) {
        int lo, hi;
        group_range(p.offsets, p.E, p.S, e, lo, hi);
        range[e] = make_int2(lo, hi);
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += NT) {
        const int n = range[e].y - range[e].x;
        int rank = 0;
        for (int o = 0; o < p.E; ++o) {
            const int no = range[o].y - range[o].x;
            rank += no > n || (no == n && o < e);
        }
        order[rank] = (int16_t)e;
    }
    __syncthreads();
    auto count = [&](int r) {
        const int2 g = range[order[r]];
        return (g.y - g.x + BM - 1) / BM * p.tiles_n;
    };
    const int tiles = scan_counts<NT>(p.E, count, first, wsum);
    // Units: the tiles of the first piece of K, then those of the next.
    const int splits = SUMS ? p.splits : 1;
    const int KT = (p.K + BK - 1) / BK, piece_steps = (KT + splits - 1) / splits;
    const int units = tiles * splits;
    // Queue x holds hands x, x + 8, ... of TK_HAND units (an eighth of the units
    // where they are few: 8 groups of 512 rows, K 7168, N 1792 on two queues
    // took 305 us, on eight 122).
    const int hand = max(min(TK_HAND, (units + TK_QUEUES - 1) / TK_QUEUES), 1);
    int x = blockIdx.x & (TK_QUEUES - 1), tried = 0;
    Share share(blockIdx.x, G);
    // Next unit for this workgroup, or -1 (thread 0 only).
    auto draw = [&]() {
        if (!p.count)                           // no workspace
            return share.draw(hand, units);
        for (; tried < TK_QUEUES; ++tried, x = (x + 1) & (TK_QUEUES - 1)) {
            const int t = queue_unit(x, (int)__hip_atomic_fetch_add(p.count + x * TK_TICKET_STRIDE, 1u,
                                                                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
                                     hand);
            if (t < units)
                return t;
        }
        return -1;
    };
    if (tid == 0)
        s_next = draw();
    const uint32_t lds0 = lds_addr(stages);
    for (;;) {
        __syncthreads();
        const int unit = __builtin_amdgcn_readfirstlane(s_next);
        __syncthreads();
        if (unit < 0)
            break;
        if (tid == 0)
            s_next = draw();
        TileAt at;
        at.piece = SUMS ? unit / max(tiles, 1) : 0;
        at.k_begin = at.piece * piece_steps;
        at.steps = max(min(piece_steps, KT - at.k_begin), 0);
        const int t = unit - at.piece * tiles;
        const int rank = __builtin_amdgcn_readfirstlane(find_group(first, p.E, t, lane));
        at.e = __builtin_amdgcn_readfirstlane(order[rank]);
        at.lo = __builtin_amdgcn_readfirstlane(range[at.e].x);
        at.hi = __builtin_amdgcn_readfirstlane(range[at.e].y);
        const int in = t - __builtin_amdgcn_readfirstlane(first[rank]);
        const int tiles_m = max((at.hi - at.lo + BM - 1) / BM, 1);
        const int band = in / (TK_GROUP_M * p.tiles_n);
        const int rest = in - band * TK_GROUP_M * p.tiles_n;
        const int high = min(TK_GROUP_M, tiles_m - band * TK_GROUP_M);
        at.nt = rest / max(high, 1);
        at.m0 = at.lo + (band * TK_GROUP_M + rest - at.nt * high) * BM;
        switch (min(8, (at.hi - at.m0 + 31) / 32)) {
        case 1: run_tile<1, GLU, SUMS>(p, lds0, at, wave, lane); break;
        case 2: run_tile<2, GLU, SUMS>(p, lds0, at, wave, lane); break;
        case 3: run_tile<3, GLU, SUMS>(p, lds0, at, wave, lane); break;
        case 4: run_tile<4, GLU, SUMS>(p, lds0, at, wave, lane); break;
        case 5: run_tile<5, GLU, SUMS>(p, lds0, at, wave, lane); break;
        case 6: run_tile<6, GLU, SUMS>(p, lds0, at, wave, lane); break;
        case 7: run_tile<7, GLU, SUMS>(p, lds0, at, wave, lane); break;
        default: run_tile<8, GLU, SUMS>(p, lds0, at, wave, lane); break;
        }
        wait_vmcnt<0>();                         // the stages are free for the next tile
    }
    // The last workgroup through leaves the counters at zero.
    if (p.count && tid == 0) {
        const uint32_t n = __hip_atomic_fetch_add(p.count + TK_DONE, 1u, __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT);
        if (n == (uint32_t)G - 1) {
            for (int q = 0; q < TK_QUEUES; ++q)
                __hip_atomic_store(p.count + q * TK_TICKET_STRIDE, 0u, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(p.count + TK_DONE, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
}

// out = the end of the sums of every position in a group, 8 columns a thread.
constexpr int FINISH_THREADS = 256;
template <bool GLU>
__global__ __launch_bounds__(FINISH_THREADS) void finish_kernel(GroupedArgs p)
{
    const int F = GLU ? p.N / 2 : p.N, vecs = F / 8;
    const int lo = min(max(p.offsets[0], 0), p.S), hi = min(max(p.offsets[p.E], lo), p.S);
    const int64_t n = (int64_t)(hi - lo) * vecs, step = (int64_t)gridDim.x * FINISH_THREADS;
    const size_t plane = (size_t)p.S * p.N;
    for (int64_t i = (int64_t)blockIdx.x * FINISH_THREADS + threadIdx.x; i < n; i += step) {
        const int m = lo + (int)(i / vecs), c = (int)(i % vecs) * 8;
        auto sum = [&](int col) {
            const float *at = p.sums + (size_t)m * p.N + col;
            f32x4_t x = *(const f32x4_t *)at;
            for (int s = 1; s < p.splits; ++s)
                x += *(const f32x4_t *)(at + s * plane);
            return x;
        };
        f32x4_t x = sum(c), y = sum(c + 4);
        if (GLU) {
            x = silu_mul(x, sum(F + c));
            y = silu_mul(y, sum(F + c + 4));
        }
        const u32x2_t a = pack_bf16x4(x), b = pack_bf16x4(y);
        *(u32x4_t *)(p.out + (size_t)m * F + c) = (u32x4_t){a[0], a[1], b[0], b[1]};
    }
}

}  // namespace gc
