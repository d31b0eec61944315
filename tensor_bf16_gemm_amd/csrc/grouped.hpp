// grouped.hpp -- gfx950 device code of the matrix products grouped by expert
// (or adapter): for every group e and every position i in
// [offsets[e], offsets[e+1])
//   y[i] = X[rows[i]] . W[e]              (rows[i] = i without a row list)
// with one of three ends:
//   PLAIN  out[i] = bf16(y[i])
//   GLU    out[i] = bf16(silu(y[i][:N/2]) * y[i][N/2:])
//   SUMS   fp32 y[i] over each of `splits` equal pieces of K, the adapters'
//          middle activations, which their reader adds up in the order of K
//
// stream_kernel: few rows per group, so the weights' bytes bound it.  A tile
// is 16*RB positions of one group by 16*NB columns of W[e]; the four waves of
// a workgroup take alternate K-steps of 32, each through a ring of D slots in
// LDS of its own, so that no barrier stands between a wave and its loads and
// (D - 1) * 4 steps of weights are in flight per CU all the time.  The waves'
// sums are added through LDS at the end of the tile.
//
// PLAIN and GLU: work is dealt out evenly whatever the groups' sizes: the
// K-steps of all tiles, counted in quads of 4 (one per wave), form one line,
// and workgroup w takes the w-th of equal pieces of it.  A tile whose K range is cut by a
// piece's end is finished by the last of its workgroups to arrive, which adds
// the others' fp32 partial tiles in the order of K: nobody waits for anybody,
// and the order of the sum does not depend on who was last.  (8 experts of one
// row each, K 7168, N 1792: 206 MB in 46.3 us,
// 4.4 TB/s with launch, look-up and hand-over.  Two workgroups per CU took
// 53 us, tiles of 256 columns 51, a ring of 3 steps the same 46.)
#pragma once

#include "deal.hpp"
#include "gc_kernel.hpp"

namespace gc {

enum Epilogue { EPI_PLAIN = 0, EPI_GLU = 1, EPI_SUMS = 2 };

constexpr int GR_GROUPS = 1024;           // groups at most

struct GroupedArgs {
    const uint16_t *X;         // [T][K]
    const uint16_t *W;         // [E][K][N]
    const int32_t *offsets;    // [E + 1]
    const int32_t *rows;       // [S] or null
    uint16_t *out;             // PLAIN [S][N], GLU [S][N/2]
    float *sums;               // sums over pieces of K [splits][S][N]
    int splits;
    int T, S, K, N, E;
    int tiles_n;               // column tiles
    int min_quads;             // smallest piece of a tile that a workgroup takes
    // Partial tiles: two slots per workgroup (a tile it ends, a tile it
    // begins) of `part_slots` / 2 workgroups, and one arrival counter per
    // workgroup for the tile it begins; counters are zero between launches.
    float *part;
    uint32_t *count;
    int part_slots;
};

// Range of group e, made safe whatever the offsets hold.  Group E is the
// positions past the last group.
__device__ __forceinline__ void group_range(const int32_t *offsets, int E, int S, int e, int &lo, int &hi)
{
    lo = min(max(offsets[e], 0), S);
    hi = e < E ? min(max(offsets[e + 1], lo), S) : S;
}

// first[i] = the sum of count(0 .. i - 1), i = 0 .. n (by add_tiles, so that it
// never falls); returns the whole sum.
// NTH threads; n <= 1024.
template <int NTH, class F>
__device__ __forceinline__ int scan_counts(int n, F &&count, int *first, int *wsum)
{
    constexpr int PER = GR_GROUPS / NTH;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = PER * tid + i;
        c[i] = at < n ? count(at) : 0;
        sum = add_tiles(sum, c[i]);
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(inc, d);
        if (lane >= d)
            inc = add_tiles(inc, o);
    }
    if (lane == 63)
        wsum[wave] = inc;
    const int prev = __shfl_up(inc, 1);
    __syncthreads();
    int at = lane > 0 ? prev : 0, before = 0, all = 0;
    for (int w = 0; w < NTH / 64; ++w) {
        if (w < wave)
            before = add_tiles(before, wsum[w]);
        all = add_tiles(all, wsum[w]);
    }
    at = add_tiles(before, at);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (PER * tid + i < n)
            first[PER * tid + i] = at;
        at = add_tiles(at, c[i]);
    }
    if (tid == 0)
        first[n] = all;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(all);
}

// first[e] = tiles of the groups before e, for tiles of `bm` positions and
// tiles_n columns tiles, and starts[e] = the clamped offsets; returns the
// number of tiles.  groups: E, or E + 1 with the positions past the last.
template <int NTH>
__device__ __forceinline__ int scan_tiles(const int32_t *offsets, int E, int S, int groups, int bm,
                                          int tiles_n, int *first, int *starts, int *wsum)
{
    auto count = [&](int e) {
        int lo, hi;
        group_range(offsets, E, S, e, lo, hi);
        starts[e] = lo;
        return (hi - lo + bm - 1) / bm * tiles_n;
    };
    if (threadIdx.x == 0)
        starts[groups] = groups == E ? min(max(offsets[E], 0), S) : S;
    return scan_counts<NTH>(groups, count, first, wsum);
}

// group_range from the starts that scan_tiles has left in LDS.
__device__ __forceinline__ void group_bounds(const int *starts, int e, int &lo, int &hi)
{
    lo = __builtin_amdgcn_readfirstlane(starts[e]);
    hi = max(__builtin_amdgcn_readfirstlane(starts[e + 1]), lo);
}

// Group of tile t: the last e with first[e] <= t (two looks of a whole wave).
__device__ __forceinline__ int find_group(const int *first, int groups, int t, int lane)
{
    const int c = min(16 * lane, groups);
    const uint64_t a = __builtin_amdgcn_ballot_w64(16 * lane < groups && first[c] <= t);
    const int base = 16 * (max(__builtin_popcountll(a), 1) - 1);
    const int f = min(base + 1 + (lane & 15), groups);
    const uint64_t b =
        __builtin_amdgcn_ballot_w64(lane < 16 && base + 1 + lane < groups && first[f] <= t);
    return base + __builtin_popcountll(b);
}

// In fp32, with the exponential as 2^(x log2 e) of the hardware: its argument
// is rounded once, which moves the result by |x| 2^-24 of itself, so by less
// than 2^-17 where e^-x is finite.  What becomes of it is rounded to bf16
// (2^-9) at once; expf would take some ten instructions more per value.
__device__ __forceinline__ float silu(float x) { return x / (1.0f + __expf(-x)); }

__device__ __forceinline__ f32x4_t silu_mul(f32x4_t g, f32x4_t u)
{
    return (f32x4_t){silu(g[0]) * u[0], silu(g[1]) * u[1], silu(g[2]) * u[2], silu(g[3]) * u[3]};
}

constexpr int ST_THREADS = 256, ST_WAVES = 4;

// NB, RB: 16-column and 16-position blocks of a tile; D: slots of a ring.
template <int NB, int RB, int D, int EPI>
__global__ __launch_bounds__(ST_THREADS) void stream_kernel(GroupedArgs p)
{
    constexpr int BN = 16 * NB, BM = 16 * RB;
    constexpr int B_SLOT = NB * 1024, SLOT = (NB + RB) * 1024;
    constexpr int LOADS = NB + RB;                       // per step and wave
    constexpr int RPI = 512 / BN;                        // rows of W per load instruction
    constexpr int RING = ST_WAVES * D * SLOT, SUMS = ST_WAVES * RB * NB * 1024;
    static_assert((D - 1) * LOADS < 64, "vmcnt");
    static_assert(EPI != EPI_GLU || NB >= 4, "gate and up columns in one tile");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[RING > SUMS ? RING : SUMS];
    __shared__ int first[GR_GROUPS + 1], starts[GR_GROUPS + 1];
    __shared__ int wsum[ST_WAVES];
    __shared__ int s_last;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fi = lane & 15, fg = lane >> 4;
    const int G = gridDim.x;
    const int F = EPI == EPI_GLU ? p.N / 2 : p.N;        // output columns
    const uint32_t N2 = (uint32_t)p.N * 2u;
    const int KT = (p.K + BK - 1) / BK;

    const int tiles = scan_tiles<ST_THREADS>(p.offsets, p.E, p.S, p.E, BM, p.tiles_n, first, starts, wsum);
    if (tiles <= 0)
        return;
    constexpr bool LINE = EPI != EPI_SUMS;
    const Line line(tiles, max((KT + ST_WAVES - 1) / ST_WAVES, 1), LINE ? p.min_quads : 1,
                    LINE ? min(G, p.part_slots / 2) : 1);
    int64_t q, q_end;
    int v = blockIdx.x;
    if constexpr (EPI == EPI_SUMS) {
        q = v;                                           // units: (tile, piece of K)
        q_end = (int64_t)tiles * p.splits;
    } else {
        if (v >= line.pieces)
            return;
        v = xcd_remap(v, line.pieces);
        q = line.bound(v);
        q_end = line.bound(v + 1);
    }

    // Loads of W: lane = row lane / (64 / RPI) of the instruction's RPI rows,
    // 16-byte slot lane % (BN / 8) of the row.  The 32-byte chunk c of row k
    // is kept at chunk c ^ f(k), so that the two rows groups a pass of the
    // transposing read covers fall into different banks: f has as many bits
    // as a row has chunks, from the bits of k that vary within a pass and do
    // not move the row's own bank.
    auto fold = [](int k) {
        return NB == 8 ? (k & 3) | (((k >> 3) & 1) << 2)
             : NB == 4 ? ((k >> 1) & 1) | (((k >> 3) & 1) << 1)
             : NB == 2 ? (k >> 3) & 1
                       : 0;
    };
    const int b_row = lane / (BN / 8), b_slot = lane % (BN / 8);
    const int a_c = (lane & 3) ^ ((lane >> 3) & 3);
    const int f_lane = fold(8 * fg + (fi >> 2));
    uint32_t b_frag[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        b_frag[j] = (uint32_t)((8 * fg + (fi >> 2)) * BN * 2 + 8 * (fi & 3) + ((j ^ f_lane) * 32));
    const uint32_t a_frag = (uint32_t)(B_SLOT + fi * 64 + ((fg ^ ((fi >> 1) & 3)) << 4));
    const uint32_t my_ring = lds_addr(ring) + (uint32_t)(wave * D * SLOT);

    while (q < q_end) {
        int t, ka, kb;
        [[maybe_unused]] int piece = 0;
        if constexpr (EPI == EPI_SUMS) {
            t = (int)(q / p.splits);
            piece = (int)(q - (int64_t)t * p.splits);
            const int len = (line.per_tile + p.splits - 1) / p.splits;
            ka = min(piece * len, line.per_tile);
            kb = min(ka + len, line.per_tile);
            q += G;
        } else {
            t = (int)(q / line.per_tile);
            ka = (int)(q - (int64_t)t * line.per_tile);
            kb = (int)min((int64_t)line.per_tile, ka + (q_end - q));
            q += kb - ka;
        }
        const int e = __builtin_amdgcn_readfirstlane(find_group(first, p.E, t, lane));
        int lo, hi;
        group_bounds(starts, e, lo, hi);
        const int in = t - __builtin_amdgcn_readfirstlane(first[e]);
        const int tiles_m = max((hi - lo + BM - 1) / BM, 1);
        const int nt = in / tiles_m;
        const int m0 = lo + (in - nt * tiles_m) * BM;

        const u32x4_t rW = make_rsrc4(p.W + (size_t)e * p.K * p.N, (uint32_t)p.K * N2);
        const u32x4_t rX = make_rsrc4(p.X, (uint32_t)p.T * (uint32_t)p.K * 2u);
        uint32_t a_off[RB], b_off[NB];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int m = m0 + 16 * i + (lane >> 2);
            int src = -1;
            if (m >= lo && m < hi)
                src = p.rows ? p.rows[m] : m;
            a_off[i] = (unsigned)src < (unsigned)p.T
                           ? ((uint32_t)src * (uint32_t)p.K + (uint32_t)(8 * a_c)) * 2u
                           : OOB;
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int k = i * RPI + b_row;
            const int c = 16 * ((b_slot >> 1) ^ fold(k)) + 8 * (b_slot & 1);   // column in the tile
            int n;
            if (EPI == EPI_GLU) {
                const int h = nt * (BN / 2) + (c & (BN / 2 - 1));
                n = h >= F ? -1 : c < BN / 2 ? h : F + h;
            } else {
                n = nt * BN + c < p.N ? nt * BN + c : -1;
            }
            b_off[i] = n >= 0 ? ((uint32_t)k * (uint32_t)p.N + (uint32_t)n) * 2u : OOB;
        }
        // Steps of this wave: s0, s0 + 4, ... below s1.  Steps past the end
        // issue the same number of loads, out of range, so that the wait
        // counts stay constant.  Rows of W past K lie past the buffer; the
        // A chunks past K are masked (they would read the next row).  An offset
        // of OOB plus a step's advance, below 2^31, is still out of range.
        const int s1 = min(ST_WAVES * kb, KT);
        auto issue = [&](int s, uint32_t slot) {
            const int k0 = s * BK;
            const bool on = s < s1;
            const uint32_t ka2 = (uint32_t)k0 * 2u, kb2 = (uint32_t)k0 * N2;
            const uint32_t at = my_ring + slot * SLOT;
#pragma unroll
            for (int i = 0; i < NB; ++i)
                dma16(rW, at + i * 1024, on ? b_off[i] + kb2 : OOB);
            const bool whole = on && k0 + 8 * a_c < p.K;
#pragma unroll
            for (int i = 0; i < RB; ++i)
                dma16(rX, at + B_SLOT + i * 1024, whole ? a_off[i] + ka2 : OOB);
        };
        f32x4_t acc[RB][NB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

        int s = ST_WAVES * ka + wave;
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            issue(s + ST_WAVES * d, d);
        uint32_t cur = 0;
        for (; s < s1; s += ST_WAVES) {
            wait_lgkmcnt0();                     // the slot to be refilled is read
            issue(s + ST_WAVES * (D - 1), cur == 0 ? D - 1 : cur - 1);
            wait_vmcnt<(D - 1) * LOADS>();       // this step's loads have landed
            const uint32_t at = my_ring + cur * SLOT;
            bf16x8_t fa[NB], fb[RB];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                bf16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (lds_bf16x4_t *)lds_ptr<bf16x4_t>(at + b_frag[j]));
                bf16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (lds_bf16x4_t *)lds_ptr<bf16x4_t>(at + b_frag[j] + 4 * BN * 2));
                fa[j] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int i = 0; i < RB; ++i)
                fb[i] = *lds_ptr<bf16x8_t>(at + a_frag + i * 1024);
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[j], fb[i], acc[i][j], 0, 0, 0);
            cur = cur == D - 1 ? 0 : cur + 1;
        }
        wait_vmcnt<0>();
        __syncthreads();

        // ---- the four waves' sums ----
        f32x4_t *sums = (f32x4_t *)ring;
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                sums[((wave * RB + i) * NB + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        auto block_sum = [&](int b) {
            f32x4_t x = sums[b * 64 + lane];
#pragma unroll
            for (int w = 1; w < ST_WAVES; ++w)
                x += sums[(w * RB * NB + b) * 64 + lane];
            return x;
        };

        // ---- a cut tile: hand the partial over, the last to arrive goes on ----
        const bool cut = EPI != EPI_SUMS && (ka > 0 || kb < line.per_tile);
        int w_first = v, w_last = v;
        const __amdgpu_buffer_rsrc_t rp =
            make_rsrc(p.part, (uint32_t)p.part_slots * (uint32_t)(RB * NB * 1024));
        if (cut) {
            const int64_t t0 = (int64_t)t * line.per_tile;
            w_first = line.piece_of(t0);
            w_last = line.piece_of(t0 + line.per_tile - 1);
            // a piece that begins inside the tile uses its workgroup's slot 0
            const uint32_t slot = (uint32_t)(2 * v + (ka == 0 ? 1 : 0));
            for (int b = wave; b < RB * NB; b += ST_WAVES)
                __builtin_amdgcn_raw_buffer_store_b128(
                    __builtin_bit_cast(u32x4_t, block_sum(b)), rp,
                    (int)(slot * (uint32_t)(RB * NB * 1024) + (uint32_t)(b * 1024 + lane * 16)), 0, CPOL_SYS);
            wait_vmcnt<0>();
            __syncthreads();
            if (tid == 0) {
                const uint32_t n = __hip_atomic_fetch_add(p.count + w_first, 1u, __ATOMIC_RELAXED,
                                                          __HIP_MEMORY_SCOPE_SYSTEM);
                const int last = (int)n == w_last - w_first;
                if (last)       // everybody has been: the counter is free again
                    __hip_atomic_store(p.count + w_first, 0u, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_SYSTEM);
                s_last = last;
            }
            __syncthreads();
            if (!s_last) {
                __syncthreads();
                continue;
            }
        }
        // Sums of n blocks (numbers at[]): of a cut tile over its pieces, in the
        // order of K, every piece's blocks asked for together.
        auto final_sums = [&](auto &x, const auto &at, auto count) {
            constexpr int n = decltype(count)::value;
            if (!cut) {
#pragma unroll
                for (int i = 0; i < n; ++i)
                    x[i] = block_sum(at[i]);
                return;
            }
#pragma unroll
            for (int i = 0; i < n; ++i)
                x[i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
            for (int w = w_first; w <= w_last; ++w) {
                const uint32_t slot = (uint32_t)(2 * w + (w == w_first ? 1 : 0));
                f32x4_t y[n];
#pragma unroll
                for (int i = 0; i < n; ++i)
                    y[i] = __builtin_bit_cast(
                        f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                     rp, (int)(slot * (uint32_t)(RB * NB * 1024) + (uint32_t)(at[i] * 1024 + lane * 16)),
                                     0, CPOL_SYS));
#pragma unroll
                for (int i = 0; i < n; ++i)
                    x[i] += y[i];
            }
        };

        // ---- epilogue ----
        const int p8 = 8 * (fg >> 1) + 16 * (fg & 1);    // first column of a lane in a pair
        if constexpr (EPI == EPI_SUMS) {
            for (int b = wave; b < RB * NB; b += ST_WAVES) {
                const int i = b / NB, j = b - i * NB;
                const int m = m0 + 16 * i + fi, n = nt * BN + 16 * j + 4 * fg;
                const f32x4_t x = block_sum(b);
                if (m < hi && n < p.N)
                    *(f32x4_t *)(p.sums + ((size_t)piece * p.S + m) * p.N + n) = x;
            }
        } else {
            // A unit is a pair of neighbouring blocks (for GLU, gate and up); a
            // wave takes every fourth.
            constexpr int PAIRS = EPI == EPI_GLU ? NB / 4 : NB / 2, PER = EPI == EPI_GLU ? 4 : 2;
            constexpr int UNITS = (RB * PAIRS + ST_WAVES - 1) / ST_WAVES;
            f32x4_t x[UNITS * PER];
            int at[UNITS * PER];
#pragma unroll
            for (int k = 0; k < UNITS; ++k) {
                const int u = min(wave + ST_WAVES * k, RB * PAIRS - 1);
                const int i = u / PAIRS, j = 2 * (u - i * PAIRS);
#pragma unroll
                for (int d = 0; d < PER; ++d)
                    at[PER * k + d] = i * NB + j + (d & 1) + (d >> 1) * (NB / 2);
            }
            final_sums(x, at, std::integral_constant<int, UNITS * PER>{});
#pragma unroll
            for (int k = 0; k < UNITS; ++k) {
                const int u = wave + ST_WAVES * k;
                const int i = u / PAIRS, j = 2 * (u - i * PAIRS);
                f32x4_t a = x[PER * k], b = x[PER * k + 1];
                if constexpr (EPI == EPI_GLU) {
                    a = silu_mul(a, x[PER * k + 2]);
                    b = silu_mul(b, x[PER * k + 3]);
                }
                const u32x4_t pk = pack_pair(a, b);
                const int m = m0 + 16 * i + fi;
                const int n = nt * (EPI == EPI_GLU ? BN / 2 : BN) + 16 * j + p8;
                if (u < RB * PAIRS && m < hi && n < F)
                    *(u32x4_t *)(p.out + (size_t)m * F + n) = pk;
            }
        }
        __syncthreads();
    }
}

}  // namespace gc
