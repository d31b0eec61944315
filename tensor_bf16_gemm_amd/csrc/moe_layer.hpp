// moe_layer.hpp -- gfx950 device code of a layer of experts for up to 16
// tokens, in two launches:
//
//   moe_up_kernel    ids, w = router(logits)
//                    a[t][j] = bf16(silu(g) * u), (g, u) = X[t] . W1[ids[t][j]]
//   moe_down_kernel  out[t] = bf16( sum_j w[t][j] (a[t][j] . W2[ids[t][j]])
//                                   + sum_p partials[p][t] )
//
// The weights of the experts in use are read once and bound both: over changing
// inputs, 16 tokens, 8 of 64 experts, K 7168, F 896, N 7168, 7 peers 382 to 396 us at
// 5.6 TB/s (2.1 to 2.2 GB); one token 74 (308 MB, 60 us at the rate of a copy), the
// rest the routing (1.9 us), the list (0.8), the hand-over of cut tiles (2.2 each
// launch) and the gap between the launches (1.4).  The operators one by one (route,
// two products, combine) take 78 for one token, 394 for 16 in 382; of 256 experts
// under a biased sigmoid, F 256, 44 for one token in 38, 204 for 16 in 174.
//
// With so few tokens a tile's rows are the tokens themselves, all of them for
// every expert: the matrix cores have rows to spare, and nothing is gathered or
// grouped.  (A second row block, for 32 tokens, took 450 us where two calls took
// 423.)
// Every workgroup routes all tokens by itself (16 lanes a token, as moe_route),
// which costs less than a launch before it.
//
// Work is dealt as in stream_kernel (grouped.hpp): the K-quads of all tiles are
// one line that the workgroups take in equal pieces, each wave streams its steps
// through a ring in LDS of its own, and the last workgroup to arrive at a cut
// tile adds the pieces in the order of K.  In the second kernel a tile's K is
// that of all experts in use, one after the other; at an expert's end its sums
// enter the totals of the rows that chose it, times the weight, so that no other
// row is touched by what the expert's weights hold.
#pragma once

#include "choose.hpp"
#include "fp8_gemm.hpp"
#include "grouped.hpp"

namespace gc {

constexpr int ML_TOKENS = 16, ML_PAIRS = ML_TOKENS * RT_TOP;
constexpr int ML_THREADS = 256, ML_WAVES = 4, ML_NB = 8, ML_D = 3;

struct LayerArgs {
    RouteArgs route;
    uint32_t *chosen;          // a Chosen, workspace
    const uint16_t *X;         // [T][K]
    const uint16_t *W1;        // [local][K][2 F]
    const uint16_t *W2;        // [local][F][N]
    uint16_t *a;               // [T * k][F], workspace
    const uint16_t *partials;  // npeers blocks of [T][N], peer_stride elements apart
    int64_t peer_stride;
    int npeers;
    uint16_t *out;             // [T][N]
    int first, local;          // experts here
    int T, K, F, N;
    int tiles_n;
    int min_quads;
    float *part;               // as in GroupedArgs
    uint32_t *count;
    int part_slots;
};

// Which tokens chose which of the experts here; the first kernel leaves it for
// the second.
struct Chosen {
    float w[ML_PAIRS];                   // weights [T][k]
    int8_t slot[ML_PAIRS][ML_TOKENS];    // (place in the list, token): the token's choice that it is, or -1
    int16_t list[ML_PAIRS];              // experts in use, rising
    int32_t n;                           // experts in use
};
constexpr int ML_WORDS = sizeof(Chosen) / 4;

struct Choice {
    Chosen kept;
    uint32_t rows[RT_GROUPS];            // tokens of an expert, a bit each
    int16_t place[RT_GROUPS];            // an expert's place in the list
    int id[ML_PAIRS];
};

// From the ids of all T * k pairs, in LDS: the rest.
__device__ __forceinline__ void list_experts(Choice &x, int T, int k, int first, int local)
{
    Chosen &c = x.kept;
    const int tid = threadIdx.x, lane = tid & 63;
    for (int e = tid; e < local; e += ML_THREADS)
        x.rows[e] = 0u;
    __syncthreads();
    for (int i = tid; i < T * k; i += ML_THREADS) {
        const int e = x.id[i] - first;
        if (x.id[i] >= 0 && (unsigned)e < (unsigned)local)
            atomicOr(&x.rows[e], 1u << (i / k));
    }
    __syncthreads();
    if (tid < 64) {
        int n = 0;
        for (int e0 = 0; e0 < local; e0 += 64) {
            const int e = e0 + lane;
            const bool in = e < local && x.rows[e] != 0u;
            const uint64_t all = __builtin_amdgcn_ballot_w64(in);
            if (in) {
                const int at = n + __builtin_popcountll(all & ((1ull << lane) - 1ull));
                c.list[at] = (int16_t)e;
                x.place[e] = (int16_t)at;
            }
            n += __builtin_popcountll(all);
        }
        if (lane == 0)
            c.n = n;
    }
    __syncthreads();
    const int words = c.n * (ML_TOKENS / 4);
    for (int i = tid; i < words; i += ML_THREADS)
        ((uint32_t *)c.slot)[i] = ~0u;
    __syncthreads();
    for (int i = tid; i < T * k; i += ML_THREADS) {
        const int e = x.id[i] - first;
        if (x.id[i] >= 0 && (unsigned)e < (unsigned)local)
            c.slot[x.place[e]][i / k] = (int8_t)(i % k);
    }
    __syncthreads();
}

template <int LPT, int V, bool BF16>
__device__ __forceinline__ void route_all(const RouteArgs &p, Choice &x)
{
    constexpr int PER = ML_THREADS / LPT;
    using Pair = std::conditional_t<BF16, NarrowPair, WidePair>;
    const int j = threadIdx.x % LPT;
    for (int tb = 0; tb < p.T; tb += PER) {
        const int t = tb + threadIdx.x / LPT, tl = min(t, p.T - 1);
        int id;
        float w;
        if (BF16 && p.bias)
            route_token<LPT, V, BF16, false, WidePair>(p, tl, j, id, w);
        else if (p.vec)
            route_token<LPT, V, BF16, true, Pair>(p, tl, j, id, w);
        else
            route_token<LPT, V, BF16, false, Pair>(p, tl, j, id, w);
        if (j < p.k && t < p.T) {
            x.id[t * p.k + j] = id;
            x.kept.w[t * p.k + j] = w;
        }
    }
    __syncthreads();
}

// The four waves' sums of RB * NB blocks through LDS, and over the pieces of a
// tile that is cut: block b's sum by block(b), or by final(x, at, n) once the
// last workgroup is here.  (As at the end of stream_kernel's tiles.)
struct TileSums {
    static constexpr int NB = ML_NB, BLOCK = NB * 1024;
    f32x4_t *sums;
    __amdgpu_buffer_rsrc_t rp;
    uint32_t *count;
    int lane, wave;
    bool live;                           // the lane's row is a token's
    bool cut;
    int w_first, w_last;

    __device__ __forceinline__ void put(const f32x4_t (&x)[NB])
    {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NB; ++j)
            sums[(wave * NB + j) * 64 + lane] = x[j];
        __syncthreads();
    }
    __device__ __forceinline__ f32x4_t block(int b) const
    {
        f32x4_t x = sums[b * 64 + lane];
#pragma unroll
        for (int w = 1; w < ML_WAVES; ++w)
            x += sums[(w * NB + b) * 64 + lane];
        return x;
    }
    // Hands piece v of the tile of quads [t0, t0 + per_tile) over; whether it is
    // the last to arrive (or the tile is not cut).
    __device__ __forceinline__ bool hand_over(const Line &line, int64_t t0, int v, int ka, int kb, int *s_last)
    {
        cut = ka > 0 || kb < line.per_tile;
        w_first = w_last = v;
        if (!cut)
            return true;
        w_first = line.piece_of(t0);
        w_last = line.piece_of(t0 + line.per_tile - 1);
        const uint32_t slot = (uint32_t)(2 * v + (ka == 0 ? 1 : 0));
        for (int b = wave; b < NB; b += ML_WAVES) {
            const f32x4_t x = block(b);
            if (live)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, x), rp,
                                                       (int)(slot * BLOCK + (uint32_t)(b * 1024 + lane * 16)), 0,
                                                       CPOL_SYS);
        }
        wait_vmcnt<0>();
        __syncthreads();
        if (threadIdx.x == 0) {
            const uint32_t n = __hip_atomic_fetch_add(count + w_first, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
            const int last = (int)n == w_last - w_first;
            if (last)           // everybody has been: the counter is free again
                __hip_atomic_store(count + w_first, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
            *s_last = last;
        }
        __syncthreads();
        const bool mine = __builtin_amdgcn_readfirstlane(*s_last) != 0;
        __syncthreads();
        return mine;
    }
    template <int N>
    __device__ __forceinline__ void final(f32x4_t (&x)[N], const int (&at)[N]) const
    {
        if (!cut) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                x[i] = block(at[i]);
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        // AHEAD pieces at a time, in order: every turn is a trip to memory
        constexpr int AHEAD = 4;
        for (int w0 = w_first; w0 <= w_last; w0 += AHEAD) {
            f32x4_t y[AHEAD][N];
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                const int w = w0 + d;
                const uint32_t slot = (uint32_t)(2 * w + (w == w_first ? 1 : 0));
                // (past the last piece: past the buffer)
                const uint32_t from = live && w <= w_last ? slot * BLOCK + (uint32_t)(lane * 16) : OOB;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    y[d][i] = __builtin_bit_cast(
                        f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(from + (uint32_t)(at[i] * 1024)), 0, CPOL_SYS));
            }
#pragma unroll
            for (int d = 0; d < AHEAD; ++d)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    x[i] += y[d][i];
        }
    }
};

// One K-step of a wave from the ring's slot `at`: rows of X against 128 columns.
__device__ __forceinline__ void ring_step(uint32_t at, const uint32_t (&b_frag)[ML_NB], uint32_t a_frag,
                                          f32x4_t (&acc)[ML_NB])
{
    bf16x8_t fa[ML_NB];
#pragma unroll
    for (int j = 0; j < ML_NB; ++j) {
        bf16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t *)lds_ptr<bf16x4_t>(at + b_frag[j]));
        bf16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
            (lds_bf16x4_t *)lds_ptr<bf16x4_t>(at + b_frag[j] + 4 * 256));
        fa[j] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    const bf16x8_t fb = *lds_ptr<bf16x8_t>(at + a_frag);
#pragma unroll
    for (int j = 0; j < ML_NB; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[j], fb, acc[j], 0, 0, 0);
}

// Lane constants of a ring of NB = 8 (see stream_kernel): the 32-byte chunk c
// of row k of the weights is kept at c ^ fold(k).
__device__ __forceinline__ int ring_fold(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }

// LPT, V: lanes of a token and experts of a lane in the router.
template <int LPT, int V, bool BF16>
__global__ __launch_bounds__(ML_THREADS) void moe_up_kernel(LayerArgs p)
{
    constexpr int NB = ML_NB, D = ML_D, B_SLOT = NB * 1024, SLOT = B_SLOT + 1024, LOADS = NB + 1;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[ML_WAVES * D * SLOT];
    __shared__ Choice x;
    Chosen &c = x.kept;
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fi = lane & 15, fg = lane >> 4;
    const int k = p.route.k;

    route_all<LPT, V, BF16>(p.route, x);
    list_experts(x, p.T, k, p.first, p.local);
    if (blockIdx.x == 0) {
        for (int i = tid; i < ML_WORDS; i += ML_THREADS)
            p.chosen[i] = ((const uint32_t *)&c)[i];
    }
    const int tiles = __builtin_amdgcn_readfirstlane(c.n) * p.tiles_n;
    if (tiles <= 0)
        return;
    const int KT = (p.K + BK - 1) / BK;
    const Line line(tiles, max((KT + ML_WAVES - 1) / ML_WAVES, 1), p.min_quads, min((int)gridDim.x, p.part_slots / 2));
    if ((int)blockIdx.x >= line.pieces)
        return;
    const int v = xcd_remap(blockIdx.x, line.pieces);
    int64_t q = line.bound(v);
    const int64_t q_end = line.bound(v + 1);

    const int b_row = lane / 16, b_slot = lane % 16;
    const int a_c = (lane & 3) ^ ((lane >> 3) & 3);
    const int f_lane = ring_fold(8 * fg + (fi >> 2));
    uint32_t b_frag[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        b_frag[j] = (uint32_t)((8 * fg + (fi >> 2)) * 256 + 8 * (fi & 3) + ((j ^ f_lane) * 32));
    const uint32_t a_frag = (uint32_t)(B_SLOT + fi * 64 + ((fg ^ ((fi >> 1) & 3)) << 4));
    const uint32_t my_ring = lds_addr(ring) + (uint32_t)(wave * D * SLOT);
    const uint32_t N2 = (uint32_t)p.F * 4u;              // bytes of a row of W1
    const u32x4_t rX = make_rsrc4(p.X, (uint32_t)p.T * (uint32_t)p.K * 2u);
    const int a_tok = lane >> 2;
    const uint32_t a_off = a_tok < p.T ? ((uint32_t)a_tok * (uint32_t)p.K + (uint32_t)(8 * a_c)) * 2u : OOB;
    TileSums ts;
    ts.sums = (f32x4_t *)ring;
    ts.rp = make_rsrc(p.part, (uint32_t)p.part_slots * (uint32_t)TileSums::BLOCK);
    ts.count = p.count;
    ts.lane = lane;
    ts.wave = wave;
    ts.live = fi < p.T;

    while (q < q_end) {
        const int t = (int)(q / line.per_tile);
        const int ka = (int)(q - (int64_t)t * line.per_tile);
        const int kb = (int)min((int64_t)line.per_tile, ka + (q_end - q));
        q += kb - ka;
        const int at_list = t / p.tiles_n, nt = t - at_list * p.tiles_n;
        const int e = __builtin_amdgcn_readfirstlane((int)c.list[at_list]);
        const u32x4_t rW = make_rsrc4(p.W1 + (size_t)e * p.K * (2 * (size_t)p.F), (uint32_t)p.K * N2);
        uint32_t b_off[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int kr = i * 4 + b_row;
            const int col = 16 * ((b_slot >> 1) ^ ring_fold(kr)) + 8 * (b_slot & 1);
            const int h = nt * 64 + (col & 63), n = col < 64 ? h : p.F + h;
            b_off[i] = h < p.F ? (uint32_t)kr * N2 + (uint32_t)n * 2u : OOB;
        }
        const int s1 = min(ML_WAVES * kb, KT);
        auto issue = [&](int s, uint32_t slot) {
            const int k0 = s * BK;
            const bool on = s < s1, whole = on && k0 + 8 * a_c < p.K;
            const uint32_t at = my_ring + slot * SLOT;
#pragma unroll
            for (int i = 0; i < NB; ++i)
                dma16(rW, at + i * 1024, on ? b_off[i] + (uint32_t)k0 * N2 : OOB);
            dma16(rX, at + B_SLOT, whole ? a_off + (uint32_t)k0 * 2u : OOB);
        };
        f32x4_t acc[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        int s = ML_WAVES * ka + wave;
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            issue(s + ML_WAVES * d, d);
        uint32_t cur = 0;
        for (; s < s1; s += ML_WAVES) {
            wait_lgkmcnt0();                     // the slot to be refilled is read
            issue(s + ML_WAVES * (D - 1), cur == 0 ? D - 1 : cur - 1);
            wait_vmcnt<(D - 1) * LOADS>();       // this step's loads have landed
            ring_step(my_ring + cur * SLOT, b_frag, a_frag, acc);
            cur = cur == D - 1 ? 0 : cur + 1;
        }
        wait_vmcnt<0>();
        ts.put(acc);
        if (!ts.hand_over(line, (int64_t)t * line.per_tile, v, ka, kb, &s_last))
            continue;
        // Gate and up blocks of 32 columns: two pairs, a wave each.
        const int j = 2 * (wave & 1);
        f32x4_t y[4];
        ts.final(y, {j, j + 1, j + NB / 2, j + NB / 2 + 1});
        const u32x4_t pk = pack_pair(silu_mul(y[0], y[2]), silu_mul(y[1], y[3]));
        const int col = nt * 64 + 16 * j + pair_col(fg);
        if (wave < 2 && fi < p.T && col < p.F) {
            const int slot = c.slot[at_list][fi];
            if (slot >= 0)
                *(u32x4_t *)(p.a + (size_t)(fi * k + slot) * p.F + col) = pk;
        }
        __syncthreads();                         // the ring is free for the next tile
    }
}

__global__ __launch_bounds__(ML_THREADS) void moe_down_kernel(LayerArgs p)
{
    constexpr int NB = ML_NB, D = ML_D, B_SLOT = NB * 1024, SLOT = B_SLOT + 1024, LOADS = NB + 1;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[ML_WAVES * D * SLOT];
    __shared__ Chosen c;
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fi = lane & 15, fg = lane >> 4;
    const int k = p.route.k;
    for (int i = tid; i < ML_WORDS; i += ML_THREADS)
        ((uint32_t *)&c)[i] = p.chosen[i];
    __syncthreads();
    const int used = __builtin_amdgcn_readfirstlane(c.n);
    const int KT = (p.F + BK - 1) / BK, quads = max((KT + ML_WAVES - 1) / ML_WAVES, 1);   // of one expert
    // (no expert: the tiles are still written, from the peers alone)
    const Line line(p.tiles_n, max(used * quads, 1), p.min_quads, min((int)gridDim.x, p.part_slots / 2));
    if ((int)blockIdx.x >= line.pieces)
        return;
    const int v = xcd_remap(blockIdx.x, line.pieces);
    int64_t q = line.bound(v);
    const int64_t q_end = line.bound(v + 1);

    const int b_row = lane / 16, b_slot = lane % 16;
    const int a_c = (lane & 3) ^ ((lane >> 3) & 3);
    const int f_lane = ring_fold(8 * fg + (fi >> 2));
    uint32_t b_frag[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        b_frag[j] = (uint32_t)((8 * fg + (fi >> 2)) * 256 + 8 * (fi & 3) + ((j ^ f_lane) * 32));
    const uint32_t a_frag = (uint32_t)(B_SLOT + fi * 64 + ((fg ^ ((fi >> 1) & 3)) << 4));
    const uint32_t my_ring = lds_addr(ring) + (uint32_t)(wave * D * SLOT);
    const uint32_t N2 = (uint32_t)p.N * 2u;
    const u32x4_t rA = make_rsrc4(p.a, (uint32_t)(p.T * k) * (uint32_t)p.F * 2u);
    TileSums ts;
    ts.sums = (f32x4_t *)ring;
    ts.rp = make_rsrc(p.part, (uint32_t)p.part_slots * (uint32_t)TileSums::BLOCK);
    ts.count = p.count;
    ts.lane = lane;
    ts.wave = wave;
    ts.live = fi < p.T;

    while (q < q_end) {
        const int t = (int)(q / line.per_tile);
        const int ka = (int)(q - (int64_t)t * line.per_tile);
        const int kb = (int)min((int64_t)line.per_tile, ka + (q_end - q));
        q += kb - ka;
        uint32_t b_off[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int kr = i * 4 + b_row;
            const int n = t * 128 + 16 * ((b_slot >> 1) ^ ring_fold(kr)) + 8 * (b_slot & 1);
            b_off[i] = n < p.N ? (uint32_t)kr * N2 + (uint32_t)n * 2u : OOB;
        }
        // Quad qi of the tile: step 4 (qi % quads) + wave of expert qi / quads of the list.
        const int q1 = used > 0 ? kb : 0;
        int ahead = -1, ahead_q = ka, ahead_s = 0;       // loads: expert, quad, step
        u32x4_t rW = {0u, 0u, 0u, 0u};
        uint32_t a_off = OOB;
        const int a_tok = lane >> 2;
        auto issue = [&](uint32_t slot) {
            const bool on = ahead_q < q1;
            if (on) {
                const int g = ahead_q / quads;
                ahead_s = ML_WAVES * (ahead_q - g * quads) + wave;
                if (g != ahead) {
                    ahead = g;
                    const int e = __builtin_amdgcn_readfirstlane((int)c.list[g]);
                    rW = make_rsrc4(p.W2 + (size_t)e * p.F * p.N, (uint32_t)p.F * N2);
                    const int j = a_tok < p.T ? c.slot[g][a_tok] : -1;
                    a_off = j >= 0 ? ((uint32_t)(a_tok * k + j) * (uint32_t)p.F + (uint32_t)(8 * a_c)) * 2u : OOB;
                }
            }
            ++ahead_q;
            const int k0 = ahead_s * BK;
            const bool live = on && ahead_s < KT, whole = live && k0 + 8 * a_c < p.F;
            const uint32_t at = my_ring + slot * SLOT;
            // (the same in all lanes, which the compiler does not see here)
            const u32x4_t r = {(uint32_t)__builtin_amdgcn_readfirstlane((int)rW[0]),
                               (uint32_t)__builtin_amdgcn_readfirstlane((int)rW[1]),
                               (uint32_t)__builtin_amdgcn_readfirstlane((int)rW[2]), (uint32_t)BUFFER_FLAGS};
#pragma unroll
            for (int i = 0; i < NB; ++i)
                dma16(r, at + i * 1024, live ? b_off[i] + (uint32_t)k0 * N2 : OOB);
            dma16(rA, at + B_SLOT, whole ? a_off + (uint32_t)k0 * 2u : OOB);
        };
        f32x4_t acc[NB], total[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n)
            acc[n] = total[n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        // The sums of expert g of the list enter the rows that chose it.
        auto flush = [&](int g) {
            const int j = fi < p.T ? c.slot[g][fi] : -1;
            const float w = j >= 0 ? c.w[fi * k + j] : 0.f;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    total[n][d] = j >= 0 ? total[n][d] + w * acc[n][d] : total[n][d];
                acc[n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
            }
        };
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            issue(d);
        uint32_t cur = 0;
        int in = ka % quads, g = ka / quads;
        for (int qi = ka; qi < q1; ++qi) {
            wait_lgkmcnt0();
            issue(cur == 0 ? D - 1 : cur - 1);
            wait_vmcnt<(D - 1) * LOADS>();
            ring_step(my_ring + cur * SLOT, b_frag, a_frag, acc);
            cur = cur == D - 1 ? 0 : cur + 1;
            if (++in == quads || qi + 1 == q1) {
                flush(g);
                in = 0;
                ++g;
            }
        }
        wait_vmcnt<0>();
        ts.put(total);
        if (!ts.hand_over(line, (int64_t)t * line.per_tile, v, ka, kb, &s_last))
            continue;
        // Pairs of 32 columns, a wave each.
        const int j = 2 * wave;
        f32x4_t x[2];
        ts.final(x, {j, j + 1});
        float o[8];
        pair_f32(x[0], x[1], o);
        const int col = t * 128 + 16 * j + pair_col(fg);
        if (fi < p.T && col < p.N) {
            const int64_t to = (int64_t)fi * p.N + col;
            add_peers(o, p.partials, p.peer_stride, p.npeers, to);
            *(u32x4_t *)(p.out + to) = pack_bf16x8(o);
        }
        __syncthreads();                         // the ring is free for the next tile
    }
}

}  // namespace gc
