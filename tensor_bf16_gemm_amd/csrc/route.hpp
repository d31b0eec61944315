// route.hpp -- gfx950 device code of the expert router and of the grouping of
// row indices by a small integer (expert of a routed pair, adapter of a row).
//
// Router: for every token the k experts of largest key, in falling order
// (equal keys: the lower index first), where the key is the logit or, with a
// selection bias, score + bias; the score is softmax(logits) or
// sigmoid(logit) in fp32.  A logit of NaN or -inf is never chosen; a place
// that is left over gets id -1 and weight 0.
//
// A token is a row of 16 lanes (four tokens per wave) for up to 256 experts,
// else a whole wave; each lane holds V experts.  A (key, index)
// pair is packed into one number -- an order-preserving key, then the index
// counted downwards -- so that one maximum compares both and no two are
// equal: 16 + 16 bits of a word for bf16 logits, else 32 + 20 bits of the
// mantissa of a double in [1, 2).  Every lane sorts its V pairs once (a
// network of min/max); a round of the choice is then a maximum over the
// lanes' heads (four row rotations) and the winner's lane moves its list up
// by one.  The issue rate bounds it: 16384 tokens of 256 bf16 logits, k = 8,
// take 7.7 us here, and took 16.8 us with a whole wave per token and a scan of
// its keys in every round.
//
// Grouping: a stable counting sort by blocks of consecutive items.  Counts
// per block first (LDS integer atomics: order does not matter to a sum), then
// every block adds up the counts of the blocks before it by itself -- 256
// rows of 2-byte counts, read from the L2 -- which costs less than a scan
// launch between the two kernels would (the same 131072 pairs: 7 us).  Inside a
// block, the items of a wave that share a group find one another with one
// ballot per bit of the group number.  Up to ROUTE_ONE_ITEMS items of few tokens
// take one workgroup and one launch for everything (64 tokens of 64 experts,
// k = 8: 5.8 us, of which launch and memory latencies are most).
#pragma once

#include "choose.hpp"

namespace gc {

constexpr int RT_THREADS = 1024, RT_WAVES = RT_THREADS / 64;
constexpr int RT_BLOCKS = 256;           // blocks of a many-block grouping, unless
constexpr int RT_ITEMS = 8191;           // a block's items were more than this (8 counts add up in 16 bits)
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
// Items that one workgroup routes and groups in a single launch.
constexpr int ROUTE_ONE_ITEMS = 1024;

// Inclusive prefix sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    return v;
}

// LDS of the grouping.
struct GroupLds {
    int base[RT_GROUPS + 8];                 // next position of every group
    int total[RT_GROUPS + 8];
    int wave_at[RT_WAVES][RT_GROUPS + 1];    // a pass: counts, then positions, per wave
    int wave_sum[RT_WAVES];
    int grouped_before, none;                // items before the block in a group; next position of those in none
};

// Exclusive prefix sum of v over threads 0 .. RT_THREADS - 1, and the whole
// sum (one barrier).
__device__ __forceinline__ int block_scan(GroupLds &l, int v, int &all)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int inc = wave_scan(v);
    if (lane == 63)
        l.wave_sum[wave] = inc;
    __syncthreads();
    int before = 0;
    all = 0;
    for (int w = 0; w < RT_WAVES; ++w) {
        if (w < wave)
            before += l.wave_sum[w];
        all += l.wave_sum[w];
    }
    return before + inc - v;
}

__device__ __forceinline__ void clear_wave_at(GroupLds &l, int waves, int groups)
{
    for (int w = 0; w < waves; ++w)
        for (int e = threadIdx.x; e <= groups; e += RT_THREADS)
            l.wave_at[w][e] = 0;
}

// Rank of the lane's item among the earlier items of its wave in the same
// group g, the group's count in the wave written to l.wave_at (cleared
// before): one ballot per bit of the group number.
__device__ __forceinline__ int rank_in_wave(GroupLds &l, bool live, int g, int groups)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int bits = 32 - __builtin_clz(groups);       // groups itself is a value
    uint64_t same = __builtin_amdgcn_ballot_w64(live);
    for (int b = 0; b < bits; ++b) {
        const uint64_t on = __builtin_amdgcn_ballot_w64((g >> b) & 1);
        same &= (g >> b) & 1 ? on : ~on;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1ull));
    if (live && rank == 0)
        l.wave_at[wave][g] = __builtin_popcountll(same);
    return rank;
}

// Counts of group e in the waves to positions from `at` on; returns the next.
__device__ __forceinline__ int counts_to_positions(GroupLds &l, int waves, int e, int at)
{
    int c[RT_WAVES];                                     // (all read before any is written)
#pragma unroll
    for (int w = 0; w < RT_WAVES; ++w)
        c[w] = w < waves ? l.wave_at[w][e] : 0;
#pragma unroll
    for (int w = 0; w < RT_WAVES; ++w) {
        if (w < waves)
            l.wave_at[w][e] = at;
        at += c[w];
    }
    return at;
}

__device__ __forceinline__ void place(const RouteArgs &p, int flat, int g, int pos)
{
    p.rows[pos] = (int)((unsigned)flat / (unsigned)p.per_row);
    p.slots[flat] = g == p.E ? -1 : pos;
}

// Group of an id from outside: ids past the groups are in none.
__device__ __forceinline__ int group_of(int id, int groups)
{
    return (unsigned)id < (unsigned)groups ? id : groups;
}

// Routes the tokens of this block (V > 0) or reads their ids (V == 0),
// then: ONE (a single workgroup, at most ROUTE_ONE_ITEMS items) groups them,
// else counts them per group.
template <int LPT, int V, bool BF16, bool ONE>
__global__ __launch_bounds__(RT_THREADS) void route_kernel(RouteArgs p)
{
    static_assert(ROUTE_ONE_ITEMS <= RT_THREADS, "one item per thread");
    __shared__ GroupLds l;
    __shared__ int s_id[ONE ? ROUTE_ONE_ITEMS : 1];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = ONE ? 0 : blockIdx.x * p.block_tokens;
    const int t1 = ONE ? p.T : min(p.T, t0 + p.block_tokens);
    const bool group = p.offsets != nullptr;
    const int n = p.T * p.k, waves = (n + 63) / 64;      // (ONE)
    if (group) {
        if (ONE) {
            clear_wave_at(l, waves, p.E);
        } else {
            for (int e = tid; e <= p.E; e += RT_THREADS)
                l.total[e] = 0;
            __syncthreads();
        }
    }
    if constexpr (V > 0) {
        constexpr int PER = RT_THREADS / LPT;            // tokens at a time
        const int j = tid % LPT;
        for (int tb = t0; tb < t1; tb += PER) {
            const int t = tb + tid / LPT;
            if (tb + wave * (64 / LPT) >= t1)
                break;                                   // no token in this wave
            int id;
            float w;
            const int tl = min(t, t1 - 1);
            if constexpr (BF16) {
                if (p.bias)
                    route_token<LPT, V, BF16, false, WidePair>(p, tl, j, id, w);
                else if (p.vec)
                    route_token<LPT, V, BF16, true, NarrowPair>(p, tl, j, id, w);
                else
                    route_token<LPT, V, BF16, false, NarrowPair>(p, tl, j, id, w);
            } else {
                if (p.vec)
                    route_token<LPT, V, BF16, true, WidePair>(p, tl, j, id, w);
                else
                    route_token<LPT, V, BF16, false, WidePair>(p, tl, j, id, w);
            }
            if (j < p.k && t < t1) {
                const int flat = t * p.k + j;
                p.ids[flat] = id;
                p.weights[flat] = w;
                if (group) {
                    const int g = id < 0 ? p.E : id;
                    if (ONE)
                        s_id[flat] = g;
                    else
                        atomicAdd(&l.total[g], 1);
                }
            }
        }
    } else {
        for (int i = t0 * p.k + tid; i < t1 * p.k; i += RT_THREADS) {
            const int g = group_of(p.ids[i], p.E);
            if (ONE)
                s_id[i] = g;
            else
                atomicAdd(&l.total[g], 1);
        }
    }
    if (!group)
        return;
    __syncthreads();
    if constexpr (ONE) {
        const bool live = tid < n;
        const int g = live ? s_id[tid] : 0;
        const int rank = rank_in_wave(l, live, g, p.E);
        __syncthreads();
        int sum = 0, all;
        if (tid < p.E) {
#pragma unroll
            for (int w = 0; w < RT_WAVES; ++w)
                sum += w < waves ? l.wave_at[w][tid] : 0;
        }
        const int at = block_scan(l, sum, all);
        if (tid < p.E) {
            counts_to_positions(l, waves, tid, at);
            p.offsets[tid] = at;
        }
        if (tid == RT_THREADS - 1) {
            counts_to_positions(l, waves, p.E, all);
            p.offsets[p.E] = all;
        }
        __syncthreads();
        if (live)
            place(p, tid, g, l.wave_at[wave][g] + rank);
    } else {
        for (int e = tid; e < p.cstride; e += RT_THREADS)
            p.counts[(int64_t)blockIdx.x * p.cstride + e] = e < p.E ? (uint16_t)l.total[e] : (uint16_t)0;
    }
}

// Second kernel of a many-block grouping: positions of this block's items.
__global__ __launch_bounds__(RT_THREADS) void place_kernel(RouteArgs p)
{
    __shared__ GroupLds l;
    const int tid = threadIdx.x, wave = tid >> 6;
    const int blocks = gridDim.x, b = blockIdx.x;
    for (int e = tid; e < p.cstride; e += RT_THREADS) {
        l.base[e] = 0;
        l.total[e] = 0;
    }
    if (tid == 0)
        l.grouped_before = 0;
    const int first = b * p.block_tokens * p.k;
    const int n = (min(p.T, (b + 1) * p.block_tokens) - b * p.block_tokens) * p.k;
    auto group_at = [&](int i) { return i < n ? group_of(p.ids[first + i], p.E) : 0; };
    int g = group_at(tid);                               // (asked for before the counts)
    __syncthreads();
    // Counts of the blocks before this one (base) and of all (total): a
    // thread adds 8 neighbouring groups over every per_pass-th block.  In the
    // LDS, group 8 c + i is kept at i * lanes + c, so that the lanes of an
    // addition, whose c differ, fall into different banks.
    const int lanes = p.cstride / 8, per_pass = RT_THREADS / lanes;
    const int r0 = tid / lanes, c = tid - r0 * lanes;
    int before = 0;
    if (r0 < per_pass) {
        constexpr int AHEAD = 8;                         // rows asked for at once
        int pre[8] = {}, tot[8] = {};
        for (int q = r0; q < blocks; q += AHEAD * per_pass) {
            u32x4_t v[AHEAD];
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                const int r = q + d * per_pass;
                v[d] = *(const u32x4_t *)(p.counts + (int64_t)min(r, blocks - 1) * p.cstride + 8 * c);
            }
            // two counts a word: AHEAD of them stay below 2^16
            u16x2_t pre2[4] = {}, tot2[4] = {};
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                const int r = q + d * per_pass;
                const uint32_t in = r < blocks ? ~0u : 0u, early = r < b ? ~0u : 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    tot2[i] += __builtin_bit_cast(u16x2_t, v[d][i] & in);
                    pre2[i] += __builtin_bit_cast(u16x2_t, v[d][i] & early);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                tot[i] += tot2[i >> 1][i & 1];
                pre[i] += pre2[i >> 1][i & 1];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            atomicAdd(&l.total[i * lanes + c], tot[i]);
            atomicAdd(&l.base[i * lanes + c], pre[i]);
            before += pre[i];
        }
    }
    // What the blocks before have in no group is the rest of their items.
    before = wave_scan(before);
    if ((tid & 63) == 63)
        atomicAdd(&l.grouped_before, before);
    __syncthreads();
    auto kept = [&](int e) { return (e & 7) * lanes + (e >> 3); };
    int all;
    const int at = block_scan(l, tid < p.E ? l.total[kept(tid)] : 0, all);
    if (tid < p.E) {
        l.base[kept(tid)] += at;
        if (b == 0)
            p.offsets[tid] = at;
    }
    if (tid == RT_THREADS - 1) {
        l.none = all + first - l.grouped_before;
        if (b == 0)
            p.offsets[p.E] = all;
    }
    for (int i0 = 0; i0 < n; i0 += RT_THREADS) {
        const int waves = min(RT_WAVES, (n - i0 + 63) / 64);
        clear_wave_at(l, waves, p.E);
        const bool live = i0 + tid < n;
        if (i0 > 0)
            g = group_at(i0 + tid);
        __syncthreads();
        const int rank = rank_in_wave(l, live, g, p.E);
        __syncthreads();
        if (tid < p.E)
            l.base[kept(tid)] = counts_to_positions(l, waves, tid, l.base[kept(tid)]);
        if (tid == RT_THREADS - 1)
            l.none = counts_to_positions(l, waves, p.E, l.none);
        __syncthreads();
        if (live)
            place(p, first + i0 + tid, g, l.wave_at[wave][g] + rank);
        __syncthreads();
    }
}

}  // namespace gc
