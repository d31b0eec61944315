// route.hpp -- gfx950 device code of the expert router and of the grouping of
// row indices by a small integer (expert of a routed pair, adapter of a row).
//
// Router: for every token the k experts of largest key, in falling order
// (equal keys: the lower index first), where the key is the logit or, with a
// selection bias, score + bias; the score is softmax(logits) or
// sigmoid(logit) in fp32.  A logit of NaN or -inf is never chosen; a place
// that is left over gets id -1 and weight 0.
//
// One wave per token: lane l holds the VPL consecutive experts VPL*l ..
// VPL*l + VPL-1 as order-preserving 32-bit keys, so "lowest index first" is
// "lowest lane first".  Each of the k rounds is one maximum over the wave
// (six DPP steps), one ballot, and the removal of the winner; nothing is
// sorted and nothing leaves the registers.
//
// Grouping: a stable counting sort by blocks of consecutive items.  Counts
// per block first (LDS integer atomics: order does not matter to a sum), then
// every block adds up the counts of the blocks before it by itself -- at
// most 256 rows of 2-byte counts, read from the L2 -- which costs
// less than a scan launch between the two kernels would.  Inside a block,
// the items of a wave that share a group find one another with one ballot per
// bit of the group number.  Up to ROUTE_ONE_ITEMS items take one workgroup and
// one launch for everything.
#pragma once

#include "gc_kernel.hpp"

namespace gc {

constexpr int RT_THREADS = 1024, RT_WAVES = RT_THREADS / 64;
constexpr int RT_GROUPS = 1024;          // groups (experts, adapters) at most
constexpr int RT_BLOCKS = 256;           // blocks of a many-block grouping at most
constexpr int RT_TOP = 16;               // k at most
// Items that one workgroup routes and groups in a single launch.
constexpr int ROUTE_ONE_ITEMS = 1024;

enum Score { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };

struct RouteArgs {
    const void *logits;      // [T] rows of E, row stride `stride` elements
    int64_t stride;
    const float *bias;       // [E] or null
    int T, E, k;
    int score, renorm;
    float scale;
    int32_t *ids;            // [T][k]
    float *weights;          // [T][k]
    // grouping (null offsets: none)
    int32_t *offsets;        // [E + 1]
    int32_t *rows;           // [T * k]
    int32_t *slots;          // [T * k]
    uint16_t *counts;        // [blocks][cstride]
    int cstride;             // E + 1 rounded up to 8
    int block_tokens;        // tokens (items / k) per block
    bool vec;                // a lane's VPL logits are whole aligned vectors
};

// Lane 63 of the wave's running maximum / sum (DPP row shifts, then the two
// row broadcasts), as a uniform value.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    auto mx = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));
    v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
    v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
    v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
    v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));
    v = mx(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
}

__device__ __forceinline__ float wave_sum(float v)
{
    v = dpp_add<0x111, 0xf>(v);
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);
    v = dpp_add<0x143, 0xc>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

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

// fp32 -> uint32 with the same order (-0 and +0 alike); NaN becomes -inf.
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (!(x == x))
        return KEY_NEG_INF;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// e^(x - high), the terms of a softmax whose maximum is `high`; with an
// infinite maximum the infinite terms share the weight equally.
__device__ __forceinline__ float soft_term(float x, float high)
{
    if (high == __builtin_huge_valf())
        return x == high ? 1.0f : 0.0f;
    return expf(x - high);
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Tokens that a wave routes side by side: a round is a chain of some twenty
// dependent steps (the maximum over the wave, the ballot, the removal), which
// one token alone would wait through.
template <int VPL>
constexpr int ROUTE_TOK = VPL <= 4 ? 4 : VPL == 8 ? 2 : 1;

// Routes tokens t, t + RT_WAVES, ... (those below t1) in one wave.  Lane j < k
// returns with the j-th choice's expert (-1: none) in id[] and its weight in w[].
template <int VPL, bool BF16, int TOK>
__device__ __forceinline__ void route_tokens(const RouteArgs &p, int t, int t1, int lane, int (&id)[TOK],
                                             float (&w)[TOK])
{
    const int e0 = lane * VPL;
    const bool soft = p.score == SCORE_SOFTMAX;
    float x[TOK][VPL], high[TOK], val[TOK];
    uint32_t key[TOK][VPL];
#pragma unroll
    for (int q = 0; q < TOK; ++q) {
        const int tq = t + q * RT_WAVES;
        const bool live = tq < t1;
        if constexpr (BF16) {
            const uint16_t *row = (const uint16_t *)p.logits + (int64_t)(live ? tq : t) * p.stride;
            uint16_t b[VPL];
            if (p.vec && e0 < p.E) {
                __builtin_memcpy(b, __builtin_assume_aligned(row + e0, VPL * 2 < 16 ? VPL * 2 : 16), sizeof b);
            } else {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    b[i] = e0 + i < p.E ? row[e0 + i] : (uint16_t)0xFF80;
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                x[q][i] = __uint_as_float((uint32_t)b[i] << 16);
        } else {
            const float *row = (const float *)p.logits + (int64_t)(live ? tq : t) * p.stride;
            if (p.vec && e0 < p.E) {
                __builtin_memcpy(x[q], __builtin_assume_aligned(row + e0, VPL * 4 < 16 ? VPL * 4 : 16),
                                 sizeof x[q]);
            } else {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    x[q][i] = e0 + i < p.E ? row[e0 + i] : -__builtin_huge_valf();
            }
        }
    }
#pragma unroll
    for (int q = 0; q < TOK; ++q) {
        high[q] = val[q] = 0.f;
        id[q] = -1;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            key[q][i] = e0 + i < p.E ? order_key(x[q][i]) : 0u;
        if (p.bias) {
            // scores first, for their sum with the bias is what is compared
            float total = 1.f;
            if (soft) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    m = max(m, key[q][i]);
                high[q] = key_value(wave_max_u32(m));
                float part = 0.f;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    part += key[q][i] > KEY_NEG_INF ? soft_term(x[q][i], high[q]) : 0.f;
                total = wave_sum(part);
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const bool any = key[q][i] > KEY_NEG_INF;
                x[q][i] = !any ? 0.f : soft ? soft_term(x[q][i], high[q]) / total : sigmoid(x[q][i]);
                key[q][i] = any ? order_key(x[q][i] + p.bias[e0 + i]) : 0u;
            }
        }
    }
    for (int j = 0; j < p.k; ++j) {
        uint32_t m[TOK], top[TOK];
        int at[TOK];
        float s[TOK];
#pragma unroll
        for (int q = 0; q < TOK; ++q) {
            m[q] = key[q][0];
            at[q] = 0;
            s[q] = x[q][0];
#pragma unroll
            for (int i = 1; i < VPL; ++i)
                if (key[q][i] > m[q]) {
                    m[q] = key[q][i];
                    at[q] = i;
                    s[q] = x[q][i];
                }
        }
#pragma unroll
        for (int q = 0; q < TOK; ++q)
            top[q] = wave_max_u32(m[q]);
#pragma unroll
        for (int q = 0; q < TOK; ++q) {
            // (with nothing left, the lane found is given no choice below)
            const int wl = __builtin_ctzll(__builtin_amdgcn_ballot_w64(m[q] == top[q]));
            const int won = wl * VPL + __builtin_amdgcn_readlane(at[q], wl);
            const float ws = p.bias ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s[q]), wl))
                                    : key_value(top[q]);
            const bool any = top[q] > KEY_NEG_INF;
            if (j == 0 && !p.bias)
                high[q] = ws;
            id[q] = any && lane == j ? won : id[q];
            val[q] = any && lane == j ? ws : val[q];
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                key[q][i] = lane == wl && i == at[q] ? 0u : key[q][i];
        }
    }
#pragma unroll
    for (int q = 0; q < TOK; ++q) {
        w[q] = id[q] < 0 ? 0.f : p.bias ? val[q] : soft ? soft_term(val[q], high[q]) : sigmoid(val[q]);
        if (p.renorm) {
            const float total = wave_sum(w[q]);
            w[q] = total > 0.f ? w[q] / total : 0.f;
        } else if (soft && !p.bias) {
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                part += e0 + i < p.E && order_key(x[q][i]) > KEY_NEG_INF ? soft_term(x[q][i], high[q]) : 0.f;
            const float total = wave_sum(part);
            w[q] = total > 0.f ? w[q] / total : 0.f;
        }
        w[q] *= p.scale;
    }
}

// LDS of the grouping.
struct GroupLds {
    int base[RT_GROUPS + 8];                 // next position of every group
    int total[RT_GROUPS + 8];
    int wave_at[RT_WAVES][RT_GROUPS + 1];    // a pass: counts, then positions, per wave
    int wave_sum[RT_WAVES];
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
    for (int w = 0; w < waves; ++w) {
        const int c = l.wave_at[w][e];
        l.wave_at[w][e] = at;
        at += c;
    }
    return at;
}

__device__ __forceinline__ void place(const RouteArgs &p, int flat, int g, int pos)
{
    p.rows[pos] = (int)((unsigned)flat / (unsigned)p.k);
    p.slots[flat] = g == p.E ? -1 : pos;
}

// Group of an id from outside: ids past the groups are in none.
__device__ __forceinline__ int group_of(int id, int groups)
{
    return (unsigned)id < (unsigned)groups ? id : groups;
}

// Routes the tokens of this block (VPL > 0) or reads their ids (VPL == 0),
// then: ONE (a single workgroup, at most ROUTE_ONE_ITEMS items) groups them,
// else counts them per group.
template <int VPL, bool BF16, bool ONE>
__global__ __launch_bounds__(RT_THREADS) void route_kernel(RouteArgs p)
{
    static_assert(ROUTE_ONE_ITEMS <= RT_THREADS, "one item per thread");
    __shared__ GroupLds l;
    __shared__ int s_id[ONE ? ROUTE_ONE_ITEMS : 1];
    const int tid = threadIdx.x, lane = tid & 63;
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
    if constexpr (VPL > 0) {
        constexpr int TOK = ROUTE_TOK<VPL>;
        for (int t = t0 + wave; t < t1; t += RT_WAVES * TOK) {
            int id[TOK];
            float w[TOK];
            route_tokens<VPL, BF16, TOK>(p, t, t1, lane, id, w);
#pragma unroll
            for (int q = 0; q < TOK; ++q) {
                const int tq = t + q * RT_WAVES;
                if (lane < p.k && tq < t1) {
                    const int flat = tq * p.k + lane;
                    p.ids[flat] = id[q];
                    p.weights[flat] = w[q];
                    if (group) {
                        const int g = id[q] < 0 ? p.E : id[q];
                        if (ONE)
                            s_id[flat] = g;
                        else
                            atomicAdd(&l.total[g], 1);
                    }
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
        if (tid < p.E)
            for (int w = 0; w < waves; ++w)
                sum += l.wave_at[w][tid];
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
            p.counts[(int64_t)blockIdx.x * p.cstride + e] = e <= p.E ? (uint16_t)l.total[e] : (uint16_t)0;
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
    __syncthreads();
    // Counts of the blocks before this one (base) and of all (total): a
    // thread adds 8 neighbouring groups over every per_pass-th block.  In the
    // LDS, group 8 c + i is kept at i * lanes + c, so that the lanes of an
    // addition, whose c differ, fall into different banks.
    const int lanes = p.cstride / 8, per_pass = RT_THREADS / lanes;
    const int r0 = tid / lanes, c = tid - r0 * lanes;
    if (r0 < per_pass) {
        int pre[8] = {}, tot[8] = {};
#pragma unroll 4
        for (int r = r0; r < blocks; r += per_pass) {
            const u32x4_t v = *(const u32x4_t *)(p.counts + (int64_t)r * p.cstride + 8 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int n = (int)((v[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
                tot[i] += n;
                pre[i] += r < b ? n : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            atomicAdd(&l.total[i * lanes + c], tot[i]);
            atomicAdd(&l.base[i * lanes + c], pre[i]);
        }
    }
    __syncthreads();
    auto kept = [&](int e) { return (e & 7) * lanes + (e >> 3); };
    int all;
    const int at = block_scan(l, tid < p.E ? l.total[kept(tid)] : 0, all);
    if (tid < p.E) {
        l.base[kept(tid)] += at;
        if (b == 0)
            p.offsets[tid] = at;
    }
    if (tid == 0) {
        l.base[kept(p.E)] += all;
        if (b == 0)
            p.offsets[p.E] = all;
    }
    const int first = b * p.block_tokens * p.k;
    const int n = (min(p.T, (b + 1) * p.block_tokens) - b * p.block_tokens) * p.k;
    for (int i0 = 0; i0 < n; i0 += RT_THREADS) {
        const int waves = min(RT_WAVES, (n - i0 + 63) / 64);
        clear_wave_at(l, waves, p.E);
        const bool live = i0 + tid < n;
        const int g = live ? group_of(p.ids[first + i0 + tid], p.E) : 0;
        __syncthreads();
        const int rank = rank_in_wave(l, live, g, p.E);
        __syncthreads();
        for (int e = tid; e <= p.E; e += RT_THREADS)
            l.base[kept(e)] = counts_to_positions(l, waves, e, l.base[kept(e)]);
        __syncthreads();
        if (live)
            place(p, first + i0 + tid, g, l.wave_at[wave][g] + rank);
        __syncthreads();
    }
}

}  // namespace gc
