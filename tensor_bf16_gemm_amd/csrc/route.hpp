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

// Routes one token in one wave.  Lane j < k returns with the j-th choice's
// expert (-1: none) in `id` and its weight in `w`.
template <int VPL, bool BF16>
__device__ __forceinline__ void route_token(const RouteArgs &p, int t, int lane, int &id, float &w)
{
    const int e0 = lane * VPL;
    float x[VPL];
    if constexpr (BF16) {
        const uint16_t *row = (const uint16_t *)p.logits + (int64_t)t * p.stride;
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
            x[i] = __uint_as_float((uint32_t)b[i] << 16);
    } else {
        const float *row = (const float *)p.logits + (int64_t)t * p.stride;
        if (p.vec && e0 < p.E) {
            __builtin_memcpy(x, __builtin_assume_aligned(row + e0, VPL * 4 < 16 ? VPL * 4 : 16), sizeof x);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                x[i] = e0 + i < p.E ? row[e0 + i] : -__builtin_huge_valf();
        }
    }
    uint32_t key[VPL];
    float high = 0.f;
    const bool soft = p.score == SCORE_SOFTMAX;
    if (p.bias) {
        // scores first, for their sum with the bias is what is compared
        if (soft) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                m = max(m, e0 + i < p.E ? order_key(x[i]) : 0u);
            high = key_value(wave_max_u32(m));
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                part += e0 + i < p.E && order_key(x[i]) > KEY_NEG_INF ? soft_term(x[i], high) : 0.f;
            const float total = wave_sum(part);
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const bool any = e0 + i < p.E && order_key(x[i]) > KEY_NEG_INF;
                x[i] = any ? soft_term(x[i], high) / total : 0.f;
                key[i] = any ? order_key(x[i] + p.bias[e0 + i]) : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const bool any = e0 + i < p.E && order_key(x[i]) > KEY_NEG_INF;
                x[i] = any ? sigmoid(x[i]) : 0.f;
                key[i] = any ? order_key(x[i] + p.bias[e0 + i]) : 0u;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            key[i] = e0 + i < p.E ? order_key(x[i]) : 0u;
    }
    id = -1;
    float val = 0.f;
    for (int j = 0; j < p.k; ++j) {
        uint32_t m = key[0];
        int at = 0;
        float s = x[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i)
            if (key[i] > m) {
                m = key[i];
                at = i;
                s = x[i];
            }
        const uint32_t top = wave_max_u32(m);
        if (top <= KEY_NEG_INF)
            break;
        const int wl = __builtin_ctzll(__builtin_amdgcn_ballot_w64(m == top));
        const int won = wl * VPL + __builtin_amdgcn_readlane(at, wl);
        const float ws =
            p.bias ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), wl)) : key_value(top);
        if (j == 0 && !p.bias)
            high = ws;
        if (lane == j) {
            id = won;
            val = ws;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane == wl && i == at)
                key[i] = 0u;
    }
    w = id < 0 ? 0.f : p.bias ? val : soft ? soft_term(val, high) : sigmoid(val);
    if (p.renorm) {
        const float total = wave_sum(w);
        w = total > 0.f ? w / total : 0.f;
    } else if (soft && !p.bias) {
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            part += e0 + i < p.E && order_key(x[i]) > KEY_NEG_INF ? soft_term(x[i], high) : 0.f;
        const float total = wave_sum(part);
        w = total > 0.f ? w / total : 0.f;
    }
    w *= p.scale;
}

// LDS of the grouping.
struct GroupLds {
    int base[RT_GROUPS + 8];                 // next position of every group
    int total[RT_GROUPS + 8];
    int wave_at[RT_WAVES][RT_GROUPS + 1];    // a pass: counts, then positions, per wave
    int wave_sum[RT_WAVES];
};

// Exclusive prefix sum of l.total[0 .. groups) over the workgroup; returns it
// for group threadIdx.x (any value past the groups), and the whole sum to
// every thread.
__device__ __forceinline__ int group_scan(GroupLds &l, int groups, int &all)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int v = tid < groups ? l.total[tid] : 0;
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

// Places n items of consecutive flat numbers first, first + 1, ...: item i of
// group get(i) (`groups` for none) goes to the next position of its group,
// in the order of the items.  l.base holds each group's next position.
template <class F>
__device__ __forceinline__ void place_items(GroupLds &l, F &&get, int n, int first, int k, int groups,
                                            int32_t *rows, int32_t *slots)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int bits = 32 - __builtin_clz(groups);       // groups itself is a value
    for (int i0 = 0; i0 < n; i0 += RT_THREADS) {
        for (int w = 0; w < RT_WAVES; ++w)
            for (int e = tid; e <= groups; e += RT_THREADS)
                l.wave_at[w][e] = 0;
        __syncthreads();
        const int i = i0 + tid;
        const bool live = i < n;
        const int g = live ? get(i) : 0;
        uint64_t same = __builtin_amdgcn_ballot_w64(live);
        for (int b = 0; b < bits; ++b) {
            const uint64_t on = __builtin_amdgcn_ballot_w64((g >> b) & 1);
            same &= (g >> b) & 1 ? on : ~on;
        }
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1ull));
        if (live && rank == 0)
            l.wave_at[wave][g] = __builtin_popcountll(same);
        __syncthreads();
        for (int e = tid; e <= groups; e += RT_THREADS) {
            int at = l.base[e];
            for (int w = 0; w < RT_WAVES; ++w) {
                const int c = l.wave_at[w][e];
                l.wave_at[w][e] = at;
                at += c;
            }
            l.base[e] = at;
        }
        __syncthreads();
        if (live) {
            const int pos = l.wave_at[wave][g] + rank;
            const int flat = first + i;
            rows[pos] = (int)((unsigned)flat / (unsigned)k);
            slots[flat] = g == groups ? -1 : pos;
        }
        __syncthreads();
    }
}

// Group of an id from outside: ids past the groups are in none.
__device__ __forceinline__ int group_of(int id, int groups)
{
    return (unsigned)id < (unsigned)groups ? id : groups;
}

// Routes the tokens of this block (VPL > 0) or reads their ids (VPL == 0),
// then: ONE (a single workgroup) groups them, else counts them per group.
template <int VPL, bool BF16, bool ONE>
__global__ __launch_bounds__(RT_THREADS) void route_kernel(RouteArgs p)
{
    __shared__ GroupLds l;
    __shared__ int s_id[ONE ? ROUTE_ONE_ITEMS : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = ONE ? 0 : blockIdx.x * p.block_tokens;
    const int t1 = ONE ? p.T : min(p.T, t0 + p.block_tokens);
    const bool group = p.offsets != nullptr;
    if (group) {
        for (int e = tid; e <= p.E; e += RT_THREADS)
            l.total[e] = 0;
        __syncthreads();
    }
    if constexpr (VPL > 0) {
        for (int t = t0 + wave; t < t1; t += RT_WAVES) {
            int id;
            float w;
            route_token<VPL, BF16>(p, t, lane, id, w);
            if (lane < p.k) {
                const int flat = t * p.k + lane;
                p.ids[flat] = id;
                p.weights[flat] = w;
                if (group) {
                    const int g = id < 0 ? p.E : id;
                    atomicAdd(&l.total[g], 1);
                    if (ONE)
                        s_id[flat] = g;
                }
            }
        }
    } else {
        for (int i = t0 * p.k + tid; i < t1 * p.k; i += RT_THREADS) {
            const int g = group_of(p.ids[i], p.E);
            atomicAdd(&l.total[g], 1);
            if (ONE)
                s_id[i] = g;
        }
    }
    if (!group)
        return;
    __syncthreads();
    if constexpr (ONE) {
        int all;
        const int at = group_scan(l, p.E, all);
        if (tid < p.E) {
            l.base[tid] = at;
            p.offsets[tid] = at;
        }
        if (tid == 0) {
            l.base[p.E] = all;
            p.offsets[p.E] = all;
        }
        __syncthreads();
        place_items(l, [&](int i) { return s_id[i]; }, p.T * p.k, 0, p.k, p.E, p.rows, p.slots);
    } else {
        for (int e = tid; e < p.cstride; e += RT_THREADS)
            p.counts[(int64_t)blockIdx.x * p.cstride + e] = e <= p.E ? (uint16_t)l.total[e] : (uint16_t)0;
    }
}

// Second kernel of a many-block grouping: positions of this block's items.
__global__ __launch_bounds__(RT_THREADS) void place_kernel(RouteArgs p)
{
    __shared__ GroupLds l;
    const int tid = threadIdx.x;
    const int blocks = gridDim.x, b = blockIdx.x;
    for (int e = tid; e < p.cstride; e += RT_THREADS) {
        l.base[e] = 0;
        l.total[e] = 0;
    }
    __syncthreads();
    // Counts of the blocks before this one (base) and of all (total): a
    // thread adds 8 neighbouring groups over every per_pass-th block.
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
            atomicAdd(&l.total[8 * c + i], tot[i]);
            atomicAdd(&l.base[8 * c + i], pre[i]);
        }
    }
    __syncthreads();
    int all;
    const int at = group_scan(l, p.E, all);
    if (tid < p.E) {
        l.base[tid] += at;
        if (b == 0)
            p.offsets[tid] = at;
    }
    if (tid == 0) {
        l.base[p.E] += all;
        if (b == 0)
            p.offsets[p.E] = all;
    }
    __syncthreads();
    const int first = b * p.block_tokens * p.k;
    const int n = (min(p.T, (b + 1) * p.block_tokens) - b * p.block_tokens) * p.k;
    place_items(l, [&](int i) { return group_of(p.ids[first + i], p.E); }, n, first, p.k, p.E, p.rows,
                p.slots);
}

}  // namespace gc
