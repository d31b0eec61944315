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

#include <utility>

#include "gc_kernel.hpp"

namespace gc {

constexpr int RT_THREADS = 1024, RT_WAVES = RT_THREADS / 64;
constexpr int RT_GROUPS = 1024;          // groups (experts, adapters) at most
constexpr int RT_BLOCKS = 256;           // blocks of a many-block grouping, unless
constexpr int RT_ITEMS = 8191;           // a block's items were more than this (8 counts add up in 16 bits)
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
constexpr int RT_TOP = 16;               // k at most
// Items that one workgroup routes and groups in a single launch.
constexpr int ROUTE_ONE_ITEMS = 1024;

enum Score { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };

struct RouteArgs {
    const void *logits;      // [T] rows of E, row stride `stride` elements
    int64_t stride;
    const float *bias;       // [E] or null
    int T, E, k;             // (grouping alone: T items, k = 1)
    int score, renorm;
    float scale;
    int32_t *ids;            // [T][k]
    float *weights;          // [T][k]
    // grouping (null offsets: none)
    int per_row;             // items of a row
    int32_t *offsets;        // [E + 1]
    int32_t *rows;           // [T * k]
    int32_t *slots;          // [T * k]
    uint16_t *counts;        // [blocks][cstride]
    int cstride;             // E rounded up to 8
    int block_tokens;        // tokens (items / k) per block
    bool vec;                // a lane's VPL logits are whole aligned vectors
};

// v of the lane ROR places down in the row of 16 (cyclic).
template <int ROR>
__device__ __forceinline__ uint32_t row_ror(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ROR, 0xf, 0xf, true);
}
template <int ROR>
__device__ __forceinline__ double row_ror(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint64_t o = ((uint64_t)row_ror<ROR>((uint32_t)(b >> 32)) << 32) | row_ror<ROR>((uint32_t)b);
    return __longlong_as_double((long long)o);
}

// (pairs are never NaN)
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b) { return a < b ? a : b; }
__device__ __forceinline__ double pair_max(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double pair_min(double a, double b) { return fmin(a, b); }

// Maximum of v and its partner's: the neighbouring row of 16, or (HALVES) the
// other half of the wave (both halves of a swap with itself).
template <bool HALVES>
__device__ __forceinline__ uint32_t swap_max(uint32_t v)
{
    if (HALVES) {
        const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return pair_max((uint32_t)s[0], (uint32_t)s[1]);
    }
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return pair_max((uint32_t)s[0], (uint32_t)s[1]);
}
template <bool HALVES>
__device__ __forceinline__ double swap_max(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
    uint64_t x, y;
    if (HALVES) {
        const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
        const auto h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
        x = ((uint64_t)h[0] << 32) | l[0];
        y = ((uint64_t)h[1] << 32) | l[1];
    } else {
        const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
        const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        x = ((uint64_t)h[0] << 32) | l[0];
        y = ((uint64_t)h[1] << 32) | l[1];
    }
    return pair_max(__longlong_as_double((long long)x), __longlong_as_double((long long)y));
}
// Maximum over the LPT lanes of a token (a row of 16, or the wave), in all of
// them.
template <int LPT, class P>
__device__ __forceinline__ P token_max(P v)
{
    v = pair_max(v, row_ror<8>(v));
    v = pair_max(v, row_ror<4>(v));
    v = pair_max(v, row_ror<2>(v));
    v = pair_max(v, row_ror<1>(v));
    if (LPT == 64) {
        v = swap_max<false>(v);
        v = swap_max<true>(v);
    }
    return v;
}

template <int LPT>
__device__ __forceinline__ float token_sum(float v)
{
    auto ror = [](float x, auto c) {
        return __uint_as_float(row_ror<decltype(c)::value>(__float_as_uint(x)));
    };
    v += ror(v, std::integral_constant<int, 8>{});
    v += ror(v, std::integral_constant<int, 4>{});
    v += ror(v, std::integral_constant<int, 2>{});
    v += ror(v, std::integral_constant<int, 1>{});
    if (LPT == 64) {
        const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
        const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
    }
    return v;
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

// The pair of an expert; none() is the least, for one that cannot be chosen.
// Wide: any key.  Narrow: the key of a bf16 value (its low 16 bits say nothing).
struct WidePair {
    using P = double;
    static constexpr uint64_t ONE = 0x3FF0000000000000ull;
    static __device__ __forceinline__ P none() { return __longlong_as_double((long long)ONE); }
    static __device__ __forceinline__ P make(uint32_t key, int e)
    {
        const uint64_t b =
            key > KEY_NEG_INF ? ONE | ((uint64_t)key << 20) | (uint32_t)(RT_GROUPS - 1 - e) : ONE;
        return __longlong_as_double((long long)b);
    }
    static __device__ __forceinline__ uint32_t key(P v)
    {
        return (uint32_t)((uint64_t)__double_as_longlong(v) >> 20);
    }
    static __device__ __forceinline__ int expert(P v)
    {
        return RT_GROUPS - 1 - (int)((uint64_t)__double_as_longlong(v) & 0xFFFFFu);
    }
    // mask ? x : y by bits.  (A conditional between neighbours of an array in
    // registers is turned into an index and a chain of compares.)
    static __device__ __forceinline__ P pick(bool c, P x, P y)
    {
        const uint64_t mask = c ? ~0ull : 0ull;
        const uint64_t a = (uint64_t)__double_as_longlong(x), b = (uint64_t)__double_as_longlong(y);
        return __longlong_as_double((long long)((a & mask) | (b & ~mask)));
    }
};
struct NarrowPair {
    using P = uint32_t;
    static __device__ __forceinline__ P none() { return 0u; }
    static __device__ __forceinline__ P make(uint32_t key, int e)
    {
        return key > KEY_NEG_INF ? (key & 0xFFFF0000u) | (uint32_t)(RT_GROUPS - 1 - e) : 0u;
    }
    // (a negative value's key has ones in its low half)
    static __device__ __forceinline__ uint32_t key(P v)
    {
        return v == 0u ? 0u : (v & 0x80000000u) ? v & 0xFFFF0000u : v | 0xFFFFu;
    }
    static __device__ __forceinline__ int expert(P v) { return RT_GROUPS - 1 - (int)(v & 0xFFFFu); }
    static __device__ __forceinline__ P pick(bool c, P x, P y)
    {
        const uint32_t mask = c ? ~0u : 0u;
        return (x & mask) | (y & ~mask);
    }
};

// Odd-even merge network (Batcher) for V a power of two: its comparators, as
// a table the compiler unrolls.
template <int V>
struct MergeNetwork {
    struct Pair {
        int lo, hi;
    };
    static constexpr int count()
    {
        int n = 0;
        for (int p = 1; p < V; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < V; j += 2 * k)
                    for (int i = 0; i < k && i + j + k < V; ++i)
                        n += (i + j) / (2 * p) == (i + j + k) / (2 * p);
        return n;
    }
    static constexpr Pair pair(int which)
    {
        int n = 0;
        for (int p = 1; p < V; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < V; j += 2 * k)
                    for (int i = 0; i < k && i + j + k < V; ++i)
                        if ((i + j) / (2 * p) == (i + j + k) / (2 * p) && n++ == which)
                            return Pair{i + j, i + j + k};
        return Pair{0, 0};
    }
};

template <int V, class P, int... I>
__device__ __forceinline__ void sort_steps(P (&a)[V], std::integer_sequence<int, I...>)
{
    auto step = [&](auto c) {
        constexpr auto at = MergeNetwork<V>::pair(decltype(c)::value);
        const P hi = pair_max(a[at.lo], a[at.hi]), lo = pair_min(a[at.lo], a[at.hi]);
        a[at.lo] = hi;
        a[at.hi] = lo;
    };
    (step(std::integral_constant<int, I>{}), ...);
}

// Falling order.
template <int V, class P>
__device__ __forceinline__ void sort_pairs(P (&a)[V])
{
    if constexpr (V > 1)
        sort_steps(a, std::make_integer_sequence<int, MergeNetwork<V>::count()>{});
}

template <bool BF16>
__device__ __forceinline__ float logit(const RouteArgs &p, int t, int e)
{
    if (BF16)
        return __uint_as_float((uint32_t)((const uint16_t *)p.logits)[(int64_t)t * p.stride + e] << 16);
    return ((const float *)p.logits)[(int64_t)t * p.stride + e];
}

// Routes one token per LPT lanes.  Lane j < k of the token returns with the
// j-th choice's expert (-1: none) in `id` and its weight in `w`.  `t` is the
// lane's token, which must exist.
template <int LPT, int V, bool BF16, bool VEC, class Pair>
__device__ __forceinline__ void route_token(const RouteArgs &p, int t, int j, int &id, float &w)
{
    // The lane's experts: V neighbours where they are whole aligned vectors
    // (VEC), else every LPT-th (which the lanes of a token read side by side).
    constexpr int es = VEC ? 1 : LPT;
    const int e0 = VEC ? j * V : j;
    const bool soft = p.score == SCORE_SOFTMAX;
    float x[V];
    if (VEC && e0 < p.E) {
        if constexpr (BF16) {
            uint16_t b[V];
            __builtin_memcpy(b, __builtin_assume_aligned((const uint16_t *)p.logits + (int64_t)t * p.stride + e0,
                                                         V * 2 < 16 ? V * 2 : 16), sizeof b);
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] = __uint_as_float((uint32_t)b[i] << 16);
        } else {
            __builtin_memcpy(x, __builtin_assume_aligned((const float *)p.logits + (int64_t)t * p.stride + e0,
                                                         V * 4 < 16 ? V * 4 : 16), sizeof x);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = e0 + i * es < p.E ? logit<BF16>(p, t, e0 + i * es) : -__builtin_huge_valf();
    }
    typename Pair::P a[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        a[i] = Pair::make(order_key(x[i]), e0 + i * es);
    // For a softmax over all experts: its maximum and its sum.
    float high = 0.f, total = 1.f;
    if (soft && (p.bias || !p.renorm)) {
        auto m = a[0];
#pragma unroll
        for (int i = 1; i < V; ++i)
            m = pair_max(m, a[i]);
        high = key_value(Pair::key(token_max<LPT>(m)));
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            part += a[i] != Pair::none() ? soft_term(x[i], high) : 0.f;
        total = token_sum<LPT>(part);
    }
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (a[i] != Pair::none()) {
                const float s = soft ? soft_term(x[i], high) / total : sigmoid(x[i]);
                a[i] = Pair::make(order_key(s + p.bias[e0 + i * es]), e0 + i * es);
            }
    }
    sort_pairs(a);
    const auto none = Pair::none();
    auto mine = none, best = none;
    // (a list is never asked for more than k of its pairs)
    auto rounds = [&](auto deep) {
        constexpr int D = decltype(deep)::value;
        for (int r = 0; r < p.k; ++r) {
            const auto top = token_max<LPT>(a[0]);
            if (r == 0)
                best = top;
            mine = Pair::pick(j == r, top, mine);
            const bool won = a[0] == top;        // (none: its list is empty, moving it changes nothing)
#pragma unroll
            for (int i = 0; i + 1 < D; ++i)
                a[i] = Pair::pick(won, a[i + 1], a[i]);
            a[D - 1] = Pair::pick(won, none, a[D - 1]);
        }
    };
    if (V > 8 && p.k <= 8)
        rounds(std::integral_constant<int, (V > 8 ? 8 : V)>{});
    else
        rounds(std::integral_constant<int, V>{});
    const bool chosen = mine != none;
    id = chosen ? Pair::expert(mine) : -1;
    float val = key_value(Pair::key(mine));
    if (p.bias)
        val = logit<BF16>(p, t, chosen ? id : 0);
    // Renormalized, the chosen terms are relative to the largest of them: with
    // a bias it may lie so far below the row's maximum that e^(x - high) is 0.
    if (soft && p.renorm)
        high = key_value(p.bias ? token_max<LPT>(chosen ? order_key(val) : 0u) : Pair::key(best));
    w = !chosen ? 0.f : soft ? soft_term(val, high) : sigmoid(val);
    if (p.renorm)
        total = token_sum<LPT>(w);
    else if (!soft)
        total = 1.f;
    w = chosen && total > 0.f ? w / total * p.scale : 0.f;
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
