// choose.hpp -- gfx950 device code of the router's choice: for one token the k
// experts of largest key and their weights (route_token).  What it computes,
// how and what bounds it stands in route.hpp.
#pragma once

#include <utility>

#include "gc_kernel.hpp"

namespace gc {

constexpr int RT_GROUPS = 1024;          // groups (experts, adapters) at most
constexpr int RT_TOP = 16;               // k at most

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

}  // namespace gc
