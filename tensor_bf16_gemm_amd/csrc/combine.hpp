// combine.hpp -- gfx950 device code of moe_combine: for every token t
//   out[t] = bf16( sum_j w[t][j] * Y[slots[t][j]] + sum_p partials[p][t] ),
// summed in fp32 in that order and rounded once.
//
// Every row of Y that a slot names and every peer row is read once: the
// kernel is bound by HBM.  A wave takes one token and 64 vectors of 8
// columns.  Its lanes hold the token's terms (one lane per slot or peer: the
// address of the row and its weight); the terms that exist are walked in
// order, eight rows in flight at a time, so that a slot of -1 costs neither
// a load nor a branch per lane.  (4096 tokens, N 7168, k 8, 7 peers: 940 MB in
// 158 us, 5.9 TB/s; a copy kernel moves 5.2.  16 tokens: 4 us, a launch.)
#pragma once

#include "gc_kernel.hpp"

namespace gc {

constexpr int CB_THREADS = 256, CB_WAVES = CB_THREADS / 64;

struct CombineArgs {
    const uint16_t *Y;           // [S][N]
    const int32_t *slots;        // [T][k]
    const float *weights;        // [T][k]
    const uint16_t *partials;    // npeers blocks of [T][N], peer_stride elements apart
    int64_t peer_stride;
    uint16_t *out;               // [T][N]
    int T, S, N, k, npeers;
    int col_groups;              // groups of 64 vectors in a row
    int64_t items;               // T * col_groups
};

__device__ __forceinline__ void combine_item(const CombineArgs &p, int64_t item, int lane)
{
    const int t = (int)(item / p.col_groups);
    const int cg = (int)(item - (int64_t)t * p.col_groups);
    // terms: lane j < k slot j, then the peers
    uint64_t addr = 0;
    float w = 0.f;
    bool have = false;
    if (lane < p.k) {
        const int s = p.slots[(int64_t)t * p.k + lane];
        w = p.weights[(int64_t)t * p.k + lane];
        have = (unsigned)s < (unsigned)p.S;
        addr = (uint64_t)(p.Y + (int64_t)(have ? s : 0) * p.N);
    } else if (lane < p.k + p.npeers) {
        have = true;
        w = 1.f;
        addr = (uint64_t)(p.partials + (lane - p.k) * p.peer_stride + (int64_t)t * p.N);
    }
    uint64_t left = __builtin_amdgcn_ballot_w64(have);
    const int v = cg * 64 + lane;
    const bool live = v < p.N / 8;
    f32x4_t lo = {0.f, 0.f, 0.f, 0.f}, hi = {0.f, 0.f, 0.f, 0.f};
    constexpr int DEPTH = 8;
    while (left) {
        u32x4_t x[DEPTH];
        float f[DEPTH];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            x[d] = (u32x4_t){0u, 0u, 0u, 0u};
            f[d] = 0.f;
            if (left) {
                const int j = __builtin_ctzll(left);
                left &= left - 1;
                const uint64_t a = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(addr >> 32), j) << 32) |
                                   (uint32_t)__builtin_amdgcn_readlane((int)addr, j);
                f[d] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), j));
                if (live)
                    x[d] = __builtin_nontemporal_load((const u32x4_t *)a + v);
            }
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            lo += f[d] * unpack_bf16x4((u32x2_t){x[d][0], x[d][1]});
            hi += f[d] * unpack_bf16x4((u32x2_t){x[d][2], x[d][3]});
        }
    }
    if (live) {
        const u32x2_t a = pack_bf16x4(lo), b = pack_bf16x4(hi);
        __builtin_nontemporal_store((u32x4_t){a[0], a[1], b[0], b[1]},
                                    (u32x4_t *)(p.out + (int64_t)t * p.N) + v);
    }
}

__global__ __launch_bounds__(CB_THREADS) void combine_kernel(CombineArgs p)
{
    const int lane = threadIdx.x & 63;
    const int64_t first =
        (int64_t)blockIdx.x * CB_WAVES + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    // (one item but for more than 2^26 of them)
    for (int64_t item = first; item < p.items; item += (int64_t)gridDim.x * CB_WAVES)
        combine_item(p, item, lane);
}

}  // namespace gc
