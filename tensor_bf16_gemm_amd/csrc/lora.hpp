// lora.hpp -- gfx950 device code of the second half of lora_add: for every
// position i of the rows grouped by adapter, with m = rows[i],
//   out[m] = bf16(base[m] + H[i] . up[a(i)]),   H[i] = scale[a] X[m] . down[a],
// where stream_kernel has left X[m] . down[a] as fp32 sums over pieces of K.
// H enters the matrix cores as the sum of two bf16 (the rounded value and the
// rounded rest), which keeps 16 bits of it: with one bf16 the middle
// rounding would be as large as that of the output.
//
// Rows are read and written once and there are at most r <= 128 products per
// output: the kernel is bound by the traffic of base and out.  A wave takes
// 16*RB positions, whose H it adds up and keeps in registers, and walks over
// blocks of 64 columns by itself, without a barrier: while it multiplies and
// stores one block, the next block's rows of base (into registers) and r x 64
// values of up (into LDS, in the layout the transposing read wants) are on
// their way.
#pragma once

#include "grouped.hpp"

namespace gc {

constexpr int EX_THREADS = 256, EX_WAVES = 4, EX_COLS = 64 * EX_WAVES;

struct ExpandArgs {
    const uint16_t *base;      // [M][N]
    uint16_t *out;             // [M][N]; base itself or apart from it
    const float *sums;         // [splits][M][r]
    const float *scale;        // [E]
    const uint16_t *up;        // [E][r][N]
    const int32_t *offsets;    // [E + 1]
    const int32_t *rows;       // [M]
    int M, N, r, E, splits;
    int copy;                  // out is not base: rows without adapter are copied
    int span, spans;           // column tiles of EX_COLS a workgroup walks; spans per row tile
};

// KS: steps of 32 that cover r.
template <int RB, int KS>
__global__ __launch_bounds__(EX_THREADS) void expand_kernel(ExpandArgs p)
{
    constexpr int BM = 16 * RB, NB = 4, BN = 64;
    __shared__ __attribute__((aligned(1024))) uint8_t ups[EX_WAVES * KS * 4096];
    __shared__ int first[GR_GROUPS + 1];
    __shared__ int wsum[EX_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fi = lane & 15, fg = lane >> 4;
    const int groups = p.E + (p.copy ? 1 : 0);
    const int units =
        scan_tiles<EX_THREADS>(p.offsets, p.E, p.M, groups, BM, p.spans, first, wsum);
    const uint32_t N2 = (uint32_t)p.N * 2u;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.base, (uint32_t)p.M * N2);
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.out, (uint32_t)p.M * N2);
    const uint32_t mine = lds_addr(ups) + (uint32_t)(wave * KS * 4096);
    // layout of a 32 x 64 block as in stream_kernel for NB = 4
    auto fold = [](int k) { return ((k >> 1) & 1) | (((k >> 3) & 1) << 1); };
    const int b_row = lane >> 3, b_slot = lane & 7;
    const int f_lane = fold(8 * fg + (fi >> 2));
    const int p8 = 8 * (fg >> 1) + 16 * (fg & 1);

    for (int t = blockIdx.x; t < units; t += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(find_group(first, groups, t, lane));
        int lo, hi;
        group_range(p.offsets, p.E, p.M, e, lo, hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
        const int in = t - __builtin_amdgcn_readfirstlane(first[e]);
        const int mt = in / p.spans;
        int n0 = (in - mt * p.spans) * p.span * EX_COLS + wave * BN;
        const int n_end = min(p.N, n0 - wave * BN + p.span * EX_COLS);
        const int m0 = lo + mt * BM;
        const bool delta = e < p.E;
        const u32x4_t ru = make_rsrc4(p.up + (size_t)(delta ? e : 0) * p.r * p.N, delta ? (uint32_t)p.r * N2 : 0u);
        auto load_up = [&](int n0) {
#pragma unroll
            for (int i = 0; i < 4 * KS; ++i) {
                const int k = 8 * i + b_row;
                const int n = n0 + 16 * ((b_slot >> 1) ^ fold(k)) + 8 * (b_slot & 1);
                dma16(ru, mine + i * 1024, n < n_end ? (uint32_t)k * N2 + (uint32_t)n * 2u : OOB);
            }
        };
        uint32_t row_off[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int m = m0 + 16 * i + fi;
            int row = -1;
            if (m >= lo && m < hi)
                row = p.rows[m];
            row_off[i] = (unsigned)row < (unsigned)p.M ? (uint32_t)row * N2 + (uint32_t)p8 * 2u : OOB;
        }
        auto offset = [&](int i, int h, int n0) {
            return n0 + p8 + 32 * h < n_end ? row_off[i] + (uint32_t)(n0 + 32 * h) * 2u : OOB;
        };
        auto load_base = [&](u32x4_t (&old)[RB][2], int n0) {
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    old[i][h] = __builtin_amdgcn_raw_buffer_load_b128(rb, (int)offset(i, h, n0), 0, 0);
        };
        wait_lgkmcnt0();                         // the last unit's block of up is read
        load_up(n0);
        u32x4_t old[RB][2];
        load_base(old, n0);
        // H of the rows, as two bf16 fragments
        bf16x8_t h[RB][KS], l[RB][KS];
        {
            const float sc = delta ? p.scale[e] : 0.f;
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int m = m0 + 16 * i + fi, k = 32 * s + 8 * fg;
                    f32x4_t x = {0.f, 0.f, 0.f, 0.f}, y = x;
                    if (delta && m < hi && k < p.r) {
                        const float *at = p.sums + (size_t)m * p.r + k;
                        for (int c = 0; c < p.splits; ++c, at += (size_t)p.M * p.r) {
                            x += *(const f32x4_t *)at;
                            y += *(const f32x4_t *)(at + 4);
                        }
                    }
                    x *= sc;
                    y *= sc;
                    const u32x2_t hx = pack_bf16x4(x), hy = pack_bf16x4(y);
                    const u32x2_t lx = pack_bf16x4(x - unpack_bf16x4(hx)), ly = pack_bf16x4(y - unpack_bf16x4(hy));
                    h[i][s] = __builtin_bit_cast(bf16x8_t, (u32x4_t){hx[0], hx[1], hy[0], hy[1]});
                    l[i][s] = __builtin_bit_cast(bf16x8_t, (u32x4_t){lx[0], lx[1], ly[0], ly[1]});
                }
        }
        for (; n0 < n_end; n0 += EX_COLS) {
            wait_vmcnt<0>();                     // this block of up has landed
            bf16x8_t fa[KS][NB];
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const uint32_t a = mine + (uint32_t)(s * 4096 + (8 * fg + (fi >> 2)) * 128 + 8 * (fi & 3) +
                                                         ((j ^ f_lane) * 32));
                    bf16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                        (lds_bf16x4_t *)lds_ptr<bf16x4_t>(a));
                    bf16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                        (lds_bf16x4_t *)lds_ptr<bf16x4_t>(a + 4 * 128));
                    fa[s][j] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
                }
            wait_lgkmcnt0();
            u32x4_t next[RB][2];
            load_up(n0 + EX_COLS);               // (past the end: empty)
            load_base(next, n0 + EX_COLS);
            f32x4_t acc[RB][NB];
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[s][j], h[i][s], acc[i][j], 0, 0, 0);
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[s][j], l[i][s], acc[i][j], 0, 0, 0);
                    }
            // fp32 sums regrouped as in pack_pair (lanes trade halves so that
            // each holds 8 consecutive columns), base added, one rounding
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    f32x4_t a, b;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const auto sw = __builtin_amdgcn_permlane16_swap(
                            __float_as_uint(acc[i][2 * g][c]), __float_as_uint(acc[i][2 * g + 1][c]), false, false);
                        a[c] = __uint_as_float(sw[0]);
                        b[c] = __uint_as_float(sw[1]);
                    }
                    const u32x4_t o = old[i][g];
                    const u32x2_t x = pack_bf16x4(a + unpack_bf16x4((u32x2_t){o[0], o[1]}));
                    const u32x2_t y = pack_bf16x4(b + unpack_bf16x4((u32x2_t){o[2], o[3]}));
                    store16(ro, offset(i, g, n0), (u32x4_t){x[0], x[1], y[0], y[1]});
                }
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    old[i][g] = next[i][g];
        }
        wait_vmcnt<0>();                         // the empty loads have written their zeros
    }
}

}  // namespace gc
