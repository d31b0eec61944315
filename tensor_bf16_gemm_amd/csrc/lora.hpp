// lora.hpp -- gfx950 device code of the second half of lora_add: for every
// position i of the rows grouped by adapter, with m = rows[i],
//   out[m] = bf16(base[m] + H[i] . up[a(i)]),   H[i] = scale[a] X[m] . down[a]
// (H from stream_kernel, kept as two bf16 whose sum carries 16 bits).
//
// Rows are read and written once and there are at most r <= 128 products per
// output: the kernel is bound by the traffic of base and out.  A wave takes
// 16*RB positions by 64 columns by itself: it asks for its rows of base, its
// r x 64 block of up (into LDS, in the layout the transposing read wants) and
// its rows of H all at once, and meets no barrier.
#pragma once

#include "grouped.hpp"

namespace gc {

constexpr int EX_THREADS = 256, EX_WAVES = 4, EX_COLS = 64 * EX_WAVES;

struct ExpandArgs {
    const uint16_t *base;      // [M][N]
    uint16_t *out;             // [M][N]; base itself or apart from it
    const uint16_t *h, *h_lo;  // [M][r]
    const uint16_t *up;        // [E][r][N]
    const int32_t *offsets;    // [E + 1]
    const int32_t *rows;       // [M]
    int M, N, r, E;
    int copy;                  // out is not base: rows without adapter are copied
    int tiles_n;               // column tiles of EX_COLS
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
    const int tiles =
        scan_tiles<EX_THREADS>(p.offsets, p.E, p.M, groups, BM, p.tiles_n, first, wsum);
    const uint32_t N2 = (uint32_t)p.N * 2u;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.base, (uint32_t)p.M * N2);
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.out, (uint32_t)p.M * N2);
    const uint32_t h_bytes = (uint32_t)p.M * (uint32_t)p.r * 2u;
    const __amdgpu_buffer_rsrc_t rh = make_rsrc(p.h, h_bytes), rl = make_rsrc(p.h_lo, h_bytes);
    const uint32_t mine = lds_addr(ups) + (uint32_t)(wave * KS * 4096);
    // layout of a 32 x 64 block as in stream_kernel for NB = 4
    auto fold = [](int k) { return ((k >> 1) & 1) | (((k >> 3) & 1) << 1); };
    const int b_row = lane >> 3, b_slot = lane & 7;
    const int f_lane = fold(8 * fg + (fi >> 2));
    const int p8 = 8 * (fg >> 1) + 16 * (fg & 1);

    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(find_group(first, groups, t, lane));
        int lo, hi;
        group_range(p.offsets, p.E, p.M, e, lo, hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
        // neighbouring workgroups take neighbouring columns of the same rows
        const int in = t - __builtin_amdgcn_readfirstlane(first[e]);
        const int mt = in / p.tiles_n;
        const int n0 = (in - mt * p.tiles_n) * EX_COLS + wave * BN;
        const int m0 = lo + mt * BM;
        if (n0 >= p.N)
            continue;
        const bool delta = e < p.E;
        wait_lgkmcnt0();                         // the last tile's block of up is read
        if (delta) {
            const u32x4_t ru = make_rsrc4(p.up + (size_t)e * p.r * p.N, (uint32_t)p.r * N2);
#pragma unroll
            for (int i = 0; i < 4 * KS; ++i) {
                const int k = 8 * i + b_row;
                const int n = n0 + 16 * ((b_slot >> 1) ^ fold(k)) + 8 * (b_slot & 1);
                dma16(ru, mine + i * 1024, n < p.N ? (uint32_t)k * N2 + (uint32_t)n * 2u : OOB);
            }
        }
        uint32_t row_off[RB];
        u32x4_t old[RB][2];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int m = m0 + 16 * i + fi;
            int row = -1;
            if (m >= lo && m < hi)
                row = p.rows[m];
            row_off[i] = (unsigned)row < (unsigned)p.M ? (uint32_t)row * N2 + (uint32_t)(n0 + p8) * 2u : OOB;
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                old[i][h] = __builtin_amdgcn_raw_buffer_load_b128(
                    rb, (int)(n0 + p8 + 32 * h < p.N && row_off[i] != OOB ? row_off[i] + 64 * h : OOB), 0, 0);
        f32x4_t acc[RB][NB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        if (delta) {
            u32x4_t h[RB][KS], l[RB][KS];
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int m = m0 + 16 * i + fi, k = 32 * s + 8 * fg;
                    const uint32_t off =
                        m < hi && k < p.r ? ((uint32_t)m * (uint32_t)p.r + (uint32_t)k) * 2u : OOB;
                    h[i][s] = __builtin_amdgcn_raw_buffer_load_b128(rh, (int)off, 0, 0);
                    l[i][s] = __builtin_amdgcn_raw_buffer_load_b128(rl, (int)off, 0, 0);
                }
            wait_vmcnt<0>();                     // the block of up has landed
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const uint32_t at = mine + s * 4096;
                bf16x8_t fa[NB];
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const uint32_t a = at + (uint32_t)((8 * fg + (fi >> 2)) * 128 + 8 * (fi & 3) +
                                                       ((j ^ f_lane) * 32));
                    bf16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                        (lds_bf16x4_t *)lds_ptr<bf16x4_t>(a));
                    bf16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                        (lds_bf16x4_t *)lds_ptr<bf16x4_t>(a + 4 * 128));
                    fa[j] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
                }
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            fa[j], __builtin_bit_cast(bf16x8_t, h[i][s]), acc[i][j], 0, 0, 0);
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            fa[j], __builtin_bit_cast(bf16x8_t, l[i][s]), acc[i][j], 0, 0, 0);
                    }
            }
        }
        // fp32 sums regrouped as in pack_pair (lanes trade halves so that
        // each holds 8 consecutive columns), base added, one rounding
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4_t a, b;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const auto sw = __builtin_amdgcn_permlane16_swap(
                        __float_as_uint(acc[i][2 * h][c]), __float_as_uint(acc[i][2 * h + 1][c]), false, false);
                    a[c] = __uint_as_float(sw[0]);
                    b[c] = __uint_as_float(sw[1]);
                }
                const u32x4_t o = old[i][h];
                const u32x2_t x = pack_bf16x4(a + unpack_bf16x4((u32x2_t){o[0], o[1]}));
                const u32x2_t y = pack_bf16x4(b + unpack_bf16x4((u32x2_t){o[2], o[3]}));
                const uint32_t off =
                    n0 + p8 + 32 * h < p.N && row_off[i] != OOB ? row_off[i] + 64 * h : OOB;
                store16(ro, off, (u32x4_t){x[0], x[1], y[0], y[1]});
            }
    }
}

}  // namespace gc
