// lora.hpp -- gfx950 device code of the second half of lora_add: for every
// position i of the rows grouped by adapter, with m = rows[i],
//   out[m] = bf16(base[m] + H[i] . up[a(i)]),   H[i] = scale[a] X[m] . down[a],
// where stream_kernel has left X[m] . down[a] as fp32 sums over pieces of K.
// H enters the matrix cores as three bf16 that take 8 leading bits each and
// add up to all 24 of the fp32 value: nothing is rounded between the fp32
// sums and the output.  (Two bf16 would leave an error of 2^-16 of
// H, enough to round one output in a thousand the other way.  The third costs
// 0.1 to 0.6 us: 56.4 -> 57.1 at M = 4096, N = 6288, r = 64.)
//
// Rows are read and written once and there are at most r <= 128 products per
// output: the kernels are bound by the traffic of base and out.  In both, the
// products pass through LDS from the matrix cores' layout (a lane: 4 columns
// of a row) to whole lines, so that a wave's load of base and its store of
// out cover rows of 128 bytes and more.
//
// expand_rows_kernel, many rows per group: a wave keeps r x 128 values of up
// in registers and walks down the rows of its workgroup, whose H stands in LDS
// as fp32; nothing but rows of base and out moves in the loop, and the next
// rows are on their way while these are multiplied.  (With up in LDS and the
// walk along the columns, every tile of 256 columns waited for its block of
// up, its base and the last stores in turn: M = 4096, N = 6288, r = 64 took
// 44 us.)
// It takes 34 us: 26 at 4.1 TB/s, and 8 before the first row, for the look-up
// and the sums.
// expand_kernel, few rows per group: 16 positions, walking along the columns
// (64 rows of 32 adapters, r = 32: 8 us; one row: 6 us, latencies).
#pragma once

#include "grouped.hpp"

namespace gc {

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
    int span, spans;           // expand_kernel: column tiles of EX_COLS a workgroup walks, spans
                               // per row tile; expand_rows_kernel: rows a workgroup walks,
                               // column tiles of XR_COLS
};

// Eight neighbouring outputs: fp32 products a, b plus base, rounded once.
__device__ __forceinline__ u32x4_t add_base(f32x4_t a, f32x4_t b, u32x4_t base)
{
    const u32x2_t x = pack_bf16x4(a + unpack_bf16x4((u32x2_t){base[0], base[1]}));
    const u32x2_t y = pack_bf16x4(b + unpack_bf16x4((u32x2_t){base[2], base[3]}));
    return (u32x4_t){x[0], x[1], y[0], y[1]};
}

// Eight neighbouring values of H for position m: the sums over the pieces of
// K, in order, times the scale.
template <int AHEAD>
__device__ __forceinline__ void load_h(const ExpandArgs &p, bool on, int m, int k, float scale, f32x4_t &x,
                                       f32x4_t &y)
{
    x = y = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    const float *at = p.sums + (on ? (size_t)m * p.r + k : 0);
    for (int c = 0; c < p.splits; c += AHEAD) {
        f32x4_t a[AHEAD], b[AHEAD];
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            a[d] = b[d] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
            if (on && c + d < p.splits) {
                const float *q = at + (size_t)(c + d) * p.M * p.r;
                a[d] = *(const f32x4_t *)q;
                b[d] = *(const f32x4_t *)(q + 4);
            }
        }
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            x += a[d];
            y += b[d];
        }
    }
    x *= scale;
    y *= scale;
}

// The leading 8 bits of eight fp32 values as bf16 (cut off, so that no finite
// value becomes infinite and the rest keeps its sign), the values left as the
// rest.  Three times leaves nothing of 24 bits.
__device__ __forceinline__ bf16x8_t take_bf16(f32x4_t &x, f32x4_t &y)
{
    u32x4_t r;
    const u32x4_t a = __builtin_bit_cast(u32x4_t, x), b = __builtin_bit_cast(u32x4_t, y);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r[i] = __builtin_amdgcn_perm(a[2 * i + 1], a[2 * i], 0x07060302u);
        r[i + 2] = __builtin_amdgcn_perm(b[2 * i + 1], b[2 * i], 0x07060302u);
    }
    x -= __builtin_bit_cast(f32x4_t, a & 0xFFFF0000u);
    y -= __builtin_bit_cast(f32x4_t, b & 0xFFFF0000u);
    return __builtin_bit_cast(bf16x8_t, r);
}

// The product of the leading parts plus that of the rests.  Where H or up holds
// infinities the first alone is what the whole product is (its parts have the
// signs of their values), while the rest is inf - inf or 0 * inf.
__device__ __forceinline__ f32x4_t whole_product(f32x4_t lead, f32x4_t rest)
{
    f32x4_t s = lead + rest;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = s[i] == s[i] ? s[i] : lead[i];
    return s;
}

// KS: steps of 32 that cover r.
template <int KS>
__global__ __launch_bounds__(EX_THREADS, expand_resident(KS)) void expand_kernel(ExpandArgs p)
{
    constexpr int BM = 16;
    constexpr int UP = KS * 32 * EX_COLS * 2;            // bytes of a block of up
    constexpr int LOADS = KS * 16 / EX_WAVES;            // of up, per wave
    constexpr int PITCH = 64 * 4 + 16;                   // bytes of a row in the exchange
    __shared__ __attribute__((aligned(1024))) uint8_t ups[UP];
    __shared__ __attribute__((aligned(16))) uint8_t exchange[EX_WAVES * 16 * PITCH];
    __shared__ int first[GR_GROUPS + 1], starts[GR_GROUPS + 1];
    __shared__ int wsum[EX_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fi = lane & 15, fg = lane >> 4;
    const int groups = p.E + (p.copy ? 1 : 0);
    const int units =
        scan_tiles<EX_THREADS>(p.offsets, p.E, p.M, groups, BM, p.spans, first, starts, wsum);
    const uint32_t N2 = (uint32_t)p.N * 2u;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.base, (uint32_t)p.M * N2);
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.out, (uint32_t)p.M * N2);
    const uint32_t ups0 = lds_addr(ups);
    uint8_t *const ex = exchange + wave * 16 * PITCH;
    // block of up: 512-byte rows, the 32-byte chunk c of row k kept at chunk
    // c ^ f(k) (see run_tile)
    const int slot = lane & 31;
    const int fB = (fi >> 2) | ((fg & 1) << 2);

    for (int t = blockIdx.x; t < units; t += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(find_group(first, groups, t, lane));
        int lo, hi;
        group_bounds(starts, e, lo, hi);
        const int in = t - __builtin_amdgcn_readfirstlane(first[e]);
        const int mt = in / p.spans;
        const int n_begin = (in - mt * p.spans) * p.span * EX_COLS;
        const int n_end = min(p.N, n_begin + p.span * EX_COLS);
        const int m0 = lo + mt * BM;
        const bool delta = e < p.E;
        const u32x4_t ru =
            make_rsrc4(p.up + (size_t)(delta ? e : 0) * p.r * p.N, delta ? (uint32_t)p.r * N2 : 0u);
        auto load_up = [&](int n0) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int k = 2 * (wave * LOADS + i) + (lane >> 5);
                const int fk = (k & 3) | (((k >> 3) & 1) << 2);
                const int n = n0 + 16 * ((slot >> 1) ^ fk) + 8 * (slot & 1);
                dma16(ru, ups0 + (uint32_t)((wave * LOADS + i) * 1024),
                      n < n_end ? (uint32_t)k * N2 + (uint32_t)n * 2u : OOB);
            }
        };
        // base and out: instruction i covers rows 8 i + lane / 8 of the wave's
        // 16, columns 8 (lane % 8) .. + 7 of a group of 64
        uint32_t row_off[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = m0 + 8 * i + (lane >> 3);
            int row = -1;
            if (m >= lo && m < hi)
                row = p.rows[m];
            row_off[i] =
                (unsigned)row < (unsigned)p.M ? (uint32_t)row * N2 + (uint32_t)(lane & 7) * 16u : OOB;
        }
        auto offset = [&](int i, int n0) {
            const int n = n0 + 64 * wave;
            return n + 8 * (lane & 7) < n_end ? row_off[i] + (uint32_t)n * 2u : OOB;
        };
        load_up(n_begin);
        u32x4_t old[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            old[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, (int)offset(i, n_begin), 0, 0);
        // H of the rows, as three bf16 fragments
        bf16x8_t h[KS][3];
        const float sc = delta ? p.scale[e] : 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int m = m0 + fi, k = 32 * s + 8 * fg;
            f32x4_t x, y;
            load_h<KS == 1 ? 8 : 4>(p, delta && m < hi && k < p.r, m, k, sc, x, y);
#pragma unroll
            for (int d = 0; d < 3; ++d)
                h[s][d] = take_bf16(x, y);
        }
        for (int n0 = n_begin; n0 < n_end; n0 += EX_COLS) {
            wait_vmcnt<0>();                     // this wave's part of the block of up has landed,
            __syncthreads();                     // now everybody's
            f32x4_t acc[4], rest[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] = rest[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int q = 4 * wave + j;                        // 32-byte chunk
                    const uint32_t a = ups0 + (uint32_t)((32 * s + 8 * fg + (fi >> 2)) * 512 + 8 * (fi & 3) +
                                                         (q >> 3) * 256 + (((q & 7) ^ fB) * 32));
                    bf16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                        (lds_bf16x4_t *)lds_ptr<bf16x4_t>(a));
                    bf16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                        (lds_bf16x4_t *)lds_ptr<bf16x4_t>(a + 4 * 512));
                    const bf16x8_t fa = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, h[s][0], acc[j], 0, 0, 0);
#pragma unroll
                    for (int d = 1; d < 3; ++d)
                        rest[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, h[s][d], rest[j], 0, 0, 0);
                }
            // (LDS operations of a wave are done in order: no wait between them)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *(f32x4_t *)(ex + fi * PITCH + (16 * j + 4 * fg) * 4) = whole_product(acc[j], rest[j]);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *at = ex + (8 * i + (lane >> 3)) * PITCH + (lane & 7) * 32;
                store16(ro, offset(i, n0),
                        delta ? add_base(*(const f32x4_t *)at, *(const f32x4_t *)(at + 16), old[i]) : old[i]);
                // (past the end: an empty load)
                old[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, (int)offset(i, n0 + EX_COLS), 0, 0);
            }
            __builtin_amdgcn_wave_barrier();
            __syncthreads();                     // the block of up is read
            if (n0 + EX_COLS < n_end)
                load_up(n0 + EX_COLS);
        }
    }
}

template <int KS>
__global__ __launch_bounds__(EX_THREADS, KS <= 2 ? 2 : 1) void expand_rows_kernel(ExpandArgs p)
{
    constexpr int NB = 8;                                // 16-column blocks of a wave
    constexpr int H_PITCH = 128 * KS + 16;               // bytes of a row of H in LDS
    constexpr int PITCH = 128 * 4 + 16;                  // bytes of a row in the exchange
    constexpr int MINE = 16 * PITCH;                     // bytes of a wave: a block of up, later the exchange
    static_assert(MINE >= 32 * 256, "a block of up");
    __shared__ __attribute__((aligned(1024))) uint8_t own[EX_WAVES * MINE];
    __shared__ __attribute__((aligned(16))) uint8_t hs[XR_ROWS * H_PITCH];
    __shared__ uint32_t s_row[XR_ROWS + 16];             // byte offset of each row in base and out
    __shared__ int first[GR_GROUPS + 1], starts[GR_GROUPS + 1];
    __shared__ int wsum[EX_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fi = lane & 15, fg = lane >> 4;
    const int groups = p.E + (p.copy ? 1 : 0);
    const int units =
        scan_tiles<EX_THREADS>(p.offsets, p.E, p.M, groups, p.span, p.spans, first, starts, wsum);
    const uint32_t N2 = (uint32_t)p.N * 2u;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.base, (uint32_t)p.M * N2);
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.out, (uint32_t)p.M * N2);
    const uint32_t mine = lds_addr(own) + (uint32_t)(wave * MINE);
    uint8_t *const ex = own + wave * MINE;
    // block of up: 32 rows of 256 bytes, as stream_kernel's for NB = 8
    auto fold = [](int k) { return (k & 3) | (((k >> 3) & 1) << 2); };
    const int b_row = lane >> 4, b_slot = lane & 15;
    const int f_lane = fold(8 * fg + (fi >> 2));

    for (int t = blockIdx.x; t < units; t += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(find_group(first, groups, t, lane));
        int lo, hi;
        group_bounds(starts, e, lo, hi);
        const int in = t - __builtin_amdgcn_readfirstlane(first[e]);
        const int mt = in / p.spans;
        const int n0 = (in - mt * p.spans) * XR_COLS + 128 * wave;
        const int m0 = lo + mt * p.span;
        const int count = min(hi - m0, p.span);          // rows of this workgroup
        const bool delta = e < p.E;
        const u32x4_t ru =
            make_rsrc4(p.up + (size_t)(delta ? e : 0) * p.r * p.N, delta ? (uint32_t)p.r * N2 : 0u);
        auto load_up = [&](int s) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int k = 4 * i + b_row;
                const int n = n0 + 16 * ((b_slot >> 1) ^ fold(k)) + 8 * (b_slot & 1);
                dma16(ru, mine + i * 1024, n < p.N ? (uint32_t)(32 * s + k) * N2 + (uint32_t)n * 2u : OOB);
            }
        };
        load_up(0);
        for (int i = tid; i < XR_ROWS + 16; i += EX_THREADS) {
            int row = -1;
            if (i < count)
                row = p.rows[m0 + i];
            s_row[i] = (unsigned)row < (unsigned)p.M ? (uint32_t)row * N2 : OOB;
        }
        // H of the workgroup's rows, 8 values a time
        if (delta) {
            const float sc = p.scale[e];
            for (int i = tid; i < (count + 15) / 16 * 16 * 4 * KS; i += EX_THREADS) {
                const int r = i / (4 * KS), k = 8 * (i - r * 4 * KS);
                f32x4_t x, y;
                load_h<4>(p, r < count && k < p.r, m0 + r, k, sc, x, y);
                *(f32x4_t *)(hs + r * H_PITCH + 4 * k) = x;
                *(f32x4_t *)(hs + r * H_PITCH + 4 * k + 16) = y;
            }
        }
        bf16x8_t fa[KS][NB];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            wait_vmcnt<0>();
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const uint32_t a =
                    mine + (uint32_t)((8 * fg + (fi >> 2)) * 256 + 8 * (fi & 3) + ((j ^ f_lane) * 32));
                bf16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (lds_bf16x4_t *)lds_ptr<bf16x4_t>(a));
                bf16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (lds_bf16x4_t *)lds_ptr<bf16x4_t>(a + 4 * 256));
                fa[s][j] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
            }
            wait_lgkmcnt0();                             // read before it is filled again
            if (s + 1 < KS)
                load_up(s + 1);
        }
        __syncthreads();                                 // rows and H are there
        // instruction i of a block of 16 rows: rows 4 i + lane / 16, columns
        // 8 (lane % 16) .. + 7 of the wave's 128
        const int nc = n0 + 8 * (lane & 15);
        auto offset = [&](int b, int i) {
            const uint32_t o = s_row[16 * b + 4 * i + (lane >> 4)];
            return nc < p.N && o != OOB ? o + (uint32_t)nc * 2u : OOB;
        };
        const int blocks = (count + 15) / 16;
        u32x4_t old[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            old[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, (int)offset(0, i), 0, 0);
        for (int b = 0; b < blocks; ++b) {
            // the next block's rows (past the last: s_row holds none)
            u32x4_t next[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                next[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, (int)offset(b + 1, i), 0, 0);
            f32x4_t acc[NB], rest[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j)
                acc[j] = rest[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
            if (delta) {
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const uint8_t *at = hs + (16 * b + fi) * H_PITCH + 4 * (32 * s + 8 * fg);
                    f32x4_t x = *(const f32x4_t *)at, y = *(const f32x4_t *)(at + 16);
                    const bf16x8_t h = take_bf16(x, y);
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[s][j], h, acc[j], 0, 0, 0);
#pragma unroll
                    for (int d = 1; d < 3; ++d) {
                        const bf16x8_t l = take_bf16(x, y);
#pragma unroll
                        for (int j = 0; j < NB; ++j)
                            rest[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[s][j], l, rest[j], 0, 0, 0);
                    }
                }
            }
            // (LDS operations of a wave are done in order: no wait between them)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                *(f32x4_t *)(ex + fi * PITCH + (16 * j + 4 * fg) * 4) = whole_product(acc[j], rest[j]);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *at = ex + (4 * i + (lane >> 4)) * PITCH + (lane & 15) * 32;
                store16(ro, offset(b, i),
                        delta ? add_base(*(const f32x4_t *)at, *(const f32x4_t *)(at + 16), old[i]) : old[i]);
                old[i] = next[i];
            }
            __builtin_amdgcn_wave_barrier();
        }
        __syncthreads();                                 // rows and H are read
    }
}

}  // namespace gc
