// fp8_gemm.hpp -- gfx950 device code of gemm_fp8:
//   out[m][n] = bf16( sum_b sa[m][b] sb[n/128][b] sum_{k in b} A[m][k] B[n][k]
//                     + sum_p partials[p][m][n] )
// with e4m3 A [M][K] and B [N][K], b the blocks of 128 of K.
//
// A block of K is the K of one v_mfma_f32_16x16x128_f8f6f4: its 16 x 16 sums
// start from zero and enter the fp32 accumulators with one multiply-add per
// value by sa * sb, in the shadow of the next matrix instruction (4 vector
// instructions of 4 cycles beside one of 32).  The first operand is B (n rows),
// the second A (m rows), so that a lane holds one row m and four neighbouring
// columns and needs one scale per 16 rows.
//
// Inside the instruction the products of 8 neighbouring k are added first, cut
// off below 2^-13 of the largest (measured; the 16x16x32 form of the matrix
// cores does the same), their sums in fp32.  Over random values that is 1.5e-5 of
// a block's sum, a hundredth of the output's rounding, without bias; widening
// the codes to bf16 would avoid it at half the rate.
//
// The order of k inside a block does not matter as long as both operands have
// the same: lane (fi, fg) holds bytes 16 fg .. +15 and 64 + 16 fg .. +15 of its
// row's 128, so that the lanes of a load together read whole 64-byte pieces.
#pragma once

#include "gc_kernel.hpp"

namespace gc {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct Fp8Args {
    const uint8_t *A;          // [M][K]
    const float *sa;           // element (m, b) at m * sa_row + b * sa_block bytes
    uint32_t sa_row, sa_block, sa_bytes;
    const uint8_t *B;          // [N][K]
    const float *sb;           // [ceil(N / 128)][blocks]
    const uint16_t *partials;  // npeers blocks of [M][N], peer_stride elements apart
    int64_t peer_stride;
    int npeers;
    uint16_t *out;             // [M][N]
    float *sums;               // [splits][M][N]
    int M, N, K;
    int blocks;                // of K
    int tiles_m, tiles_n;
    int splits, piece;         // pieces of K, blocks in each (the last may have fewer)
};

// 4 bytes global -> LDS at lds + 4 * lane (see dma16).
__device__ __forceinline__ void dma4(u32x4_t r, uint32_t lds, uint32_t off)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(r)
                 : "memory");
}

__device__ __forceinline__ f32x4_t mfma_e4m3(i32x8_t a, i32x8_t b)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, (f32x4_t){0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8_t join(u32x4_t lo, u32x4_t hi)
{
    return (i32x8_t){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Two neighbouring accumulator blocks of a row block (32 columns), regrouped as
// by pack_pair but in fp32: lane (fi, fg) gets the 8 columns from pair_col(fg).
__device__ __forceinline__ void pair_f32(f32x4_t x, f32x4_t y, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[i]), __float_as_uint(y[i]), false, false);
        v[i] = __uint_as_float(s[0]);
        v[4 + i] = __uint_as_float(s[1]);
    }
}
__device__ __forceinline__ int pair_col(int fg) { return 8 * (fg >> 1) + 16 * (fg & 1); }

__device__ __forceinline__ void add8(float (&v)[8], u32x4_t w)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] += __uint_as_float(w[i] << 16);
        v[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// v += the peers' 8 values at element `at` of their blocks.
__device__ __forceinline__ void add_peers(float (&v)[8], const uint16_t *partials, int64_t stride, int npeers, int64_t at)
{
    int q = 0;
    for (; q + 4 <= npeers; q += 4) {
        u32x4_t w[4];
#pragma unroll
        for (int d = 0; d < 4; ++d)
            w[d] = __builtin_nontemporal_load((const u32x4_t *)(partials + (q + d) * stride + at));
#pragma unroll
        for (int d = 0; d < 4; ++d)
            add8(v, w[d]);
    }
    for (; q < npeers; ++q)
        add8(v, __builtin_nontemporal_load((const u32x4_t *)(partials + q * stride + at)));
}

__device__ __forceinline__ u32x4_t pack_bf16x8(const float (&v)[8])
{
    const u32x2_t a = pack_bf16x4((f32x4_t){v[0], v[1], v[2], v[3]});
    const u32x2_t b = pack_bf16x4((f32x4_t){v[4], v[5], v[6], v[7]});
    return (u32x4_t){a[0], a[1], b[0], b[1]};
}

// ---- few rows: streaming ----
//
// A workgroup of W waves takes 16 * RB rows by 16 * NB columns; its waves take
// alternate blocks of K, D of them in flight in registers, and add their sums
// through LDS.
template <int RB, int NB, int W, int D>
__global__ __launch_bounds__(64 * W) void fp8_stream_kernel(Fp8Args p)
{
    __shared__ f32x4_t sums[W * RB * NB * 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fi = lane & 15, fg = lane >> 4;
    const int nt = blockIdx.x % p.tiles_n, mt = blockIdx.x / p.tiles_n;
    const int m0 = mt * 16 * RB, n0 = nt * 16 * NB;
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(p.A, (uint32_t)p.M * (uint32_t)p.K);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(p.B, (uint32_t)p.N * (uint32_t)p.K);
    const __amdgpu_buffer_rsrc_t rSA = make_rsrc(p.sa, p.sa_bytes);
    const __amdgpu_buffer_rsrc_t rSB =
        make_rsrc(p.sb, (uint32_t)((p.N + 127) / 128) * (uint32_t)p.blocks * 4u);
    uint32_t a_off[RB], s_off[RB], b_off[NB], t_off[NB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int m = m0 + 16 * i + fi;
        a_off[i] = m < p.M ? (uint32_t)m * (uint32_t)p.K + 16u * fg : OOB;
        s_off[i] = m < p.M ? (uint32_t)m * p.sa_row : OOB;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int n = n0 + 16 * j + fi;
        b_off[j] = n < p.N ? (uint32_t)n * (uint32_t)p.K + 16u * fg : OOB;
        t_off[j] = (uint32_t)((n0 + 16 * j) / 128) * (uint32_t)p.blocks * 4u;
    }
    struct Slot {
        u32x4_t a[RB][2], b[NB][2];
        float sa[RB], sb[NB];
    } slot[D];
    auto load = [&](Slot &s, int b) {
        const int k0 = 128 * b;
        const bool on0 = k0 + 16 * fg < p.K, on1 = k0 + 64 + 16 * fg < p.K, on = b < p.blocks;
        auto get = [](__amdgpu_buffer_rsrc_t r, uint32_t off) {
            return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
        };
        auto num = [](__amdgpu_buffer_rsrc_t r, uint32_t off) {
            return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
        };
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            s.b[j][0] = get(rB, on0 ? b_off[j] + k0 : OOB);
            s.b[j][1] = get(rB, on1 ? b_off[j] + k0 + 64 : OOB);
            s.sb[j] = num(rSB, on ? t_off[j] + 4u * b : OOB);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            s.a[i][0] = get(rA, on0 ? a_off[i] + k0 : OOB);
            s.a[i][1] = get(rA, on1 ? a_off[i] + k0 + 64 : OOB);
            s.sa[i] = num(rSA, on ? s_off[i] + p.sa_block * b : OOB);
        }
    };
    f32x4_t acc[RB][NB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < D; ++d)
        load(slot[d], wave + W * d);
    for (int b = wave; b < p.blocks; b += W * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] += mfma_e4m3(join(slot[d].b[j][0], slot[d].b[j][1]),
                                           join(slot[d].a[i][0], slot[d].a[i][1])) *
                                 (slot[d].sa[i] * slot[d].sb[j]);
            load(slot[d], b + W * (d + D));
        }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            sums[((wave * RB + i) * NB + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    // 4 columns of a row per lane and block
    for (int c = wave; c < RB * NB; c += W) {
        const int i = c / NB, j = c - i * NB;
        f32x4_t x = sums[c * 64 + lane];
        for (int w = 1; w < W; ++w)
            x += sums[(w * RB * NB + c) * 64 + lane];
        const int m = m0 + 16 * i + fi, n = n0 + 16 * j + 4 * fg;
        if (m >= p.M || n >= p.N)
            continue;
        const int64_t at = (int64_t)m * p.N + n;
        for (int q = 0; q < p.npeers; ++q)
            x += unpack_bf16x4(*(const u32x2_t *)(p.partials + q * p.peer_stride + at));
        *(u32x2_t *)(p.out + at) = pack_bf16x4(x);
    }
}

// ---- many rows: tiles through LDS ----
//
// Eight waves, 2 along rows and 4 along columns, each 16 * FMT rows by 64
// columns of a tile of 32 * FMT by 256.  One block of K per step, two stages:
// the loads of a step are under way while the step before is multiplied.  A row
// of a stage is 128 bytes, its 16-byte chunk c kept at c ^ (row / 2 % 8), which
// spreads the 16 lanes of a fragment read's pass over all 64 banks.
constexpr int F8_THREADS = 512, F8_BN = 256;
constexpr int F8_A = 256 * 128, F8_B = 256 * 128, F8_SCALES = 8 * 256;
constexpr int F8_STAGE = F8_A + F8_B + F8_SCALES;

template <int FMT, bool SUMS>
__global__ __launch_bounds__(F8_THREADS, 2) void fp8_tile_kernel(Fp8Args p)
{
    constexpr int BMt = 32 * FMT, A_LOADS = (FMT + 1) / 2;
    __shared__ __attribute__((aligned(1024))) uint8_t stages[2 * F8_STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3, fi = lane & 15, fg = lane >> 4;
    const int unit = xcd_remap(blockIdx.x, gridDim.x);
    const int tiles = p.tiles_m * p.tiles_n;
    const int pc = unit / tiles, t = unit - pc * tiles;
    // bands of 4 row tiles, columns next, rows of the band last
    const int band = t / (4 * p.tiles_n), rest = t - band * 4 * p.tiles_n;
    const int high = min(4, p.tiles_m - 4 * band);
    const int nt = rest / high, mt = 4 * band + rest - nt * high;
    const int m0 = mt * BMt, n0 = nt * F8_BN;
    const int b0 = pc * p.piece, b1 = min(b0 + p.piece, p.blocks);
    const u32x4_t rA = make_rsrc4(p.A, (uint32_t)p.M * (uint32_t)p.K);
    const u32x4_t rB = make_rsrc4(p.B, (uint32_t)p.N * (uint32_t)p.K);
    const uint32_t lds0 = lds_addr(stages);

    // Instruction i of a wave fills rows 8 * (wave + 8 i) .. + 7 of a stage.
    const int row8 = lane >> 3;
    uint32_t a_off[A_LOADS], b_off[4];
    int chunk = (lane & 7) ^ ((row8 >> 1) | ((wave & 1) << 2));
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) {
        const int r = 8 * (wave + 8 * i) + row8, m = m0 + r;
        a_off[i] = r < BMt && m < p.M ? (uint32_t)m * (uint32_t)p.K + 16u * chunk : OOB;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + 8 * (wave + 8 * i) + row8;
        b_off[i] = n < p.N ? (uint32_t)n * (uint32_t)p.K + 16u * chunk : OOB;
    }
    // Scales: waves 0 to 3 those of 64 rows each, wave 4 those of B's two blocks.
    u32x4_t rS = make_rsrc4(p.sa, p.sa_bytes);
    uint32_t s_off = OOB, s_step = p.sa_block;
    if (wave < 4) {
        const int m = m0 + 64 * wave + lane;
        if (m < p.M)
            s_off = (uint32_t)m * p.sa_row;
    } else if (wave == 4) {
        rS = make_rsrc4(p.sb, (uint32_t)((p.N + 127) / 128) * (uint32_t)p.blocks * 4u);
        s_step = 4;
        const int nb = 2 * nt + lane;
        if (lane < 2 && 128 * nb < p.N)
            s_off = (uint32_t)nb * (uint32_t)p.blocks * 4u;
    }
    auto load = [&](int b, uint32_t st) {
        const bool on = b < b1 && 128 * b + 16 * chunk < p.K;
        const uint32_t k0 = 128u * (uint32_t)b;
#pragma unroll
        for (int i = 0; i < A_LOADS; ++i)
            if (8 * i + wave < 4 * FMT)
                dma16(rA, st + (uint32_t)((wave + 8 * i) * 1024), on ? a_off[i] + k0 : OOB);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dma16(rB, st + (uint32_t)(F8_A + (wave + 8 * i) * 1024), on ? b_off[i] + k0 : OOB);
        dma4(rS, st + (uint32_t)(F8_A + F8_B + wave * 256), b < b1 ? s_off + s_step * (uint32_t)b : OOB);
    };
    const uint32_t key = (uint32_t)((fi >> 1) & 7);
    const uint32_t frag = (uint32_t)(fi * 128) + ((fg ^ key) << 4);
    const uint32_t a_frag = (uint32_t)(wm * 16 * FMT * 128) + frag;
    const uint32_t b_frag = (uint32_t)(F8_A + wn * 64 * 128) + frag;
    const uint32_t s_frag = (uint32_t)(F8_A + F8_B + (wm * 16 * FMT + fi) * 4);
    const uint32_t t_frag = (uint32_t)(F8_A + F8_B + 4 * 256 + (wn >> 1) * 4);

    f32x4_t acc[FMT][4];
#pragma unroll
    for (int i = 0; i < FMT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    auto fragment = [&](uint32_t at) { return join(*lds_ptr<u32x4_t>(at), *lds_ptr<u32x4_t>(at ^ 64)); };
    load(b0, lds0);
    int cur = 0;
    for (int b = b0; b < b1; ++b) {
        wait_vmcnt<0>();
        barrier_only();
        const uint32_t st = opaque(lds0 + (uint32_t)(cur * F8_STAGE));
        cur ^= 1;
        load(b + 1, lds0 + (uint32_t)(cur * F8_STAGE));
        const float sb = *lds_ptr<float>(st + t_frag);
        i32x8_t fb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            fb[j] = fragment(st + b_frag + j * 2048);
#pragma unroll
        for (int i = 0; i < FMT; ++i) {
            const i32x8_t fa = fragment(st + a_frag + i * 2048);
            const float s = *lds_ptr<float>(st + s_frag + i * 64) * sb;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] += mfma_e4m3(fb[j], fa) * s;
        }
        wait_lgkmcnt0();
    }
    wait_vmcnt<0>();

    const int ln = opaque_v(lane);
    const int fi2 = ln & 15, fg2 = ln >> 4;
#pragma unroll
    for (int i = 0; i < FMT; ++i) {
        const int m = m0 + wm * 16 * FMT + 16 * i + fi2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = n0 + 64 * wn + 32 * h + pair_col(fg2);
            float v[8];
            pair_f32(acc[i][2 * h], acc[i][2 * h + 1], v);
            if (m >= p.M || n >= p.N)
                continue;
            const int64_t at = (int64_t)m * p.N + n;
            if constexpr (SUMS) {
                float *to = p.sums + (size_t)pc * p.M * p.N + at;
                *(f32x4_t *)to = (f32x4_t){v[0], v[1], v[2], v[3]};
                *(f32x4_t *)(to + 4) = (f32x4_t){v[4], v[5], v[6], v[7]};
            } else {
                add_peers(v, p.partials, p.peer_stride, p.npeers, at);
                *(u32x4_t *)(p.out + at) = pack_bf16x8(v);
            }
        }
    }
}

// out = the sums of all pieces in the order of K, plus the peers, 8 columns a thread.
constexpr int F8_FINISH = 256;
__global__ __launch_bounds__(F8_FINISH) void fp8_finish_kernel(Fp8Args p)
{
    const int64_t n = (int64_t)p.M * p.N / 8, step = (int64_t)gridDim.x * F8_FINISH;
    const size_t plane = (size_t)p.M * p.N;
    for (int64_t i = (int64_t)blockIdx.x * F8_FINISH + threadIdx.x; i < n; i += step) {
        f32x4_t x = {0.f, 0.f, 0.f, 0.f}, y = x;
        for (int s = 0; s < p.splits; ++s) {
            x += *(const f32x4_t *)(p.sums + s * plane + 8 * i);
            y += *(const f32x4_t *)(p.sums + s * plane + 8 * i + 4);
        }
        float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        add_peers(v, p.partials, p.peer_stride, p.npeers, 8 * i);
        *(u32x4_t *)(p.out + 8 * i) = pack_bf16x8(v);
    }
}

}  // namespace gc
