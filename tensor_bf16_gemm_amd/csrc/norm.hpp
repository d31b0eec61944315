// norm.hpp -- gfx950 device code of rms_norm and quantize_fp8.
//
//   h = x + residual + sum_p partials[p]        sum = bf16(h)
//   y = h / sqrt(mean(h^2) + eps) * weight      y, or e4m3 codes and scales
//
// HBM bounds both: every input is read once, into registers, and every output
// written once.  16384 rows of 7168 with a residual to e4m3 take 160 us (826 MB, 5.2
// TB/s, the rate of a copy), 4096 rows of 7168 quantised 17 us (88 MB), 6288 x 7168
// by blocks 24 (135 MB); 16 rows with 7 peers 5.2 in the kernel and 6.3 a call over
// changing inputs, a launch and two trips to memory.
// A row is a wave, 256 or 1024 threads (TPR) of V vectors of 8
// columns each; vector i of a row is thread i % TPR's, so that a wave's loads
// are whole lines and the 128 columns of a scale are 16 neighbouring lanes: the
// largest value of a block is four row rotations, without LDS.
#pragma once

#include "gc_kernel.hpp"

namespace gc {

struct NormArgs {
    const uint16_t *x;          // [M][N]
    const uint16_t *residual;   // [M][N] or null
    const uint16_t *partials;   // npeers blocks of [M][N], peer_stride elements apart
    int64_t peer_stride;
    int npeers;
    const void *weight;         // [N], float or bf16
    bool weight_f32;
    float eps;
    int M, N;
    uint16_t *sum;              // [M][N] or null
    uint16_t *y;                // [M][N]           (FP8: unused)
    uint8_t *codes;             // [M][N]           (FP8)
    float *scales;              // [M] rows of scale_stride
    int64_t scale_stride;
};

constexpr float E4M3_MAX = 448.0f;
constexpr uint32_t LEAST_BITS = 0x0D800000u;     // 2^-100: a block's largest value counts as at least this
constexpr uint32_t INF_BITS = 0x7F800000u;

// Largest of v over the row of 16 lanes, in all of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t v)
{
    auto step = [&](auto c) {
        const uint32_t o =
            (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + decltype(c)::value, 0xf, 0xf, true);
        v = v > o ? v : o;
    };
    step(std::integral_constant<int, 8>{});
    step(std::integral_constant<int, 4>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 1>{});
    return v;
}

// Largest magnitude, as bits: their order is that of the magnitudes, with
// infinity and NaN above all numbers.
__device__ __forceinline__ uint32_t most_bits(uint32_t most, float v)
{
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b > most ? b : most;
}

// Scale of a block of that largest magnitude, and its inverse.
__device__ __forceinline__ float block_scale(uint32_t most, float &inverse)
{
    const float top = __uint_as_float(most < LEAST_BITS ? LEAST_BITS : most);
    if (most >= INF_BITS)
        return inverse = __builtin_nanf("");
    inverse = E4M3_MAX / top;
    return top / E4M3_MAX;
}

// Eight codes.  (value * inverse is at most 448 (1 + 2^-22), which rounds to 448.)
__device__ __forceinline__ u32x2_t codes8(const float (&v)[8], float inverse)
{
    u32x2_t r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inverse, v[4 * h + 1] * inverse, 0, false);
        r[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inverse, v[4 * h + 3] * inverse, w, true);
    }
    return r;
}

__device__ __forceinline__ void unpack8(u32x4_t w, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Eight codes of bf16 values in a block of largest magnitude `top`: the quotient
// 448 v / top with a step of correction, so that one that lies between two codes
// stays there and goes to the even one (bf16 values often do; 448 v is exact).
// Values near the largest float are brought down first, by a power of two.
__device__ __forceinline__ u32x2_t codes8_bf16(const float (&v)[8], uint32_t most, float inverse)
{
    const bool large = most >= 0x71800000u;              // from 2^100 on
    const float down = large ? 0x1p-64f : 1.0f, up = large ? 0x1p64f : 1.0f;
    const float top = __uint_as_float(most < LEAST_BITS ? LEAST_BITS : most) * down;
    const float inv = inverse * up, part = inv * (1.0f / E4M3_MAX);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = v[i] * down, q0 = x * inv;
        q[i] = __builtin_fmaf(__builtin_fmaf(-q0, top, x * E4M3_MAX), part, q0);
    }
    return codes8(q, 1.0f);
}

// Sum of v over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

template <int TPR>
constexpr int norm_threads() { return TPR < 256 ? 256 : TPR; }

template <int TPR, int V, bool FP8>
__global__ __launch_bounds__(norm_threads<TPR>(), 4) void norm_kernel(NormArgs p)
{
    constexpr int NTH = norm_threads<TPR>(), ROWS = NTH / TPR, WPR = TPR / 64;
    __shared__ float part[NTH / 64];
    const int t = threadIdx.x % TPR, wave = threadIdx.x >> 6;
    const int vecs = p.N / 8;
    auto load_weight = [&](int v, float (&w)[8]) {
        const int at = t + TPR * v;
        if (at >= vecs)
            return;
        if (p.weight_f32) {
            const f32x4_t a = ((const f32x4_t *)p.weight)[2 * at], b = ((const f32x4_t *)p.weight)[2 * at + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = a[i], w[4 + i] = b[i];
        } else {
            unpack8(((const u32x4_t *)p.weight)[at], w);
        }
    };
    float w[V][8] = {};
#pragma unroll
    for (int v = 0; v < V; ++v)
        load_weight(v, w[v]);
    for (int r0 = blockIdx.x * ROWS; r0 < p.M; r0 += gridDim.x * ROWS) {
        const int r = r0 + threadIdx.x / TPR;
        const bool live = r < p.M;
        const int64_t row = (int64_t)r * p.N;
        float h[V][8] = {};
        // BATCH sources at a time, all asked for before the first is added: with few
        // rows the trips to memory are the time.
        constexpr int BATCH = V == 1 ? 8 : V == 2 ? 4 : 2;
        auto add = [&](auto count, auto source) {
            constexpr int n = decltype(count)::value;
            u32x4_t raw[n][V];
#pragma unroll
            for (int d = 0; d < n; ++d) {
                const uint16_t *src = source(d);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    raw[d][v] = (u32x4_t){0u, 0u, 0u, 0u};
                    if (src && live && t + TPR * v < vecs)
                        raw[d][v] = *((const u32x4_t *)(src + row) + t + TPR * v);
                }
            }
#pragma unroll
            for (int d = 0; d < n; ++d)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float f[8];
                    unpack8(raw[d][v], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        h[v][i] += f[i];
                }
        };
        add(std::integral_constant<int, 2>{}, [&](int d) { return d == 0 ? p.x : p.residual; });
        for (int q = 0; q < p.npeers; q += BATCH)
            add(std::integral_constant<int, BATCH>{}, [&](int d) {
                return q + d < p.npeers ? p.partials + (q + d) * p.peer_stride : nullptr;
            });
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s += h[v][i] * h[v][i];
        }
        s = wave_sum(s);
        if constexpr (WPR > 1) {
            __syncthreads();                             // (the row before has been read)
            if ((threadIdx.x & 63) == 0)
                part[wave] = s;
            __syncthreads();
            s = 0.f;
#pragma unroll
            for (int q = 0; q < WPR; ++q)
                s += part[q];
        }
        const float inv = 1.0f / sqrtf(s / (float)p.N + p.eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = t + TPR * v;
            const bool on = live && at < vecs;
            if (p.sum && on)
                *((u32x4_t *)(p.sum + row) + at) = pack_bf16x8(h[v]);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = h[v][i] * inv * w[v][i];
            if constexpr (FP8) {
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    most = most_bits(most, y[i]);
                if (!on)
                    most = 0;                            // (a row of infinite scale: 0 * inf)
                most = row16_max(most);
                float inverse;
                const float scale = block_scale(most, inverse);
                if (on) {
                    *((u32x2_t *)(p.codes + row) + at) = codes8(y, inverse);
                    if (at % 16 == 0)
                        p.scales[r * p.scale_stride + at / 16] = scale;
                }
            } else if (on) {
                *((u32x4_t *)(p.y + row) + at) = pack_bf16x8(y);
            }
        }
    }
}

struct QuantArgs {
    const uint16_t *x;          // [M][K]
    uint8_t *codes;             // [M][K]
    float *scales;
    int64_t scale_stride;
    int M, K, blocks_k;
};

constexpr int QT_THREADS = 256;

// A scale per row and 128 columns: 16 lanes, a vector of 8 each.
__global__ __launch_bounds__(QT_THREADS) void quant_rows_kernel(QuantArgs p)
{
    const int64_t items = (int64_t)p.M * p.blocks_k, step = (int64_t)gridDim.x * (QT_THREADS / 16);
    for (int64_t i = (int64_t)blockIdx.x * (QT_THREADS / 16) + threadIdx.x / 16; i < items; i += step) {
        const int m = (int)(i / p.blocks_k), b = (int)(i - (int64_t)m * p.blocks_k);
        const int c = 128 * b + 8 * (threadIdx.x & 15);
        const bool on = c < p.K;
        u32x4_t raw = {0u, 0u, 0u, 0u};
        if (on)
            raw = *(const u32x4_t *)(p.x + (int64_t)m * p.K + c);
        float v[8];
        unpack8(raw, v);
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            most = most_bits(most, v[j]);
        most = row16_max(most);
        float inverse;
        const float scale = block_scale(most, inverse);
        if (on)
            *(u32x2_t *)(p.codes + (int64_t)m * p.K + c) = codes8_bf16(v, most, inverse);
        if ((threadIdx.x & 15) == 0)
            p.scales[m * p.scale_stride + b] = scale;
    }
}

// A scale per block of 128 x 128: a workgroup, which keeps the block in
// registers between its largest value and its codes.
__global__ __launch_bounds__(QT_THREADS) void quant_blocks_kernel(QuantArgs p)
{
    constexpr int RPT = 128 * 16 / QT_THREADS;           // rows of a thread
    __shared__ uint32_t part[QT_THREADS / 64];
    const int bm = blockIdx.x / p.blocks_k, bk = blockIdx.x - bm * p.blocks_k;
    const int c = 128 * bk + 8 * (threadIdx.x & 15), m0 = 128 * bm + (threadIdx.x >> 4);
    u32x4_t raw[RPT];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int m = m0 + 16 * i;
        raw[i] = (u32x4_t){0u, 0u, 0u, 0u};
        if (c < p.K && m < p.M)
            raw[i] = *(const u32x4_t *)(p.x + (int64_t)m * p.K + c);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        float v[8];
        unpack8(raw[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            most = most_bits(most, v[j]);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)most, d);
        most = most > o ? most : o;
    }
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < QT_THREADS / 64; ++q)
        most = most > part[q] ? most : part[q];
    float inverse;
    const float scale = block_scale(most, inverse);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int m = m0 + 16 * i;
        float v[8];
        unpack8(raw[i], v);
        if (c < p.K && m < p.M)
            *(u32x2_t *)(p.codes + (int64_t)m * p.K + c) = codes8_bf16(v, most, inverse);
    }
    if (threadIdx.x == 0)
        p.scales[bm * p.scale_stride + bk] = scale;
}

}  // namespace gc
