// layer.hip -- host side of the C ABI declared in include/gemm_coll_layer.h:
// argument validation, choice of the kernel instance, launches.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "fp8_gemm.hpp"
#include "gemm_coll_layer.h"
#include "host.hpp"
#include "moe_layer.hpp"
#include "norm.hpp"

static_assert(GC_LAYER_TOKENS_MAX == gc::ML_TOKENS, "tokens");

namespace {

using namespace gc::host;

bool good_peers(const gc_bf16 *partials, int npeers, int64_t stride, int64_t elements)
{
    return npeers == 0 || (good16(partials) && stride % 8 == 0 && (npeers == 1 || stride >= elements));
}

// Bytes below 2 GiB (see fits) for matrices of one byte an element.
bool fits1(int64_t rows, int64_t cols) { return cols == 0 || rows < ((int64_t)1 << 31) / cols; }

template <int TPR, int V>
void launch_norm(const gc::NormArgs &a, int cus, hipStream_t st)
{
    constexpr int nth = gc::norm_threads<TPR>(), rows = nth / TPR;
    const int grid = (int)std::min<int64_t>(((int64_t)a.M + rows - 1) / rows, (int64_t)cus * (2048 / nth));
    if (a.codes)
        hipLaunchKernelGGL((gc::norm_kernel<TPR, V, true>), dim3(grid), dim3(nth), 0, st, a);
    else
        hipLaunchKernelGGL((gc::norm_kernel<TPR, V, false>), dim3(grid), dim3(nth), 0, st, a);
}

template <int RB, int NB, int W, int D>
void launch_fp8_stream(gc::Fp8Args &a, hipStream_t st)
{
    a.tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
    a.tiles_m = (a.M + 16 * RB - 1) / (16 * RB);
    hipLaunchKernelGGL((gc::fp8_stream_kernel<RB, NB, W, D>), dim3(a.tiles_n * a.tiles_m), dim3(64 * W), 0, st, a);
}

template <int FMT>
void launch_fp8_tiles(gc::Fp8Args &a, int cus, hipStream_t st)
{
    a.tiles_m = (a.M + 32 * FMT - 1) / (32 * FMT);
    a.tiles_n = (a.N + gc::F8_BN - 1) / gc::F8_BN;
    a.piece = std::max(1, (a.blocks + a.splits - 1) / a.splits);
    a.splits = std::max(1, (a.blocks + a.piece - 1) / a.piece);
    const dim3 grid(a.tiles_m * a.tiles_n * a.splits), b(gc::F8_THREADS);
    if (a.splits == 1) {
        if (a.npeers > 0)
            hipLaunchKernelGGL((gc::fp8_tile_kernel<FMT, gc::F8_PEERS>), grid, b, 0, st, a);
        else
            hipLaunchKernelGGL((gc::fp8_tile_kernel<FMT, gc::F8_PLAIN>), grid, b, 0, st, a);
        return;
    }
    hipLaunchKernelGGL((gc::fp8_tile_kernel<FMT, gc::F8_SUMS>), grid, b, 0, st, a);
    const int64_t vecs = (int64_t)a.M * a.N / 8;
    const int fin = (int)std::min<int64_t>((vecs + gc::F8_FINISH - 1) / gc::F8_FINISH, 8 * cus);
    hipLaunchKernelGGL(gc::fp8_finish_kernel, dim3(fin), dim3(gc::F8_FINISH), 0, st, a);
}

struct Fp8Plan {
    int rows, cols, splits;
};

// The cheapest by estimates in us, fitted to 14 sizes (M 100 to 8192, N 1024 to
// 8192, K 896 to 7168, up to 7 peers) run in every way:
//   streaming  3.5, and for every round of workgroups 0.8 and their operands'
//              bytes at 85 GB/s a CU; the weights from HBM at 5.2 TB/s
//   tiles      3, and for every round 3 and the steps of K: 0.75, 0.87, 1.5 or
//              1.75 each for 64, 128, 224 or 256 rows (0.85, 1.2, 1.9, 1.95 with
//              the peers in it)
//   cut in K   2 to 8 pieces of at least 4 steps: the tiles' steps, 3.5 for the
//              second launch, and at 6 TB/s the sums, written and read, and the
//              peers; where the sums have room
// us measured, the best of each kind, streaming / tiles / cut: N 6288, K 7168, 16
// rows 9.6 / - / -, 64 rows 12 / 41 / 18, 100 rows 20.8 / 40 / 20.1, 512 rows with 7
// peers 77 / 55 / 51, 2048 rows with 7 peers 297 / 118 / -; 200 rows, N 2048, K 4096,
// 8.2 / 25 / 17; 256 rows, N 3648, K 7168, 21 / 42 / 22, with 7 peers 22 / 50 / 25;
// 777 rows, N 3640, K 1040, 24 / 12.9 / 25, with 3 peers 26 / 17.5 / 28 (estimated
// 22 / 13.6 / 24).
Fp8Plan plan_fp8(int64_t M, int64_t N, int64_t K, int npeers, bool workspace, int cus)
{
    const int64_t blocks = (K + 127) / 128;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    Fp8Plan best = {};
    double least = 1e300;
    auto take = [&](double t, int rows, int cols, int splits) {
        if (t < least) {
            least = t;
            best = {rows, cols, splits};
        }
    };
    for (const auto &c : {std::pair<int, int>{16, 16}, {16, 32}, {32, 16}, {32, 32}, {32, 64}, {64, 32}}) {
        if (c.first > 16 && 2 * M <= c.first)
            continue;                                    // half of the rows would be empty
        const int64_t units = up(M, c.first) * up(N, c.second);
        if (units > (int64_t)1 << 22)                    // (a launch counts its threads in 32 bits)
            continue;
        const double round = 0.8 + (double)(c.first + c.second) * K / 85e3;
        const double rounds = (double)up(units, cus) * round;
        take(3.5 + std::max(rounds, 0.1 * rounds + (double)N * K / 5.2e6), c.first, c.second, 1);
    }
    static const int heights[] = {64, 128, 224, 256};
    static const double plain[] = {0.75, 0.87, 1.5, 1.75}, peers[] = {0.85, 1.2, 1.9, 1.95};
    const double bytes = (double)M * N;
    for (int h = 0; h < 4 && M > 32; ++h) {
        const int64_t tiles = up(M, heights[h]) * up(N, gc::F8_BN);
        take(3 + (double)up(tiles, cus) * (3 + blocks * (npeers ? peers : plain)[h]), heights[h], gc::F8_BN, 1);
        for (int q = 2; workspace && q <= 8 && blocks / q >= 4 && q * M * N * 4 <= kSumBytes; ++q) {
            const double steps = (double)up(blocks, q) * plain[h];
            take(6.5 + (double)up(tiles * q, cus) * (3 + steps) + bytes * (8 * q + 2 * npeers) / 6e6, heights[h],
                 gc::F8_BN, q);
        }
    }
    return best;
}

// Middle activations of moe_layer: their room in the workspace beside the
// partial tiles of all workgroups.
constexpr int64_t kMaxMiddle = (int64_t)1 << 24;
constexpr int kLayerWorkers = 256;                   // workgroups of a launch, at most
constexpr int64_t kLayerParts = 2 * 8192;            // two partial tiles of 16 x 128
constexpr int64_t kLayerChosen = (sizeof(gc::Chosen) + 255) / 256 * 256;
static_assert(kLayerParts * kLayerWorkers + kLayerChosen + 2 * kMaxMiddle <= kSumBytes, "workspace");
static_assert(kLayerWorkers <= kMaxWorkers, "counters");

// Lanes per token and experts per lane of the router.
template <bool BF16>
void launch_up(const gc::LayerArgs &a, int grid, hipStream_t st)
{
    const dim3 g(grid), b(gc::ML_THREADS);
    if (a.route.E <= 64)
        hipLaunchKernelGGL((gc::moe_up_kernel<16, 4, BF16>), g, b, 0, st, a);
    else if (a.route.E <= 256)
        hipLaunchKernelGGL((gc::moe_up_kernel<16, 16, BF16>), g, b, 0, st, a);
    else
        hipLaunchKernelGGL((gc::moe_up_kernel<64, 16, BF16>), g, b, 0, st, a);
}

void launch_layer(gc::LayerArgs &a, bool bf16, int cus, hipStream_t st)
{
    const int grid = std::min(cus, kLayerWorkers);
    a.part_slots = 2 * grid;
    a.min_quads = 4;                                 // (8, 12, 24: one token 73, 76, 96 us; 3: as 4)
    a.tiles_n = (a.F + 63) / 64;
    if (bf16)
        launch_up<true>(a, grid, st);
    else
        launch_up<false>(a, grid, st);
    a.tiles_n = (a.N + 127) / 128;
    hipLaunchKernelGGL(gc::moe_down_kernel, dim3(grid), dim3(gc::ML_THREADS), 0, st, a);
}

}  // namespace

extern "C" {

int gemm_coll_rms_norm(const gc_bf16 *x, const gc_bf16 *residual, const gc_bf16 *partials, int npeers,
                       int64_t peer_stride, const void *weight, int weight_type, float eps, int64_t M,
                       int64_t N, gc_bf16 *sum, gc_bf16 *y, gc_e4m3 *codes, float *scales,
                       int64_t scale_stride, void *stream)
{
    if (M < 0 || N < 0 || npeers < 0 || npeers > 15 || N % (codes ? 16 : 8) != 0 || !(eps >= 0.0f))
        return GC_EINVAL;
    if (weight_type != GC_F32 && weight_type != GC_BF16)
        return GC_EINVAL;
    if (codes && scale_stride < (N + 127) / 128)
        return GC_EINVAL;
    if (M > INT32_MAX / 2 || N > GC_NORM_MAX)
        return GC_ENOTSUP;
    if (M == 0 || N == 0)
        return GC_OK;
    if (!good16(x) || !aligned(residual, 16) || !good16(weight) || !aligned(sum, 16))
        return GC_EINVAL;
    if (codes ? !good16(codes) || !good4(scales) : !good16(y))
        return GC_EINVAL;
    if (!good_peers(partials, npeers, peer_stride, M * N) || (!codes && y == sum))
        return GC_EINVAL;
    int cus = 0;
    if (int err = cu_count(cus))
        return err;
    gc::NormArgs a = {};
    a.x = x;
    a.residual = residual;
    a.partials = partials;
    a.peer_stride = peer_stride;
    a.npeers = npeers;
    a.weight = weight;
    a.weight_f32 = weight_type == GC_F32;
    a.eps = eps;
    a.M = (int)M;
    a.N = (int)N;
    a.sum = sum;
    a.y = y;
    a.codes = codes;
    a.scales = scales;
    a.scale_stride = scale_stride;
    // Threads of a row: a wave where one holds it (65536 rows of 512 38 us against 78
    // with 256 threads, of 1024 90 against 110; few rows the same), then 256, then
    // 1024.  With at most a row per CU, 1024 threads of one vector from 4097 columns
    // on: calls over changing inputs, rows of 7168, 7 peers, 16 rows 6.3 us against
    // 8.2, 256 rows 9.7 against 11.6 (320 rows 14.4 against 13.2, 16384 without peers
    // 169 against 160; up to 4096 columns the same).
    const hipStream_t st = (hipStream_t)stream;
    if (N <= 512)
        launch_norm<64, 1>(a, cus, st);
    else if (N <= 1024)
        launch_norm<64, 2>(a, cus, st);
    else if (N <= 2048)
        launch_norm<256, 1>(a, cus, st);
    else if (N <= 4096)
        launch_norm<256, 2>(a, cus, st);
    else if (N <= 8192 && M <= cus)
        launch_norm<1024, 1>(a, cus, st);
    else if (N <= 8192)
        launch_norm<256, 4>(a, cus, st);
    else if (N <= 16384)
        launch_norm<1024, 2>(a, cus, st);
    else
        launch_norm<1024, 4>(a, cus, st);
    return launched();
}

int gemm_coll_quantize_fp8(const gc_bf16 *x, int64_t M, int64_t K, int block_rows, gc_e4m3 *codes,
                           float *scales, int64_t scale_stride, void *stream)
{
    if (M < 0 || K < 0 || K % 16 != 0 || (block_rows != 1 && block_rows != 128) || scale_stride < (K + 127) / 128)
        return GC_EINVAL;
    if (M > INT32_MAX / 2 || K > INT32_MAX / 2)
        return GC_ENOTSUP;
    if (M == 0 || K == 0)
        return GC_OK;
    if (!good16(x) || !good16(codes) || !good4(scales))
        return GC_EINVAL;
    gc::QuantArgs a = {};
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.scale_stride = scale_stride;
    a.M = (int)M;
    a.K = (int)K;
    a.blocks_k = (int)((K + 127) / 128);
    const hipStream_t st = (hipStream_t)stream;
    if (block_rows == 1) {
        const int64_t items = M * a.blocks_k, per = gc::QT_THREADS / 16;
        const int grid = (int)std::min<int64_t>((items + per - 1) / per, 1 << 16);
        hipLaunchKernelGGL(gc::quant_rows_kernel, dim3(grid), dim3(gc::QT_THREADS), 0, st, a);
    } else {
        const int64_t blocks = (M + 127) / 128 * a.blocks_k;
        if (blocks > UINT32_MAX / gc::QT_THREADS)
            return GC_ENOTSUP;
        hipLaunchKernelGGL(gc::quant_blocks_kernel, dim3((unsigned)blocks), dim3(gc::QT_THREADS), 0, st, a);
    }
    return launched();
}

static int check_fp8(int64_t M, int64_t N, int64_t K, int npeers)
{
    if (M < 0 || N < 0 || K < 0 || K % 16 != 0 || N % 8 != 0 || npeers < 0 || npeers > 15)
        return GC_EINVAL;
    if (M > INT32_MAX / 2 || N >= 1 << 27 || K > INT32_MAX / 2 || !fits1(M, K) || !fits1(N, K) || !fits(M, N))
        return GC_ENOTSUP;
    return GC_OK;
}

int gemm_coll_gemm_fp8_plan(int64_t M, int64_t N, int64_t K, int npeers, int with_workspace, int cus,
                            gc_fp8_plan *plan)
{
    if (!plan || cus < 1 || cus > 4096)
        return GC_EINVAL;
    if (int err = check_fp8(M, N, K, npeers))
        return err;
    *plan = {0, 0, 1};
    if (M == 0 || N == 0)
        return GC_OK;
    const Fp8Plan pl = plan_fp8(M, N, K, npeers, with_workspace != 0, cus);
    *plan = {pl.rows, pl.cols, pl.splits};
    return GC_OK;
}

int gemm_coll_gemm_fp8(const gc_e4m3 *A, const float *a_scales, int64_t a_row_stride,
                       int64_t a_block_stride, const gc_e4m3 *B, const float *b_scales, int64_t M,
                       int64_t N, int64_t K, const gc_bf16 *partials, int npeers, int64_t peer_stride,
                       gc_bf16 *out, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (int err = check_fp8(M, N, K, npeers))
        return err;
    if (a_row_stride < 0 || a_block_stride < 0)
        return GC_EINVAL;
    const int64_t blocks = (K + 127) / 128, most = (int64_t)1 << 28;
    if (a_row_stride > most || a_block_stride > most)
        return GC_ENOTSUP;
    const int64_t extent = M > 0 && blocks > 0 ? (M - 1) * a_row_stride + (blocks - 1) * a_block_stride + 1 : 0;
    if (extent >= (int64_t)1 << 29 || !fits((N + 127) / 128, 2 * blocks))
        return GC_ENOTSUP;
    if (M == 0 || N == 0)
        return GC_OK;
    if (!good16(out) || !aligned(workspace, 16) || !good_peers(partials, npeers, peer_stride, M * N))
        return GC_EINVAL;
    if (K > 0 && (!good16(A) || !good16(B) || !good4(a_scales) || !good4(b_scales)))
        return GC_EINVAL;
    int cus = 0;
    if (int err = cu_count(cus))
        return err;
    gc::Fp8Args a = {};
    if (workspace) {
        if (workspace_bytes < (uint64_t)base_bytes(cus))
            return GC_EINVAL;
        a.sums = (float *)((char *)workspace + kCountBytes);
    }
    a.A = A;
    a.sa = a_scales;
    a.sa_row = (uint32_t)a_row_stride * 4u;
    a.sa_block = (uint32_t)a_block_stride * 4u;
    a.sa_bytes = (uint32_t)extent * 4u;
    a.B = B;
    a.sb = b_scales;
    a.partials = partials;
    a.peer_stride = peer_stride;
    a.npeers = npeers;
    a.out = out;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.blocks = (int)blocks;
    const hipStream_t st = (hipStream_t)stream;
    const Fp8Plan pl = plan_fp8(M, N, K, npeers, workspace != nullptr, cus);
    a.splits = pl.splits;
    if (pl.cols == 256) {
        switch (pl.rows) {
        case 64: launch_fp8_tiles<2>(a, cus, st); break;
        case 128: launch_fp8_tiles<4>(a, cus, st); break;
        case 224: launch_fp8_tiles<7>(a, cus, st); break;
        default: launch_fp8_tiles<8>(a, cus, st); break;
        }
    } else {
        switch (pl.rows * 256 + pl.cols) {
        case 16 * 256 + 16: launch_fp8_stream<1, 1, 8, 3>(a, st); break;
        case 16 * 256 + 32: launch_fp8_stream<1, 2, 4, 3>(a, st); break;
        case 32 * 256 + 16: launch_fp8_stream<2, 1, 4, 3>(a, st); break;
        case 32 * 256 + 32: launch_fp8_stream<2, 2, 4, 2>(a, st); break;
        case 32 * 256 + 64: launch_fp8_stream<2, 4, 4, 2>(a, st); break;
        default: launch_fp8_stream<4, 2, 4, 2>(a, st); break;
        }
    }
    return launched();
}

int gemm_coll_moe_layer(const gc_bf16 *X, const void *logits, int logits_type, int64_t stride, int64_t T,
                        int E, int k, int score, const float *bias, int renormalize, float scale,
                        const gc_bf16 *W1, const gc_bf16 *W2, int first, int local, int64_t K, int64_t F,
                        int64_t N, const gc_bf16 *partials, int npeers, int64_t peer_stride, gc_bf16 *out,
                        void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (T < 0 || E < 1 || E > GC_GROUPS_MAX || k < 1 || k > GC_TOPK_MAX || stride < E)
        return GC_EINVAL;
    if ((logits_type != GC_F32 && logits_type != GC_BF16) ||
        (score != GC_SCORE_SOFTMAX && score != GC_SCORE_SIGMOID))
        return GC_EINVAL;
    if (first < 0 || local < 1 || first > E - local || K < 0 || F < 0 || N < 0 || npeers < 0 || npeers > 15)
        return GC_EINVAL;
    if (K % 8 != 0 || F % 8 != 0 || N % 8 != 0)
        return GC_EINVAL;
    if (T > GC_LAYER_TOKENS_MAX || K > INT32_MAX || 2 * F > kMaxCols || N > kMaxCols)
        return GC_ENOTSUP;
    if (!fits(T, K) || !fits(K, 2 * F) || !fits(F, N) || !fits(T, N) || T * k * F > kMaxMiddle)
        return GC_ENOTSUP;
    if (T == 0 || N == 0)
        return GC_OK;
    const uintptr_t elem = logits_type == GC_BF16 ? 2 : 4;
    if (!logits || !aligned(logits, elem) || !aligned(bias, 4) || !good16(out))
        return GC_EINVAL;
    if ((K > 0 && (!good16(X) || (F > 0 && !good16(W1)))) || (F > 0 && !good16(W2)))
        return GC_EINVAL;
    if (!good16(workspace) || !good_peers(partials, npeers, peer_stride, T * N))
        return GC_EINVAL;
    int cus = 0;
    if (int err = cu_count(cus))
        return err;
    // Workspace: the counters, the partial tiles, who chose what, the middle activations.
    if (workspace_bytes < (uint64_t)base_bytes(cus))
        return GC_EINVAL;
    const int64_t parts = kLayerParts * kLayerWorkers;
    char *at = (char *)workspace + kCountBytes;
    gc::LayerArgs a = {};
    a.count = (uint32_t *)workspace;
    a.part = (float *)at;
    a.chosen = (uint32_t *)(at + parts);
    a.a = (uint16_t *)(at + parts + kLayerChosen);
    const int v = E <= 64 ? 4 : 16;                  // experts of a lane
    a.route.logits = logits;
    a.route.stride = stride;
    a.route.bias = bias;
    a.route.T = (int)T;
    a.route.E = E;
    a.route.k = k;
    a.route.score = score;
    a.route.renorm = renormalize != 0;
    a.route.scale = scale;
    a.route.vec = E % v == 0 && stride % v == 0 && aligned(logits, std::min<uintptr_t>(16, v * elem));
    a.X = X;
    a.W1 = W1;
    a.W2 = W2;
    a.partials = partials;
    a.peer_stride = peer_stride;
    a.npeers = npeers;
    a.out = out;
    a.first = first;
    a.local = local;
    a.T = (int)T;
    a.K = (int)K;
    a.F = (int)F;
    a.N = (int)N;
    const hipStream_t st = (hipStream_t)stream;
    launch_layer(a, logits_type == GC_BF16, cus, st);
    return launched();
}

}  // extern "C"
