/*
 * gemm_coll_grouped.h -- routed and grouped operators beside the fused
 * projections of gemm_coll.h, for AMD MI355X (gfx950).
 *
 * What a transformer layer with experts or adapters runs next to its
 * projections on one tensor- or expert-parallel rank:
 *
 *   gemm_coll_moe_route     the router: k experts per token, their weights,
 *                           and the chosen pairs grouped by expert
 *   gemm_coll_group_rows    the grouping alone (rows by adapter)
 *   gemm_coll_grouped_gemm  one product per expert, ragged row counts, with
 *                           an optional gather of rows and silu(gate) * up
 *   gemm_coll_moe_combine   the weighted sum of every token's expert rows
 *                           plus the other ranks' partial sums
 *   gemm_coll_lora_add      low-rank adapters of many requests, added to a
 *                           projection's output
 *
 * Conventions are those of gemm_coll.h: bf16 data, fp32 sums, one rounding
 * to nearest-even at each output; dense row-major layouts ([K][N] weights);
 * device pointers on the current HIP device, 16-byte aligned for bf16 data
 * and 4-byte aligned for int32 and float; row lengths (K, N, ranks of
 * adapters) multiples of 8; work enqueued on `stream`, nothing synchronized,
 * no device memory allocated; a negative return launches nothing.  Outputs
 * must not overlap inputs (lora_add's out may be its base).  A buffer
 * addressed as one (X, out, one expert's weights) must be below 2 GiB
 * (GC_ENOTSUP; so are weights of more than 2^24 columns); the weights of all
 * experts together may be larger.
 *
 * Groups.  A grouping of n items into `groups` groups is
 *   offsets  int32 [groups + 1]: group g owns positions [offsets[g], offsets[g+1])
 *   rows     int32 [n]: row of the item at each position (items in no group
 *            come last, after offsets[groups], in their order)
 *   slots    int32 [n]: position of each item, -1 for an item in no group
 * With the experts first .. first + local - 1 on this rank, the grouping of
 * ids - first into `local` groups (group_rows) is what the products and the
 * combine take: the other ranks' pairs get slot -1 and come last.  (The
 * router's own slots count the pairs of all experts; with a part of its
 * offsets they would name rows that no product has written.)
 * Groups keep the order of their items.  offsets do not fall.  Kernels read
 * offsets and rows on the device and stay in bounds whatever they hold: an
 * offset is clamped to [0, S], a row outside its matrix reads as zeros (and is
 * not written by lora_add).
 *
 * Workspace.  `workspace` points to workspace_bytes of device memory, zeroed
 * before its first use and not used by two calls at the same time; calls on
 * one stream may share one.  Each call says below how much it needs.
 */
#ifndef GEMM_COLL_GROUPED_H
#define GEMM_COLL_GROUPED_H

#include "gemm_coll.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GC_GROUPS_MAX 1024   /* groups (experts, adapters) */
#define GC_TOPK_MAX 16       /* experts per token */

#define GC_F32 0
#define GC_BF16 1

#define GC_SCORE_SOFTMAX 0
#define GC_SCORE_SIGMOID 1

#define GC_ACT_NONE 0
#define GC_ACT_SILU_GLU 1

/* Bytes of workspace that every call here can be given on the current device
 * (64 MiB; lora_add of very many rows needs more); negative on a
 * HIP error. */
int64_t gemm_coll_grouped_workspace_bytes(void);

/*
 * Router.  For each of T tokens (rows of logits, `stride` elements apart,
 * of type GC_F32 or GC_BF16), scores s = softmax or sigmoid of its E logits
 * in fp32, and the k experts of largest key, in falling order, equal keys in
 * the order of their index; the key is the logit (bias NULL) or s + bias
 * (bias float [E]).  An expert whose logit (or key) is NaN or -inf is never
 * chosen.
 *   ids      int32 [T][k]  the experts; -1 where none was left
 *   weights  float [T][k]  s of each, divided by their sum if `renormalize`,
 *                          times `scale`; 0 where the id is -1.  (Infinite
 *                          logits share a softmax equally; a sum of 0 gives 0.)
 *   offsets, rows, slots   the grouping of the T * k pairs by expert, rows
 *                          holding token numbers; all three NULL for none
 * 1 <= E <= 1024, 1 <= k <= 16 (k may exceed E), T * k <= 2^24 (GC_ENOTSUP
 * beyond).  T == 0 writes offsets only.  More than 1024 pairs need the workspace
 * (GC_EINVAL without).
 */
int gemm_coll_moe_route(const void *logits, int logits_type, int64_t stride, int64_t T, int E, int k,
                        int score, const float *bias, int renormalize, float scale, int32_t *ids,
                        float *weights, int32_t *offsets, int32_t *rows, int32_t *slots,
                        void *workspace, uint64_t workspace_bytes, void *stream);

/*
 * Grouping of the ids [T][k] (a row is item / k) into `groups` groups; an id
 * outside [0, groups) is in none.  1 <= groups <= 1024, k >= 1 of any size,
 * T * k <= 2^24 (GC_ENOTSUP beyond).  More than 1024 ids need the workspace
 * (GC_EINVAL without).
 */
int gemm_coll_group_rows(const int32_t *ids, int64_t T, int k, int groups, int32_t *offsets,
                         int32_t *rows, int32_t *slots, void *workspace, uint64_t workspace_bytes,
                         void *stream);

/*
 * Grouped product.  For every position i of group e,
 *   y = X[rows[i]] . W[e]     (X[i] with rows NULL)
 *   out[i] = bf16(y)                                  GC_ACT_NONE
 *   out[i] = bf16(silu(y[:N/2]) * y[N/2:])            GC_ACT_SILU_GLU
 * with X [T][K], W [E][K][N], rows [S], out [S][N] or [S][N/2].  Positions in
 * no group are left untouched.  The way it runs is chosen for S rows, as if
 * all were in groups: where most are not, it may be slower than on the rows
 * that are.  N is a multiple of 16 for GC_ACT_SILU_GLU.
 * With workspace NULL no product is split along K (slower for few rows); the
 * result differs only by the order of fp32 sums, and for given sizes, offsets
 * and device it is the same in every call.
 */
int gemm_coll_grouped_gemm(const gc_bf16 *X, int64_t T, const gc_bf16 *W, const int32_t *offsets,
                           const int32_t *rows, int64_t S, int64_t K, int64_t N, int E, int act,
                           gc_bf16 *out, void *workspace, uint64_t workspace_bytes, void *stream);

/* How gemm_coll_grouped_gemm runs these sizes on a device of `cus` compute
 * units (host arithmetic only; GC_EINVAL for sizes it would refuse). */
typedef struct gc_grouped_plan {
    int32_t tiles;       /* 1: 256-column tiles of up to 256 rows; 0: streaming tiles of 128 columns */
    int32_t splits;      /* tiles: pieces of K, summed by a second launch (1: none) */
    int32_t block_rows;  /* streaming: rows of a tile, 16, 32 or 64 */
} gc_grouped_plan;
int gemm_coll_grouped_plan(int64_t S, int64_t K, int64_t N, int E, int act, int with_workspace, int cus,
                           gc_grouped_plan *plan);

/*
 * Combine.  out[t] = bf16( sum_j weights[t][j] * Y[slots[t][j]]
 *                          + sum_p partials[p][t] ),
 * fp32, summed in that order; slots outside [0, S) are skipped whatever
 * their weight.  Y [S][N], slots and weights [T][k], out [T][N]; partials:
 * npeers blocks of [T][N], peer_stride elements apart (a row slice of the
 * peers' partials, as for GEMM-RS, is a pointer offset and the full stride),
 * NULL for npeers 0.  0 <= npeers <= 15, 1 <= k <= 16.
 */
int gemm_coll_moe_combine(const gc_bf16 *Y, int64_t S, const int32_t *slots, const float *weights,
                          int64_t T, int k, int64_t N, const gc_bf16 *partials, int npeers,
                          int64_t peer_stride, gc_bf16 *out, void *stream);

/*
 * Adapters.  For every position i of group a, with m = rows[i],
 *   out[m] = bf16( base[m] + (scale[a] * X[m] . down[a]) . up[a] )
 * with X [M][K], base and out [M][N], down [G][K][r], up [G][r][N],
 * scale float [G], offsets and rows [M] a grouping of all M rows by adapter
 * (offsets[0] is 0).
 * The middle activations are fp32 sums and are multiplied as such (all 24
 * bits).  Rows in no group: out is base (base == out: untouched).
 * r <= 128, a multiple of 8; G <= 1023.  Needs
 * gemm_coll_lora_workspace_bytes(M, r) bytes of workspace.
 */
int gemm_coll_lora_add(const gc_bf16 *base, const gc_bf16 *X, const gc_bf16 *down, const gc_bf16 *up,
                       const float *scale, const int32_t *offsets, const int32_t *rows, int64_t M,
                       int64_t K, int64_t N, int r, int G, gc_bf16 *out, void *workspace,
                       uint64_t workspace_bytes, void *stream);
int64_t gemm_coll_lora_workspace_bytes(int64_t M, int r);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_COLL_GROUPED_H */
