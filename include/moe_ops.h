/*
 * moe_ops.h -- C ABI of the expert path's operators on their own, beside the
 * whole layer of moe_layer.h: FP4 quantisation, the grouped product of FP4
 * operands, tokens sorted by expert, and rows sent to their experts and
 * brought back with their gates, with the gradients of both.
 *
 * They make up an expert path that is not the layer's own (another activation,
 * gates that are trained, a dense FP4 projection) and the bytes that the layer
 * reads (moe_fp4_quantize writes checkpoint layout).  Used together:
 *   moe_route_topk_noalloc -> moe_sort_tokens -> moe_fp4_quantize ->
 *   moe_dispatch (codes, scales) -> moe_fp4_matmul -> activation ->
 *   moe_fp4_quantize -> moe_fp4_matmul -> moe_combine.
 *
 * Conventions (those of moe_layer.h, and):
 *  - Every pointer is memory of the calling thread's current device, and so is
 *    `stream`.  A call only enqueues kernels on `stream`: it allocates no device
 *    memory, keeps no workspace, never waits, and may be captured into a graph.
 *    Calls on different streams are independent of one another.
 *  - Rows are contiguous along their last axis; ld* is the distance between two
 *    rows in elements, at least the row's length.  Outputs must not overlap
 *    inputs or one another.
 *  - Every index that is read from device memory (ids, inv, offsets) is checked
 *    before it is used: one out of range drops its pair or row.
 *  - A call with no rows is a no-op that returns MOE_OK.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types; MOE_DT_U8 (quantised codes and scales) for moe_dispatch only. */
typedef enum { MOE_DT_F32 = 0, MOE_DT_BF16 = 1, MOE_DT_F16 = 2, MOE_DT_U8 = 3 } moe_dtype_t;

/* Rows of FP4 values in checkpoint layout: codes uint8 [rows, K/2] (low nibble =
 * even element), scales uint8 [rows, K/32] (MXFP4, E8M0) or [rows, K/16] (NVFP4,
 * E4M3), global_scale fp32, one for each `rows_per_scale` rows (NVFP4; NULL for
 * MXFP4).  A value is code * scale * global_scale. */

/* Quantise x [rows, K] (F32, BF16 or F16) to MOE_FMT_MXFP4 or MOE_FMT_NVFP4.
 * K is a multiple of 32, rows a multiple of rows_per_scale, rows * K < 2^35.
 *  - MXFP4, a block of 32: X = clamp(floor(log2 amax) - 2, -126, 127) (-126 when
 *    amax = 0), scale code X + 127, code = v / 2^X rounded to E2M1, ties to even,
 *    saturating at 6.
 *  - NVFP4, a group of rows_per_scale rows: G = the least power of two that is
 *    not below amax / 2688, at least 2^-100 (1 when amax = 0); a block of 16: s =
 *    amax / (6 G) rounded to E4M3; code = v / (s G) rounded to E2M1 (0 when s = 0).
 * Each rounding is that of the real quotient.  rows_per_scale = 1 gives each
 * token its scale, rows_per_scale = the matrix's rows the layer's per-matrix
 * scales.  A block that holds a NaN or an infinity becomes NaN (scale code 255 /
 * 127, zero codes) and takes no part in G; moe_admit refuses such a block.
 * codes must be 16-byte aligned.  With rows_per_scale > 1 an NVFP4 call runs two
 * passes over x. */
moe_status_t moe_fp4_quantize(const void *x, int32_t dtype, int64_t rows, int64_t K, int64_t ldx, int32_t fmt,
                              int64_t rows_per_scale, uint8_t *codes, uint8_t *scales, float *global_scale,
                              void *stream);

/* The values that codes stand for, code * scale * global_scale, each rounded once to
 * dtype (F32, BF16 or F16), whatever fp32 number the global scale is.  F32 is exact
 * where the value has an fp32 number: with MXFP4 up to its range (scale code 254 is
 * 2^127, and 4 or 6 of it infinite), with NVFP4 where global_scale has at most 18 digits
 * and the value is no subnormal.  Same shapes and limits as moe_fp4_quantize. */
moe_status_t moe_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, const float *global_scale, int32_t fmt,
                                int64_t rows, int64_t K, int64_t rows_per_scale, void *out, int32_t dtype,
                                int64_t ldo, void *stream);

/* Grouped product of two FP4 operands on the block-scaled tensor cores:
 *   y[r, n] = xG[r] * wG[g] * sum_k x[r, k] * w[g, n, k]
 * for the rows r in [offsets[g], offsets[g + 1]) of each group g, accumulated in
 * fp32 and rounded once to dtype (F32, BF16 or F16).  The factor xG wG rounds to fp32
 * first, and where it leaves fp32's normal numbers the scales meet the sum one by one,
 * so that y has its value whenever y itself is in range.  x: codes and scales of
 * `rows` rows with one fp32 scale per row (rows_per_scale = 1); w: of n_groups
 * matrices of N rows with one fp32 scale per matrix (xG and wG NULL for MXFP4).
 * offsets: device int32 [n_groups + 1], non-decreasing (moe_sort_tokens writes
 * them); NULL: n_groups = 1 and every row is in it.  Rows of y before offsets[0]
 * or behind offsets[n_groups] are left as they were.  Sums do not depend on the
 * order in which the GPU runs them: equal calls give equal bits.
 * Scale codes are read as in moe_admit: a NaN code makes its block NaN, NVFP4
 * scales must not be negative.
 * K is a multiple of 32, 1 <= n_groups <= 1024; codes are 16-byte aligned and y
 * aligned to its type; rows <= 2^27; N and K <= 2^30; n_groups * N below 2^31.  The scale rows
 * are read fastest when they start on 16 bytes (K a multiple of 512, with NVFP4 of
 * 256).  Every wait inside the kernel is bounded, by two seconds and more where rows are
 * very long.  Should one give up, that launch's y is invalid, and that launch's alone:
 * whatever else is queued, runs beside it or replays it later is right.  The first
 * moe_fp4_matmul on the device that begins after that returns MOE_ERR_CUDA, having
 * enqueued nothing; one such return covers every failure up to it, and the calls after it
 * run.  A replay of a captured product is no call: a program that only replays asks with
 * a call of rows = 0, which enqueues nothing. */
moe_status_t moe_fp4_matmul(const uint8_t *x_codes, const uint8_t *x_scales, const float *x_global, int32_t rows,
                            const uint8_t *w_codes, const uint8_t *w_scales, const float *w_global, int32_t n_groups,
                            int32_t N, int32_t K, int32_t fmt, const int32_t *offsets, void *y, int32_t dtype,
                            int64_t ldy, void *stream);

/* Test hook, beside moe_debug_inject: enqueue a kernel whose one wait, on a barrier
 * that nothing completes, gives up after a millisecond, as a wait of moe_fp4_matmul
 * does at its limit of two seconds.  To both come 4 us for each of `stages` stages of 256
 * elements that are waited for (here 0 to 250000).  Causes no GPU fault and writes
 * nothing but the error. */
moe_status_t moe_debug_give_up(int32_t stages, void *stream);

/* Sort the T * k pairs p = t * k + j by their expert ids[p], ties by ascending p
 * (the order of moe_forward's routing).  An id outside [0, E), a sink target or
 * the mark of a padded token, drops its pair.  counts int32 [E]; offsets int32
 * [E + 1], the exclusive scan of counts; perm int32 [T * k]: sorted position ->
 * pair, -1 from offsets[E] on; inv int32 [T * k]: pair -> sorted position, -1
 * for a dropped one.  1 <= k <= 32, 1 <= E <= 1024, T * k <= 2^30. */
moe_status_t moe_sort_tokens(const int32_t *ids, int32_t T, int32_t k, int32_t E, int32_t *counts, int32_t *offsets,
                             int32_t *perm, int32_t *inv, void *stream);

/* Send each token's row to its pairs: xs[inv[t * k + j]] = x[t] for every pair
 * with inv in [0, rows).  x [T, H], xs [rows, H], any element type.  Rows of xs
 * that no pair names are left as they were.  The positions in inv must differ
 * from one another (moe_sort_tokens writes such an inv).  1 <= k <= 32,
 * 1 <= H <= 2^28 and T * k < 2^31 here and in the three calls below. */
moe_status_t moe_dispatch(const void *x, int32_t dtype, int32_t T, int32_t k, int32_t H, int64_t ldx,
                          const int32_t *inv, int32_t rows, void *xs, int64_t ldxs, void *stream);

/* Its gradient: dx[t] = sum_j dxs[inv[t * k + j]], in fp32 and ascending j,
 * rounded once (0 where every pair was dropped).  F32, BF16 or F16. */
moe_status_t moe_dispatch_backward(const void *dxs, int32_t dtype, int32_t rows, int32_t T, int32_t k, int32_t H,
                                   int64_t lddxs, const int32_t *inv, void *dx, int64_t lddx, void *stream);

/* Bring the rows back: y[t] = sum_j gates[t * k + j] * ys[inv[t * k + j]] over the
 * pairs with inv in [0, rows), in fp32 and ascending j, rounded once to y_dtype
 * (0 where every pair was dropped; the gates of dropped pairs are not read into
 * the sum).  ys [rows, H] and y [T, H] are F32, BF16 or F16; gates fp32 [T, k] or
 * NULL for ones. */
moe_status_t moe_combine(const void *ys, int32_t ys_dtype, int32_t rows, int32_t T, int32_t k, int32_t H,
                         int64_t ldys, const int32_t *inv, const float *gates, void *y, int32_t y_dtype, int64_t ldy,
                         void *stream);

/* Its gradients, from dy [T, H] (dy_dtype): dys[inv[t * k + j]] = gates * dy[t],
 * rounded once to ys_dtype (rows that no pair names are left as they were), and
 * dgates[t * k + j] = sum_h dy[t, h] * ys[inv, h] in fp32 (0 for a dropped pair).
 * dys or dgates may be NULL when it is not wanted (ys may then be NULL too when
 * dgates is); gates NULL stands for ones.  The positions in inv must differ. */
moe_status_t moe_combine_backward(const void *dy, int32_t dy_dtype, int64_t lddy, const void *ys, int32_t ys_dtype,
                                  int64_t ldys, int32_t rows, int32_t T, int32_t k, int32_t H, const int32_t *inv,
                                  const float *gates, void *dys, int64_t lddys, float *dgates, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
