/*
 * xpose_block -- what stands around a linear layer in a residual stream, for
 * MI355X (gfx950): root-mean-square norm with the residual's addition before
 * it (as a tensor, straight to e4m3, and its backward pass), low-rank adapters
 * of many requests beside the layer's shared product with their gradients, and
 * dropout from a counter-based generator.
 *
 * C ABI of libxpose.so.  Status codes and error rules are include/xpose.h's;
 * quantised matrices, memory, streams, errors and what "in place" means are
 * include/linear/xpose_linear.h's: DEVICE pointers, sizes and pitches in
 * elements, everything asynchronous on `stream`, nothing allocated, results
 * that repeat bit for bit, no memset or copy recorded.
 */
#ifndef XPOSE_BLOCK_H
#define XPOSE_BLOCK_H

#include <stdint.h>

#include "xpose_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* h = x + residual, y = h rstd weight, rstd = 1 / sqrt(sum h^2 / cols + eps)
 *
 * over each row of x (rows x cols).  The sum is formed in float32 and rounded
 * to dtype, x's; that is what h receives and what is normalised, in float32.
 * residual and h are both given or both NULL (h is x then).  y has x's dtype.
 * weight (NULL: ones) is cols values of param_dtype.  rstd (NULL: not wanted)
 * is `rows` float32 values.  eps >= 0.  y and h may each be x or residual
 * themselves (same pitch), not the same one.  A row whose squares sum to over
 * float32 has rstd 0; with eps 0, one whose squares are all under it has an
 * infinite one, and y is infinite or NaN.  This and the next two: rows <=
 * 2^31 - 1. */
int xpose_rms_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                   int32_t dtype, const void *residual, int64_t ld_residual,
                   void *h, int64_t ldh, const void *weight,
                   int32_t param_dtype, float eps, void *y, int64_t ldy,
                   float *rstd, void *stream);

/* The same, with y quantised from float32 (block rows 1) instead of stored.
 * flags: XPOSE_LINEAR_POW2.  q is 8-byte aligned with ldq a multiple of 8. */
int xpose_rms_norm_quantize(int64_t rows, int64_t cols, const void *x,
                            int64_t ldx, int32_t dtype, const void *residual,
                            int64_t ld_residual, void *h, int64_t ldh,
                            const void *weight, int32_t param_dtype, float eps,
                            int32_t flags, void *q, int64_t ldq, float *scale,
                            int64_t ld_scale, float *rstd, void *stream);

/* With xhat = h rstd and g = dy weight, over rows of `cols`:
 *
 *   dx      = rstd (g - xhat sum(g xhat) / cols) + dresidual
 *   dweight = sum over rows of dy xhat      (NULL: not wanted)
 *
 * h is what the norm normalised.  dresidual (NULL: zeros) is the gradient that
 * h has from elsewhere; dx is then the gradient of x and of residual alike,
 * rounded once.  dy, h, dresidual and dx are of dtype; dweight is `cols`
 * float32 values, zeros when there are no rows (the workspace is needed without
 * it too).  dx may be dy or dresidual itself (same pitch).  Over 8192 columns:
 * ceil(cols / 2048) min(rows, 256) < 2^24. */
int xpose_rms_norm_backward(int64_t rows, int64_t cols, const void *dy,
                            int64_t lddy, const void *h, int64_t ldh,
                            int32_t dtype, const float *rstd,
                            const void *dresidual, int64_t ld_dresidual,
                            const void *weight, int32_t param_dtype, void *dx,
                            int64_t lddx, float *dweight, void *workspace,
                            int64_t workspace_bytes, void *stream);
int xpose_rms_norm_backward_workspace(int64_t rows, int64_t cols,
                                      int64_t *bytes);

/* Low-rank adapters: row i of x has adapter l = ids[i], and where 0 <= l <
 * count
 *
 *   hidden[i] = x[i] A[l]^T
 *   out[i]    = base[i] + alpha scale[l] hidden[i] B[l]^T
 *
 * Rows of any other id have none: out is base there (not written where out is
 * base itself) and hidden is 0.  Ids come in any order and any mixture.
 *
 * x: m x k of dtype, or, where scale_x is not NULL, e4m3 quantised with block
 * rows 1 (16-byte aligned with ldx a multiple of 16; the 16-byte line of
 * memory that holds a row's last element is read whole).  a: `count` matrices
 * of rank x k, row pitch lda, stride_a from one to the next; b: of n x rank,
 * ldb, stride_b; both of dtype.  scale (NULL: ones): count float32 values.
 * base (NULL: zeros) and out: m x n of out_dtype, which is dtype or XPOSE_F32;
 * out may be base itself (same pitch), and base x.  hidden (NULL: not wanted):
 * m x rank float32 values, dense.  ids: m values.
 *
 * hidden is summed in float32 and stays float32; out is formed in float32 and
 * rounded once.  Where hidden, B or scale holds an infinity, what it goes into
 * is infinite or NaN.  Nothing of a row goes into another one.
 *
 * m <= 2^26, n and k <= 2^30, rank <= 4096, count <= 65535. */
int xpose_adapters(int64_t m, int64_t n, int64_t k, int64_t rank,
                   int64_t count, const void *x, int64_t ldx,
                   const float *scale_x, int64_t ld_scale_x, const void *a,
                   int64_t lda, int64_t stride_a, const void *b, int64_t ldb,
                   int64_t stride_b, int32_t dtype, const int32_t *ids,
                   const float *scale, float alpha, const void *base,
                   int64_t ld_base, void *out, int64_t ld_out,
                   int32_t out_dtype, float *hidden, void *workspace,
                   int64_t workspace_bytes, void *stream);
/* The workspace, 16-byte aligned, of a call with x of x_size bytes an element
 * (1: e4m3, 2 or 4), with or without `hidden`. */
int xpose_adapters_workspace(int64_t m, int64_t k, int64_t rank, int64_t count,
                             int32_t x_size, int32_t hidden, int64_t *bytes);

/* The gradients for dout, that of out; with dh[i] = alpha scale[l] dout[i] B[l]:
 *
 *   dx[i] = base[i] + dh[i] A[l]            (base[i] where there is no adapter)
 *   da[l] = sum of dh[i]^T x[i]
 *   db[l] = sum of alpha scale[l] dout[i]^T hidden[i]   over the rows of l
 *
 * x and dout are of dtype (x is the forward call's, or what it was quantised
 * from), hidden is the forward call's.  base (NULL: zeros) and dx: m x k of
 * dx_dtype, dtype or XPOSE_F32; dx may be base itself (same pitch), and base
 * dout or x: the gradients are then formed before dx.  da and db: dense float32
 * of count x rank x k and count x n x rank, zeros for adapters of no row.  dx,
 * da and db may each be NULL: not wanted (the workspace is the same).  Sums are
 * float32, in an order of their own for each set of sizes and ids; where a term
 * holds an infinity, its sum is infinite or NaN.  Limits as above, and
 * (m / 4096 + count + 1) (ceil(n / 128) + ceil(k / 128)) < 2^23 - 256. */
int xpose_adapters_backward(int64_t m, int64_t n, int64_t k, int64_t rank,
                            int64_t count, const void *dout, int64_t lddout,
                            const void *x, int64_t ldx, const void *a,
                            int64_t lda, int64_t stride_a, const void *b,
                            int64_t ldb, int64_t stride_b, int32_t dtype,
                            const int32_t *ids, const float *scale, float alpha,
                            const float *hidden, const void *base,
                            int64_t ld_base, void *dx, int64_t lddx,
                            int32_t dx_dtype, float *da, float *db,
                            void *workspace, int64_t workspace_bytes,
                            void *stream);
int xpose_adapters_backward_workspace(int64_t m, int64_t n, int64_t k,
                                      int64_t rank, int64_t count,
                                      int32_t dtype, int64_t *bytes);

/* y = residual + x / (1 - p) where an element stays, residual where it is
 * dropped (residual NULL: zeros), formed in float32 and rounded once.
 *
 * Element (row, col) takes the 16 bits number col % 8, the first word's low
 * half first, of the Philox4x32-10 block with the counter (col / 8, row, low
 * and high word of offset) and the key (low and high word of the seed), and
 * stays where they are at least t = floor(65536 p + 1/2): p counts in steps of
 * 2^-16, and what stays is multiplied by 65536 / (65536 - t).  The mask does
 * not depend on types, pitches or the other sizes.  The gradient of x is the
 * same call on that of y without residual.  device_seed, where it is not NULL,
 * is read on the GPU instead of `seed`, so that a graph gets a new mask from
 * each replay.  0 <= p <= 1 (1: all dropped).  y may be x or residual itself (same pitch).
 * rows <= 2^31 - 1, cols < 2^34. */
int xpose_dropout(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                  int32_t dtype, double p, uint64_t seed,
                  const uint64_t *device_seed, uint64_t offset,
                  const void *residual, int64_t ld_residual, void *y,
                  int64_t ldy, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* XPOSE_BLOCK_H */
