/*
 * xpose_linear -- the operators of a normalised linear layer trained and
 * served in 8-bit floating point, for MI355X (gfx950): matrix product with
 * block scales, block quantisation, layer norm with its backward pass, and
 * the clipping of many gradients by their global norm.
 *
 * C ABI of libxpose.so (the same library as include/xpose.h, whose status
 * codes and error rules apply here too).
 *
 * Numbers.  An 8-bit value is e4m3: 1 sign, 4 exponent, 3 mantissa bits, no
 * infinity, largest magnitude 448, one NaN (0x7f).  A QUANTISED matrix is
 * rows x cols e4m3 values (row pitch ldq) and its scales: a matrix of
 * ceil(cols / 128) rows (pitch ld_scale >= the number of its columns), whose
 * element [kb][r] belongs to columns 128 kb .. 128 kb + 127 of row r (block
 * rows 1: `rows` columns) or of rows 128 r .. 128 r + 127 (block rows 128:
 * ceil(rows / 128) columns).  An element stands for value * scale.  Along a
 * row, scales of neighbouring rows are neighbours in memory, which is what a
 * tile of the product reads.
 *
 *     scale = max(amax / 448, 2^-126)      amax: the block's largest |x|
 *     with XPOSE_LINEAR_POW2 the least power of two at or above that
 *     value = e4m3(float32(x / scale))     both roundings to nearest even
 *
 * A block that holds an infinity has scale inf, finite elements 0 and the
 * others NaN; one that holds a NaN has scale NaN and only NaN elements.
 *
 * Memory and streams.  Pointers are DEVICE pointers on the current HIP device
 * unless a comment says host.  Sizes and pitches count elements.  Calls are
 * asynchronous on `stream` (NULL = the null stream), never synchronise, never
 * allocate device memory, keep nothing of one call for the next (but how many
 * workgroups of a kernel run at once, asked for once), record no memset or
 * copy, and may be captured into a graph.  A workspace is written and read by the call's own kernels only;
 * it may be reused once the call's work on the stream has finished.  Results
 * repeat bit for bit: no sum depends on the order in which workgroups run.
 * Offsets are 64 bits wide.
 *
 * Errors (validated on the host before anything is launched):
 *   XPOSE_EINVAL  a negative size, a pitch below its row, a NULL pointer that
 *                 the call would use, an extent that overflows, unknown flags,
 *                 a size that one launch of 2^32 - 1 threads cannot cover
 *                 (stated per call)
 *   XPOSE_EDTYPE  a dtype that is not XPOSE_F32, XPOSE_F16 or XPOSE_BF16
 *   XPOSE_EALIGN  a pointer off its element's size (stated per call where
 *                 more is needed)
 *   XPOSE_EALIAS  an output overlaps an input, another output or the
 *                 workspace (stated per call where it may)
 *   XPOSE_EWORKSPACE  workspace_bytes below what the call needs
 *   XPOSE_EHIP    a launch failed (xpose_last_hip_error())
 */
#ifndef XPOSE_LINEAR_H
#define XPOSE_LINEAR_H

#include <stdint.h>

#include "../xpose.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags of the calls below. */
enum {
  XPOSE_LINEAR_POW2 = 1 /* quantisation: make the scales powers of two.
                           Product: every scale IS a power of two from 2^-126
                           on (or inf, NaN); the matrix cores then apply it
                           themselves.  They read a scale's exponent only, so
                           of any other scale the mantissa would be lost.    */
};

/* What a product launches. */
typedef struct xpose_fp8_gemm_info {
  int32_t tile_m, tile_n;  /* outputs per workgroup                          */
  int32_t threads;         /* threads per workgroup                          */
  int32_t splits;          /* slices of k (1: none)                          */
  int64_t workgroups;      /* of the product's launch, all slices            */
  int64_t workspace_bytes; /* what xpose_fp8_gemm needs for this plan        */
} xpose_fp8_gemm_info;

/* c[i][j] = sum_l (a[i][l] scale_a[l / 128][i]) (b[j][l] scale_b[l / 128][j'])
 *
 * a: m x k, block rows 1.  b: n x k, block rows b_block_rows (1: j' = j, 128:
 * j' = j / 128).  c: m x n, pitch ldc, of out_dtype.  a and b are 16-byte
 * aligned with lda and ldb multiples of 16, each at most 2^23 - 16
 * (XPOSE_EALIGN, XPOSE_EINVAL); bytes between k and the pitch do not come
 * into any sum (the 16-byte line of memory that holds a row's last element is
 * read whole).  Sums of products and of blocks are float32, and the result is
 * rounded once to out_dtype.  For a 16-bit out_dtype the matrix cores' 8-bit
 * instructions multiply: among each 8 neighbouring products they drop what
 * lies under 2^-13 of the largest one's leading bit, at most 2^-10 of the
 * products' magnitudes (1.4e-5 of the result's norm on normal data, where
 * bfloat16's rounding is 1.6e-3).  For float32 the products are summed in
 * full, at half the rate.  A block's sum takes one scale after the other, each
 * step in float32: while scales lie between 2^-100 and 2^100 (or are 0) nothing
 * is lost to that, whatever their product.  k == 0 gives zeros.  A workspace
 * lets few tiles with a long k run as several slices; xpose_fp8_gemm_plan says
 * how many bytes (0: none needed); with less, the call fails with
 * XPOSE_EWORKSPACE.  The workspace is 16-byte aligned.  a and b may overlap.
 * ceil(m / 128) ceil(n / 128) < 2^24. */
int xpose_fp8_gemm(int64_t m, int64_t n, int64_t k, const void *a, int64_t lda,
                   const float *scale_a, int64_t ld_scale_a, const void *b,
                   int64_t ldb, const float *scale_b, int64_t ld_scale_b,
                   int32_t b_block_rows, void *c, int64_t ldc,
                   int32_t out_dtype, int32_t flags, void *workspace,
                   int64_t workspace_bytes, void *stream);

/* The kernel and the workspace that these sizes and flags lead to; touches no
 * GPU. */
int xpose_fp8_gemm_plan(int64_t m, int64_t n, int64_t k, int32_t b_block_rows,
                        int32_t out_dtype, int32_t flags,
                        xpose_fp8_gemm_info *info);

/* Quantises x (rows x cols, pitch ldx, of dtype) into q and scale, and, where
 * qt is not NULL, its transpose (cols x rows) into qt and scale_t, in one
 * pass over x.  block_rows: 1 or 128, of both.  q and qt are 8-byte aligned
 * with ldq and ldqt multiples of 8.  ceil(rows / 128) ceil(cols / 128) < 2^24. */
int xpose_fp8_quantize(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                       int32_t dtype, int32_t block_rows, int32_t flags,
                       void *q, int64_t ldq, float *scale, int64_t ld_scale,
                       void *qt, int64_t ldqt, float *scale_t,
                       int64_t ld_scale_t, void *stream);

/* y = (x - mean) rstd weight + bias over each row of x (rows x cols), with
 * mean = sum x / cols and rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps), in
 * float32; y has x's dtype.  weight (NULL: ones) and bias (NULL: zeros) are
 * cols values of param_dtype.  mean and rstd (rows float32 values each) are
 * both given or both NULL.  eps >= 0.  y may be x itself (same pitch).  This
 * and the next two: rows <= 2^31 - 1. */
int xpose_layer_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                     int32_t dtype, const void *weight, const void *bias,
                     int32_t param_dtype, float eps, void *y, int64_t ldy,
                     float *mean, float *rstd, void *stream);

/* The same, with y quantised from float32 (block rows 1) instead of stored.
 * q is 8-byte aligned with ldq a multiple of 8. */
int xpose_layer_norm_quantize(int64_t rows, int64_t cols, const void *x,
                              int64_t ldx, int32_t dtype, const void *weight,
                              const void *bias, int32_t param_dtype, float eps,
                              int32_t flags, void *q, int64_t ldq,
                              float *scale, int64_t ld_scale, float *mean,
                              float *rstd, void *stream);

/* With xhat = (x - mean) rstd and g = dy weight, over rows of `cols`:
 *
 *   dx      = rstd (g - sum g / cols - xhat sum(g xhat) / cols)
 *   dweight = sum over rows of dy xhat      (NULL: not wanted)
 *   dbias   = sum over rows of dy           (NULL: not wanted)
 *
 * dy, x and dx are of dtype; dweight and dbias are `cols` float32 values,
 * zeros when there are no rows.  dx may be dy itself (same pitch).  Over 8192
 * columns: ceil(cols / 2048) min(rows, 256) < 2^24. */
int xpose_layer_norm_backward(int64_t rows, int64_t cols, const void *dy,
                              int64_t lddy, const void *x, int64_t ldx,
                              int32_t dtype, const float *mean,
                              const float *rstd, const void *weight,
                              int32_t param_dtype, void *dx, int64_t lddx,
                              float *dweight, float *dbias, void *workspace,
                              int64_t workspace_bytes, void *stream);
int xpose_layer_norm_backward_workspace(int64_t rows, int64_t cols,
                                        int64_t *bytes);

/* One gradient of a clip: `count` contiguous values at `in` go to `out`. */
typedef struct xpose_clip_tensor {
  const void *in;
  void *out;
  int64_t count;
  int32_t dtype;
  int32_t reserved; /* 0 */
} xpose_clip_tensor;

/* norm = sqrt(sum of all squares), held in 64 bits and stored as float32;
 * out = in min(1, max_norm / (norm + eps)), the factor rounded to float32.
 * A norm of inf gives the factor 0, one of NaN gives NaN.  `list` is HOST
 * memory, read before the call returns.  out == in clips in place; outputs
 * overlap nothing else.  The workspace is 8-byte aligned. */
int xpose_clip_grad_norm(int64_t tensors, const xpose_clip_tensor *list,
                         double max_norm, double eps, float *norm,
                         void *workspace, int64_t workspace_bytes,
                         void *stream);
int xpose_clip_grad_norm_workspace(int64_t tensors,
                                   const xpose_clip_tensor *list,
                                   int64_t *bytes);

#ifdef __cplusplus
}
#endif
#endif /* XPOSE_LINEAR_H */
