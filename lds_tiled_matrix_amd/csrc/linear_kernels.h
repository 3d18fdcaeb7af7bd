// Internal interface between the front end of the FP8 linear layer's
// operators (linear_api.cpp) and their gfx950 kernels.  Not installed, not
// part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace xpose {

constexpr int64_t kMaxThreads = UINT32_MAX;  // of a launch

// ----- matrix product (fp8_gemm_kernels.hip) --------------------------------

struct Fp8GemmArgs {
  const uint8_t *a, *b;
  const float *scale_a, *scale_b;
  void *c;          // the output, or the first slice's partial sums
  int64_t m, n, k;
  int64_t lda, ldb, ld_scale_a, ld_scale_b, ldc;
  int64_t slice;    // elements from one slice's partial sums to the next's
  int32_t out;      // xpose_dtype of c
  int32_t b_shift;  // 0 or 7: scale_b's column of row j is j >> b_shift
  uint32_t tiles_m, tiles_n;
  int32_t splits, blocks_per_split;  // of the ceil(k / 128) blocks
};

enum Fp8GemmMode { kFp8Rows, kFp8Tiles, kFp8Pow2 };  // what scale_b looks like

struct Fp8GemmKernel {
  int tile_m, tile_n, threads;
  bool skinny;  // waves share out k among themselves
  bool exact;   // for float32 results: products summed in full
  hipError_t (*launch)(const Fp8GemmArgs &, Fp8GemmMode, hipStream_t);
};
const Fp8GemmKernel *fp8_gemm_kernels(int *count);

// c = sum over slices of partial, rounded to `out`.
struct Fp8ReduceArgs {
  const float *partial;
  void *c;
  int64_t m, n, ldc;
  int32_t splits, out;
};
hipError_t launch_fp8_reduce(const Fp8ReduceArgs &, hipStream_t);

// ----- quantisation and clipping (quantize_kernels.hip) ----------------------

struct QuantizeArgs {
  const void *x;
  uint8_t *q, *qt;  // qt may be null
  float *scale, *scale_t;
  int64_t rows, cols, ldx, ldq, ld_scale, ldqt, ld_scale_t;
  uint32_t tiles_r, tiles_c;
};
constexpr int kQuantThreads = 256;  // of the workgroup that each tile takes
hipError_t launch_quantize(const QuantizeArgs &, int dtype, int block_rows,
                           bool pow2, hipStream_t);

constexpr int kClipTable = 96;     // tensors per launch: 3 KiB of arguments
constexpr int kClipGroups = 2048;  // workgroups, and partial sums, per launch
constexpr int64_t kClipChunk = 16384;  // elements of one workgroup's step

struct ClipArgs {
  const void *in[kClipTable];
  void *out[kClipTable];
  int64_t count[kClipTable];
  uint32_t end[kClipTable];  // chunks of tensors 0..i together
  uint8_t dtype[kClipTable];
  int32_t tensors;
  uint32_t chunks;
  double *partial;     // all launches' partial sums
  int32_t first;       // where this launch's begin
  int32_t partials;    // how many there are
  double max_norm, eps;
  float *norm;         // null but in one launch
};
hipError_t launch_clip_squares(const ClipArgs &, uint32_t groups, hipStream_t);
hipError_t launch_clip_scale(const ClipArgs &, uint32_t groups, hipStream_t);

// ----- layer norm (norm_kernels.hip) -----------------------------------------

struct NormArgs {
  const void *x, *weight, *bias;
  void *y;  // of x's dtype, or e4m3
  float *scale, *mean, *rstd;
  int64_t rows, cols, ldx, ldy, ld_scale;
  int32_t param_dtype;
  float eps;
};
hipError_t launch_layer_norm(const NormArgs &, int dtype, hipStream_t);
hipError_t launch_layer_norm_quantize(const NormArgs &, int dtype, bool pow2,
                                      hipStream_t);

struct NormBwdArgs {
  const void *dy, *x, *weight;
  const float *mean, *rstd;
  void *dx;
  float *dweight, *dbias, *partial;
  int64_t rows, cols, lddy, ldx, lddx;
  int32_t param_dtype;
  int32_t parts;  // partial sums of each gradient
};
// How many partial sums of `cols` values the backward pass of these sizes
// takes, and how many floats of row sums before them.
int norm_bwd_parts(int64_t rows, int64_t cols);
// Whether its launches are possible: rows of many columns take a workgroup for
// each block of them and partial sum.
bool norm_bwd_fits(int64_t rows, int64_t cols);
int64_t norm_bwd_row_floats(int64_t rows, int64_t cols);
hipError_t launch_layer_norm_backward(const NormBwdArgs &, int dtype,
                                      hipStream_t);

int record_hip_error(hipError_t e);  // kept by xpose_api.cpp

}  // namespace xpose
