// Internal interface between the front end of a residual block's operators
// (block_api.cpp) and their gfx950 kernels.  Not installed, not part of the
// ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace xpose {

// ----- root-mean-square norm (rms_norm_kernels.hip) ---------------------------

struct RmsNormArgs {
  const void *x, *residual, *weight;  // residual: null, or h is stored
  void *h, *y;                        // y of x's dtype, or e4m3
  float *scale, *rstd;
  int64_t rows, cols, ldx, ldr, ldh, ldy, ld_scale;
  int32_t param_dtype;
  float eps;
};
hipError_t launch_rms_norm(const RmsNormArgs &, int dtype, hipStream_t);
hipError_t launch_rms_norm_quantize(const RmsNormArgs &, int dtype, bool pow2, hipStream_t);

struct RmsNormBwdArgs {
  const void *dy, *h, *dresidual, *weight;
  const float *rstd;
  void *dx;
  float *dweight, *partial;
  int64_t rows, cols, lddy, ldh, lddr, lddx;
  int32_t param_dtype;
  int32_t parts;  // partial sums of dweight
};
// As for layer norm: partial sums of `cols` values, floats of row sums before
// them, and whether the launches are possible.
int rms_norm_bwd_parts(int64_t rows, int64_t cols);
int64_t rms_norm_bwd_row_floats(int64_t rows, int64_t cols);
bool rms_norm_bwd_fits(int64_t rows, int64_t cols);
hipError_t launch_rms_norm_backward(const RmsNormBwdArgs &, int dtype, hipStream_t);

// ----- low-rank adapters (adapter_kernels.hip) ---------------------------------

// h[row][r] = factor sum_c x[row][c] w[ids[row]][r][c]: zeros in rows without an
// adapter.  factor: 1, or alpha scale[ids[row]] where `scaled`.  And, where
// order is not null, the rows of each adapter.
struct ShrinkArgs {
  const void *x, *w;
  const float *scale_x;  // of e4m3 x
  const int32_t *ids;
  const float *scale;
  float *h;        // the first slice's sums; null: not wanted
  int32_t *order, *starts;  // rows by adapter; where each adapter's begin (count + 1)
  int64_t m, k;
  int64_t ldx, ld_scale_x, ldw, stride_w;
  int64_t slice;   // floats from one slice's sums to the next's
  int32_t rank, count;
  int32_t steps_per_slice;  // steps of 128 bytes of a row of x
  int32_t slots;   // workgroups of a tile and slice, adapters in turn
  uint32_t tiles;  // of rows; set by the launch
  float alpha;
  bool scaled;
  bool turned;     // w is (columns, rank) in memory
};
struct ShrinkPlan {
  int row_tiles;  // of 16, of a workgroup
  int slots, slices, steps_per_slice;
};
// x_size: bytes of an element of x.  whole: no slices.
ShrinkPlan shrink_plan(int64_t m, int64_t k, int64_t rank, int64_t count, int x_size, bool whole);
hipError_t launch_shrink(const ShrinkArgs &, const ShrinkPlan &, int dtype, hipStream_t);

// out[row][c] = base[row][c] + alpha scale[ids[row]] sum_r h[row][r] w[ids[row]][c][r]
struct ExpandArgs {
  const float *h;
  const void *w;
  const int32_t *ids;
  const float *scale;
  const void *base;  // may be null
  void *out;
  int64_t m, n;
  int64_t ldw, stride_w, ld_base, ld_out;
  int64_t slice;
  int32_t slices;
  int32_t rank, count;
  int32_t slots;
  int32_t strips;  // of a workgroup's columns
  int32_t tiles;   // of rows, of a workgroup; set by the launch
  float alpha;
  bool turned;     // w is (rank, columns) in memory
};
struct ExpandPlan {
  int waves_down;  // of a workgroup, 16 rows each
  int slots;
  int64_t strips, tiles;
};
// beside: for launch_adapter_both.
ExpandPlan expand_plan(int64_t m, int64_t n, int64_t count, bool beside);
hipError_t launch_expand(const ExpandArgs &, const ExpandPlan &, int dtype, int out_dtype, hipStream_t);

// da[l][r][c] = sum over l's rows of dh[row][r] x[row][c]
// db[l][c][r] = alpha scale[l] sum over l's rows of dout[row][c] h[row][r]
struct AdapterGradArgs {
  const float *dh, *h;
  const void *x, *dout;
  const int32_t *order, *starts;
  const float *scale;
  float *da, *db;    // null: not wanted
  float *partial;
  int64_t m, n, k;
  int64_t ldx, lddout;
  int32_t rank, count;
  int32_t piece;     // rows of one workgroup
  int32_t tiles_k, tiles;  // of columns, of x and of both; set by the launch
  float alpha;
};
int adapter_grad_piece(int64_t m, int64_t n, int64_t k);
int64_t adapter_grad_slots(int64_t m, int piece);
hipError_t launch_adapter_grad(const AdapterGradArgs &, int dtype, hipStream_t);
// Both at once.
hipError_t launch_adapter_both(const ExpandArgs &, const ExpandPlan &, const AdapterGradArgs &, int dtype,
                               int dx_dtype, hipStream_t);

// ----- dropout (adapter_kernels.hip) -------------------------------------------

struct DropoutArgs {
  const void *x, *residual;
  void *y;
  const uint64_t *device_seed;  // null: `seed`
  uint64_t seed, offset;
  int64_t rows, cols, ldx, ldr, ldy;
  uint32_t threshold;  // of 65536
  float factor;
  int32_t lanes;       // a power of two: neighbours that share a row
};
hipError_t launch_dropout(const DropoutArgs &, int dtype, hipStream_t);

}  // namespace xpose
