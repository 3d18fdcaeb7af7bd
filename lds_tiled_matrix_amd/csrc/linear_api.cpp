// C-ABI front end of the FP8 linear layer's operators
// (include/linear/xpose_linear.h): argument validation, choice of kernels and
// launch.  Validation and planning are host code that never touches the GPU.

#include "../../include/linear/xpose_linear.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>
#include <vector>

#include "linear_kernels.h"

namespace {

using xpose::record_hip_error;

constexpr int64_t kBlock = 128;
constexpr int64_t kMaxFp8Pitch = ((int64_t)1 << 23) - 16;
constexpr int64_t kMaxRows = INT32_MAX;

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

int size_of(int dtype) {
  return dtype == XPOSE_F32 ? 4 : dtype == XPOSE_F16 || dtype == XPOSE_BF16 ? 2 : 0;
}

int hip(hipError_t e) { return e == hipSuccess ? XPOSE_OK : record_hip_error(e); }

// What a call reads and writes, checked together: every range is there, fits
// 64 bits and starts at a multiple of its alignment, and no output overlaps
// anything else of the call.
class Ranges {
 public:
  // rows x cols elements of `size` bytes with a pitch of ld elements.  The
  // pitch is checked for empty matrices too, as far as it has rows to bridge.
  void matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int size,
              int align, bool output) {
    if (ld < (cols > 1 ? cols : 1)) rc_ = XPOSE_EINVAL;
    if (rc_ != XPOSE_OK || rows == 0 || cols == 0) return;
    int64_t last, bytes;
    uintptr_t end;
    if (!p || __builtin_mul_overflow(rows - 1, ld, &last) ||
        __builtin_add_overflow(last, cols, &last) ||
        __builtin_mul_overflow(last, (int64_t)size, &bytes) ||
        __builtin_add_overflow((uintptr_t)p, (uintptr_t)bytes, &end)) {
      rc_ = XPOSE_EINVAL;
      return;
    }
    if ((uintptr_t)p % align) late(XPOSE_EALIGN);
    if (rows > 1 && ld * size % align) late(XPOSE_EALIGN);
    all_[count_++] = {(uintptr_t)p, end, output, ld};
  }
  void vector(const void *p, int64_t n, int size, bool output) {
    matrix(p, 1, n, n > 1 ? n : 1, size, size, output);
  }
  // `out` may also be `in` itself.
  void same(const void *in, const void *out) { in_place_ = in == out; }
  int check() const {
    if (rc_ != XPOSE_OK || late_ != XPOSE_OK) return rc_ != XPOSE_OK ? rc_ : late_;
    for (int i = 0; i < count_; ++i)
      for (int j = i + 1; j < count_; ++j) {
        const Range &a = all_[i], &b = all_[j];
        if (!(a.output || b.output) || a.lo >= b.hi || b.lo >= a.hi) continue;
        if (in_place_ && a.lo == b.lo && a.hi == b.hi && a.ld == b.ld &&
            a.output != b.output)
          continue;
        return XPOSE_EALIAS;
      }
    return XPOSE_OK;
  }

 private:
  struct Range {
    uintptr_t lo, hi;
    bool output;
    int64_t ld;
  };
  void late(int rc) { if (late_ == XPOSE_OK) late_ = rc; }
  Range all_[12];  // no call has more
  int count_ = 0;
  int rc_ = XPOSE_OK, late_ = XPOSE_OK;
  bool in_place_ = false;
};

// ----- matrix product -----------------------------------------------------------

struct GemmPlan {
  const xpose::Fp8GemmKernel *kernel = nullptr;
  int64_t tiles_m = 0, tiles_n = 0;
  int64_t blocks_per_split = 0, splits = 1;
  int64_t workspace = 0;
};

constexpr int64_t kMaxSplits = 16;

// Estimated microseconds of a product on MI355X, for choosing among kernels,
// fitted to timings of products with m up to 500 and n up to 4096.  Of 435 shapes
// from 1 x 64 x 128 to 4352 x 28672 x 8192 (128 x 128 scales of b), each timed
// with every kernel, with eight counts of slices from 1 to 16 and as chosen here,
// the choice is within 12% of the fastest for 417 with bfloat16 results and 424
// with float32 ones.  The worst at n <= 4096 takes 16% (float32 25%) more.  Past
// that, where nothing was fitted, a few rows may take half as much again:
// 1 x 14336 x 2048 takes 15.9 us in 16 slices as chosen, 10.5 in 4.
//
// Tiles: a start, then a block of k takes `one` while the compute units hold a
// workgroup each and `two` with two of the 128 x 128 tiles on each (of 256 x
// 256 only one fits); a lone workgroup waits for memory, so that the second
// costs about half as much again.
double tile_time(const xpose::Fp8GemmKernel &kern, int64_t tiles, int64_t splits,
                 int64_t blocks, double outputs, int out_size) {
  const bool large = kern.tile_m == 256;
  const double one = large ? 1.75 : kern.exact ? 1.2 : 0.8;
  const double two = large ? 3.5 : kern.exact ? 1.75 : 1.15;
  const int64_t groups = tiles * splits, rest = groups % 512;
  const double rounds = (double)(groups / 512) * two + (rest > 256 ? two : rest ? one : 0);
  return (large ? 5.0 : 3.3) + rounds * (double)ceil_div(blocks, splits) + outputs * out_size / 4e6;
}

// Few rows: rounds of a workgroup a compute unit; a block of k costs more
// where it is not among the first 16, which are on their way together, and with
// more rows of a to read for it.
double skinny_time(const xpose::Fp8GemmKernel &kern, int64_t groups, int64_t blocks) {
  const bool wide = kern.tile_m == 64;
  const double first = wide ? 0.17 : kern.tile_m == 32 ? 0.12 : 0.04;
  const double later = wide ? 0.25 : kern.tile_m == 32 ? 0.165 : 0.085;
  const double b = (double)std::min<int64_t>(blocks, 16), more = (double)blocks - b;
  return 0.8 + (double)ceil_div(groups, 256) * ((wide ? 2.9 : 2.5) + first * b + later * more);
}

int plan_gemm(int64_t m, int64_t n, int64_t k, int out_dtype, GemmPlan &plan) {
  const bool exact = out_dtype == XPOSE_F32;
  const int64_t blocks = std::max<int64_t>(1, ceil_div(k, kBlock));
  const double outputs = (double)m * (double)n;
  const int skinny_rows = m <= 16 ? 16 : m <= 32 ? 32 : 64;
  int count = 0;
  const xpose::Fp8GemmKernel *table = xpose::fp8_gemm_kernels(&count);
  double best = 0;
  for (int i = 0; i < count; ++i) {
    const xpose::Fp8GemmKernel &kern = table[i];
    if (kern.exact != exact || (kern.skinny && kern.tile_m != skinny_rows)) continue;
    const int64_t tiles_m = ceil_div(m, kern.tile_m), tiles_n = ceil_div(n, kern.tile_n);
    int64_t tiles;
    if (__builtin_mul_overflow(tiles_m, tiles_n, &tiles)) continue;
    const int64_t most = kern.tile_m == 256 ? 1 : kMaxSplits;
    for (int64_t want = 1; want <= most && want <= blocks; ++want) {
      const int64_t per = ceil_div(blocks, want), splits = ceil_div(blocks, per);
      if (splits != want || tiles > xpose::kMaxThreads / kern.threads / splits) continue;
      int64_t bytes = 0;
      if (splits > 1 && (__builtin_mul_overflow(m, n, &bytes) ||
                         __builtin_mul_overflow(bytes, 4 * splits, &bytes)))
        continue;
      double t = kern.skinny ? skinny_time(kern, tiles * splits, per)
                             : tile_time(kern, tiles, splits, blocks, outputs, exact ? 4 : 2);
      // slices are written and read as float32, the latter by a launch of its own
      if (splits > 1) t += 2.2 + outputs * (8.0 * (double)splits + (exact ? 4 : 2)) / 4e6;
      if (!plan.kernel || t < best) {
        best = t;
        plan = GemmPlan{&kern, tiles_m, tiles_n, per, splits, bytes};
      }
    }
  }
  return plan.kernel ? XPOSE_OK : XPOSE_EINVAL;
}

int check_gemm(int64_t m, int64_t n, int64_t k, int32_t b_block_rows,
               int32_t out_dtype, int32_t flags) {
  if (m < 0 || n < 0 || k < 0 || k > kMaxFp8Pitch) return XPOSE_EINVAL;
  if (b_block_rows != 1 && b_block_rows != 128) return XPOSE_EINVAL;
  if (flags & ~XPOSE_LINEAR_POW2) return XPOSE_EINVAL;
  return size_of(out_dtype) ? XPOSE_OK : XPOSE_EDTYPE;
}

}  // namespace

extern "C" {

int xpose_fp8_gemm_plan(int64_t m, int64_t n, int64_t k, int32_t b_block_rows,
                        int32_t out_dtype, int32_t flags,
                        xpose_fp8_gemm_info *info) {
  int rc = check_gemm(m, n, k, b_block_rows, out_dtype, flags);
  if (rc != XPOSE_OK) return rc;
  if (!info) return XPOSE_EINVAL;
  *info = xpose_fp8_gemm_info{};
  if (m == 0 || n == 0) return XPOSE_OK;
  GemmPlan plan;
  rc = plan_gemm(m, n, k, out_dtype, plan);
  if (rc != XPOSE_OK) return rc;
  info->tile_m = plan.kernel->tile_m;
  info->tile_n = plan.kernel->tile_n;
  info->threads = plan.kernel->threads;
  info->splits = (int32_t)plan.splits;
  info->workgroups = plan.tiles_m * plan.tiles_n * plan.splits;
  info->workspace_bytes = plan.workspace;
  return XPOSE_OK;
}

int xpose_fp8_gemm(int64_t m, int64_t n, int64_t k, const void *a, int64_t lda,
                   const float *scale_a, int64_t ld_scale_a, const void *b,
                   int64_t ldb, const float *scale_b, int64_t ld_scale_b,
                   int32_t b_block_rows, void *c, int64_t ldc,
                   int32_t out_dtype, int32_t flags, void *workspace,
                   int64_t workspace_bytes, void *stream) {
  int rc = check_gemm(m, n, k, b_block_rows, out_dtype, flags);
  if (rc != XPOSE_OK) return rc;
  if (lda > kMaxFp8Pitch || ldb > kMaxFp8Pitch || workspace_bytes < 0) return XPOSE_EINVAL;
  const int64_t blocks = ceil_div(k, kBlock);
  const int64_t b_cols = b_block_rows == 1 ? n : ceil_div(n, kBlock);
  const bool empty = m == 0 || n == 0;
  GemmPlan plan;
  if (!empty) {
    rc = plan_gemm(m, n, k, out_dtype, plan);
    if (rc != XPOSE_OK) return rc;
  }
  Ranges r;
  r.matrix(a, empty ? 0 : m, k, lda, 1, 16, false);
  r.matrix(b, empty ? 0 : n, k, ldb, 1, 16, false);
  r.matrix(scale_a, empty ? 0 : blocks, m, ld_scale_a, 4, 4, false);
  r.matrix(scale_b, empty ? 0 : blocks, b_cols, ld_scale_b, 4, 4, false);
  r.matrix(c, m, n, ldc, size_of(out_dtype), size_of(out_dtype), true);
  if (plan.workspace && workspace && workspace_bytes >= plan.workspace)
    r.matrix(workspace, 1, plan.workspace, plan.workspace, 1, 16, true);
  rc = r.check();
  if (rc != XPOSE_OK || empty) return rc;
  if (plan.workspace && (!workspace || workspace_bytes < plan.workspace))
    return XPOSE_EWORKSPACE;

  xpose::Fp8GemmArgs g{};
  g.a = (const uint8_t *)a;
  g.b = (const uint8_t *)b;
  g.scale_a = scale_a;
  g.scale_b = scale_b;
  g.m = m;
  g.n = n;
  g.k = k;
  g.lda = lda;
  g.ldb = ldb;
  g.ld_scale_a = ld_scale_a;
  g.ld_scale_b = ld_scale_b;
  g.b_shift = b_block_rows == 1 ? 0 : 7;
  g.tiles_m = (uint32_t)plan.tiles_m;
  g.tiles_n = (uint32_t)plan.tiles_n;
  g.splits = (int32_t)plan.splits;
  g.blocks_per_split = (int32_t)plan.blocks_per_split;
  const bool split = plan.splits > 1;
  g.c = split ? workspace : c;
  g.ldc = split ? n : ldc;
  g.out = split ? (int32_t)XPOSE_F32 : out_dtype;
  g.slice = m * n;
  const bool pow2 = (flags & XPOSE_LINEAR_POW2) && !plan.kernel->exact;
  const xpose::Fp8GemmMode mode = pow2                ? xpose::kFp8Pow2
                                  : b_block_rows == 1 ? xpose::kFp8Rows
                                                      : xpose::kFp8Tiles;
  hipError_t e = plan.kernel->launch(g, mode, (hipStream_t)stream);
  if (e == hipSuccess && split) {
    xpose::Fp8ReduceArgs s{};
    s.partial = (const float *)workspace;
    s.c = c;
    s.m = m;
    s.n = n;
    s.ldc = ldc;
    s.splits = (int32_t)plan.splits;
    s.out = out_dtype;
    e = xpose::launch_fp8_reduce(s, (hipStream_t)stream);
  }
  return hip(e);
}

// ----- quantisation ---------------------------------------------------------------

int xpose_fp8_quantize(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                       int32_t dtype, int32_t block_rows, int32_t flags,
                       void *q, int64_t ldq, float *scale, int64_t ld_scale,
                       void *qt, int64_t ldqt, float *scale_t,
                       int64_t ld_scale_t, void *stream) {
  if (rows < 0 || cols < 0 || (block_rows != 1 && block_rows != 128) ||
      (flags & ~XPOSE_LINEAR_POW2))
    return XPOSE_EINVAL;
  const int size = size_of(dtype);
  if (!size) return XPOSE_EDTYPE;
  const int64_t tiles_r = ceil_div(rows, kBlock), tiles_c = ceil_div(cols, kBlock);
  int64_t tiles;
  if (__builtin_mul_overflow(tiles_r, tiles_c, &tiles) ||
      tiles > xpose::kMaxThreads / xpose::kQuantThreads)
    return XPOSE_EINVAL;
  Ranges r;
  r.matrix(x, rows, cols, ldx, size, size, false);
  r.matrix(q, rows, cols, ldq, 1, 8, true);
  r.matrix(scale, tiles_c, block_rows == 1 ? rows : tiles_r, ld_scale, 4, 4, true);
  if (qt) {
    r.matrix(qt, cols, rows, ldqt, 1, 8, true);
    r.matrix(scale_t, tiles_r, block_rows == 1 ? cols : tiles_c, ld_scale_t, 4, 4, true);
  }
  const int rc = r.check();
  if (rc != XPOSE_OK || tiles == 0) return rc;
  xpose::QuantizeArgs a{};
  a.x = x;
  a.q = (uint8_t *)q;
  a.qt = (uint8_t *)qt;
  a.scale = scale;
  a.scale_t = scale_t;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldq = ldq;
  a.ld_scale = ld_scale;
  a.ldqt = ldqt;
  a.ld_scale_t = ld_scale_t;
  a.tiles_r = (uint32_t)tiles_r;
  a.tiles_c = (uint32_t)tiles_c;
  return hip(xpose::launch_quantize(a, dtype, block_rows, flags & XPOSE_LINEAR_POW2,
                                    (hipStream_t)stream));
}

// ----- layer norm -------------------------------------------------------------------

static int layer_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                      int32_t dtype, const void *weight, const void *bias,
                      int32_t param_dtype, float eps, bool quantized,
                      int32_t flags, void *y, int64_t ldy, float *scale,
                      int64_t ld_scale, float *mean, float *rstd, void *stream) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || (flags & ~XPOSE_LINEAR_POW2) ||
      !(eps >= 0) || (mean == nullptr) != (rstd == nullptr))
    return XPOSE_EINVAL;
  const int size = size_of(dtype), param = size_of(param_dtype);
  if (!size || !param) return XPOSE_EDTYPE;
  Ranges r;
  r.matrix(x, rows, cols, ldx, size, size, false);
  if (weight) r.vector(weight, cols, param, false);
  if (bias) r.vector(bias, cols, param, false);
  r.matrix(y, rows, cols, ldy, quantized ? 1 : size, quantized ? 8 : size, true);
  if (quantized) r.matrix(scale, ceil_div(cols, kBlock), rows, ld_scale, 4, 4, true);
  else r.same(x, y);
  if (mean && cols) {
    r.vector(mean, rows, 4, true);
    r.vector(rstd, rows, 4, true);
  }
  const int rc = r.check();
  if (rc != XPOSE_OK || rows == 0 || cols == 0) return rc;
  xpose::NormArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.scale = scale;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldy = ldy;
  a.ld_scale = ld_scale;
  a.param_dtype = param_dtype;
  a.eps = eps;
  return hip(quantized ? xpose::launch_layer_norm_quantize(a, dtype, flags & XPOSE_LINEAR_POW2,
                                                           (hipStream_t)stream)
                       : xpose::launch_layer_norm(a, dtype, (hipStream_t)stream));
}

int xpose_layer_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                     int32_t dtype, const void *weight, const void *bias,
                     int32_t param_dtype, float eps, void *y, int64_t ldy,
                     float *mean, float *rstd, void *stream) {
  return layer_norm(rows, cols, x, ldx, dtype, weight, bias, param_dtype, eps, false, 0,
                    y, ldy, nullptr, 0, mean, rstd, stream);
}

int xpose_layer_norm_quantize(int64_t rows, int64_t cols, const void *x,
                              int64_t ldx, int32_t dtype, const void *weight,
                              const void *bias, int32_t param_dtype, float eps,
                              int32_t flags, void *q, int64_t ldq,
                              float *scale, int64_t ld_scale, float *mean,
                              float *rstd, void *stream) {
  return layer_norm(rows, cols, x, ldx, dtype, weight, bias, param_dtype, eps, true, flags,
                    q, ldq, scale, ld_scale, mean, rstd, stream);
}

// Floats of workspace: the rows' sums where the kernel needs them, then two
// partial gradients a workgroup.
static int bwd_floats(int64_t rows, int64_t cols, int64_t *floats) {
  const int64_t parts = xpose::norm_bwd_parts(rows, cols);
  int64_t f;
  if (__builtin_mul_overflow(2 * parts, cols, &f) ||
      __builtin_add_overflow(f, xpose::norm_bwd_row_floats(rows, cols), &f) ||
      f > INT64_MAX / 4)
    return XPOSE_EINVAL;
  *floats = f;
  return XPOSE_OK;
}

int xpose_layer_norm_backward_workspace(int64_t rows, int64_t cols, int64_t *bytes) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || !bytes) return XPOSE_EINVAL;
  int64_t floats = 0;
  const int rc = bwd_floats(rows, cols, &floats);
  if (rc == XPOSE_OK) *bytes = 4 * floats;
  return rc;
}

int xpose_layer_norm_backward(int64_t rows, int64_t cols, const void *dy,
                              int64_t lddy, const void *x, int64_t ldx,
                              int32_t dtype, const float *mean,
                              const float *rstd, const void *weight,
                              int32_t param_dtype, void *dx, int64_t lddx,
                              float *dweight, float *dbias, void *workspace,
                              int64_t workspace_bytes, void *stream) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || workspace_bytes < 0) return XPOSE_EINVAL;
  const int size = size_of(dtype), param = size_of(param_dtype);
  if (!size || !param) return XPOSE_EDTYPE;
  int64_t floats = 0;
  int rc = bwd_floats(rows, cols, &floats);
  if (rc != XPOSE_OK) return rc;
  if (!xpose::norm_bwd_fits(rows, cols)) return XPOSE_EINVAL;
  Ranges r;
  r.matrix(dy, rows, cols, lddy, size, size, false);
  r.matrix(x, rows, cols, ldx, size, size, false);
  if (cols) {
    r.vector(mean, rows, 4, false);
    r.vector(rstd, rows, 4, false);
  }
  if (weight) r.vector(weight, cols, param, false);
  r.matrix(dx, rows, cols, lddx, size, size, true);
  r.same(dy, dx);
  if (dweight) r.vector(dweight, cols, 4, true);
  if (dbias) r.vector(dbias, cols, 4, true);
  const bool enough = workspace && workspace_bytes / 4 >= floats;
  if (enough && floats) r.matrix(workspace, 1, floats, floats, 4, 4, true);
  rc = r.check();
  if (rc != XPOSE_OK || cols == 0) return rc;
  if (floats && !enough) return XPOSE_EWORKSPACE;
  xpose::NormBwdArgs a{};
  a.dy = dy;
  a.x = x;
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partial = (float *)workspace;
  a.rows = rows;
  a.cols = cols;
  a.lddy = lddy;
  a.ldx = ldx;
  a.lddx = lddx;
  a.param_dtype = param_dtype;
  a.parts = xpose::norm_bwd_parts(rows, cols);
  return hip(xpose::launch_layer_norm_backward(a, dtype, (hipStream_t)stream));
}

// ----- clipping -------------------------------------------------------------------------

// The launches of a list: runs of its tensors that are not empty, each of at
// most kClipTable tensors and 2^32 - 1 chunks.
static int clip_launches(int64_t tensors, const xpose_clip_tensor *list,
                         std::vector<xpose::ClipArgs> &launches, int64_t *partials) {
  if (tensors < 0 || (tensors && !list)) return XPOSE_EINVAL;
  *partials = 0;
  int64_t chunks = 0;
  auto close = [&] {
    if (launches.empty()) return;
    xpose::ClipArgs &a = launches.back();
    a.chunks = (uint32_t)chunks;
    a.first = (int32_t)*partials;
    *partials += std::min<int64_t>(chunks, xpose::kClipGroups);
  };
  for (int64_t i = 0; i < tensors; ++i) {
    const xpose_clip_tensor &t = list[i];
    if (t.count < 0 || t.reserved) return XPOSE_EINVAL;
    if (!size_of(t.dtype)) return XPOSE_EDTYPE;
    if (t.count == 0) continue;
    const int64_t more = ceil_div(t.count, xpose::kClipChunk);
    if (more > UINT32_MAX) return XPOSE_EINVAL;
    if (launches.empty() || launches.back().tensors == xpose::kClipTable ||
        chunks + more > UINT32_MAX) {
      close();
      if (*partials > INT32_MAX - xpose::kClipGroups) return XPOSE_EINVAL;
      launches.emplace_back();
      chunks = 0;
    }
    chunks += more;
    xpose::ClipArgs &a = launches.back();
    a.in[a.tensors] = t.in;
    a.out[a.tensors] = t.out;
    a.count[a.tensors] = t.count;
    a.dtype[a.tensors] = (uint8_t)t.dtype;
    a.end[a.tensors] = (uint32_t)chunks;
    ++a.tensors;
  }
  close();
  return XPOSE_OK;
}

// Errors as for matrices: outputs overlap nothing but their own input.  One
// sort instead of all pairs: a model has hundreds of gradients.
static int check_clip(int64_t tensors, const xpose_clip_tensor *list, const float *norm,
                      const void *workspace, int64_t workspace_bytes) {
  struct Range {
    uintptr_t lo, hi;
    bool output;
    int64_t owner;
  };
  std::vector<Range> all;
  all.reserve(2 * tensors + 2);
  bool aligned = (uintptr_t)norm % 4 == 0 && (uintptr_t)workspace % 8 == 0;
  if (!norm) return XPOSE_EINVAL;
  for (int64_t i = 0; i < tensors; ++i) {
    const xpose_clip_tensor &t = list[i];
    if (t.count == 0) continue;
    const int size = size_of(t.dtype);
    int64_t bytes;
    uintptr_t in_end, out_end;
    if (!t.in || !t.out || __builtin_mul_overflow(t.count, (int64_t)size, &bytes) ||
        __builtin_add_overflow((uintptr_t)t.in, (uintptr_t)bytes, &in_end) ||
        __builtin_add_overflow((uintptr_t)t.out, (uintptr_t)bytes, &out_end))
      return XPOSE_EINVAL;
    aligned &= (uintptr_t)t.in % size == 0 && (uintptr_t)t.out % size == 0;
    if (t.in != t.out) all.push_back({(uintptr_t)t.in, in_end, false, i});
    all.push_back({(uintptr_t)t.out, out_end, true, i});
  }
  if (!aligned) return XPOSE_EALIGN;
  all.push_back({(uintptr_t)norm, (uintptr_t)norm + 4, true, -1});
  if (workspace && workspace_bytes > 0)
    all.push_back({(uintptr_t)workspace, (uintptr_t)workspace + (uintptr_t)workspace_bytes, true, -2});
  std::sort(all.begin(), all.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
  uintptr_t end = 0, out_end = 0;  // of all ranges so far, and of the outputs
  for (const Range &x : all) {
    if (x.lo < out_end || (x.output && x.lo < end)) return XPOSE_EALIAS;
    end = std::max(end, x.hi);
    if (x.output) out_end = std::max(out_end, x.hi);
  }
  return XPOSE_OK;
}

int xpose_clip_grad_norm_workspace(int64_t tensors, const xpose_clip_tensor *list,
                                   int64_t *bytes) {
  if (!bytes) return XPOSE_EINVAL;
  try {
    std::vector<xpose::ClipArgs> launches;
    int64_t partials = 0;
    const int rc = clip_launches(tensors, list, launches, &partials);
    if (rc == XPOSE_OK) *bytes = 8 * partials;
    return rc;
  } catch (...) {  // no host memory
    return XPOSE_EINVAL;
  }
}

int xpose_clip_grad_norm(int64_t tensors, const xpose_clip_tensor *list,
                         double max_norm, double eps, float *norm,
                         void *workspace, int64_t workspace_bytes, void *stream) {
  if (!(max_norm >= 0) || !(eps >= 0) || workspace_bytes < 0) return XPOSE_EINVAL;
  try {
    std::vector<xpose::ClipArgs> launches;
    int64_t partials = 0;
    int rc = clip_launches(tensors, list, launches, &partials);
    if (rc != XPOSE_OK) return rc;
    const bool enough = partials == 0 || (workspace && workspace_bytes / 8 >= partials);
    rc = check_clip(tensors, list, norm, workspace, enough ? 8 * partials : 0);
    if (rc != XPOSE_OK) return rc;
    if (!enough) return XPOSE_EWORKSPACE;
    if (launches.empty()) launches.emplace_back();  // the norm of nothing is 0
    auto groups = [](const xpose::ClipArgs &a) {
      return std::max<uint32_t>(1, std::min<uint32_t>(a.chunks, xpose::kClipGroups));
    };
    hipError_t e = hipSuccess;
    for (xpose::ClipArgs &a : launches) {
      a.partial = (double *)workspace;
      a.partials = (int32_t)partials;
      a.max_norm = max_norm;
      a.eps = eps;
      if (e == hipSuccess && a.chunks)
        e = xpose::launch_clip_squares(a, groups(a), (hipStream_t)stream);
    }
    launches.back().norm = norm;
    for (size_t i = launches.size(); i-- > 0 && e == hipSuccess;)
      e = xpose::launch_clip_scale(launches[i], groups(launches[i]), (hipStream_t)stream);
    return hip(e);
  } catch (...) {
    return XPOSE_EINVAL;
  }
}

}  // extern "C"
