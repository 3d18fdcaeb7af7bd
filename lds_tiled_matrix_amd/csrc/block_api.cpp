// C-ABI front end of a residual block's operators
// (include/linear/xpose_block.h): argument validation, workspaces and launch.
// Validation and planning are host code that never touches the GPU.

#include "../../include/linear/xpose_block.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "block_kernels.h"
#include "linear_checks.h"
#include "linear_kernels.h"

namespace {

// Under 2^32 threads of a launch: 512 for 16 rows and for an adapter's list; 256
// for 128 columns of n or k, at least, and as many workgroups again beside them.
constexpr int64_t kMaxAdapterRows = (int64_t)1 << 26, kMaxAdapterCols = (int64_t)1 << 30;
constexpr int64_t kMaxRank = 4096, kMaxAdapters = 65535;
constexpr int64_t kMaxGradGroups = (int64_t)1 << 23;

// Parts of a workspace, one after the other, each at a multiple of 16 bytes.
class Parts {
 public:
  // `count` x `more` elements of `size`; where they begin.
  int64_t add(int64_t count, int64_t more, int64_t size) {
    int64_t bytes;
    const int64_t at = total_;
    if (__builtin_mul_overflow(count, more, &bytes) || __builtin_mul_overflow(bytes, size, &bytes) ||
        __builtin_add_overflow(bytes, 15, &bytes) || __builtin_add_overflow(total_, bytes / 16 * 16, &total_))
      fits_ = false;
    return at;
  }
  bool fits() const { return fits_; }
  int64_t total() const { return total_; }

 private:
  int64_t total_ = 0;
  bool fits_ = true;
};

}  // namespace

extern "C" {

// ----- root-mean-square norm ------------------------------------------------------

static int rms_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t dtype, const void *residual,
                    int64_t ldr, void *h, int64_t ldh, const void *weight, int32_t param_dtype, float eps,
                    bool quantized, int32_t flags, void *y, int64_t ldy, float *scale, int64_t ld_scale, float *rstd,
                    void *stream) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || (flags & ~XPOSE_LINEAR_POW2) || !(eps >= 0) ||
      (residual == nullptr) != (h == nullptr))
    return XPOSE_EINVAL;
  const int size = size_of(dtype), param = size_of(param_dtype);
  if (!size || !param) return XPOSE_EDTYPE;
  Ranges r;
  const int in = r.matrix(x, rows, cols, ldx, size, size, false);
  int res = -1;
  if (residual) {
    res = r.matrix(residual, rows, cols, ldr, size, size, false);
    const int sum = r.matrix(h, rows, cols, ldh, size, size, true);
    r.same(in, sum);
    r.same(res, sum);
  }
  if (weight) r.vector(weight, cols, param, false);
  const int out = r.matrix(y, rows, cols, ldy, quantized ? 1 : size, quantized ? 8 : size, true);
  if (quantized) {
    r.matrix(scale, ceil_div(cols, kBlock), rows, ld_scale, 4, 4, true);
  } else {
    r.same(in, out);
    r.same(res, out);
  }
  if (rstd && cols) r.vector(rstd, rows, 4, true);
  const int rc = r.check();
  if (rc != XPOSE_OK || rows == 0 || cols == 0) return rc;
  xpose::RmsNormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.h = h;
  a.y = y;
  a.scale = scale;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldh = ldh;
  a.ldy = ldy;
  a.ld_scale = ld_scale;
  a.param_dtype = param_dtype;
  a.eps = eps;
  return hip(quantized ? xpose::launch_rms_norm_quantize(a, dtype, flags & XPOSE_LINEAR_POW2, (hipStream_t)stream)
                       : xpose::launch_rms_norm(a, dtype, (hipStream_t)stream));
}

int xpose_rms_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t dtype, const void *residual,
                   int64_t ld_residual, void *h, int64_t ldh, const void *weight, int32_t param_dtype, float eps,
                   void *y, int64_t ldy, float *rstd, void *stream) {
  return rms_norm(rows, cols, x, ldx, dtype, residual, ld_residual, h, ldh, weight, param_dtype, eps, false, 0, y, ldy,
                  nullptr, 0, rstd, stream);
}

int xpose_rms_norm_quantize(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t dtype, const void *residual,
                            int64_t ld_residual, void *h, int64_t ldh, const void *weight, int32_t param_dtype,
                            float eps, int32_t flags, void *q, int64_t ldq, float *scale, int64_t ld_scale, float *rstd,
                            void *stream) {
  return rms_norm(rows, cols, x, ldx, dtype, residual, ld_residual, h, ldh, weight, param_dtype, eps, true, flags, q,
                  ldq, scale, ld_scale, rstd, stream);
}

// Floats of workspace: the rows' sums where the kernel needs them, then a
// partial gradient a workgroup.
static int rms_bwd_floats(int64_t rows, int64_t cols, int64_t *floats) {
  const int64_t parts = xpose::rms_norm_bwd_parts(rows, cols);
  int64_t f;
  if (__builtin_mul_overflow(parts, cols, &f) ||
      __builtin_add_overflow(f, xpose::rms_norm_bwd_row_floats(rows, cols), &f) || f > INT64_MAX / 4)
    return XPOSE_EINVAL;
  *floats = f;
  return XPOSE_OK;
}

int xpose_rms_norm_backward_workspace(int64_t rows, int64_t cols, int64_t *bytes) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || !bytes) return XPOSE_EINVAL;
  int64_t floats = 0;
  const int rc = rms_bwd_floats(rows, cols, &floats);
  if (rc == XPOSE_OK) *bytes = 4 * floats;
  return rc;
}

int xpose_rms_norm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy, const void *h, int64_t ldh,
                            int32_t dtype, const float *rstd, const void *dresidual, int64_t ld_dresidual,
                            const void *weight, int32_t param_dtype, void *dx, int64_t lddx, float *dweight,
                            void *workspace, int64_t workspace_bytes, void *stream) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || workspace_bytes < 0) return XPOSE_EINVAL;
  const int size = size_of(dtype), param = size_of(param_dtype);
  if (!size || !param) return XPOSE_EDTYPE;
  int64_t floats = 0;
  int rc = rms_bwd_floats(rows, cols, &floats);
  if (rc != XPOSE_OK) return rc;
  if (!xpose::rms_norm_bwd_fits(rows, cols)) return XPOSE_EINVAL;
  Ranges r;
  const int in = r.matrix(dy, rows, cols, lddy, size, size, false);
  const int in_h = r.matrix(h, rows, cols, ldh, size, size, false);
  const int res = dresidual ? r.matrix(dresidual, rows, cols, ld_dresidual, size, size, false) : -1;
  if (cols) r.vector(rstd, rows, 4, false);
  if (weight) r.vector(weight, cols, param, false);
  const int out = r.matrix(dx, rows, cols, lddx, size, size, true);
  r.same(in, out);
  r.same(res, out);
  if (dx == dy || dx == dresidual) r.same(in_h, out);  // h may be either: all are read before dx is written there
  if (dweight) r.vector(dweight, cols, 4, true);
  const bool enough = workspace && workspace_bytes / 4 >= floats;
  if (enough && floats) r.matrix(workspace, 1, floats, floats, 4, 4, true);
  rc = r.check();
  if (rc != XPOSE_OK || cols == 0) return rc;
  if (floats && !enough) return XPOSE_EWORKSPACE;
  xpose::RmsNormBwdArgs a{};
  a.dy = dy;
  a.h = h;
  a.dresidual = dresidual;
  a.weight = weight;
  a.rstd = rstd;
  a.dx = dx;
  a.dweight = dweight;
  a.partial = (float *)workspace;
  a.rows = rows;
  a.cols = cols;
  a.lddy = lddy;
  a.ldh = ldh;
  a.lddr = ld_dresidual;
  a.lddx = lddx;
  a.param_dtype = param_dtype;
  a.parts = xpose::rms_norm_bwd_parts(rows, cols);
  return hip(xpose::launch_rms_norm_backward(a, dtype, (hipStream_t)stream));
}

// ----- low-rank adapters --------------------------------------------------------------

static bool adapter_sizes(int64_t m, int64_t n, int64_t k, int64_t rank, int64_t count) {
  return m >= 0 && n >= 0 && k >= 0 && rank >= 0 && count >= 0 && m <= kMaxAdapterRows && n <= kMaxAdapterCols &&
         k <= kMaxAdapterCols && rank <= kMaxRank && count <= kMaxAdapters;
}

int xpose_adapters_workspace(int64_t m, int64_t k, int64_t rank, int64_t count, int32_t x_size, int32_t hidden,
                             int64_t *bytes) {
  if (!adapter_sizes(m, 0, k, rank, count) || !bytes || (x_size != 1 && x_size != 2 && x_size != 4)) return XPOSE_EINVAL;
  Parts p;
  if (m && rank) {
    if (!hidden) p.add(m * rank, xpose::shrink_plan(m, k, rank, count, x_size, false).slices, 4);
  }
  *bytes = p.total();
  return XPOSE_OK;
}

int xpose_adapters(int64_t m, int64_t n, int64_t k, int64_t rank, int64_t count, const void *x, int64_t ldx,
                   const float *scale_x, int64_t ld_scale_x, const void *a, int64_t lda, int64_t stride_a,
                   const void *b, int64_t ldb, int64_t stride_b, int32_t dtype, const int32_t *ids, const float *scale,
                   float alpha, const void *base, int64_t ld_base, void *out, int64_t ld_out, int32_t out_dtype,
                   float *hidden, void *workspace, int64_t workspace_bytes, void *stream) {
  if (!adapter_sizes(m, n, k, rank, count) || workspace_bytes < 0) return XPOSE_EINVAL;
  const int size = size_of(dtype), out_size = size_of(out_dtype);
  if (!size || !out_size || (out_dtype != dtype && out_dtype != XPOSE_F32)) return XPOSE_EDTYPE;
  const int x_size = scale_x ? 1 : size;
  int64_t need = 0;
  int rc = xpose_adapters_workspace(m, k, rank, count, x_size, hidden != nullptr, &need);
  if (rc != XPOSE_OK) return rc;
  const bool some = m && rank && count;  // whether anything of A and x is read
  Ranges r;
  const int in = r.matrix(x, some ? m : 0, k, ldx, x_size, scale_x ? 16 : size, false);
  if (scale_x) r.matrix(scale_x, some ? ceil_div(k, kBlock) : 0, m, ld_scale_x, 4, 4, false);
  r.matrices(a, some ? count : 0, stride_a, rank, k, lda, size);
  r.matrices(b, some ? count : 0, stride_b, n, rank, ldb, size);
  r.vector(ids, m, 4, false);
  if (scale) r.vector(scale, count, 4, false);
  const int from = base ? r.matrix(base, m, n, ld_base, out_size, out_size, false) : -1;
  const int to = r.matrix(out, m, n, ld_out, out_size, out_size, true);
  r.same(from, to);
  if (base == out) r.same(in, to);  // base may be x, which only the first launch reads
  if (hidden) r.vector(hidden, m * rank, 4, true);
  const bool enough = need == 0 || (workspace && workspace_bytes >= need);
  if (need && enough) r.matrix(workspace, 1, need, need, 1, 16, true);
  rc = r.check();
  if (rc != XPOSE_OK || m == 0) return rc;
  if (!enough) return XPOSE_EWORKSPACE;

  const float *h = hidden ? hidden : (const float *)workspace;
  int slices = 1;
  if (rank) {
    const xpose::ShrinkPlan plan = xpose::shrink_plan(m, k, rank, count, x_size, hidden != nullptr);
    xpose::ShrinkArgs s{};
    s.x = x;
    s.w = a;
    s.scale_x = scale_x;
    s.ids = ids;
    s.h = hidden ? hidden : (float *)workspace;
    s.m = m;
    s.k = k;
    s.ldx = ldx;
    s.ld_scale_x = ld_scale_x;
    s.ldw = lda;
    s.stride_w = stride_a;
    s.slice = m * rank;
    s.rank = (int32_t)rank;
    s.count = (int32_t)count;
    s.steps_per_slice = plan.steps_per_slice;
    s.slots = plan.slots;
    rc = hip(xpose::launch_shrink(s, plan, dtype, (hipStream_t)stream));
    if (rc != XPOSE_OK) return rc;
    slices = plan.slices;
  }
  if (n == 0 || ((rank == 0 || count == 0) && base == out)) return XPOSE_OK;
  const int64_t used = rank ? count : 0;  // with no rank, no row has an adapter
  const xpose::ExpandPlan plan = xpose::expand_plan(m, n, used, false);
  xpose::ExpandArgs e{};
  e.h = h;
  e.w = b;
  e.ids = ids;
  e.scale = scale;
  e.base = base;
  e.out = out;
  e.m = m;
  e.n = n;
  e.ldw = ldb;
  e.stride_w = stride_b;
  e.ld_base = ld_base;
  e.ld_out = ld_out;
  e.slice = m * rank;
  e.slices = slices;
  e.rank = (int32_t)rank;
  e.count = (int32_t)used;
  e.slots = plan.slots;
  e.strips = (int32_t)plan.strips;
  e.alpha = alpha;
  return hip(xpose::launch_expand(e, plan, dtype, out_dtype, (hipStream_t)stream));
}

namespace {
// Where the backward pass keeps what.
struct BackwardParts {
  int64_t order, starts, dh, partial, bytes;
  xpose::ShrinkPlan plan;
  int piece;
};
bool backward_parts(int64_t m, int64_t n, int64_t k, int64_t rank, int64_t count, int size, BackwardParts &w) {
  // pieces of 4096 rows, or shorter ones, 256 workgroups at most
  if ((m / 4096 + count + 1) * (ceil_div(n, 128) + ceil_div(k, 128)) >= kMaxGradGroups - 256) return false;
  Parts p;
  w.plan = xpose::shrink_plan(std::max<int64_t>(m, 1), n, rank, count, size, true);
  w.piece = xpose::adapter_grad_piece(m, n, k);
  w.order = p.add(m, 1, 4);
  w.starts = p.add(count + 1, 1, 4);
  w.dh = p.add(m * rank, 1, 4);
  w.partial = p.add(xpose::adapter_grad_slots(m, w.piece) * rank, k + n, 4);
  w.bytes = p.total();
  return p.fits();
}
}  // namespace

int xpose_adapters_backward_workspace(int64_t m, int64_t n, int64_t k, int64_t rank, int64_t count, int32_t dtype,
                                      int64_t *bytes) {
  if (!adapter_sizes(m, n, k, rank, count) || !bytes) return XPOSE_EINVAL;
  const int size = size_of(dtype);
  if (!size) return XPOSE_EDTYPE;
  BackwardParts w;
  if (!backward_parts(m, n, k, rank, count, size, w)) return XPOSE_EINVAL;
  *bytes = w.bytes;
  return XPOSE_OK;
}

int xpose_adapters_backward(int64_t m, int64_t n, int64_t k, int64_t rank, int64_t count, const void *dout,
                            int64_t lddout, const void *x, int64_t ldx, const void *a, int64_t lda, int64_t stride_a,
                            const void *b, int64_t ldb, int64_t stride_b, int32_t dtype, const int32_t *ids,
                            const float *scale, float alpha, const float *hidden, const void *base, int64_t ld_base,
                            void *dx, int64_t lddx, int32_t dx_dtype, float *da, float *db, void *workspace,
                            int64_t workspace_bytes, void *stream) {
  if (!adapter_sizes(m, n, k, rank, count) || workspace_bytes < 0) return XPOSE_EINVAL;
  const int size = size_of(dtype), dx_size = size_of(dx_dtype);
  if (!size || !dx_size || (dx_dtype != dtype && dx_dtype != XPOSE_F32)) return XPOSE_EDTYPE;
  BackwardParts w;
  if (!backward_parts(m, n, k, rank, count, size, w)) return XPOSE_EINVAL;
  const bool some = m && rank && count;
  Ranges r;
  const int in_dout = r.matrix(dout, some ? m : 0, n, lddout, size, size, false);
  const int in_x = da ? r.matrix(x, some ? m : 0, k, ldx, size, size, false) : -1;
  if (dx) r.matrices(a, some ? count : 0, stride_a, rank, k, lda, size);
  if (dx || da) r.matrices(b, some ? count : 0, stride_b, n, rank, ldb, size);
  r.vector(ids, m, 4, false);
  if (scale) r.vector(scale, count, 4, false);
  if (db) r.vector(hidden, some ? m * rank : 0, 4, false);
  if (dx) {
    const int from = base ? r.matrix(base, m, k, ld_base, dx_size, dx_size, false) : -1;
    const int to = r.matrix(dx, m, k, lddx, dx_size, dx_size, true);
    r.same(from, to);
    if (base == dx) {  // base may be dout or x
      r.same(in_dout, to);
      r.same(in_x, to);
    }
  }
  const bool weights = count && rank && ((da && k) || (db && n));
  if (da) r.vector(da, count * rank * k, 4, true);
  if (db) r.vector(db, count * n * rank, 4, true);
  const bool enough = workspace && workspace_bytes >= w.bytes;
  if (enough && w.bytes) r.matrix(workspace, 1, w.bytes, w.bytes, 1, 16, true);
  int rc = r.check();
  if (rc != XPOSE_OK) return rc;
  const bool copies = dx && m && k && !(some ? false : base == dx);
  if (!weights && !copies) return XPOSE_OK;
  if (w.bytes && !enough) return XPOSE_EWORKSPACE;

  uint8_t *ws = (uint8_t *)workspace;
  const bool back = some && ((dx && k) || (da && k));  // dh is needed
  float *dh = (float *)(ws + w.dh);
  if (weights || back) {
    xpose::ShrinkArgs s{};
    s.x = dout;
    s.w = b;
    s.turned = true;
    s.ids = ids;
    s.scale = scale;
    s.alpha = alpha;
    s.scaled = true;
    s.h = back ? dh : nullptr;
    s.order = weights ? (int32_t *)(ws + w.order) : nullptr;
    s.starts = (int32_t *)(ws + w.starts);
    s.m = m;
    s.k = n;
    s.ldx = lddout;
    s.ldw = ldb;
    s.stride_w = stride_b;
    s.rank = (int32_t)rank;
    s.count = (int32_t)count;
    s.steps_per_slice = w.plan.steps_per_slice;
    s.slots = w.plan.slots;
    rc = hip(xpose::launch_shrink(s, w.plan, dtype, (hipStream_t)stream));
    if (rc != XPOSE_OK) return rc;
  }
  const int64_t used = some ? count : 0;
  // Over dout or x, dx waits for the gradients, which read them.
  const bool over = dx == dout || dx == x;
  const bool beside = copies && weights && rank <= 32 && !over;
  const xpose::ExpandPlan plan = xpose::expand_plan(m, k, used, beside);
  xpose::ExpandArgs e{};
  e.h = dh;
  e.w = a;
  e.turned = true;
  e.ids = ids;
  e.base = base;
  e.out = dx;
  e.m = m;
  e.n = k;
  e.ldw = lda;
  e.stride_w = stride_a;
  e.ld_base = ld_base;
  e.ld_out = lddx;
  e.slice = m * rank;
  e.slices = 1;
  e.rank = (int32_t)rank;
  e.count = (int32_t)used;
  e.slots = plan.slots;
  e.strips = (int32_t)plan.strips;
  e.alpha = 1.f;
  xpose::AdapterGradArgs g{};
  g.dh = dh;
  g.h = hidden;
  g.x = x;
  g.dout = dout;
  g.order = (const int32_t *)(ws + w.order);
  g.starts = (const int32_t *)(ws + w.starts);
  g.scale = scale;
  g.da = k ? da : nullptr;
  g.db = n ? db : nullptr;
  g.partial = (float *)(ws + w.partial);
  g.m = m;
  g.n = n;
  g.k = k;
  g.ldx = ldx;
  g.lddout = lddout;
  g.rank = (int32_t)rank;
  g.count = (int32_t)count;
  g.piece = w.piece;
  g.alpha = alpha;
  if (beside) return hip(xpose::launch_adapter_both(e, plan, g, dtype, dx_dtype, (hipStream_t)stream));
  if (weights) {
    rc = hip(xpose::launch_adapter_grad(g, dtype, (hipStream_t)stream));
    if (rc != XPOSE_OK) return rc;
  }
  return copies ? hip(xpose::launch_expand(e, plan, dtype, dx_dtype, (hipStream_t)stream)) : XPOSE_OK;
}

// ----- dropout ---------------------------------------------------------------------------

int xpose_dropout(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t dtype, double p, uint64_t seed,
                  const uint64_t *device_seed, uint64_t offset, const void *residual, int64_t ld_residual, void *y,
                  int64_t ldy, void *stream) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols >= (int64_t)1 << 34 || !(p >= 0 && p <= 1)) return XPOSE_EINVAL;
  const int size = size_of(dtype);
  if (!size) return XPOSE_EDTYPE;
  Ranges r;
  const int in = r.matrix(x, rows, cols, ldx, size, size, false);
  const int res = residual ? r.matrix(residual, rows, cols, ld_residual, size, size, false) : -1;
  const int out = r.matrix(y, rows, cols, ldy, size, size, true);
  r.same(in, out);
  r.same(res, out);
  if (device_seed) r.vector(device_seed, 1, 8, false);
  const int rc = r.check();
  if (rc != XPOSE_OK || rows == 0 || cols == 0) return rc;
  xpose::DropoutArgs a{};
  a.x = x;
  a.residual = residual;
  a.y = y;
  a.device_seed = device_seed;
  a.seed = seed;
  a.offset = offset;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldr = ld_residual;
  a.ldy = ldy;
  a.threshold = (uint32_t)(p * 65536 + 0.5);
  a.factor = a.threshold < 65536 ? (float)(65536.0 / (65536 - (double)a.threshold)) : 0.f;
  return hip(xpose::launch_dropout(a, dtype, (hipStream_t)stream));
}

}  // extern "C"
