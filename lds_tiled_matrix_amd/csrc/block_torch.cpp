// The torch side of a residual block's operators: checks of tensors, outputs
// and workspaces from torch's allocator, torch's streams.  All work is the C
// ABI's (include/linear/xpose_block.h).

#include "linear_torch.h"

#include <array>

#include "../../include/linear/xpose_block.h"

void bind_block(py::module_ &m);  // called by linear_torch.cpp

namespace {

// ----- root-mean-square norm ------------------------------------------------------

struct Weight {
  const void *data;
  int code;
};
Weight norm_weight(const Tensor &x, const OptTensor &weight) {
  if (x.dim() == 2 && x.size(1) == 0) bad_value("norm over no columns");
  same_device(x, weight);
  return {vector(weight, x.dim() == 2 ? x.size(1) : 0, "weight"),
          weight ? dtype_code(weight->scalar_type(), "weight") : (int)XPOSE_F32};
}

void like(const Tensor &x, const OptTensor &t, const char *what) {
  if (!t) return;
  same_device(x, *t);
  if (t->scalar_type() != x.scalar_type() || t->sizes() != x.sizes())
    bad_value(std::string(what) + " must match x's dtype and shape");
}

// The residual stream's side of a norm: what is added and where the sum goes.
struct Sum {
  Tensor h;
  Matrix residual{0, 0, 0}, out{0, 0, 0};
  const void *from = nullptr;
  void *to = nullptr;
};
Sum residual_sum(const Tensor &x, const OptTensor &residual, const OptTensor &given) {
  Sum s;
  if (!residual) {
    if (given) bad_value("residual_out without a residual");
    return s;
  }
  s.h = given ? *given : empty({x.size(0), x.size(1)}, x.scalar_type(), x);
  s.residual = matrix(*residual, "residual");
  s.out = matrix(s.h, "residual_out");
  s.from = residual->data_ptr();
  s.to = s.h.data_ptr();
  return s;
}

std::vector<Tensor> rms_norm(const Tensor &x, const OptTensor &weight, const OptTensor &residual, double eps, bool stats,
                             const OptTensor &given, const OptTensor &residual_out, const py::object &stream) {
  on_device(x);
  const int code = dtype_code(x.scalar_type(), "x");
  const Matrix mx = matrix(x, "x");
  const Weight w = norm_weight(x, weight);
  like(x, residual, "residual");
  like(x, residual_out, "residual_out");
  like(x, given, "out");
  const Stream on(x, stream);
  const Sum sum = residual_sum(x, residual, residual_out);
  Tensor out = given ? *given : empty({mx.rows, mx.cols}, x.scalar_type(), x), rstd;
  const Matrix my = matrix(out, "out");
  if (stats) rstd = empty({mx.rows}, at::kFloat, x);
  check(xpose_rms_norm(mx.rows, mx.cols, x.data_ptr(), mx.ld, code, sum.from, sum.residual.ld, sum.to, sum.out.ld,
                       w.data, w.code, (float)eps, out.data_ptr(), my.ld, stats ? rstd.data_ptr<float>() : nullptr,
                       on.raw()),
        "xpose_rms_norm");
  modified(given);
  modified(residual_out);
  on.uses(x, weight, residual, residual_out, given);
  on.returns(rstd);
  if (!given) on.returns(out);
  if (!residual_out) on.returns(sum.h);
  std::vector<Tensor> got{out};
  if (residual) got.push_back(sum.h);
  if (stats) got.push_back(rstd);
  return got;
}

std::vector<Tensor> rms_norm_quantize(const Tensor &x, const OptTensor &weight, const OptTensor &residual, double eps,
                                      bool pow2, bool stats, const OptTensor &residual_out, const py::object &stream) {
  on_device(x);
  const int code = dtype_code(x.scalar_type(), "x");
  const Matrix mx = matrix(x, "x");
  const Weight w = norm_weight(x, weight);
  like(x, residual, "residual");
  like(x, residual_out, "residual_out");
  const Stream on(x, stream);
  const Sum sum = residual_sum(x, residual, residual_out);
  Tensor q = empty_e4m3(mx.rows, mx.cols, x), scale = empty({blocks(mx.cols), mx.rows}, at::kFloat, x), rstd;
  if (stats) rstd = empty({mx.rows}, at::kFloat, x);
  check(xpose_rms_norm_quantize(mx.rows, mx.cols, x.data_ptr(), mx.ld, code, sum.from, sum.residual.ld, sum.to,
                                sum.out.ld, w.data, w.code, (float)eps, pow2 ? XPOSE_LINEAR_POW2 : 0, q.data_ptr(),
                                q.stride(0), scale.data_ptr<float>(), std::max<int64_t>(mx.rows, 1),
                                stats ? rstd.data_ptr<float>() : nullptr, on.raw()),
        "xpose_rms_norm_quantize");
  modified(residual_out);
  on.uses(x, weight, residual, residual_out);
  on.returns(q, scale, rstd);
  if (!residual_out) on.returns(sum.h);
  std::vector<Tensor> got{q, scale};
  if (residual) got.push_back(sum.h);
  if (stats) got.push_back(rstd);
  return got;
}

std::tuple<Tensor, Tensor> rms_norm_backward(const Tensor &dy, const Tensor &h, const Tensor &rstd,
                                             const OptTensor &weight, const OptTensor &dresidual,
                                             const py::object &stream) {
  on_device(h);
  same_device(h, dy);
  same_device(h, rstd);
  const int code = dtype_code(h.scalar_type(), "h");
  const Matrix mh = matrix(h, "h");
  const Weight w = norm_weight(h, weight);
  if (dy.scalar_type() != h.scalar_type() || dy.sizes() != h.sizes()) bad_value("dy must match h's dtype and shape");
  if (dresidual && (dresidual->scalar_type() != h.scalar_type() || dresidual->sizes() != h.sizes()))
    bad_value("dresidual must match h's dtype and shape");
  same_device(h, dresidual);
  const Matrix mdy = matrix(dy, "dy");
  const Matrix mr = dresidual ? matrix(*dresidual, "dresidual") : Matrix{0, 0, 0};
  const float *r = statistics(rstd, mh.rows, "rstd");
  const Stream on(h, stream);
  int64_t size = 0;
  check(xpose_rms_norm_backward_workspace(mh.rows, mh.cols, &size), "xpose_rms_norm_backward_workspace");
  Tensor dx = empty({mh.rows, mh.cols}, h.scalar_type(), h), dweight = empty({mh.cols}, at::kFloat, h);
  Tensor ws = empty({size}, at::kByte, h);
  check(xpose_rms_norm_backward(mh.rows, mh.cols, dy.data_ptr(), mdy.ld, h.data_ptr(), mh.ld, code, r,
                                dresidual ? dresidual->data_ptr() : nullptr, mr.ld, w.data, w.code, dx.data_ptr(),
                                std::max<int64_t>(mh.cols, 1), dweight.data_ptr<float>(), ws.data_ptr(), size,
                                on.raw()),
        "xpose_rms_norm_backward");
  on.uses(dy, h, rstd, weight, dresidual);
  on.returns(dx, dweight);
  return {dx, dweight};
}

// ----- low-rank adapters --------------------------------------------------------------

// `count` matrices one after the other.
struct Matrices {
  int64_t count, rows, cols, ld, stride;
};
Matrices matrices(const Tensor &t, const char *what) {
  if (t.dim() != 3) bad_value(std::string(what) + ": expected a 3-D tensor");
  const int64_t count = t.size(0), rows = t.size(1), cols = t.size(2);
  if (cols > 1 && t.stride(2) != 1) bad_value(std::string(what) + ": the last dimension must be contiguous");
  return {count, rows, cols, rows > 1 ? t.stride(1) : std::max<int64_t>(cols, 1), count > 1 ? t.stride(0) : 0};
}

// A number of the caller's that may be a tensor too; of another type it is a TypeError.
template <typename T>
T number(const py::object &given, const char *what) {
  try {
    return given.cast<T>();
  } catch (const py::cast_error &) {
    bad_type(std::string(what) + ": expected a number or a tensor, got " +
             py::str(py::type::of(given).attr("__name__")).cast<std::string>());
  }
}

// What a row's adapter is and is worth.
struct Adapters {
  Matrices a, b;
  int code;
  const int32_t *ids;
  const float *scale = nullptr;
  float alpha = 1.f;
  OptTensor scales;  // kept for its stream
};
Adapters adapters_of(const Tensor &first, const Tensor &a, const Tensor &b, const Tensor &ids, int64_t m, int64_t k,
                     int64_t n, const py::object &scale) {
  same_device(first, a);
  same_device(first, b);
  same_device(first, ids);
  Adapters r;
  r.a = matrices(a, "a");
  r.b = matrices(b, "b");
  if (a.scalar_type() != b.scalar_type()) bad_type("a and b have different dtypes");
  r.code = dtype_code(a.scalar_type(), "a, b");
  if (r.a.cols != k) bad_value("a: expected " + std::to_string(k) + " columns, got " + std::to_string(r.a.cols));
  if (r.b.count != r.a.count || r.b.cols != r.a.rows)
    bad_value("a and b differ in their number or rank");
  if (n >= 0 && r.b.rows != n) bad_value("b: expected " + std::to_string(n) + " rows, got " + std::to_string(r.b.rows));
  if (ids.scalar_type() != at::kInt) bad_type(std::string("ids: expected int32, got ") + c10::toString(ids.scalar_type()));
  r.ids = (const int32_t *)vector(ids, m, "ids");
  if (THPVariable_Check(scale.ptr())) {
    r.scales = THPVariable_Unpack(scale.ptr());
    same_device(first, *r.scales);
    r.scale = statistics(*r.scales, r.a.count, "scale");
  } else {
    r.alpha = (float)number<double>(scale, "scale");
  }
  return r;
}

// The call's out or its base's sum: its type and pitch.
at::ScalarType out_type(const OptTensor &base, const OptTensor &given, const Tensor &weights, int64_t rows, int64_t cols) {
  for (const OptTensor *t : {&base, &given})
    if (*t && ((*t)->dim() != 2 || (*t)->size(0) != rows || (*t)->size(1) != cols))
      bad_value(std::string(t == &base ? "base" : "out") + ": expected " + shape(rows, cols));
  if (base && given && base->scalar_type() != given->scalar_type()) bad_type("base and out have different dtypes");
  const at::ScalarType type = base ? base->scalar_type() : given ? given->scalar_type() : weights.scalar_type();
  if (type != at::kFloat && type != weights.scalar_type())
    bad_type(std::string("base, out: expected float32 or the adapters' dtype, got ") + c10::toString(type));
  return type;
}

std::vector<Tensor> adapters(const Tensor &x, const Tensor &a, const Tensor &b, const Tensor &ids,
                             const OptTensor &base, const py::object &scale, const OptTensor &scale_x, bool hidden,
                             const OptTensor &given, const py::object &stream) {
  on_device(x);
  same_device(x, scale_x);
  same_device(x, base);
  same_device(x, given);
  const Matrix mx = matrix(x, "x");
  const int64_t m = mx.rows, k = mx.cols;
  const Adapters w = adapters_of(x, a, b, ids, m, k, -1, scale);
  const int64_t n = w.b.rows, rank = w.a.rows, count = w.a.count;
  Matrix msx{0, 0, 0};
  if (scale_x) {
    if (x.scalar_type() != at::kFloat8_e4m3fn || scale_x->scalar_type() != at::kFloat)
      bad_type("x with scale_x: expected float8_e4m3fn and float32");
    msx = matrix(*scale_x, "scale_x");
    if (msx.rows != blocks(k) || msx.cols != m)
      bad_value("scale_x: expected " + shape(blocks(k), m) + ", got " + shape(msx.rows, msx.cols));
  } else if (x.scalar_type() != a.scalar_type()) {
    bad_type(std::string("x: expected the adapters' dtype, got ") + c10::toString(x.scalar_type()));
  }
  const at::ScalarType type = out_type(base, given, a, m, n);
  const Matrix mb = base ? matrix(*base, "base") : Matrix{0, 0, 0};
  const Stream on(x, stream);
  Tensor out = given ? *given : empty({m, n}, type, x), h, ws;
  const Matrix mo = matrix(out, "out");
  int64_t size = 0;
  check(xpose_adapters_workspace(m, k, rank, count, (int)x.element_size(), hidden, &size), "xpose_adapters_workspace");
  if (hidden) h = empty({m, rank}, at::kFloat, x);
  if (size) ws = empty({size}, at::kByte, x);
  check(xpose_adapters(m, n, k, rank, count, x.data_ptr(), mx.ld, scale_x ? scale_x->data_ptr<float>() : nullptr,
                       msx.ld, a.data_ptr(), w.a.ld, w.a.stride, b.data_ptr(), w.b.ld, w.b.stride, w.code, w.ids,
                       w.scale, w.alpha, base ? base->data_ptr() : nullptr, mb.ld, out.data_ptr(), mo.ld,
                       dtype_code(type, "out"), hidden ? h.data_ptr<float>() : nullptr,
                       size ? ws.data_ptr() : nullptr, size, on.raw()),
        "xpose_adapters");
  modified(given);
  on.uses(x, a, b, ids, base, w.scales, scale_x, given);
  on.returns(h);
  if (!given) on.returns(out);
  if (hidden) return {out, h};
  return {out};
}

std::vector<OptTensor> adapters_backward(const Tensor &dout, const Tensor &x, const Tensor &a, const Tensor &b,
                                         const Tensor &ids, const Tensor &hidden, const OptTensor &base,
                                         const py::object &scale, const std::array<bool, 3> &wanted,
                                         const OptTensor &given, const py::object &stream) {
  on_device(x);
  same_device(x, dout);
  same_device(x, hidden);
  same_device(x, base);
  same_device(x, given);
  const Matrix mx = matrix(x, "x"), mdout = matrix(dout, "dout"), mh = matrix(hidden, "hidden");
  const int64_t m = mx.rows, k = mx.cols, n = mdout.cols;
  if (mdout.rows != m) bad_value("x and dout differ in their rows");
  const Adapters w = adapters_of(x, a, b, ids, m, k, n, scale);
  const int64_t rank = w.a.rows, count = w.a.count;
  if (x.scalar_type() != a.scalar_type() || dout.scalar_type() != a.scalar_type())
    bad_type("x, dout: expected the adapters' dtype");
  if (hidden.scalar_type() != at::kFloat) bad_type("hidden: expected float32");
  if (mh.rows != m || mh.cols != rank || (m > 1 && mh.ld != std::max<int64_t>(rank, 1)))
    bad_value("hidden: expected " + shape(m, rank) + ", contiguous");
  if (!wanted[0] && (base || given)) bad_value("base or out without dx");
  const at::ScalarType type = out_type(base, given, a, m, k);
  const Matrix mb = base ? matrix(*base, "base") : Matrix{0, 0, 0};
  const Stream on(x, stream);
  OptTensor dx, da, db;
  Matrix mdx{0, 0, 1};
  if (wanted[0]) {
    dx = given ? *given : empty({m, k}, type, x);
    mdx = matrix(*dx, "out");
  }
  if (wanted[1]) da = empty({count, rank, k}, at::kFloat, x);
  if (wanted[2]) db = empty({count, n, rank}, at::kFloat, x);
  int64_t size = 0;
  check(xpose_adapters_backward_workspace(m, n, k, rank, count, w.code, &size), "xpose_adapters_backward_workspace");
  Tensor ws = empty({size}, at::kByte, x);
  check(xpose_adapters_backward(m, n, k, rank, count, dout.data_ptr(), mdout.ld, x.data_ptr(), mx.ld, a.data_ptr(),
                                w.a.ld, w.a.stride, b.data_ptr(), w.b.ld, w.b.stride, w.code, w.ids, w.scale, w.alpha,
                                hidden.data_ptr<float>(), base ? base->data_ptr() : nullptr, mb.ld,
                                dx ? dx->data_ptr() : nullptr, mdx.ld, dtype_code(type, "dx"),
                                da ? da->data_ptr<float>() : nullptr, db ? db->data_ptr<float>() : nullptr,
                                ws.data_ptr(), size, on.raw()),
        "xpose_adapters_backward");
  modified(given);
  on.uses(dout, x, a, b, ids, hidden, base, w.scales, given);
  if (!given && dx) on.returns(*dx);
  if (da) on.returns(*da);
  if (db) on.returns(*db);
  return {dx, da, db};
}

// ----- dropout ---------------------------------------------------------------------------

Tensor dropout(const Tensor &x, double p, const py::object &seed, uint64_t offset, const OptTensor &residual,
               const OptTensor &given, const py::object &stream) {
  on_device(x);
  const int code = dtype_code(x.scalar_type(), "x");
  const Matrix mx = matrix(x, "x");
  like(x, residual, "residual");
  like(x, given, "out");
  const Matrix mr = residual ? matrix(*residual, "residual") : Matrix{0, 0, 0};
  OptTensor device_seed;
  uint64_t host_seed = 0;
  if (THPVariable_Check(seed.ptr())) {
    device_seed = THPVariable_Unpack(seed.ptr());
    same_device(x, *device_seed);
    if (device_seed->scalar_type() != at::kLong)
      bad_type(std::string("seed: expected int64, got ") + c10::toString(device_seed->scalar_type()));
    if (device_seed->numel() != 1) bad_value("seed: expected one value");
  } else {
    host_seed = number<uint64_t>(seed, "seed");
  }
  const Stream on(x, stream);
  Tensor out = given ? *given : empty({mx.rows, mx.cols}, x.scalar_type(), x);
  const Matrix my = matrix(out, "out");
  check(xpose_dropout(mx.rows, mx.cols, x.data_ptr(), mx.ld, code, p, host_seed,
                      device_seed ? (const uint64_t *)device_seed->data_ptr() : nullptr, offset,
                      residual ? residual->data_ptr() : nullptr, mr.ld, out.data_ptr(), my.ld, on.raw()),
        "xpose_dropout");
  modified(given);
  on.uses(x, device_seed, residual, given);
  if (!given) on.returns(out);
  return out;
}

}  // namespace

void bind_block(py::module_ &m) {
  m.def("rms_norm", torch::wrap_pybind_function(rms_norm));
  m.def("rms_norm_quantize", torch::wrap_pybind_function(rms_norm_quantize));
  m.def("rms_norm_backward", torch::wrap_pybind_function(rms_norm_backward));
  m.def("adapters", torch::wrap_pybind_function(adapters));
  m.def("adapters_backward", torch::wrap_pybind_function(adapters_backward));
  m.def("dropout", torch::wrap_pybind_function(dropout));
}
