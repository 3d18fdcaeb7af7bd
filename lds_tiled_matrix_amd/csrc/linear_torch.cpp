// The torch side of the FP8 linear layer's operators: checks of tensors,
// outputs and workspaces from torch's allocator, torch's streams.  All work is
// the C ABI's (include/linear/xpose_linear.h).  It is compiled code because
// the smallest calls (one token, a handful of small gradients) take the GPU
// 4 to 6 us, less than the same checks take in Python (14 and 41 us).

#include "linear_torch.h"

void bind_block(py::module_ &m);  // block_torch.cpp

namespace {

Tensor fp8_gemm(const Tensor &a, const Tensor &scale_a, const Tensor &b, const Tensor &scale_b,
                const OptTensor &given, const std::optional<at::ScalarType> &out_dtype, bool pow2,
                const py::object &stream) {
  on_device(a);
  same_device(a, scale_a);
  same_device(a, b);
  same_device(a, scale_b);
  same_device(a, given);
  if (a.scalar_type() != at::kFloat8_e4m3fn || b.scalar_type() != at::kFloat8_e4m3fn)
    bad_type(std::string("a, b: expected float8_e4m3fn, got ") + c10::toString(a.scalar_type()) + ", " +
             c10::toString(b.scalar_type()));
  if (scale_a.scalar_type() != at::kFloat || scale_b.scalar_type() != at::kFloat)
    bad_type("scale_a, scale_b: expected float32");
  const Matrix ma = matrix(a, "a"), mb = matrix(b, "b");
  const Matrix sa = matrix(scale_a, "scale_a"), sb = matrix(scale_b, "scale_b");
  const int64_t m = ma.rows, n = mb.rows, k = ma.cols, kb = blocks(k);
  if (mb.cols != k) bad_value("inner dimensions differ");
  if (sa.rows != kb || sa.cols != m)
    bad_value("scale_a: expected " + shape(kb, m) + ", got " + shape(sa.rows, sa.cols));
  const int block_rows = sb.cols == n ? 1 : sb.cols == blocks(n) ? 128 : 0;
  if (sb.rows != kb || !block_rows)
    bad_value("scale_b: expected " + shape(kb, n) + " or " + shape(kb, blocks(n)) + ", got " +
              shape(sb.rows, sb.cols));
  if (given) {
    if (given->dim() != 2 || given->size(0) != m || given->size(1) != n) bad_value("out has the wrong shape");
    if (out_dtype && given->scalar_type() != *out_dtype) bad_type("out and out_dtype differ");
  }
  const at::ScalarType type = given ? given->scalar_type() : out_dtype.value_or(at::kBFloat16);
  const int code = dtype_code(type, "out");
  const Stream on(a, stream);
  Tensor out = given ? *given : empty({m, n}, type, a), ws;
  const Matrix mc = matrix(out, "out");
  const int flags = pow2 ? XPOSE_LINEAR_POW2 : 0;
  xpose_fp8_gemm_info info;
  check(xpose_fp8_gemm_plan(m, n, k, block_rows, code, flags, &info), "xpose_fp8_gemm_plan");
  if (info.workspace_bytes) ws = empty({info.workspace_bytes}, at::kByte, a);
  check(xpose_fp8_gemm(m, n, k, a.data_ptr(), ma.ld, scale_a.data_ptr<float>(), sa.ld, b.data_ptr(), mb.ld,
                       scale_b.data_ptr<float>(), sb.ld, block_rows, out.data_ptr(), mc.ld, code, flags,
                       ws.defined() ? ws.data_ptr() : nullptr, info.workspace_bytes, on.raw()),
        "xpose_fp8_gemm");
  modified(given);
  on.uses(a, scale_a, b, scale_b, given);
  if (!given) on.returns(out);
  return out;
}

std::vector<Tensor> fp8_quantize(const Tensor &x, int64_t block_rows, bool pow2, bool transposed,
                                 const py::object &stream) {
  on_device(x);
  const int code = dtype_code(x.scalar_type(), "x");
  const Matrix mx = matrix(x, "x");
  if (block_rows != 1 && block_rows != 128) bad_value("block_rows is 1 or 128");
  const Stream on(x, stream);
  const bool tiles = block_rows == 128;
  const int64_t rows = mx.rows, cols = mx.cols, rb = blocks(rows), cb = blocks(cols);
  Tensor q = empty_e4m3(rows, cols, x), scale = empty({cb, tiles ? rb : rows}, at::kFloat, x), qt, scale_t;
  if (transposed) {
    qt = empty_e4m3(cols, rows, x);
    scale_t = empty({rb, tiles ? cb : cols}, at::kFloat, x);
  }
  if (rows && cols)
    check(xpose_fp8_quantize(rows, cols, x.data_ptr(), mx.ld, code, (int)block_rows, pow2 ? XPOSE_LINEAR_POW2 : 0,
                             q.data_ptr(), q.stride(0), scale.data_ptr<float>(), scale.size(1),
                             transposed ? qt.data_ptr() : nullptr, transposed ? qt.stride(0) : 0,
                             transposed ? scale_t.data_ptr<float>() : nullptr,
                             transposed ? scale_t.size(1) : 0, on.raw()),
          "xpose_fp8_quantize");
  on.uses(x);
  on.returns(q, scale, qt, scale_t);
  if (transposed) return {q, scale, qt, scale_t};
  return {q, scale};
}

struct Parameters {
  const void *weight, *bias;
  int code;
};
Parameters parameters(const Tensor &x, const OptTensor &weight, const OptTensor &bias, int64_t cols) {
  on_device(x);
  same_device(x, weight);
  same_device(x, bias);
  if (weight && bias && weight->scalar_type() != bias->scalar_type())
    bad_type("weight and bias have different dtypes");
  const OptTensor &one = weight ? weight : bias;
  return {vector(weight, cols, "weight"), vector(bias, cols, "bias"),
          one ? dtype_code(one->scalar_type(), "weight, bias") : (int)XPOSE_F32};
}

int64_t some_columns(const Tensor &x) {
  if (x.dim() == 2 && x.size(1) == 0) bad_value("layer norm over no columns");
  return x.dim() == 2 ? x.size(1) : 0;
}

std::vector<Tensor> layer_norm(const Tensor &x, const OptTensor &weight, const OptTensor &bias, double eps, bool stats,
                               const OptTensor &given, const py::object &stream) {
  on_device(x);
  const int code = dtype_code(x.scalar_type(), "x");
  const Matrix mx = matrix(x, "x");
  const Parameters p = parameters(x, weight, bias, some_columns(x));
  same_device(x, given);
  if (given && (given->scalar_type() != x.scalar_type() || given->sizes() != x.sizes()))
    bad_value("out must match x's dtype and shape");
  const Stream on(x, stream);
  Tensor out = given ? *given : empty({mx.rows, mx.cols}, x.scalar_type(), x), mean, rstd;
  const Matrix my = matrix(out, "out");
  if (stats) {
    mean = empty({mx.rows}, at::kFloat, x);
    rstd = empty({mx.rows}, at::kFloat, x);
  }
  check(xpose_layer_norm(mx.rows, mx.cols, x.data_ptr(), mx.ld, code, p.weight, p.bias, p.code, (float)eps,
                         out.data_ptr(), my.ld, stats ? mean.data_ptr<float>() : nullptr,
                         stats ? rstd.data_ptr<float>() : nullptr, on.raw()),
        "xpose_layer_norm");
  modified(given);
  on.uses(x, weight, bias, given);
  on.returns(mean, rstd);
  if (!given) on.returns(out);
  if (stats) return {out, mean, rstd};
  return {out};
}

std::vector<Tensor> layer_norm_quantize(const Tensor &x, const OptTensor &weight, const OptTensor &bias, double eps,
                                        bool pow2, bool stats, const py::object &stream) {
  on_device(x);
  const int code = dtype_code(x.scalar_type(), "x");
  const Matrix mx = matrix(x, "x");
  const Parameters p = parameters(x, weight, bias, some_columns(x));
  const Stream on(x, stream);
  Tensor q = empty_e4m3(mx.rows, mx.cols, x), scale = empty({blocks(mx.cols), mx.rows}, at::kFloat, x), mean, rstd;
  if (stats) {
    mean = empty({mx.rows}, at::kFloat, x);
    rstd = empty({mx.rows}, at::kFloat, x);
  }
  check(xpose_layer_norm_quantize(mx.rows, mx.cols, x.data_ptr(), mx.ld, code, p.weight, p.bias, p.code, (float)eps,
                                  pow2 ? XPOSE_LINEAR_POW2 : 0, q.data_ptr(), q.stride(0), scale.data_ptr<float>(),
                                  std::max<int64_t>(mx.rows, 1), stats ? mean.data_ptr<float>() : nullptr,
                                  stats ? rstd.data_ptr<float>() : nullptr, on.raw()),
        "xpose_layer_norm_quantize");
  on.uses(x, weight, bias);
  on.returns(q, scale, mean, rstd);
  if (stats) return {q, scale, mean, rstd};
  return {q, scale};
}

std::tuple<Tensor, Tensor, Tensor> layer_norm_backward(const Tensor &dy, const Tensor &x, const Tensor &mean,
                                                       const Tensor &rstd, const OptTensor &weight,
                                                       const py::object &stream) {
  on_device(x);
  same_device(x, dy);
  same_device(x, mean);
  same_device(x, rstd);
  const int code = dtype_code(x.scalar_type(), "x");
  const Matrix mx = matrix(x, "x");
  const Parameters p = parameters(x, weight, std::nullopt, some_columns(x));
  if (dy.scalar_type() != x.scalar_type() || dy.sizes() != x.sizes()) bad_value("dy must match x's dtype and shape");
  const Matrix mdy = matrix(dy, "dy");
  const float *m = statistics(mean, mx.rows, "mean"), *r = statistics(rstd, mx.rows, "rstd");
  const Stream on(x, stream);
  int64_t size = 0;
  check(xpose_layer_norm_backward_workspace(mx.rows, mx.cols, &size), "xpose_layer_norm_backward_workspace");
  Tensor dx = empty({mx.rows, mx.cols}, x.scalar_type(), x);
  Tensor dweight = empty({mx.cols}, at::kFloat, x), dbias = empty({mx.cols}, at::kFloat, x);
  Tensor ws = empty({size}, at::kByte, x);
  check(xpose_layer_norm_backward(mx.rows, mx.cols, dy.data_ptr(), mdy.ld, x.data_ptr(), mx.ld, code, m, r, p.weight,
                                  p.code, dx.data_ptr(), mx.cols, dweight.data_ptr<float>(), dbias.data_ptr<float>(),
                                  ws.data_ptr(), size, on.raw()),
        "xpose_layer_norm_backward");
  on.uses(dy, x, mean, rstd, weight);
  on.returns(dx, dweight, dbias);
  return {dx, dweight, dbias};
}

const Tensor &tensor_of(PyObject *o, const char *what) {
  if (!THPVariable_Check(o)) bad_type(std::string(what) + ": expected tensors");
  return THPVariable_Unpack(o);
}

// Whether a gradient's elements fill one stretch of memory, in any order.
bool is_dense(const Tensor &t) { return t.is_non_overlapping_and_dense(); }

// (norm, out): `out` is the caller's own sequence, or a new list.
py::tuple clip_grad_norm(const py::object &given_grads, double max_norm, double eps, const py::object &given_out,
                         const py::object &stream) {
  const py::object grads = py::reinterpret_steal<py::object>(PySequence_Fast(given_grads.ptr(), "grads: expected tensors"));
  if (!grads) throw py::error_already_set();
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(grads.ptr());
  if (n == 0) bad_value("no gradients");
  const bool make = given_out.is_none();
  py::object out;
  if (make) {
    out = py::list(n);
  } else {
    out = py::reinterpret_steal<py::object>(PySequence_Fast(given_out.ptr(), "out: expected tensors"));
    if (!out) throw py::error_already_set();
    if (PySequence_Fast_GET_SIZE(out.ptr()) != n)
      bad_value(std::to_string(n) + " gradients, " + std::to_string(PySequence_Fast_GET_SIZE(out.ptr())) + " outputs");
  }
  const Tensor &first = tensor_of(PySequence_Fast_GET_ITEM(grads.ptr(), 0), "grads");
  on_device(first);
  const Stream on(first, stream);
  std::vector<xpose_clip_tensor> table((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor &g = tensor_of(PySequence_Fast_GET_ITEM(grads.ptr(), i), "grads");
    same_device(first, g);
    const int code = dtype_code(g.scalar_type(), "grads");
    if (!is_dense(g)) bad_value("a gradient does not fill one stretch of memory");
    if (make) PyList_SET_ITEM(out.ptr(), i, THPVariable_Wrap(at::empty_like(g)));
    const Tensor &o = tensor_of(PySequence_Fast_GET_ITEM(out.ptr(), i), "out");
    if (!make && !o.is_same(g)) {
      same_device(first, o);
      if (o.scalar_type() != g.scalar_type() || o.sizes() != g.sizes())
        bad_value("an output differs from its gradient in dtype or shape");
      if (g.numel() && o.strides() != g.strides()) bad_value("an output differs from its gradient in strides");
    }
    table[(size_t)i] = {g.data_ptr(), o.data_ptr(), g.numel(), code, 0};
    on.uses(g);
    if (make) on.returns(o); else on.uses(o);
  }
  int64_t size = 0;
  check(xpose_clip_grad_norm_workspace(n, table.data(), &size), "xpose_clip_grad_norm_workspace");
  Tensor norm = empty({}, at::kFloat, first), ws;
  if (size) ws = empty({size / 8}, at::kDouble, first);
  check(xpose_clip_grad_norm(n, table.data(), max_norm, eps, norm.data_ptr<float>(),
                             size ? ws.data_ptr() : nullptr, size, on.raw()),
        "xpose_clip_grad_norm");
  for (Py_ssize_t i = 0; i < n && !make; ++i) modified(tensor_of(PySequence_Fast_GET_ITEM(out.ptr(), i), "out"));
  on.returns(norm);
  return py::make_tuple(norm, make ? out : given_out);
}

}  // namespace

PYBIND11_MODULE(_linear, m) {
  m.def("fp8_gemm", torch::wrap_pybind_function(fp8_gemm));
  m.def("fp8_quantize", torch::wrap_pybind_function(fp8_quantize));
  m.def("layer_norm", torch::wrap_pybind_function(layer_norm));
  m.def("layer_norm_quantize", torch::wrap_pybind_function(layer_norm_quantize));
  m.def("layer_norm_backward", torch::wrap_pybind_function(layer_norm_backward));
  m.def("clip_grad_norm", torch::wrap_pybind_function(clip_grad_norm));
  m.def("is_dense", torch::wrap_pybind_function(is_dense));
  bind_block(m);
}
