// What the torch sides of the linear layer's and the residual block's operators
// share: checks of tensors, outputs from torch's allocator, torch's streams.
#pragma once

#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>
#include <ATen/ATen.h>

#include <optional>
#include <string>
#include <tuple>
#include <vector>

#include "../../include/linear/xpose_linear.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

[[noreturn]] void bad_value(const std::string &what) { throw py::value_error(what); }
[[noreturn]] void bad_type(const std::string &what) { throw py::type_error(what); }

void check(int rc, const char *what) {
  if (rc == XPOSE_OK) return;
  const py::object cls = py::module_::import("lds_tiled_matrix_amd").attr("XposeError");
  PyErr_SetObject(cls.ptr(), cls(rc, what).ptr());
  throw py::error_already_set();
}

int dtype_code(at::ScalarType t, const char *what) {
  switch (t) {
    case at::kFloat: return XPOSE_F32;
    case at::kHalf: return XPOSE_F16;
    case at::kBFloat16: return XPOSE_BF16;
    default:
      bad_type(std::string(what) + ": expected float32, float16 or bfloat16, got " + c10::toString(t));
  }
}

// Device tensors of one device: checked before anything is launched, so a
// host tensor is an error here, not a fault on the GPU.
void on_device(const Tensor &first) {
  if (!first.is_cuda()) bad_value("expected a CUDA tensor, got one on " + first.device().str());
}
void same_device(const Tensor &first, const Tensor &t) {
  if (t.device() != first.device())
    bad_value("tensors on different devices: " + first.device().str() + ", " + t.device().str());
}
void same_device(const Tensor &first, const OptTensor &t) {
  if (t) same_device(first, *t);
}

// The stream of a call: the current one of the tensors' device, or the
// caller's.  On the caller's, everything that the call allocates comes from
// that stream's memory: what the current stream's pool hands out may still be
// in use by work queued there, which the call does not wait for.
class Stream {
 public:
  Stream(const Tensor &t, const py::object &given) {
    const auto current = c10::hip::current_device();
    if (t.device().index() != current)
      bad_value("tensors on " + t.device().str() + ", but the current device is cuda:" +
                std::to_string(current));
    raw_ = c10::hip::getCurrentHIPStream(current).stream();
    if (given.is_none()) return;
    const auto other = c10::Stream::unpack3(given.attr("stream_id").cast<int64_t>(),
                                            (c10::DeviceIndex)given.attr("device_index").cast<int>(),
                                            (c10::DeviceType)given.attr("device_type").cast<int>());
    if (other.device() != t.device())
      bad_value("tensors on " + t.device().str() + ", but a stream of " + other.device().str());
    raw_ = reinterpret_cast<void *>(given.attr("cuda_stream").cast<uintptr_t>());
    guard_.emplace(other);
  }
  void *raw() const { return raw_; }
  // The caller's tensors: kept from being reused before the call's work has run.
  template <typename... Ts>
  void uses(const Ts &...tensors) const {
    if (guard_) (..., record(tensors, guard_->current_stream()));
  }
  // Tensors that the call allocated and returns: the caller goes on with them
  // on the stream that was current.
  template <typename... Ts>
  void returns(const Ts &...tensors) const {
    if (guard_) (..., record(tensors, guard_->original_stream()));
  }

 private:
  static void record(const Tensor &t, const c10::Stream &s) {
    if (t.defined()) t.record_stream(s);
  }
  static void record(const OptTensor &t, const c10::Stream &s) {
    if (t) record(*t, s);
  }
  void *raw_ = nullptr;
  std::optional<c10::StreamGuard> guard_;
};

struct Matrix {
  int64_t rows, cols, ld;
};
Matrix matrix(const Tensor &t, const char *what) {
  if (t.dim() != 2) bad_value(std::string(what) + ": expected a 2-D tensor");
  const int64_t rows = t.size(0), cols = t.size(1);
  if (cols > 1 && t.stride(1) != 1)
    bad_value(std::string(what) + ": the last dimension must be contiguous");
  return {rows, cols, rows > 1 ? t.stride(0) : std::max<int64_t>(cols, 1)};
}

const void *vector(const OptTensor &t, int64_t n, const char *what) {
  if (!t) return nullptr;
  if (t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1))
    bad_value(std::string(what) + ": expected " + std::to_string(n) + " contiguous values");
  return t->data_ptr();
}
const float *statistics(const Tensor &t, int64_t n, const char *what) {
  if (t.scalar_type() != at::kFloat)
    bad_type(std::string(what) + ": expected float32, got " + c10::toString(t.scalar_type()));
  return (const float *)vector(t, n, what);
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const Tensor &like) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

// Uninitialised e4m3 values, rows at multiples of 16 bytes, long ones at whole
// 128-byte lines.
Tensor empty_e4m3(int64_t rows, int64_t cols, const Tensor &like) {
  const int64_t to = cols < 1024 ? 16 : 128, pitch = (cols + to - 1) / to * to;
  Tensor q = empty({rows, pitch}, at::kFloat8_e4m3fn, like);
  return pitch == cols ? q : q.narrow(1, 0, cols);
}

// A tensor of the caller's that the call writes: autograd sees that what it
// saved of it is gone.  (Inference tensors have no versions.)
void modified(const Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void modified(const OptTensor &t) {
  if (t) modified(*t);
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }
std::string shape(int64_t a, int64_t b) {
  return "(" + std::to_string(a) + ", " + std::to_string(b) + ")";
}

}  // namespace
