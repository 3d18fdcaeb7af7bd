// Argument checks shared by the front ends of the linear layer's and the
// residual block's operators.  Host code that never touches the GPU.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/linear/xpose_linear.h"
#include "linear_kernels.h"

namespace {

using xpose::record_hip_error;

constexpr int64_t kBlock = 128;
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
  // The range's number, -1 where there is none.
  int matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int size,
             int align, bool output) {
    if (ld < (cols > 1 ? cols : 1)) rc_ = XPOSE_EINVAL;
    if (rc_ != XPOSE_OK || rows == 0 || cols == 0) return -1;
    int64_t last, bytes;
    uintptr_t end;
    if (!p || __builtin_mul_overflow(rows - 1, ld, &last) ||
        __builtin_add_overflow(last, cols, &last) ||
        __builtin_mul_overflow(last, (int64_t)size, &bytes) ||
        __builtin_add_overflow((uintptr_t)p, (uintptr_t)bytes, &end)) {
      rc_ = XPOSE_EINVAL;
      return -1;
    }
    if ((uintptr_t)p % align) late(XPOSE_EALIGN);
    if (rows > 1 && ld * size % align) late(XPOSE_EALIGN);
    all_[count_] = {(uintptr_t)p, end, output, ld};
    return count_++;
  }
  // An input of `count` such matrices, `stride` elements from one to the next.
  void matrices(const void *p, int64_t count, int64_t stride, int64_t rows,
                int64_t cols, int64_t ld, int size) {
    if (stride < 0) rc_ = XPOSE_EINVAL;
    const int before = count_;
    matrix(p, count ? rows : 0, cols, ld, size, size, false);
    if (count_ == before || count < 2) return;
    int64_t more;
    if (__builtin_mul_overflow(count - 1, stride, &more) ||
        __builtin_mul_overflow(more, (int64_t)size, &more) ||
        __builtin_add_overflow(all_[before].hi, (uintptr_t)more, &all_[before].hi))
      rc_ = XPOSE_EINVAL;
  }
  int vector(const void *p, int64_t n, int size, bool output) {
    return matrix(p, 1, n, n > 1 ? n : 1, size, size, output);
  }
  // The output `out` may also be the input `in` itself: these two, not what
  // else lies there.
  void same(int in, int out) {
    if (in >= 0 && out >= 0) in_place_[places_++] = {in, out};
  }
  int check() const {
    if (rc_ != XPOSE_OK || late_ != XPOSE_OK) return rc_ != XPOSE_OK ? rc_ : late_;
    for (int i = 0; i < count_; ++i)
      for (int j = i + 1; j < count_; ++j) {
        const Range &a = all_[i], &b = all_[j];
        if (!(a.output || b.output) || a.lo >= b.hi || b.lo >= a.hi) continue;
        if (in_place(i, j) && a.lo == b.lo && a.hi == b.hi && a.ld == b.ld) continue;
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
  struct Pair {
    int in, out;
  };
  bool in_place(int i, int j) const {
    for (int p = 0; p < places_; ++p)
      if ((in_place_[p].in == i && in_place_[p].out == j) || (in_place_[p].in == j && in_place_[p].out == i)) return true;
    return false;
  }
  void late(int rc) { if (late_ == XPOSE_OK) late_ = rc; }
  Range all_[16];  // no call has more
  Pair in_place_[4];
  int count_ = 0, places_ = 0;
  int rc_ = XPOSE_OK, late_ = XPOSE_OK;
};

}  // namespace
