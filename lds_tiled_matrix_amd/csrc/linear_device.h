// Device helpers shared by the kernels of the FP8 linear layer's operators:
// vectors of eight elements, sums and maxima over lanes, and the e4m3
// rounding of x / scale.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace xpose {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Vectors that need no more than their element's alignment: gfx950 loads and
// stores global memory at any byte address, so rows of odd pitch take the
// same 16-byte accesses as aligned ones.
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef _Float16 f16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef __bf16 bf16x8_any __attribute__((ext_vector_type(8), aligned(2)));

template <typename T> struct Vec8;
template <> struct Vec8<float> { f32x4_any v[2]; };
template <> struct Vec8<_Float16> { f16x8_any v; };
template <> struct Vec8<__bf16> { bf16x8_any v; };

// Eight elements at p, of which the first `valid` exist; zeros for the rest.
// As they are in memory: 16-bit types take half of float32's registers.
template <typename T>
__device__ inline Vec8<T> load_raw8(const T *p, int valid) {
  if (valid >= 8) return *reinterpret_cast<const Vec8<T> *>(p);
  Vec8<T> r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const T v = e < valid ? p[e] : (T)0.f;
    if constexpr (sizeof(T) == 4) r.v[e / 4][e % 4] = v; else r.v[e] = v;
  }
  return r;
}
template <typename T>
__device__ inline float at8(const Vec8<T> &r, int e) {
  if constexpr (sizeof(T) == 4) return r.v[e / 4][e % 4]; else return (float)r.v[e];
}

// The same of a row of `cols` >= 8 elements, from `col` on, for loads that are to
// stay under way: element by element they would be waited for at once, to be
// put together.  Lanes at the row's end load its last eight elements, and
// `settle8` then moves them to their places.
template <typename T>
__device__ inline Vec8<T> load_row8(const T *row, int64_t cols, int64_t col) {
  return *reinterpret_cast<const Vec8<T> *>(row + (col < cols - 8 ? col : cols - 8));
}
template <typename T>
__device__ inline void settle8(Vec8<T> &v, int64_t cols, int64_t col) {
  if (col <= cols - 8) return;
  constexpr int N = 2 * sizeof(T);
  const int64_t past = col + 8 - cols;
  const int by = past < 8 ? (int)past : 8;  // elements
  uint32_t w[N + 1];
  __builtin_memcpy(w, &v, 4 * N);
  w[N] = 0;
  const int words = by * (int)sizeof(T) / 4;
#pragma unroll
  for (int d = N; d; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (words & d) w[i] = i + d < N ? w[i + d] : 0;
  if constexpr (sizeof(T) == 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (by & 1) w[i] = w[i] >> 16 | w[i + 1] << 16;
  __builtin_memcpy(&v, w, 4 * N);
}

template <typename T>
__device__ inline void load8(const T *p, int valid, float (&f)[8]) {
  const Vec8<T> r = load_raw8(p, valid);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = at8<T>(r, e);
}

template <typename T>
__device__ inline void store8(T *p, int valid, const float (&f)[8]) {
  if (valid >= 8) {
    Vec8<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e / 4][e % 4] = f[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = (T)f[e];
    }
    *reinterpret_cast<Vec8<T> *>(p) = r;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = (T)f[e];
  }
}

// The same where the values will not be read again soon: past the caches.
template <typename T>
__device__ inline void store8_past(T *p, int valid, const float (&f)[8]) {
  if (valid < 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = (T)f[e];
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __builtin_nontemporal_store(f32x4_any{f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]},
                                  reinterpret_cast<f32x4_any *>(p) + h);
  } else {
    decltype(Vec8<T>::v) r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (T)f[e];
    __builtin_nontemporal_store(r, reinterpret_cast<decltype(r) *>(p));
  }
}

// f(0) .. f(N - 1), the numbers as constants.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}

// ----- over lanes ------------------------------------------------------------

// x of the lane `N` further on in this lane's row of 16 (cyclic).
template <int N>
__device__ inline uint32_t rotate16(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + N, 0xf, 0xf,
                                               true);
}

// x of lane N of this lane's row of 16.
template <int N>
__device__ inline float from16(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)__float_as_uint(x), 0x150 + N, 0xf, 0xf, true));
}

// Magnitudes are compared as the integers that their bits are: a NaN is then
// above infinity, so that it is not lost.
__device__ inline uint32_t magnitude(float x) {
  return __float_as_uint(x) & 0x7fffffffu;
}
__device__ inline uint32_t max16(uint32_t x) {
  x = max(x, rotate16<8>(x));
  x = max(x, rotate16<4>(x));
  x = max(x, rotate16<2>(x));
  return max(x, rotate16<1>(x));
}

// The sum over this lane's row of 16, and over a wave's 64 lanes, in every lane.
__device__ inline float sum16(float x) {
  x += __uint_as_float(rotate16<8>(__float_as_uint(x)));
  x += __uint_as_float(rotate16<4>(__float_as_uint(x)));
  x += __uint_as_float(rotate16<2>(__float_as_uint(x)));
  return x + __uint_as_float(rotate16<1>(__float_as_uint(x)));
}
__device__ inline float sum64(float x) {
  x = sum16(x);
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// ----- e4m3 --------------------------------------------------------------------

constexpr float kE4m3Max = 448.f;
constexpr float kSmallestScale = 0x1p-126f;

template <bool POW2>
__device__ inline float scale_of(uint32_t amax_bits) {
  float s = __uint_as_float(amax_bits) / kE4m3Max;
  if (s < kSmallestScale) s = kSmallestScale;  // a NaN stays
  if (POW2 && s < __builtin_inff())
    s = __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u);
  return s;
}

// x / scale, rounded to float32 as a division is wherever that decides the
// e4m3 value, for three multiplications instead of a division's ten.
//
// With r = 1 / s correctly rounded, q = x r is off by a little over one unit
// in the last place; q + (x - q s) r, the remainder exact in a fused
// multiply-add, is the correctly rounded quotient unless the remainder
// underflows.  It cannot where it matters: below s = 2^-60 both x and s are
// taken times 2^64, and with s >= 2^-60 a remainder underflows only where
// x / s < 2^-40, which is 0 in e4m3 either way.  By a power of two, x r is
// x / s itself.
//
// scale inf: x / inf is 0 for a finite x and NaN for an infinite one, which
// is x * 0.  scale NaN: everything is NaN.
template <bool POW2>
struct Quotient {
  float up, s, r;
  bool tiny;  // whether any lane of the wave has up != 1 for its sake
  Quotient() = default;
  __device__ Quotient(float scale, uint32_t amax_bits) {
    if (POW2) {
      r = 1.f / scale;
    } else {
      const bool inf = scale == __builtin_inff();
      up = scale < 0x1p-60f ? 0x1p64f : 1.f;
      tiny = __any(scale < 0x1p-60f && amax_bits != 0);  // zeros need no care
      if (!tiny) up = 1.f;
      s = inf ? 0.f : scale * up;
      r = inf ? 0.f : 1.f / s;
    }
  }
  // The divisor that lane N of this lane's row of 16 has.
  template <int N>
  __device__ Quotient from() const {
    Quotient o;
    o.r = from16<N>(r);
    if (!POW2) {
      o.s = from16<N>(s);
      o.tiny = tiny;
      if (tiny) o.up = from16<N>(up);
    }
    return o;
  }
  __device__ float operator()(float x) const {
    if (POW2) return x * r;
    if (tiny) x *= up;
    const float q = x * r;
    // the remainder's negative, so that a zero keeps its sign
    return __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
  }
  // Eight at a time, so that `tiny` is a branch and not two more instructions
  // for each of them.
  __device__ void operator()(const float (&x)[8], float (&f)[8]) const {
    Quotient usual = *this;
    usual.tiny = false;
    if (!POW2 && tiny) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = usual(x[e] * up);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = usual(x[e]);
    }
  }
};

// Four values to e4m3, nearest even; |f| <= 448 or NaN.
__device__ inline uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

}  // namespace
}  // namespace xpose
