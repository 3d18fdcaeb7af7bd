// gfx950 kernels of root-mean-square norm with the residual's addition before
// it, as a tensor or straight as e4m3 with block scales, and of its backward
// pass.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/linear/xpose_linear.h"
#include "block_kernels.h"
#include "linear_device.h"
#include "linear_kernels.h"
#include "norm_device.h"

namespace xpose {
namespace {

// h = x + residual is rounded to its type before anything else happens to it:
// the stream holds it so, the backward pass and the next layer read it so, and
// the norm of another h than theirs would be a function of neither.
//
// A row stays in the registers of the TR lanes that work on it, NC chunks of
// eight neighbouring columns a lane: x and the residual are read once, h and y
// written once.  Rows of fewer columns than a load (SHORT) are read by elements.

template <typename T, bool SHORT>
__device__ inline Vec8<T> fetch8(const T *row, int64_t cols, int64_t col) {
  if constexpr (SHORT) return load_raw8(row + col, in_row(cols, col));
  return load_row8(row, cols, col);
}

// Eight elements of h from x (and the residual); zeros beyond the row.
template <typename T, bool RES, bool SHORT>
__device__ inline void sum8(Vec8<T> x, Vec8<T> res, int64_t cols, int64_t col, float (&h)[8]) {
  if constexpr (!SHORT) {
    settle8<T>(x, cols, col);
    if constexpr (RES) settle8<T>(res, cols, col);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h[e] = at8<T>(x, e);
    if constexpr (RES) h[e] = (float)(T)(h[e] + at8<T>(res, e));
  }
}

// As in layer norm, workgroups stay, with the weight in registers and the next
// row's loads under way.  Memory bounds it: 8192 x 8192 bfloat16 with the residual
// moves 537 MB in 95 us (5.6 TB/s; a copy reaches 6.3), 4096 x 8192 to e4m3
// 236 MB in 43 us.
template <typename T, Out OUT, bool RES, int TR, int NC, bool SHORT>
__global__ __launch_bounds__(norm_threads(TR)) void rms_norm_kernel(RmsNormArgs a) {
  __shared__ float lds[2][TR > 64 ? TR / 64 : 1];
  const int lane = threadIdx.x % TR;
  const int64_t first = (int64_t)blockIdx.x * (norm_threads(TR) / TR) + threadIdx.x / TR;
  const int64_t groups = (int64_t)gridDim.x * (norm_threads(TR) / TR);
  if (first >= a.rows) return;  // whole groups, and none where barriers follow
  float w[NC][8];
  Vec8<T> next_x[NC], next_res[NC];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      next_x[i] = fetch8<T, SHORT>((const T *)a.x + row * a.ldx, a.cols, col);
      if constexpr (RES) next_res[i] = fetch8<T, SHORT>((const T *)a.residual + row * a.ldr, a.cols, col);
    }
  };
  fetch(first);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t col = (i * TR + lane) * 8;
    load_param8(a.weight, a.param_dtype, col, in_row(a.cols, col), 1.f, w[i]);
  }
  int turn = 0;
  for (int64_t row = first; row < a.rows; row += groups, turn ^= 1) {
    float h[NC][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      sum8<T, RES, SHORT>(next_x[i], next_res[i], a.cols, (i * TR + lane) * 8, h[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __builtin_fmaf(h[i][e], h[i][e], s);
    }
    // unconditional: else the new row is copied, and so waited for, at once
    fetch(row + groups < a.rows ? row + groups : row);
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int64_t col = (i * TR + lane) * 8;
        store8((T *)a.h + row * a.ldh + col, in_row(a.cols, col), h[i]);
      }
    }
    const float rstd = 1.f / sqrtf(row_sum<TR>(s, lds[turn]) / (float)a.cols + a.eps);
    if (lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = h[i][e] * rstd * w[i][e];
      put_chunk<T, OUT>(a, row, col, in_row(a.cols, col), y);
    }
  }
}

// Rows of any length, in two sweeps; the second one reads h, which each lane
// has stored itself, and finds much of it in the caches.
template <typename T, Out OUT, bool RES>
__global__ __launch_bounds__(kLongThreads) void rms_norm_long_kernel(RmsNormArgs a) {
  __shared__ float lds[kLongThreads / 64];
  const int64_t row = long_index();
  if (row >= a.rows) return;
  const T *x = (const T *)a.x + row * a.ldx;
  constexpr int64_t kStep = kLongThreads * 8;
  float s = 0.f;
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += kStep) {
    const int valid = in_row(a.cols, col);
    float h[8];
    load8(x + col, valid, h);
    if constexpr (RES) {
      float r[8];
      load8((const T *)a.residual + row * a.ldr + col, valid, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (float)(T)(h[e] + r[e]);
      store8((T *)a.h + row * a.ldh + col, valid, h);
    }
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = __builtin_fmaf(h[e], h[e], t);
    s += t;
  }
  const float rstd = 1.f / sqrtf(row_sum<kLongThreads>(s, lds) / (float)a.cols + a.eps);
  if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
  const T *h = RES ? (const T *)a.h + row * a.ldh : x;
  // whole groups of 16 lanes stay together: the block maxima need them all
  for (int64_t c0 = 0; c0 < a.cols; c0 += kStep) {
    const int64_t col = c0 + threadIdx.x * 8;
    const int valid = in_row(a.cols, col);
    float v[8], w[8];
    load8(h + col, valid, v);
    load_param8(a.weight, a.param_dtype, col, valid, 1.f, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * w[e];
    put_chunk<T, OUT>(a, row, col, valid, v);
  }
}

hipError_t launch(const void *kernel, const RmsNormArgs &a, dim3 grid, int threads, hipStream_t s) {
  RmsNormArgs copy = a;
  void *args[] = {&copy};
  return hipLaunchKernel(kernel, grid, dim3(threads), args, 0, s);
}
// Whether half of the workgroups that fit on a compute unit, `half`, are enough
// for rows of `bytes` that leave as a tensor: more rows at a time than keep memory
// busy cost it.  A unit needs 24 KB of rows under way so, and 12 KB more for one
// workgroup alone, which has a row at a time and waits for its sum; 10 KB and 20 KB
// where each has 16 rows to go through, and the first and last ones count less.
// To e4m3 the arithmetic needs them all (4096 x 8192 53 us and 43).
//
// All and half, in us: bfloat16 with the residual, one workgroup of two, 14826 x
// 4519 127 and 162, 10468 x 6400 100 and 104, 9054 x 7400 102 and 104, 8723 x 7680
// 100 and 99.5, 8186 x 8184 102 and 98, 1000 x 8192 11.3 and 12.3; float32 so 7413 x
// 4519 107 and 105, 4154 x 8064 108 and 100, 700 x 6144 14.4 and 13.6.  Without it,
// four of eight, bfloat16 55833 x 1200 55 and 69, 43619 x 1536 50 and 54, 32714 x
// 2048 49 and 46, 5000 x 2048 8.2 and 9.6, 2000 x 4096 7.5 and 6.7.
bool half_will_do(int64_t rows, int64_t bytes, int half) {
  const int64_t under_way = bytes * half, kb = 1024;
  return under_way >= 24 * kb + 12 * kb / half || (rows >= 16 * 256 * half && under_way >= 10 * kb + 20 * kb / half);
}
template <typename T, Out OUT, bool RES, int TR, int NC, bool SHORT = false>
hipError_t launch_rms(const RmsNormArgs &a, hipStream_t s) {
  constexpr int per = norm_threads(TR) / TR;
  const void *kernel = reinterpret_cast<const void *>(&rms_norm_kernel<T, OUT, RES, TR, NC, SHORT>);
  // as many workgroups as run at once: a few more would run after all others
  static std::atomic<int> at_once{0};  // of a compute unit; kept once it is known
  int n = at_once.load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, norm_threads(TR), 0) == hipSuccess && n > 0)
      at_once.store(n, std::memory_order_relaxed);
    else
      n = 1;
  }
  if (OUT == kTensor && TR > 64 && half_will_do(a.rows, a.cols * (int64_t)sizeof(T) * (RES ? 2 : 1), (n + 1) / 2))
    n = (n + 1) / 2;
  const int64_t grid = (a.rows + per - 1) / per, most = 256 * (int64_t)n;
  return launch(kernel, a, dim3((uint32_t)(grid < most ? grid : most)), norm_threads(TR), s);
}
template <typename T, Out OUT, bool RES>
hipError_t rms(const RmsNormArgs &a, hipStream_t s) {
  if (a.cols < 8) return launch_rms<T, OUT, RES, 16, 1, true>(a, s);
  if (a.cols <= 128) return launch_rms<T, OUT, RES, 16, 1>(a, s);
  if (a.cols <= 256) return launch_rms<T, OUT, RES, 16, 2>(a, s);
  if (a.cols <= 512) return launch_rms<T, OUT, RES, 64, 1>(a, s);
  if (a.cols <= 1024) return launch_rms<T, OUT, RES, 64, 2>(a, s);
  if (a.cols <= 2048) return launch_rms<T, OUT, RES, 256, 1>(a, s);
  if (a.cols <= 4096) return launch_rms<T, OUT, RES, 256, 2>(a, s);
  if (a.cols <= 8192) return launch_rms<T, OUT, RES, 512, 2>(a, s);
  if (a.cols <= 16384) return launch_rms<T, OUT, RES, 1024, 2>(a, s);
  return launch(reinterpret_cast<const void *>(&rms_norm_long_kernel<T, OUT, RES>), a, long_grid(a.rows),
                kLongThreads, s);
}
template <typename T, Out OUT>
hipError_t rms(const RmsNormArgs &a, hipStream_t s) {
  return a.residual ? rms<T, OUT, true>(a, s) : rms<T, OUT, false>(a, s);
}
template <Out OUT>
hipError_t rms(const RmsNormArgs &a, int dtype, hipStream_t s) {
  if (dtype == XPOSE_F32) return rms<float, OUT>(a, s);
  if (dtype == XPOSE_F16) return rms<_Float16, OUT>(a, s);
  return rms<__bf16, OUT>(a, s);
}

// ----- the backward pass -----------------------------------------------------
//
// With xhat = h rstd and g = dy weight: dh = rstd (g - xhat mean(g xhat)) plus
// the gradient that h has from elsewhere (RES), rounded once.  A group of TR
// lanes walks over rows `groups` apart and keeps the sums for dweight of its
// columns in registers, so everything is read once; the workgroup's sums go to
// the workspace, and a second launch adds them up column by column, all in a
// fixed order.

template <typename T, bool RES, int TR, int NC, bool SHORT>
__global__ __launch_bounds__(norm_threads(TR)) void rms_norm_bwd_kernel(RmsNormBwdArgs a) {
  constexpr int kPer = norm_threads(TR) / TR;  // of a workgroup
  __shared__ float lds[2][TR > 64 ? TR / 64 : 1];
  __shared__ __align__(16) float joined[kPer > 1 ? 3 : 1][kPer > 1 ? NC * TR * 8 : 4];
  const int lane = threadIdx.x % TR, wave = threadIdx.x / 64;
  const int64_t group = (int64_t)blockIdx.x * kPer + threadIdx.x / TR, groups = (int64_t)a.parts * kPer;
  float w[NC][8], dw[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t col = (i * TR + lane) * 8;
    load_param8(a.weight, a.param_dtype, col, in_row(a.cols, col), 1.f, w[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  }
  Vec8<T> next_dy[NC], next_h[NC], next_res[NC];
  float next_rstd;
  auto fetch = [&](int64_t row) {
    next_rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      next_dy[i] = fetch8<T, SHORT>((const T *)a.dy + row * a.lddy, a.cols, col);
      next_h[i] = fetch8<T, SHORT>((const T *)a.h + row * a.ldh, a.cols, col);
      if constexpr (RES) next_res[i] = fetch8<T, SHORT>((const T *)a.dresidual + row * a.lddr, a.cols, col);
    }
  };
  if (group < a.rows) fetch(group);
  int turn = 0;
  for (int64_t row = group; row < a.rows; row += groups, turn ^= 1) {
    const float rstd = next_rstd;
    float dy[NC][8], xhat[NC][8];
    Vec8<T> res[NC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      sum8<T, false, SHORT>(next_dy[i], next_dy[i], a.cols, col, dy[i]);
      sum8<T, false, SHORT>(next_h[i], next_h[i], a.cols, col, xhat[i]);
      if constexpr (RES) res[i] = next_res[i];
    }
    // unconditional: else the new row is copied, and so waited for, at once
    fetch(row + groups < a.rows ? row + groups : row);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int valid = in_row(a.cols, (i * TR + lane) * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xhat[i][e] = e < valid ? xhat[i][e] * rstd : 0.f;  // rstd may be inf
        const float gx = dy[i][e] * xhat[i][e];
        s = __builtin_fmaf(gx, w[i][e], s);
        dw[i][e] += gx;
      }
    }
    s = row_sum<TR>(s, lds[turn]) / (float)a.cols;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      float d[8];
      if constexpr (RES && !SHORT) settle8<T>(res[i], a.cols, col);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = (dy[i][e] * w[i][e] - xhat[i][e] * s) * rstd;
        if constexpr (RES) d[e] += at8<T>(res[i], e);
      }
      store8((T *)a.dx + row * a.lddx + col, in_row(a.cols, col), d);
    }
  }
  if constexpr (kPer > 1) {  // four waves' sums, first of the groups in each
    if constexpr (TR == 16) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[i][e] += __shfl_xor(dw[i][e], 16);
          dw[i][e] += __shfl_xor(dw[i][e], 32);
        }
    }
    if (wave > 0 && threadIdx.x % 64 < TR) {
#pragma unroll
      for (int i = 0; i < NC; ++i) store8(&joined[wave - 1][(i * TR + lane) * 8], 8, dw[i]);
    }
    __syncthreads();
    if (threadIdx.x >= TR) return;
#pragma unroll
    for (int v = 0; v < 3; ++v)
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] += joined[v][(i * TR + lane) * 8 + e];
  }
  float *p = a.partial + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t col = (i * TR + lane) * 8;
    store8(p + col, in_row(a.cols, col), dw[i]);
  }
}

// Rows of any length: their sums first, then blocks of columns.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void rms_norm_bwd_sums_kernel(RmsNormBwdArgs a) {
  __shared__ float lds[kLongThreads / 64];
  const int64_t row = long_index();
  if (row >= a.rows) return;
  const float rstd = a.rstd[row];
  float s = 0.f;
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += kLongThreads * 8) {
    const int valid = in_row(a.cols, col);
    float dy[8], h[8], w[8], t = 0.f;
    load8((const T *)a.dy + row * a.lddy + col, valid, dy);
    load8((const T *)a.h + row * a.ldh + col, valid, h);
    load_param8(a.weight, a.param_dtype, col, valid, 1.f, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) t = __builtin_fmaf(dy[e] * (e < valid ? h[e] * rstd : 0.f), w[e], t);
    s += t;
  }
  s = row_sum<kLongThreads>(s, lds);
  if (threadIdx.x == 0) a.partial[row] = s / (float)a.cols;
}

constexpr int kLongBlockThreads = 256, kLongBlock = 8 * kLongBlockThreads;  // columns of a workgroup
template <typename T, bool RES>
__global__ __launch_bounds__(kLongBlockThreads) void rms_norm_bwd_long_kernel(RmsNormBwdArgs a) {
  const int64_t blocks = (a.cols + kLongBlock - 1) / kLongBlock;
  const int64_t col = (int64_t)(blockIdx.x % blocks) * kLongBlock + threadIdx.x * 8;
  const int group = (int)(blockIdx.x / blocks);
  const int valid = in_row(a.cols, col);
  float w[8], dw[8] = {};
  load_param8(a.weight, a.param_dtype, col, valid, 1.f, w);
  for (int64_t row = group; row < a.rows; row += a.parts) {
    const float rstd = a.rstd[row], s = a.partial[row];
    float dy[8], h[8], res[8], d[8];
    load8((const T *)a.dy + row * a.lddy + col, valid, dy);
    load8((const T *)a.h + row * a.ldh + col, valid, h);
    if constexpr (RES) load8((const T *)a.dresidual + row * a.lddr + col, valid, res);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xhat = h[e] * rstd;
      d[e] = (dy[e] * w[e] - xhat * s) * rstd;
      if constexpr (RES) d[e] += res[e];
      dw[e] = __builtin_fmaf(dy[e], xhat, dw[e]);
    }
    store8((T *)a.dx + row * a.lddx + col, valid, d);
  }
  store8(a.partial + a.rows + (int64_t)group * a.cols + col, valid, dw);
}

// 64 columns a workgroup: lane l of a wave has column l, the 16 waves every
// 16th partial sum.
constexpr int kParamWaves = kLongThreads / 64;
__global__ __launch_bounds__(64 * kParamWaves) void rms_norm_bwd_params_kernel(RmsNormBwdArgs a) {
  __shared__ float lds[kParamWaves][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t block = long_index(), col = block * 64 + lane;
  if (block * 64 >= a.cols) return;
  float s = 0.f;
  if (col < a.cols) {
#pragma unroll 8
    for (int g = wave; g < a.parts; g += kParamWaves) s += a.partial[(int64_t)g * a.cols + col];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < a.cols) {
#pragma unroll
    for (int v = 1; v < kParamWaves; ++v) s += lds[v][lane];
    a.dweight[col] = s;
  }
}

constexpr bool in_registers(int64_t cols) { return cols <= 8192; }

hipError_t launch(const void *kernel, const RmsNormBwdArgs &a, dim3 grid, int threads, hipStream_t s) {
  RmsNormBwdArgs copy = a;
  void *args[] = {&copy};
  return hipLaunchKernel(kernel, grid, dim3(threads), args, 0, s);
}
template <typename T, bool RES, int TR, int NC, bool SHORT = false>
hipError_t launch_bwd(const RmsNormBwdArgs &a, hipStream_t s) {
  return launch(reinterpret_cast<const void *>(&rms_norm_bwd_kernel<T, RES, TR, NC, SHORT>), a,
                dim3((uint32_t)a.parts), norm_threads(TR), s);
}
template <typename T, bool RES>
hipError_t rms_bwd(const RmsNormBwdArgs &a, hipStream_t s) {
  if (!in_registers(a.cols)) {
    const hipError_t e = launch(reinterpret_cast<const void *>(&rms_norm_bwd_sums_kernel<T>), a, long_grid(a.rows),
                                kLongThreads, s);
    if (e != hipSuccess) return e;
    return launch(reinterpret_cast<const void *>(&rms_norm_bwd_long_kernel<T, RES>), a,
                  dim3((uint32_t)((a.cols + kLongBlock - 1) / kLongBlock * a.parts)), kLongBlockThreads, s);
  }
  if (a.cols < 8) return launch_bwd<T, RES, 16, 1, true>(a, s);
  if (a.cols <= 128) return launch_bwd<T, RES, 16, 1>(a, s);
  if (a.cols <= 256) return launch_bwd<T, RES, 16, 2>(a, s);
  if (a.cols <= 512) return launch_bwd<T, RES, 64, 1>(a, s);
  if (a.cols <= 1024) return launch_bwd<T, RES, 64, 2>(a, s);
  if (a.cols <= 2048) return launch_bwd<T, RES, 256, 1>(a, s);
  if (a.cols <= 4096) return launch_bwd<T, RES, 256, 2>(a, s);
  return launch_bwd<T, RES, 512, 2>(a, s);
}
template <typename T>
hipError_t rms_bwd(const RmsNormBwdArgs &a, hipStream_t s) {
  return a.dresidual ? rms_bwd<T, true>(a, s) : rms_bwd<T, false>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const RmsNormArgs &a, int dtype, hipStream_t s) { return rms<kTensor>(a, dtype, s); }
hipError_t launch_rms_norm_quantize(const RmsNormArgs &a, int dtype, bool pow2, hipStream_t s) {
  return pow2 ? rms<kE4m3Pow2>(a, dtype, s) : rms<kE4m3>(a, dtype, s);
}

// Workgroups, each with a row of sums in the workspace: as for layer norm's
// backward pass, but that half as many do for rows of over 2048 columns
// (8192 x 4096 bfloat16 with the residual 48 us with 256, 52 with 512; 16384 x
// 4096 float32 144 and 153; but 16384 x 2048 bfloat16 65 and 45).
int rms_norm_bwd_parts(int64_t rows, int64_t cols) {
  if (cols <= 1024) {
    const int64_t per = cols <= 256 ? 16 : 4, parts = (rows + per - 1) / per;
    return (int)(parts < 256 ? parts : parts < 8 * 256 ? 256 : 512);
  }
  const int64_t most = cols <= 2048 ? 512 : 256;
  int64_t parts = 1;
  while (parts < most && parts * parts < 32 * rows) parts *= 2;
  return (int)(rows < parts ? rows : parts);
}
bool rms_norm_bwd_fits(int64_t rows, int64_t cols) {
  if (in_registers(cols)) return true;
  const int64_t blocks = cols / kLongBlock + (cols % kLongBlock != 0);
  return rms_norm_bwd_parts(rows, cols) <= kMaxThreads / kLongBlockThreads / blocks;
}
int64_t rms_norm_bwd_row_floats(int64_t rows, int64_t cols) { return in_registers(cols) ? 0 : rows; }

hipError_t launch_rms_norm_backward(const RmsNormBwdArgs &a, int dtype, hipStream_t s) {
  if (a.rows > 0) {
    const hipError_t e = dtype == XPOSE_F32   ? rms_bwd<float>(a, s)
                         : dtype == XPOSE_F16 ? rms_bwd<_Float16>(a, s)
                                              : rms_bwd<__bf16>(a, s);
    if (e != hipSuccess) return e;
  }
  if (!a.dweight) return hipSuccess;
  RmsNormBwdArgs sums = a;
  if (a.rows > 0) sums.partial += rms_norm_bwd_row_floats(a.rows, a.cols);
  return launch(reinterpret_cast<const void *>(&rms_norm_bwd_params_kernel), sums, long_grid((a.cols + 63) / 64),
                kLongThreads, s);
}

}  // namespace xpose
