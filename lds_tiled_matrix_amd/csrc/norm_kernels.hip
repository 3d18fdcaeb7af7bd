// gfx950 kernels of layer norm, as a tensor or straight as e4m3 with block
// scales, and of its backward pass.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/linear/xpose_linear.h"
#include "linear_device.h"
#include "linear_kernels.h"

namespace xpose {
namespace {

// A row stays in the registers of the TR lanes that work on it, NC chunks of
// eight neighbouring columns a lane: it is read once, and the variance is the
// mean of the centred squares, not a difference of large sums.
//
// TR is 16 (a row of up to 256 columns to a quarter of a wave), 64 (a wave a
// row) or the whole workgroup.  Short rows on 64 lanes leave most of them idle:
// 100000 x 128 bfloat16 took 32 us.

// Weights and biases: float32, or of the input's 16-bit types.
__device__ inline void load_param8(const void *p, int dtype, int64_t col, int valid, float none, float (&f)[8]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = none;
  } else if (dtype == XPOSE_F32) {
    load8((const float *)p + col, valid, f);
  } else if (dtype == XPOSE_F16) {
    load8((const _Float16 *)p + col, valid, f);
  } else {
    load8((const __bf16 *)p + col, valid, f);
  }
}

__device__ inline int in_row(int64_t cols, int64_t col) {
  const int64_t left = cols - col;
  return left < 0 ? 0 : left > 8 ? 8 : (int)left;
}

// Sums over the lanes of a row, the same in all of them.  Within a wave no LDS
// is needed; else `lds` holds a float for each wave, and two calls in
// turn use two of them, so that one barrier a call is enough: who writes to the
// first one again has passed the second's barrier, behind everybody's reads.
template <int TR>
__device__ inline float row_sum(float x, float *lds) {
  if constexpr (TR == 16) return sum16(x);
  x = sum64(x);
  if constexpr (TR > 64) {
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
    __syncthreads();
    x = lds[0];
#pragma unroll
    for (int w = 1; w < TR / 64; ++w) x += lds[w];
  }
  return x;
}

enum Out { kTensor, kE4m3, kE4m3Pow2 };

// What a lane does with eight normalised values of one chunk.
template <typename T, Out OUT>
__device__ inline void put_chunk(const NormArgs &a, int64_t row, int64_t col, int valid, const float (&y)[8]) {
  if constexpr (OUT == kTensor) {
    store8((T *)a.y + row * a.ldy + col, valid, y);
  } else {
    // the 16 lanes of a DPP row hold the 128 columns of one block
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, magnitude(y[e]));
    if (valid < 8) {
      m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, e < valid ? magnitude(y[e]) : 0u);
    }
    m = max16(m);
    const float scale = scale_of<OUT == kE4m3Pow2>(m);
    if (threadIdx.x % 16 == 0 && valid > 0) a.scale[(col >> 7) * a.ld_scale + row] = scale;
    const Quotient<OUT == kE4m3Pow2> by(scale, m);
    float f[8];
    by(y, f);
    const u32x2 w = {e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7])};
    uint8_t *q = (uint8_t *)a.y + row * a.ldy + col;
    if (valid == 8) {
      *reinterpret_cast<u32x2 *>(q) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < valid) q[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
    }
  }
}

constexpr int norm_threads(int tr) { return tr <= 64 ? 256 : tr; }

// Workgroups stay: a group of TR lanes walks over rows `groups` apart with the
// weight and bias in registers (read anew for each row they are four times a
// bfloat16 row's bytes: 8192 x 8192 took 56 us so), and the next row's loads
// are under way while this one is worked on: 43 us, 6.2 TB/s (the kernel's own
// time; a call among others 44 to 50).  Rows of odd lengths: 12345 x 6789 bfloat16
// 79 us; with loads of single elements at a row's end, which cannot stay under
// way, a quarter more.
template <typename T, Out OUT, int TR, int NC>
__global__ __launch_bounds__(norm_threads(TR)) void norm_kernel(NormArgs a) {
  __shared__ float lds[2][TR > 64 ? TR / 64 : 1];
  const int lane = threadIdx.x % TR;
  const int64_t first = (int64_t)blockIdx.x * (norm_threads(TR) / TR) + threadIdx.x / TR;
  const int64_t groups = (int64_t)gridDim.x * (norm_threads(TR) / TR);
  if (first >= a.rows) return;  // whole groups, and none where barriers follow
  float w[NC][8], b[NC][8];
  Vec8<T> ahead[NC];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      ahead[i] = load_row8((const T *)a.x + row * a.ldx, a.cols, col);
    }
  };
  fetch(first);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t col = (i * TR + lane) * 8;
    load_param8(a.weight, a.param_dtype, col, in_row(a.cols, col), 1.f, w[i]);
    load_param8(a.bias, a.param_dtype, col, in_row(a.cols, col), 0.f, b[i]);
  }
  for (int64_t row = first; row < a.rows; row += groups) {
    float v[NC][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      settle8<T>(ahead[i], a.cols, (i * TR + lane) * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] = at8<T>(ahead[i], e);
        s += v[i][e];
      }
    }
    // unconditional: else the new row is copied, and so waited for, at once
    fetch(row + groups < a.rows ? row + groups : row);
    const float mean = row_sum<TR>(s, lds[0]) / (float)a.cols;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int valid = in_row(a.cols, (i * TR + lane) * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] -= mean;
      if (valid < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= valid) v[i][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __builtin_fmaf(v[i][e], v[i][e], s);
    }
    const float rstd = 1.f / sqrtf(row_sum<TR>(s, lds[1]) / (float)a.cols + a.eps);
    if (lane == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(v[i][e] * rstd, w[i][e], b[i][e]);
      put_chunk<T, OUT>(a, row, col, in_row(a.cols, col), y);
    }
  }
}

// A workgroup of 1024 for each of `count` things.  A launch can have no more than
// 2^32 - 1 threads in one dimension, so past 4 million workgroups they go on in
// the second; the last ones may have nothing to do.
constexpr int kLongThreads = 1024;
dim3 long_grid(int64_t count, uint32_t kinds = 1) {
  const int64_t most = kMaxThreads / kLongThreads, x = count < most ? count : most;
  return dim3((uint32_t)x, (uint32_t)((count + x - 1) / x), kinds);
}
__device__ inline int64_t long_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Rows of any length, in three sweeps; the second and third find much of the
// row in the caches.
template <typename T, Out OUT>
__global__ __launch_bounds__(kLongThreads) void norm_long_kernel(NormArgs a) {
  __shared__ float lds[2][kLongThreads / 64];
  const int64_t row = long_index();
  if (row >= a.rows) return;
  const T *x = (const T *)a.x + row * a.ldx;
  constexpr int64_t kStep = kLongThreads * 8;
  float s = 0.f;
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += kStep) {
    float v[8];
    load8(x + col, in_row(a.cols, col), v);
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) t += v[e];
    s += t;
  }
  const float mean = row_sum<kLongThreads>(s, lds[0]) / (float)a.cols;
  s = 0.f;
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += kStep) {
    const int valid = in_row(a.cols, col);
    float v[8];
    load8(x + col, valid, v);
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = e < valid ? v[e] - mean : 0.f;
      t = __builtin_fmaf(d, d, t);
    }
    s += t;
  }
  const float rstd = 1.f / sqrtf(row_sum<kLongThreads>(s, lds[1]) / (float)a.cols + a.eps);
  if (threadIdx.x == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  // whole groups of 16 lanes stay together: the block maxima need them all
  for (int64_t c0 = 0; c0 < a.cols; c0 += kStep) {
    const int64_t col = c0 + threadIdx.x * 8;
    const int valid = in_row(a.cols, col);
    float v[8], w[8], b[8];
    load8(x + col, valid, v);
    load_param8(a.weight, a.param_dtype, col, valid, 1.f, w);
    load_param8(a.bias, a.param_dtype, col, valid, 0.f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf((v[e] - mean) * rstd, w[e], b[e]);
    put_chunk<T, OUT>(a, row, col, valid, v);
  }
}

hipError_t launch(const void *kernel, const NormArgs &a, dim3 grid, int threads, hipStream_t s) {
  NormArgs copy = a;
  void *args[] = {&copy};
  return hipLaunchKernel(kernel, grid, dim3(threads), args, 0, s);
}
template <typename T, Out OUT, int TR, int NC>
hipError_t launch_norm(const NormArgs &a, hipStream_t s) {
  constexpr int per = norm_threads(TR) / TR;
  const void *kernel = reinterpret_cast<const void *>(&norm_kernel<T, OUT, TR, NC>);
  // as many workgroups as run at once: a few more would run after all others
  // (16384 x 4096 bfloat16 takes 45 us, 51 with 6 of which 5 fit)
  static std::atomic<int> at_once{0};  // of a compute unit; kept once it is known
  int n = at_once.load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, norm_threads(TR), 0) == hipSuccess && n > 0)
      at_once.store(n, std::memory_order_relaxed);
    else
      n = 1;
  }
  const int64_t grid = (a.rows + per - 1) / per, most = 256 * (int64_t)n;
  return launch(kernel, a, dim3((uint32_t)(grid < most ? grid : most)), norm_threads(TR), s);
}
template <typename T, Out OUT>
hipError_t launch_long_norm(const NormArgs &a, hipStream_t s) {
  return launch(reinterpret_cast<const void *>(&norm_long_kernel<T, OUT>), a,
                long_grid(a.rows), kLongThreads, s);
}
template <typename T, Out OUT>
hipError_t norm(const NormArgs &a, hipStream_t s) {
  if (a.cols < 8) return launch_long_norm<T, OUT>(a, s);  // shorter than a load
  // Where twice the lanes would be little more than half used, three chunks a
  // lane, if rows fill the card so (five waves a SIMD): 4000 x 9000 bfloat16 30
  // us, 42 on 1024 lanes; 16384 x 2800 to e4m3 42 and 51; but 64 x 4519 5.7 and
  // 4.8.  float32 to float32 is near what memory allows without (8192 x 8192 97
  // us, of which a copy would take 85).
  if constexpr (sizeof(T) == 2 || OUT != kTensor) {
    const auto three = [&](int64_t lanes) {
      return a.cols > 2 * 8 * lanes && a.cols <= 3 * 8 * lanes && a.rows * lanes >= 256 * 1280;
    };
    if (three(64)) return launch_norm<T, OUT, 64, 3>(a, s);
    if (three(128)) return launch_norm<T, OUT, 128, 3>(a, s);
    if (three(256)) return launch_norm<T, OUT, 256, 3>(a, s);
    if (three(512)) return launch_norm<T, OUT, 512, 3>(a, s);
  }
  if (a.cols <= 128) return launch_norm<T, OUT, 16, 1>(a, s);
  if (a.cols <= 256) return launch_norm<T, OUT, 16, 2>(a, s);
  if (a.cols <= 512) return launch_norm<T, OUT, 64, 1>(a, s);
  if (a.cols <= 1024) return launch_norm<T, OUT, 64, 2>(a, s);
  if (a.cols <= 2048) return launch_norm<T, OUT, 256, 1>(a, s);
  if (a.cols <= 4096) return launch_norm<T, OUT, 256, 2>(a, s);
  if (a.cols <= 8192) return launch_norm<T, OUT, 512, 2>(a, s);
  if (a.cols <= 16384) return launch_norm<T, OUT, 1024, 2>(a, s);
  return launch_long_norm<T, OUT>(a, s);
}
template <Out OUT>
hipError_t norm(const NormArgs &a, int dtype, hipStream_t s) {
  if (dtype == XPOSE_F32) return norm<float, OUT>(a, s);
  if (dtype == XPOSE_F16) return norm<_Float16, OUT>(a, s);
  return norm<__bf16, OUT>(a, s);
}

// ----- the backward pass -----------------------------------------------------
//
// A group of TR lanes walks over rows `groups` apart and keeps the sums for
// dweight and dbias of its columns in registers, so dy and x are read once; the
// workgroup's two rows of sums go to the workspace, and a second launch adds
// them up column by column, all in a fixed order.  8192 x 4096 bfloat16 takes
// 44 us (4.6 TB/s; memory bounds it at 32).  Two rows' loads under way instead of
// one gain nothing.
// Short rows: 100000 x 128 bfloat16 takes 20 us, 75 with a wave a row and a sum
// a wave; 4096 x 1024 12 us, 17 with a sum a wave.

template <typename T, int TR, int NC>
__global__ __launch_bounds__(norm_threads(TR)) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int kPer = norm_threads(TR) / TR;  // of a workgroup
  __shared__ float lds[2][2][TR > 64 ? TR / 64 : 1];
  __shared__ __align__(16) float joined[kPer > 1 ? 3 : 1][2][kPer > 1 ? NC * TR * 8 : 4];
  const int lane = threadIdx.x % TR, wave = threadIdx.x / 64;
  const int64_t group = (int64_t)blockIdx.x * kPer + threadIdx.x / TR, groups = (int64_t)a.parts * kPer;
  float w[NC][8], dw[NC][8], db[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t col = (i * TR + lane) * 8;
    load_param8(a.weight, a.param_dtype, col, in_row(a.cols, col), 1.f, w[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.f;
  }
  // the next row's loads are under way while this one is worked on
  Vec8<T> next_dy[NC], next_x[NC];
  float next_mean, next_rstd;
  auto fetch = [&](int64_t row) {
    next_mean = a.mean[row];
    next_rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      next_dy[i] = load_row8((const T *)a.dy + row * a.lddy, a.cols, col);
      next_x[i] = load_row8((const T *)a.x + row * a.ldx, a.cols, col);
    }
  };
  if (group < a.rows) fetch(group);
  int turn = 0;
  for (int64_t row = group; row < a.rows; row += groups, turn ^= 1) {
    const float mean = next_mean, rstd = next_rstd;
    float dy[NC][8], x[NC][8];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      settle8<T>(next_dy[i], a.cols, (i * TR + lane) * 8);
      settle8<T>(next_x[i], a.cols, (i * TR + lane) * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dy[i][e] = at8<T>(next_dy[i], e);
        x[i][e] = at8<T>(next_x[i], e);
      }
    }
    // unconditional: else the new row is copied, and so waited for, at once
    fetch(row + groups < a.rows ? row + groups : row);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int valid = in_row(a.cols, (i * TR + lane) * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = (x[i][e] - mean) * rstd;
      if (valid < 8) {  // a dy of 0 beyond the row is not enough: -mean rstd may be inf
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= valid) x[i][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = dy[i][e] * w[i][e];
        s1 += g;
        s2 = __builtin_fmaf(g, x[i][e], s2);
        db[i][e] += dy[i][e];
        dw[i][e] = __builtin_fmaf(dy[i][e], x[i][e], dw[i][e]);
      }
    }
    // both sums behind one barrier; the next row uses the other half of lds
    s1 = TR == 16 ? sum16(s1) : sum64(s1);
    s2 = TR == 16 ? sum16(s2) : sum64(s2);
    if constexpr (TR > 64) {
      if (threadIdx.x % 64 == 0) {
        lds[turn][0][threadIdx.x / 64] = s1;
        lds[turn][1][threadIdx.x / 64] = s2;
      }
      __syncthreads();
      s1 = lds[turn][0][0];
      s2 = lds[turn][1][0];
#pragma unroll
      for (int v = 1; v < TR / 64; ++v) {
        s1 += lds[turn][0][v];
        s2 += lds[turn][1][v];
      }
    }
    s1 /= (float)a.cols;
    s2 /= (float)a.cols;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = (i * TR + lane) * 8;
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        d[e] = (dy[i][e] * w[i][e] - s1 - x[i][e] * s2) * rstd;
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
          db[i][e] += __shfl_xor(db[i][e], 16);
          db[i][e] += __shfl_xor(db[i][e], 32);
        }
    }
    if (wave > 0 && threadIdx.x % 64 < TR) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        store8(&joined[wave - 1][0][(i * TR + lane) * 8], 8, dw[i]);
        store8(&joined[wave - 1][1][(i * TR + lane) * 8], 8, db[i]);
      }
    }
    __syncthreads();
    if (threadIdx.x >= TR) return;
#pragma unroll
    for (int v = 0; v < 3; ++v)
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[i][e] += joined[v][0][(i * TR + lane) * 8 + e];
          db[i][e] += joined[v][1][(i * TR + lane) * 8 + e];
        }
  }
  float *p = a.partial + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t col = (i * TR + lane) * 8;
    const int valid = in_row(a.cols, col);
    store8(p + col, valid, dw[i]);
    store8(p + a.cols + col, valid, db[i]);
  }
}

// Rows of any length: their two sums first, then blocks of columns.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void norm_bwd_sums_kernel(NormBwdArgs a) {
  __shared__ float lds[2][kLongThreads / 64];
  const int64_t row = long_index();
  if (row >= a.rows) return;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += kLongThreads * 8) {
    const int valid = in_row(a.cols, col);
    float dy[8], x[8], w[8], t1 = 0.f, t2 = 0.f;
    load8((const T *)a.dy + row * a.lddy + col, valid, dy);
    load8((const T *)a.x + row * a.ldx + col, valid, x);
    load_param8(a.weight, a.param_dtype, col, valid, 1.f, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = dy[e] * w[e];
      t1 += g;
      t2 = __builtin_fmaf(g, e < valid ? (x[e] - mean) * rstd : 0.f, t2);
    }
    s1 += t1;
    s2 += t2;
  }
  s1 = row_sum<kLongThreads>(s1, lds[0]);
  s2 = row_sum<kLongThreads>(s2, lds[1]);
  if (threadIdx.x == 0) {
    a.partial[2 * row] = s1 / (float)a.cols;
    a.partial[2 * row + 1] = s2 / (float)a.cols;
  }
}

constexpr int kLongBlockThreads = 256, kLongBlock = 8 * kLongBlockThreads;  // columns of a workgroup
template <typename T>
__global__ __launch_bounds__(kLongBlockThreads) void norm_bwd_long_kernel(NormBwdArgs a) {
  const int64_t blocks = (a.cols + kLongBlock - 1) / kLongBlock;
  const int64_t col = (int64_t)(blockIdx.x % blocks) * kLongBlock + threadIdx.x * 8;
  const int group = (int)(blockIdx.x / blocks);
  const int valid = in_row(a.cols, col);
  float w[8], dw[8] = {}, db[8] = {};
  load_param8(a.weight, a.param_dtype, col, valid, 1.f, w);
  for (int64_t row = group; row < a.rows; row += a.parts) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    const float s1 = a.partial[2 * row], s2 = a.partial[2 * row + 1];
    float dy[8], x[8], d[8];
    load8((const T *)a.dy + row * a.lddy + col, valid, dy);
    load8((const T *)a.x + row * a.ldx + col, valid, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xhat = (x[e] - mean) * rstd;
      d[e] = (dy[e] * w[e] - s1 - xhat * s2) * rstd;
      db[e] += dy[e];
      dw[e] = __builtin_fmaf(dy[e], xhat, dw[e]);
    }
    store8((T *)a.dx + row * a.lddx + col, valid, d);
  }
  float *p = a.partial + 2 * a.rows + (int64_t)group * 2 * a.cols;
  store8(p + col, valid, dw);
  store8(p + a.cols + col, valid, db);
}

// 64 columns of one gradient a workgroup: lane l of a wave has column l, the
// 16 waves every 16th partial sum.
constexpr int kParamWaves = kLongThreads / 64;
__global__ __launch_bounds__(64 * kParamWaves) void norm_bwd_params_kernel(NormBwdArgs a) {
  __shared__ float lds[kParamWaves][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int which = blockIdx.z;
  const int64_t block = long_index(), col = block * 64 + lane;
  float *out = which ? a.dbias : a.dweight;
  if (!out || block * 64 >= a.cols) return;
  float s = 0.f;
  if (col < a.cols) {
    const float *p = a.partial + which * a.cols + col;
#pragma unroll 8
    for (int g = wave; g < a.parts; g += kParamWaves) s += p[(int64_t)g * 2 * a.cols];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < a.cols) {
#pragma unroll
    for (int v = 1; v < kParamWaves; ++v) s += lds[v][lane];
    out[col] = s;
  }
}

// More than 8192 columns would spill registers, under eight are less than a load.
constexpr bool in_registers(int64_t cols) { return cols >= 8 && cols <= 8192; }

hipError_t launch(const void *kernel, const NormBwdArgs &a, dim3 grid, int threads, hipStream_t s) {
  NormBwdArgs copy = a;
  void *args[] = {&copy};
  return hipLaunchKernel(kernel, grid, dim3(threads), args, 0, s);
}
template <typename T, int TR, int NC>
hipError_t launch_bwd(const NormBwdArgs &a, hipStream_t s) {
  return launch(reinterpret_cast<const void *>(&norm_bwd_kernel<T, TR, NC>), a,
                dim3((uint32_t)a.parts), norm_threads(TR), s);
}
template <typename T>
hipError_t norm_bwd(const NormBwdArgs &a, hipStream_t s) {
  if (!in_registers(a.cols)) {
    hipError_t e = launch(reinterpret_cast<const void *>(&norm_bwd_sums_kernel<T>), a, long_grid(a.rows),
                          kLongThreads, s);
    if (e != hipSuccess) return e;
    return launch(reinterpret_cast<const void *>(&norm_bwd_long_kernel<T>), a,
                  dim3((uint32_t)((a.cols + kLongBlock - 1) / kLongBlock * a.parts)), kLongBlockThreads, s);
  }
  if (a.cols <= 128) return launch_bwd<T, 16, 1>(a, s);
  if (a.cols <= 256) return launch_bwd<T, 16, 2>(a, s);
  if (a.cols <= 512) return launch_bwd<T, 64, 1>(a, s);
  if (a.cols <= 1024) return launch_bwd<T, 64, 2>(a, s);
  if (a.cols <= 2048) return launch_bwd<T, 256, 1>(a, s);
  if (a.cols <= 4096) return launch_bwd<T, 256, 2>(a, s);
  return launch_bwd<T, 512, 2>(a, s);
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs &a, int dtype, hipStream_t s) {
  return norm<kTensor>(a, dtype, s);
}
hipError_t launch_layer_norm_quantize(const NormArgs &a, int dtype, bool pow2, hipStream_t s) {
  return pow2 ? norm<kE4m3Pow2>(a, dtype, s) : norm<kE4m3>(a, dtype, s);
}

// Workgroups, each with two rows of sums in the workspace.  Its rows cost time
// one after the other, its sums are written and read again.
// - To 1024 columns (`per` rows at a time, joined into one sum): a row each up
//   to 256 workgroups, twice as many from eight rows each (bfloat16, 256 against
//   512: 4096 x 1024 11.8 and 13.2 us, 16384 x 512 20.6 and 16.9).
// - A row a workgroup: the least of both lies near sqrt(32 rows), and powers of
//   two load the 256 compute units evenly (3001 x 2999: 29 us with 512, 37 with
//   334).  No more than run at once: two on a compute unit, or one for rows over
//   4096 columns (2048 x 8192: 34 us with 512, 27 with 256; 512 x 4096: 18 us
//   with 512, 12.4 with 128).
int norm_bwd_parts(int64_t rows, int64_t cols) {
  if (cols <= 1024) {
    const int64_t per = cols <= 256 ? 16 : 4, parts = (rows + per - 1) / per;
    return (int)(parts < 256 ? parts : parts < 8 * 256 ? 256 : 512);
  }
  const int64_t most = cols <= 4096 ? 512 : 256;
  int64_t parts = 1;
  while (parts < most && parts * parts < 32 * rows) parts *= 2;
  return (int)(rows < parts ? rows : parts);
}
bool norm_bwd_fits(int64_t rows, int64_t cols) {
  if (in_registers(cols)) return true;
  const int64_t blocks = cols / kLongBlock + (cols % kLongBlock != 0);
  return blocks == 0 || norm_bwd_parts(rows, cols) <= kMaxThreads / kLongBlockThreads / blocks;
}
int64_t norm_bwd_row_floats(int64_t rows, int64_t cols) {
  return in_registers(cols) ? 0 : 2 * rows;
}

hipError_t launch_layer_norm_backward(const NormBwdArgs &a, int dtype, hipStream_t s) {
  if (a.rows > 0) {
    const hipError_t e = dtype == XPOSE_F32   ? norm_bwd<float>(a, s)
                         : dtype == XPOSE_F16 ? norm_bwd<_Float16>(a, s)
                                              : norm_bwd<__bf16>(a, s);
    if (e != hipSuccess) return e;
  }
  if (!a.dweight && !a.dbias) return hipSuccess;
  NormBwdArgs sums = a;
  if (a.rows > 0) sums.partial += norm_bwd_row_floats(a.rows, a.cols);
  return launch(reinterpret_cast<const void *>(&norm_bwd_params_kernel), sums,
                long_grid((a.cols + 63) / 64, 2), kLongThreads, s);
}

}  // namespace xpose
