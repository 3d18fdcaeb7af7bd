// Device helpers shared by the kernels of layer norm and root-mean-square norm:
// parameters, sums over the lanes of a row, and what becomes of normalised values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/linear/xpose_linear.h"
#include "linear_device.h"
#include "linear_kernels.h"

namespace xpose {
namespace {

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
template <typename T, Out OUT, typename Args>
__device__ inline void put_chunk(const Args &a, int64_t row, int64_t col, int valid, const float (&y)[8]) {
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

// A workgroup of 1024 for each of `count` things.  A launch can have no more than
// 2^32 - 1 threads in one dimension, so past 4 million workgroups they go on in
// the second; the last ones may have nothing to do.
constexpr int kLongThreads = 1024;
dim3 long_grid(int64_t count, uint32_t kinds = 1) {
  const int64_t most = kMaxThreads / kLongThreads, x = count < most ? count : most;
  return dim3((uint32_t)x, (uint32_t)((count + x - 1) / x), kinds);
}
__device__ inline int64_t long_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace
}  // namespace xpose
