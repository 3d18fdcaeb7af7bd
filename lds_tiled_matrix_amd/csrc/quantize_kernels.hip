// gfx950 kernels of block quantisation to e4m3 and of the clipping of many
// gradients by their global norm.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/linear/xpose_linear.h"
#include "linear_device.h"
#include "linear_kernels.h"

namespace xpose {
namespace {

// ----- quantisation ------------------------------------------------------------
//
// One workgroup takes a tile of 128 x 128, which holds whole blocks of the
// matrix and of its transpose: x is read once for both.  A lane holds 8 x 8
// values (rows 8 g .. 8 g + 7, columns 8 c .. 8 c + 7; 16 lanes cover a row,
// a wave 32 rows), so a row's block is a maximum over 16 lanes, a column's
// one over the 16 row groups (four in a wave, four waves through LDS), and
// either direction's bytes are eight of the lane's own.  Rows are stored from
// registers, 128 bytes a row; the transpose goes through LDS as bytes
// (16 KiB), in units of 8 rows whose place in a row of the transpose is
// swizzled by c: writes of 16 lanes (one g, all c) and 16-byte reads then
// both touch every bank once.
//
// Divisions are dear next to the rest (32 a lane made 40% of the instructions):
// each scale and its reciprocal are worked out once and handed round.
//
// 8192 x 8192 bfloat16 both ways takes 54 us (4.9 TB/s), 12345 x 6789 float32
// 90 us (5.6 TB/s); a copy of as many bytes, 43 and 80.
constexpr int kTile = 128;

template <typename T, int BLOCK_ROWS, bool POW2, bool BOTH>
__global__ __launch_bounds__(kQuantThreads) void quantize_kernel(QuantizeArgs a) {
  __shared__ uint32_t col_max[4][kTile];
  __shared__ __align__(16) uint8_t turned[BOTH ? kTile * kTile : 16];
  // of column 8 c + j at [j][c]: lanes next to each other read neighbours
  __shared__ Quotient<POW2> col_by[8][BOTH && BLOCK_ROWS == 1 ? 16 : 1];
  const int t = threadIdx.x, c = t % 16, g = t / 16, wave = t / 64;
  // Workgroups go to the 8 dies in turn: of every 64 tiles a die gets 8
  // neighbours of a row, which share lines where the pitch is odd, so that
  // they share a cache too.
  const uint32_t b = blockIdx.x, run = b / 64 * 64;
  const uint32_t tile = run + 64 <= gridDim.x ? run + b % 8 * 8 + b / 8 % 8 : b;
  const int64_t rb = tile / a.tiles_c, cb = tile % a.tiles_c;
  const int64_t r0 = rb * kTile, c0 = cb * kTile;
  const int64_t row = r0 + 8 * g, col = c0 + 8 * c;
  const int rows = (int)(a.rows - row < 0 ? 0 : a.rows - row > 8 ? 8 : a.rows - row);
  const int cols = (int)(a.cols - col < 0 ? 0 : a.cols - col > 8 ? 8 : a.cols - col);

  // as they are in memory, and widened at each use: with 16-bit values that
  // is 32 registers instead of 64, and twice the workgroups on a compute unit
  Vec8<T> x[8];
  const T *src = (const T *)a.x + row * a.ldx;
  if (r0 + kTile <= a.rows && c0 + kTile <= a.cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = load_raw8(src + i * a.ldx + col, 8);
  } else if (a.cols >= 8) {  // whole loads here too, all under way together
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = load_row8((const T *)a.x + (row + i < a.rows ? row + i : a.rows - 1) * a.ldx, a.cols, col);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      settle8<T>(x[i], a.cols, col);
      if (i >= rows) x[i] = Vec8<T>{};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = load_raw8(src + i * a.ldx + col, i < rows ? cols : 0);
  }

  uint32_t row_amax[8], tile_amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, magnitude(at8<T>(x[i], j)));
    row_amax[i] = m;
    tile_amax = max(tile_amax, m);
  }

  uint8_t *q = a.q + row * a.ldq + col;
  // Results go past the caches: 12345 x 6789 float32 takes 91 us so and 98 us
  // else, and a product right behind takes no longer (512 to 4096 rows).
  auto put8 = [](uint8_t *p, u32x2 w) { __builtin_nontemporal_store(w, reinterpret_cast<u32x2 *>(p)); };
  // The bytes of one row (or column) of the lane's values.
  auto put_row = [&](int i, const float (&f)[8]) {
    if (i >= rows || cols <= 0) return;
    const u32x2 w = {e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7])};
    uint8_t *p = q + i * a.ldq;
    if (cols == 8) {
      put8(p, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cols) p[j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
    }
  };
  auto put_turned = [&](int j, const float (&f)[8]) {
    const u32x2 w = {e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7])};
    const int unit = ((((g >> 1) ^ c) & 7) << 1) | ((g ^ (c >> 3)) & 1);
    *reinterpret_cast<u32x2 *>(turned + (8 * c + j) * kTile + unit * 8) = w;
  };

  if constexpr (BLOCK_ROWS == 128) {
    uint32_t m = max16(tile_amax);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (t % 64 == 0) col_max[wave][0] = m;
    __syncthreads();
    m = max(max(col_max[0][0], col_max[1][0]), max(col_max[2][0], col_max[3][0]));
    const float scale = scale_of<POW2>(m);
    if (t == 0) {
      a.scale[cb * a.ld_scale + rb] = scale;
      if (BOTH) a.scale_t[rb * a.ld_scale_t + cb] = scale;
    }
    const Quotient<POW2> by(scale, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = by(at8<T>(x[i], j));
      put_row(i, f);
    }
    if constexpr (BOTH) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = by(at8<T>(x[i], j));
        put_turned(j, f);
      }
    }
  } else {
    if constexpr (BOTH) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, magnitude(at8<T>(x[i], j)));
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (t % 64 < 16) col_max[wave][8 * c + j] = m;
      }
    }
    // Lane c < 8 of a row group works out the scale of its row c, for all 16.
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = max16(row_amax[i]);
      if (c % 8 == i) mine = m;
    }
    const float scale = scale_of<POW2>(mine);
    if (c < rows) a.scale[cb * a.ld_scale + row + c] = scale;
    const Quotient<POW2> by(scale, mine);
    unrolled<8>([&](auto i) {
      const Quotient<POW2> of = by.template from<i>();
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = of(at8<T>(x[i], j));
      put_row(i, f);
    });
    if constexpr (BOTH) {
      // and thread t < 128 that of column t
      __syncthreads();
      if (t < kTile) {
        const uint32_t m = max(max(col_max[0][t], col_max[1][t]), max(col_max[2][t], col_max[3][t]));
        const float scale = scale_of<POW2>(m);
        if (c0 + t < a.cols) a.scale_t[rb * a.ld_scale_t + c0 + t] = scale;
        col_by[t % 8][t / 8] = Quotient<POW2>(scale, m);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Quotient<POW2> of = col_by[j][c];
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = of(at8<T>(x[i], j));
        put_turned(j, f);
      }
    }
  }

  if constexpr (BOTH) {
    __syncthreads();
    // 8 lanes a row of the transpose, 16 bytes (two units) each
    const int p = t % 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 32 * i + t / 8;
      const int unit = p ^ ((at >> 3) & 7);
      u32x4 w = *reinterpret_cast<const u32x4 *>(turned + at * kTile + unit * 16);
      if (at >= 64) w = {w[2], w[3], w[0], w[1]};
      const int64_t qrow = c0 + at, qcol = r0 + 16 * p;
      if (qrow >= a.cols || qcol >= a.rows) continue;
      uint8_t *dst = a.qt + qrow * a.ldqt + qcol;
      if (qcol + 16 <= a.rows) {
        // rows of the transpose start at multiples of 8
        put8(dst, u32x2{w[0], w[1]});
        put8(dst + 8, u32x2{w[2], w[3]});
      } else {
        const int n = (int)(a.rows - qcol);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < n) dst[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
      }
    }
  }
}

template <typename T, int BLOCK_ROWS, bool POW2, bool BOTH>
hipError_t quantize(const QuantizeArgs &a, hipStream_t s) {
  QuantizeArgs copy = a;
  void *args[] = {&copy};
  return hipLaunchKernel(
      reinterpret_cast<const void *>(&quantize_kernel<T, BLOCK_ROWS, POW2, BOTH>),
      dim3(a.tiles_r * a.tiles_c), dim3(kQuantThreads), args, 0, s);
}
template <typename T, int BLOCK_ROWS>
hipError_t quantize(const QuantizeArgs &a, bool pow2, hipStream_t s) {
  if (pow2)
    return a.qt ? quantize<T, BLOCK_ROWS, true, true>(a, s)
                : quantize<T, BLOCK_ROWS, true, false>(a, s);
  return a.qt ? quantize<T, BLOCK_ROWS, false, true>(a, s)
              : quantize<T, BLOCK_ROWS, false, false>(a, s);
}
template <typename T>
hipError_t quantize(const QuantizeArgs &a, int block_rows, bool pow2, hipStream_t s) {
  return block_rows == 1 ? quantize<T, 1>(a, pow2, s) : quantize<T, 128>(a, pow2, s);
}

// ----- clipping ------------------------------------------------------------------
//
// Two launches: every workgroup sums the squares of its chunks into one
// number, then every workgroup adds up all of those in the same order (16 KiB
// from the L2 cache) and scales its chunks.  Squares and sums are of 64 bits:
// no square overflows, and the sum of 10^9 gradients loses nothing; their
// cost hides behind the loads.  The second launch walks backwards, so that it
// begins with what the first one left in the caches, and stores past them, so
// that this stays there (32 layers' gradients, 760 MB in bfloat16: 383 us
// without, 348 us with).
//
// Those gradients take 112 us to sum (6.0 TB/s) and 234 us to scale (5.7 TB/s).
constexpr int kClipThreads = 256;

struct Span {
  int tensor;
  int64_t begin, count;
};

__device__ inline Span chunk_span(const ClipArgs &a, uint32_t chunk) {
  int lo = 0, hi = a.tensors - 1;  // the first tensor whose chunks end after it
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.end[mid] > chunk) hi = mid; else lo = mid + 1;
  }
  const uint32_t first = lo ? a.end[lo - 1] : 0;
  const int64_t begin = (int64_t)(chunk - first) * kClipChunk;
  const int64_t rest = a.count[lo] - begin;
  return {lo, begin, rest < kClipChunk ? rest : kClipChunk};
}

__device__ inline double sum256(double x, double *lds) {
#pragma unroll
  for (int d = 32; d; d /= 2) x += __shfl_xor(x, d);
  __syncthreads();
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

template <typename T>
__device__ inline double squares(const T *p, int64_t count) {
  double s = 0;
  for (int64_t i = threadIdx.x * 8; i < count; i += kClipThreads * 8) {
    float f[8];
    load8(p + i, count - i < 8 ? (int)(count - i) : 8, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fma((double)f[e], (double)f[e], s);
  }
  return s;
}

__global__ __launch_bounds__(kClipThreads) void clip_squares_kernel(ClipArgs a) {
  __shared__ double lds[4];
  double s = 0;
  for (uint32_t chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    const Span p = chunk_span(a, chunk);
    const void *in = a.in[p.tensor];
    if (a.dtype[p.tensor] == XPOSE_F32)
      s += squares((const float *)in + p.begin, p.count);
    else if (a.dtype[p.tensor] == XPOSE_F16)
      s += squares((const _Float16 *)in + p.begin, p.count);
    else
      s += squares((const __bf16 *)in + p.begin, p.count);
  }
  s = sum256(s, lds);
  if (threadIdx.x == 0) a.partial[a.first + blockIdx.x] = s;
}

template <typename T>
__device__ inline void scale_span(const T *in, T *out, int64_t count, float factor) {
  for (int64_t i = threadIdx.x * 8; i < count; i += kClipThreads * 8) {
    const int valid = count - i < 8 ? (int)(count - i) : 8;
    float f[8];
    load8(in + i, valid, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= factor;
    store8_past(out + i, valid, f);
  }
}

__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipArgs a) {
  __shared__ double lds[4];
  double s = 0;
  for (int i = threadIdx.x; i < a.partials; i += kClipThreads) s += a.partial[i];
  const double norm = sqrt(sum256(s, lds));
  double factor = a.max_norm / (norm + a.eps);
  if (factor > 1.0) factor = 1.0;  // a NaN stays
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  for (uint32_t i = blockIdx.x; i < a.chunks; i += gridDim.x) {
    const Span p = chunk_span(a, a.chunks - 1 - i);
    const void *in = a.in[p.tensor];
    void *out = a.out[p.tensor];
    if (a.dtype[p.tensor] == XPOSE_F32)
      scale_span((const float *)in + p.begin, (float *)out + p.begin, p.count, (float)factor);
    else if (a.dtype[p.tensor] == XPOSE_F16)
      scale_span((const _Float16 *)in + p.begin, (_Float16 *)out + p.begin, p.count, (float)factor);
    else
      scale_span((const __bf16 *)in + p.begin, (__bf16 *)out + p.begin, p.count, (float)factor);
  }
}

hipError_t launch_clip(const void *kernel, const ClipArgs &a, uint32_t groups, hipStream_t s) {
  ClipArgs copy = a;
  void *args[] = {&copy};
  return hipLaunchKernel(kernel, dim3(groups), dim3(kClipThreads), args, 0, s);
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs &a, int dtype, int block_rows,
                           bool pow2, hipStream_t s) {
  if (dtype == XPOSE_F32) return quantize<float>(a, block_rows, pow2, s);
  if (dtype == XPOSE_F16) return quantize<_Float16>(a, block_rows, pow2, s);
  return quantize<__bf16>(a, block_rows, pow2, s);
}

hipError_t launch_clip_squares(const ClipArgs &a, uint32_t groups, hipStream_t s) {
  return launch_clip(reinterpret_cast<const void *>(&clip_squares_kernel), a, groups, s);
}
hipError_t launch_clip_scale(const ClipArgs &a, uint32_t groups, hipStream_t s) {
  return launch_clip(reinterpret_cast<const void *>(&clip_scale_kernel), a, groups, s);
}

}  // namespace xpose
