// gfx950 kernels of low-rank adapters beside a shared projection, forward and
// backward, and of dropout from a counter-based generator.
//
// A row of x has the adapter ids[row], (A, B) of rank r:
//
//   hidden = x A^T                      "shrink": k columns to r
//   out    = base + alpha scale hidden B^T        "expand": r columns to n
//
// and, with dh = alpha scale dout B (another shrink, over n) in the backward
// pass, dx = base + dh A (another expand), dA = sum dh^T x and dB = sum alpha
// scale dout^T hidden over an adapter's rows.
//
// Whose rows.  A workgroup has a tile of rows and takes the adapters that they
// have one after the other, in the order of their first rows: no sorting, no
// host that waits for ids, and any mixture is right.  Few rows with an adapter
// each (tokens being generated) would take 16 turns of a memory latency so;
// there a tile's adapters are dealt out to `slots` workgroups.  A row of another
// adapter, or of none, is computed and not stored: what its numbers are does
// not reach the others, as rows are columns of the matrix instructions.
//
// Rows with an id out of 0 .. count - 1 have no adapter.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/linear/xpose_block.h"
#include "block_kernels.h"
#include "linear_device.h"
#include "linear_kernels.h"

namespace xpose {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;  // columns that share a scale of e4m3 x

__device__ inline int valid8(int64_t left) { return left < 0 ? 0 : left > 8 ? 8 : (int)left; }

// Eight elements from `col` on of a row of `len`: zeros beyond it.
template <typename T>
__device__ inline Vec8<T> guarded8(const T *row, int64_t len, int64_t col) {
  if (len < 8) return load_raw8(row + col, valid8(len - col));
  Vec8<T> v = load_row8(row, len, col);
  settle8<T>(v, len, col);
  return v;
}

// sum[i][j] += sum over the lanes' eight values of w[i] x[j]: lane l has row
// l % 16 of both operands, and lanes of one l / 16 the same eight of 32 columns.
template <typename T> __device__ inline f32x4 multiply8(const Vec8<T> &w, const Vec8<T> &x, f32x4 sum);
template <> __device__ inline f32x4 multiply8<__bf16>(const Vec8<__bf16> &w, const Vec8<__bf16> &x, f32x4 sum) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16((bf16x8)w.v, (bf16x8)x.v, sum, 0, 0, 0);
}
template <>
__device__ inline f32x4 multiply8<_Float16>(const Vec8<_Float16> &w, const Vec8<_Float16> &x, f32x4 sum) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16((f16x8)w.v, (f16x8)x.v, sum, 0, 0, 0);
}
template <> __device__ inline f32x4 multiply8<float>(const Vec8<float> &w, const Vec8<float> &x, f32x4 sum) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    sum = __builtin_amdgcn_mfma_f32_16x16x4f32(w.v[e / 4][e % 4], x.v[e / 4][e % 4], sum, 0, 0, 0);
  return sum;
}

// Eight e4m3 values (two words) in a type that holds each of them.
template <typename T>
__device__ inline Vec8<T> widen8(uint32_t lo, uint32_t hi) {
  Vec8<T> r;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t b = w ? hi : lo;
    if constexpr (sizeof(T) == 4) {
      const f32x2 p = __builtin_amdgcn_cvt_pk_f32_fp8((int)b, false), q = __builtin_amdgcn_cvt_pk_f32_fp8((int)b, true);
      r.v[w] = f32x4_any{p[0], p[1], q[0], q[1]};
    } else if constexpr (std::is_same_v<T, _Float16>) {
      const f16x2 p = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false);
      const f16x2 q = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true);
      r.v[4 * w] = p[0], r.v[4 * w + 1] = p[1], r.v[4 * w + 2] = q[0], r.v[4 * w + 3] = q[1];
    } else {
      const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false);
      const bf16x2 q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
      r.v[4 * w] = p[0], r.v[4 * w + 1] = p[1], r.v[4 * w + 2] = q[0], r.v[4 * w + 3] = q[1];
    }
  }
  return r;
}

// The adapter of row t0 + lane in the lanes below ROWS, -1 for none and -2 for no row.
template <int ROWS>
__device__ inline int tile_ids(const int32_t *ids, int64_t m, int count, int64_t t0, int lane) {
  const int64_t row = t0 + lane;
  if (lane >= ROWS || row >= m) return -2;
  const int id = ids[row];
  return (uint32_t)id < (uint32_t)count ? id : -1;
}

// f(adapter, lanes whose rows have it) for every adapter of a tile that falls
// to this slot; the same in all waves of a workgroup.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int slot, int slots, F &&f) {
  uint64_t rest = __ballot(id >= 0);
  for (int j = 0; rest; ++j) {
    const int d = __builtin_amdgcn_readlane(id, __builtin_ctzll(rest));
    const uint64_t match = __ballot(id == d);
    rest &= ~match;
    if ((j & (slots - 1)) == slot) f(d, match);
  }
}

// ----- shrink -----------------------------------------------------------------------
//
// h = x w^T: the rows of w (the rank) are the instruction's first operand, the
// rows of x its second, so a lane's results are four ranks of one row.  The
// four waves of a workgroup share out its columns in blocks of 128 and add
// their sums up at the end; a lane takes chunks of 8 columns at 64 (s / 2) + 16
// (l / 16) + 8 (s % 2), which in e4m3 are 16 bytes for two of them.
constexpr int kShrinkWaves = 4, kShrinkThreads = 64 * kShrinkWaves;

template <typename T, bool Q, int NI, int NR>
__global__ __launch_bounds__(kShrinkThreads) void shrink_kernel(ShrinkArgs a) {
  constexpr int ROWS = 16 * NI;
  __shared__ f32x4 lds[kShrinkWaves][NI * NR][64];
  const int tid = threadIdx.x, lane = tid % 64, i16 = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t t0 = (int64_t)blockIdx.x * ROWS;
  const int slice = blockIdx.y / a.slots, slot = blockIdx.y % a.slots;
  const int r0 = blockIdx.z * 16 * NR;
  const int id = tile_ids<ROWS>(a.ids, a.m, a.count, t0, lane);
  float *h = a.h + slice * a.slice;
  if (slot == 0) {
    uint64_t none = __ballot(id == -1);
    if (none)
      for (int i = tid; i < ROWS * 16 * NR; i += kShrinkThreads) {
        const int row = i / (16 * NR), r = r0 + i % (16 * NR);
        if ((none >> row & 1) && r < a.rank) h[(t0 + row) * a.rank + r] = 0.f;
      }
  }
  const int64_t blocks = (a.k + kBlock - 1) / kBlock, whole = a.k / kBlock;
  const int64_t first = (int64_t)slice * a.blocks_per_slice;
  const int64_t last = min(first + a.blocks_per_slice, blocks);
  int64_t row[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) row[i] = min(t0 + 16 * i + i16, a.m - 1);

  each_adapter(id, slot, a.slots, [&](int d, uint64_t match) {
    f32x4 sum[NI][NR];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < NR; ++q) sum[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    const T *w0 = (const T *)a.w + d * a.stride_w;
    const T *w[NR];
#pragma unroll
    for (int q = 0; q < NR; ++q) w[q] = w0 + min(r0 + 16 * q + i16, a.rank - 1) * a.ldw;

    auto block = [&](int64_t kb, auto ragged) {
      constexpr bool RAGGED = decltype(ragged)::value;
      const int64_t c0 = kb * kBlock + 16 * g;
      Vec8<T> wv[NR][4];
      auto load_w = [&](int s) {
        const int64_t c = c0 + 64 * (s / 2) + 8 * (s % 2);
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          if constexpr (RAGGED) wv[q][s] = guarded8(w[q], a.k, c);
          else wv[q][s] = load_raw8(w[q] + c, 8);
        }
      };
      if constexpr (Q) {
        u32x4 xq[NI][2];
        float scale[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint8_t *x = (const uint8_t *)a.x + row[i] * a.ldx;
          scale[i] = a.scale_x[kb * a.ld_scale_x + row[i]];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int64_t col = c0 + 64 * c;
            if constexpr (RAGGED) {  // the 16 bytes that hold a row's end are all there
              const int64_t left = a.k - col;
              xq[i][c] = *reinterpret_cast<const u32x4 *>(x + (left > 0 ? col : 0));
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const int64_t in = left - 4 * b;
                xq[i][c][b] &= in >= 4 ? ~0u : in <= 0 ? 0u : (1u << (8 * (int)in)) - 1;
              }
            } else {
              xq[i][c] = *reinterpret_cast<const u32x4 *>(x + col);
            }
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) load_w(s);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          f32x4 part[NR];
#pragma unroll
          for (int q = 0; q < NR; ++q) part[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const Vec8<T> x = widen8<T>(xq[i][s / 2][s % 2 * 2], xq[i][s / 2][s % 2 * 2 + 1]);
#pragma unroll
            for (int q = 0; q < NR; ++q) part[q] = multiply8<T>(wv[q][s], x, part[q]);
          }
#pragma unroll
          for (int q = 0; q < NR; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[i][q][e] = __builtin_fmaf(part[q][e], scale[i], sum[i][q][e]);
        }
      } else {
        Vec8<T> xv[NI][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int64_t c = c0 + 64 * (s / 2) + 8 * (s % 2);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const T *x = (const T *)a.x + row[i] * a.ldx;
            if constexpr (RAGGED) xv[i][s] = guarded8(x, a.k, c);
            else xv[i][s] = load_raw8(x + c, 8);
          }
          load_w(s);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int q = 0; q < NR; ++q) sum[i][q] = multiply8<T>(wv[q][s], xv[i][s], sum[i][q]);
      }
    };
    int64_t kb = first + wave;
    for (; kb < min(last, whole); kb += kShrinkWaves) block(kb, std::false_type{});
    if (kb < last) block(kb, std::true_type{});

#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < NR; ++q) lds[wave][i * NR + q][lane] = sum[i][q];
    __syncthreads();
    const float factor = a.scaled ? a.alpha * (a.scale ? a.scale[d] : 1.f) : 1.f;
    for (int f = wave; f < NI * NR; f += kShrinkWaves) {
      f32x4 v = lds[0][f][lane];
#pragma unroll
      for (int o = 1; o < kShrinkWaves; ++o) v += lds[o][f][lane];
      const int in = f / NR * 16 + i16, r = r0 + f % NR * 16 + 4 * g;
      if (!(match >> in & 1)) continue;
      float *to = h + (t0 + in) * a.rank + r;
      v *= factor;
      if (r + 4 <= a.rank) {
        *reinterpret_cast<f32x4_any *>(to) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e < a.rank) to[e] = v[e];
      }
    }
    __syncthreads();  // before the next adapter's sums
  });
}

constexpr int kSlicesThreads = 256;
__global__ __launch_bounds__(kSlicesThreads) void slices_kernel(SlicesArgs a) {
  for (int64_t i = (int64_t)blockIdx.x * kSlicesThreads + threadIdx.x; i < a.count;
       i += (int64_t)gridDim.x * kSlicesThreads) {
    float s = a.in[i];
    for (int p = 1; p < a.slices; ++p) s += a.in[p * a.count + i];
    a.out[i] = s;
  }
}

// ----- expand ------------------------------------------------------------------------
//
// out = base + h w^T, the rows of w (columns of out) as the first operand: a
// lane's results lie in one row of out.  Which of the 32 columns of two
// instructions is which of their rows is chosen so that a lane has eight
// neighbours of them, and four lanes 32.
//
// h is float32 and stays it: for 16-bit weights it goes to the matrix cores as
// the sum of three bfloat16 numbers (24 bits; they have float32's range, which
// float16 has not), float16 weights as the sum of two.  Next to reading base
// and writing out, the products are free.
constexpr int kExpandThreads = 256, kExpandCols = 256;  // of a workgroup; 64 a wave

// Eight float32 numbers as operands of multiply_split.
template <typename T> struct Split8 {
  bf16x8 part[3];
  __device__ void set(const float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float rest = f[e];
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const __bf16 b = (__bf16)rest;
        part[p][e] = b;
        rest -= (float)b;
        // an infinity is one, and not one less itself
        if (!(__builtin_fabsf((float)b) < __builtin_inff())) rest = 0.f;
      }
    }
  }
};
template <> struct Split8<float> {
  float v[8];
  __device__ void set(const float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f[e];
  }
};
template <typename T> __device__ inline f32x4 multiply_split(const Vec8<T> &w, const Split8<T> &h, f32x4 sum);
template <>
__device__ inline f32x4 multiply_split<__bf16>(const Vec8<__bf16> &w, const Split8<__bf16> &h, f32x4 sum) {
#pragma unroll
  for (int p = 2; p >= 0; --p) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16((bf16x8)w.v, h.part[p], sum, 0, 0, 0);
  return sum;
}
template <>
__device__ inline f32x4 multiply_split<_Float16>(const Vec8<_Float16> &w, const Split8<_Float16> &h, f32x4 sum) {
  bf16x8 hi, lo;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float f = (float)w.v[e];
    hi[e] = (__bf16)f;
    lo[e] = (__bf16)(__builtin_fabsf(f) < __builtin_inff() ? f - (float)hi[e] : 0.f);
  }
#pragma unroll
  for (int p = 1; p >= 0; --p) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, h.part[p], sum, 0, 0, 0);
#pragma unroll
  for (int p = 2; p >= 0; --p) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, h.part[p], sum, 0, 0, 0);
  return sum;
}
template <> __device__ inline f32x4 multiply_split<float>(const Vec8<float> &w, const Split8<float> &h, f32x4 sum) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    sum = __builtin_amdgcn_mfma_f32_16x16x4f32(w.v[e / 4][e % 4], h.v[e], sum, 0, 0, 0);
  return sum;
}

template <typename T, typename O, int NI>
__global__ __launch_bounds__(kExpandThreads) void expand_kernel(ExpandArgs a) {
  constexpr int ROWS = 16 * NI;
  const int tid = threadIdx.x, lane = tid % 64, i16 = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t col_tiles = (a.n + kExpandCols - 1) / kExpandCols;
  const int slot = blockIdx.x % a.slots;
  const int64_t tile = blockIdx.x / a.slots;
  const int64_t t0 = tile / col_tiles * ROWS, n0 = tile % col_tiles * kExpandCols + wave * 64;
  const int id = tile_ids<ROWS>(a.ids, a.m, a.count, t0, lane);
  if (n0 >= a.n) return;

  // the 64 columns of this wave, those rows of `match`
  auto store = [&](uint64_t match, const f32x4 (&sum)[NI][4], bool add) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (!(match >> (16 * i + i16) & 1)) continue;
      const int64_t row = t0 + 16 * i + i16;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int64_t col = n0 + 32 * p + 8 * g;
        const int valid = valid8(a.n - col);
        float f[8] = {};
        if (a.base) load8((const O *)a.base + row * a.ld_base + col, valid, f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (add) f[e] += sum[i][2 * p + e / 4][e % 4];
        store8((O *)a.out + row * a.ld_out + col, valid, f);
      }
    }
  };

  if (slot == 0 && a.base != a.out) {  // rows without an adapter
    const uint64_t none = __ballot(id == -1);
    f32x4 zero[NI][4];
    if (none) store(none, zero, false);
  }
  each_adapter(id, slot, a.slots, [&](int d, uint64_t match) {
    const T *w0 = (const T *)a.w + d * a.stride_w;
    const float factor = a.alpha * (a.scale ? a.scale[d] : 1.f);
    f32x4 sum[NI][4];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int p = 0; p < 4; ++p) sum[i][p] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < a.rank; c += 32) {
      const int r = c + 8 * g, valid = valid8(a.rank - r);
      Vec8<T> w[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int64_t col = n0 + 32 * (p / 2) + 8 * (i16 / 4) + 4 * (p % 2) + i16 % 4;
        w[p] = load_raw8(w0 + min(col, a.n - 1) * a.ldw + r, valid);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float *h = a.h + min(t0 + 16 * i + i16, a.m - 1) * a.rank + r;
        float f[8];
        load8(h, valid, f);
        for (int s = 1; s < a.slices; ++s) {
          float more[8];
          load8(h + s * a.slice, valid, more);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] += more[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= factor;
        Split8<T> hs;
        hs.set(f);
#pragma unroll
        for (int p = 0; p < 4; ++p) sum[i][p] = multiply_split<T>(w[p], hs, sum[i][p]);
      }
    }
    store(match, sum, true);
  });
}

// ----- what the backward pass lays out first -------------------------------------------
//
// One launch: the first `count` workgroups find an adapter's rows each, all
// others transpose 256 columns (of A) or rows (of B) of an adapter's weights.
// An adapter's rows follow those of all adapters before it, so its workgroup
// counts those too; ids are read by each of them, from the caches.
constexpr int kPrepThreads = 256, kPrepRanks = 32;

template <typename T>
__global__ __launch_bounds__(kPrepThreads) void adapter_prep_kernel(AdapterPrepArgs a) {
  __shared__ T tile[kPrepThreads][kPrepRanks + 1];
  __shared__ int32_t waves[2][kPrepThreads / 64];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  int64_t block = blockIdx.x;
  if (a.order) {
    if (block < a.count) {
      const int l = (int)block;
      int before = 0;
      for (int64_t i = tid; i < a.m; i += kPrepThreads) before += (uint32_t)a.ids[i] < (uint32_t)l;
#pragma unroll
      for (int d = 32; d; d /= 2) before += __shfl_xor(before, d);
      if (lane == 0) waves[0][wave] = before;
      __syncthreads();
      int at = 0;
#pragma unroll
      for (int w = 0; w < kPrepThreads / 64; ++w) at += waves[0][w];
      if (tid == 0) a.starts[l] = at;
      for (int64_t i0 = 0; i0 < a.m; i0 += kPrepThreads) {
        const int64_t i = i0 + tid;
        const bool mine = i < a.m && a.ids[i] == l;
        const uint64_t in_wave = __ballot(mine);
        __syncthreads();
        if (lane == 0) waves[1][wave] = __popcll(in_wave);
        __syncthreads();
        int place = at + __popcll(in_wave & ((1ull << lane) - 1));
#pragma unroll
        for (int w = 0; w < kPrepThreads / 64; ++w) {
          if (w < wave) place += waves[1][w];
          at += waves[1][w];
        }
        if (mine) a.order[place] = (int32_t)i;
      }
      if (tid == 0 && l == a.count - 1) a.starts[a.count] = at;
      return;
    }
    block -= a.count;
  }
  const int64_t tiles_a = a.at ? (a.k + kPrepThreads - 1) / kPrepThreads * a.count : 0;
  const bool of_b = block >= tiles_a;
  if (of_b) block -= tiles_a;
  const int64_t len = of_b ? a.n : a.k, tiles = (len + kPrepThreads - 1) / kPrepThreads;
  const int64_t l = block / tiles, c0 = block % tiles * kPrepThreads;
  const int cols = (int)min(len - c0, (int64_t)kPrepThreads);
  for (int r0 = 0; r0 < a.rank; r0 += kPrepRanks) {
    const int ranks = min(a.rank - r0, kPrepRanks);
    __syncthreads();
    if (of_b) {
      const T *b = (const T *)a.b + l * a.stride_b + c0 * a.ldb + r0;
      for (int i = tid; i < cols * ranks; i += kPrepThreads) tile[i / ranks][i % ranks] = b[i / ranks * a.ldb + i % ranks];
    } else {
      const T *w = (const T *)a.a + l * a.stride_a + (int64_t)r0 * a.lda + c0;
      if (tid < cols)
        for (int r = 0; r < ranks; ++r) tile[tid][r] = w[r * a.lda + tid];
    }
    __syncthreads();
    if (of_b) {
      T *to = (T *)a.bt + (l * a.rank + r0) * a.n + c0;
      if (tid < cols)
        for (int r = 0; r < ranks; ++r) to[r * a.n + tid] = tile[tid][r];
    } else {
      T *to = (T *)a.at + (l * a.k + c0) * a.rank + r0;
      for (int i = tid; i < cols * ranks; i += kPrepThreads)
        to[(int64_t)(i / ranks) * a.rank + i % ranks] = tile[i / ranks][i % ranks];
    }
  }
}

// ----- the adapters' gradients ----------------------------------------------------------
//
// G[r][c] = sum over rows u[row][r] v[row][c], u of r columns in float32, v as
// it is: on the float32 matrix cores, whose operands need no turning around,
// as a lane has one rank or eight neighbouring columns of one row in four.
//
// An adapter's rows are cut into pieces, a workgroup for 128 columns of each.
// An adapter of one piece is done with that; the pieces of larger ones go to
// the workspace and a second launch adds them up, in their order.  Adapter l's
// pieces are the numbers starts[l] / piece + l and on: there are enough
// numbers between one adapter's first and the next one's.  Workspace slots,
// which only adapters of over a piece need, are 2 (starts[l] / piece) and on.
constexpr int kGradThreads = 256, kGradCols = 128, kGradWaves = 4;

__device__ inline int grad_pieces(int rows, int piece) { return (rows + piece - 1) / piece; }

template <typename T, int NR>
__global__ __launch_bounds__(kGradThreads) void adapter_grad_kernel(AdapterGradArgs a, int64_t tiles_k, int64_t tiles) {
  __shared__ f32x4 lds[NR][8][64];
  const int tid = threadIdx.x, lane = tid % 64, i16 = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t number = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int r0 = blockIdx.y * 16 * NR;
  int lo = 0, hi = a.count - 1;  // the last adapter whose first number is no later
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.starts[mid] / a.piece + mid <= number) lo = mid; else hi = mid - 1;
  }
  const int l = __builtin_amdgcn_readfirstlane(lo);
  const int start = a.starts[l], rows = a.starts[l + 1] - start;
  const int j = (int)(number - (start / a.piece + l));
  const int pieces = grad_pieces(rows, a.piece);
  if (j >= pieces) return;
  const int begin = start + j * a.piece, end = min(begin + a.piece, start + rows);

  const bool of_b = tile >= tiles_k;
  const int64_t cols = of_b ? a.n : a.k, c0 = (of_b ? tile - tiles_k : tile) * kGradCols;
  const T *v = (const T *)(of_b ? a.dout : a.x);
  const int64_t ldv = of_b ? a.lddout : a.ldx;
  const float *u = of_b ? a.h : a.dh;
  const float factor = of_b ? a.alpha * (a.scale ? a.scale[l] : 1.f) : 1.f;
  const int64_t col = c0 + 8 * i16;

  f32x4 sum[NR][8];
#pragma unroll
  for (int q = 0; q < NR; ++q)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[q][e] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int p0 = begin + 16 * wave; p0 < end; p0 += 16 * kGradWaves) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int at = p0 + 4 * s + g;
      const bool in = at < end;
      const int64_t row = a.order[in ? at : end - 1];
      const Vec8<T> vv = cols < 8 ? load_raw8(v + row * ldv + col, valid8(cols - col)) : load_row8(v + row * ldv, cols, col);
      float uu[NR];
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        const int r = r0 + 16 * q + i16;
        uu[q] = u[row * a.rank + min(r, a.rank - 1)];
        if (!in) uu[q] = 0.f;
      }
      Vec8<T> settled = vv;
      if (cols >= 8) settle8<T>(settled, cols, col);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = in ? at8<T>(settled, e) : 0.f;
#pragma unroll
        for (int q = 0; q < NR; ++q) sum[q][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(uu[q], f, sum[q][e], 0, 0, 0);
      }
    }
  }
  // the waves' sums, one after the other
  for (int w = 0; w < kGradWaves; ++w) {
    if (w == wave) {
#pragma unroll
      for (int q = 0; q < NR; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) lds[q][e][lane] = w == 0 ? sum[q][e] : lds[q][e][lane] + sum[q][e];
    }
    __syncthreads();
  }
  // lds[q][e][lane] has columns 8 (lane % 16) + e, ranks 16 q + 4 (lane / 16) and on
  const float *flat = (const float *)lds;
  auto value = [&](int r, int c) {
    return flat[(((r / 16) * 8 + c % 8) * 64 + r % 16 / 4 * 16 + c / 8) * 4 + r % 4] * factor;
  };
  const int ranks = min(a.rank - r0, 16 * NR), here = (int)min(cols - c0, (int64_t)kGradCols);
  const int64_t slot = 2 * (int64_t)(start / a.piece) + j, each = (int64_t)a.rank * (a.k + a.n);
  const bool done = pieces == 1;
  if (of_b) {
    float *to = done ? a.db + (int64_t)l * a.n * a.rank : a.partial + slot * each + (int64_t)a.rank * a.k;
    for (int i = tid; i < ranks * here; i += kGradThreads)
      to[(c0 + i / ranks) * a.rank + r0 + i % ranks] = value(i % ranks, i / ranks);
  } else {
    float *to = done ? a.da + (int64_t)l * a.rank * a.k : a.partial + slot * each;
    for (int i = tid; i < ranks * kGradCols; i += kGradThreads) {
      const int r = i / kGradCols, c = i % kGradCols;
      if (c < here) to[(int64_t)(r0 + r) * a.k + c0 + c] = value(r, c);
    }
  }
}

// Adapters of no rows get zeros, those of several pieces their sum.
__global__ __launch_bounds__(kGradThreads) void adapter_grad_sum_kernel(AdapterGradArgs a, int64_t groups) {
  const int l = (int)(blockIdx.x / groups);
  const int start = a.starts[l], pieces = grad_pieces(a.starts[l + 1] - start, a.piece);
  if (pieces == 1) return;
  const int64_t of_a = (int64_t)a.rank * a.k, each = of_a + (int64_t)a.rank * a.n;
  const float *p = a.partial + 2 * (int64_t)(start / a.piece) * each;
  for (int64_t i = (int64_t)(blockIdx.x % groups) * kGradThreads + threadIdx.x; i < each; i += groups * kGradThreads) {
    float *to = i < of_a ? (a.da ? a.da + l * of_a + i : nullptr)
                         : (a.db ? a.db + l * (each - of_a) + (i - of_a) : nullptr);
    if (!to) continue;
    float s = 0.f;
    for (int j = 0; j < pieces; ++j) s += p[j * each + i];
    *to = s;
  }
}

// ----- dropout ---------------------------------------------------------------------------
//
// A lane has eight neighbouring columns of a row and takes their 16 bits each
// from one Philox4x32-10 block (Salmon, Moraes, Dror and Shaw, 2011), whose
// counter is the chunk's place: nothing is stored, and the backward pass, which
// is the same call on the gradient, gets the same mask whatever the type,
// strides and launch.
constexpr int kDropThreads = 256;

struct Philox {
  uint32_t w[4];
  __device__ Philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) : w{c0, c1, c2, c3} {
#pragma unroll
    for (int round = 0; round < 10; ++round) {
      const uint64_t p = (uint64_t)w[0] * 0xD2511F53u, q = (uint64_t)w[2] * 0xCD9E8D57u;
      w[0] = (uint32_t)(q >> 32) ^ w[1] ^ (k0 + (uint32_t)round * 0x9E3779B9u);
      w[1] = (uint32_t)q;
      w[2] = (uint32_t)(p >> 32) ^ w[3] ^ (k1 + (uint32_t)round * 0xBB67AE85u);
      w[3] = (uint32_t)p;
    }
  }
  __device__ uint32_t bits(int e) const { return w[e / 2] >> (16 * (e % 2)) & 0xffffu; }
};

template <typename T, bool RES>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(DropoutArgs a) {
  const int lane = threadIdx.x & (a.lanes - 1), rows_at_once = kDropThreads / a.lanes;
  const int64_t chunk = (int64_t)blockIdx.x * a.lanes + lane, col = chunk * 8;
  if (col >= a.cols) return;
  const uint64_t seed = a.device_seed ? *a.device_seed : a.seed;
  const int valid = valid8(a.cols - col);
  const int64_t step = (int64_t)gridDim.y * rows_at_once;
  for (int64_t row = (int64_t)blockIdx.y * rows_at_once + threadIdx.x / a.lanes; row < a.rows; row += step) {
    float x[8], y[8], r[8];
    load8((const T *)a.x + row * a.ldx + col, valid, x);
    if constexpr (RES) load8((const T *)a.residual + row * a.ldr + col, valid, r);
    const Philox random((uint32_t)chunk, (uint32_t)row, (uint32_t)a.offset, (uint32_t)(a.offset >> 32), (uint32_t)seed,
                        (uint32_t)(seed >> 32));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = random.bits(e) >= a.threshold ? x[e] * a.factor : 0.f;
      if constexpr (RES) y[e] += r[e];
    }
    store8((T *)a.y + row * a.ldy + col, valid, y);
  }
}

template <typename Args, typename... More>
hipError_t launch(const void *kernel, dim3 grid, int threads, hipStream_t s, const Args &a, More... more) {
  Args copy = a;
  void *args[] = {&copy, &more...};
  return hipLaunchKernel(kernel, grid, dim3(threads), args, 0, s);
}

template <typename T, bool Q, int NI>
hipError_t shrink(const ShrinkArgs &a, dim3 grid, hipStream_t s) {
  if (a.rank <= 16) {
    return launch(reinterpret_cast<const void *>(&shrink_kernel<T, Q, NI, 1>), grid, kShrinkThreads, s, a);
  }
  if (a.rank <= 32) return launch(reinterpret_cast<const void *>(&shrink_kernel<T, Q, NI, 2>), grid, kShrinkThreads, s, a);
  grid.z = (uint32_t)((a.rank + 63) / 64);
  return launch(reinterpret_cast<const void *>(&shrink_kernel<T, Q, NI, 4>), grid, kShrinkThreads, s, a);
}
template <typename T, bool Q>
hipError_t shrink(const ShrinkArgs &a, const ShrinkPlan &p, hipStream_t s) {
  const int64_t rows = 16 * p.row_tiles;
  const dim3 grid((uint32_t)((a.m + rows - 1) / rows), (uint32_t)(p.slices * p.slots));
  return p.row_tiles == 1 ? shrink<T, Q, 1>(a, grid, s) : shrink<T, Q, 2>(a, grid, s);
}
template <typename T>
hipError_t shrink(const ShrinkArgs &a, const ShrinkPlan &p, hipStream_t s) {
  return a.scale_x ? shrink<T, true>(a, p, s) : shrink<T, false>(a, p, s);
}

template <typename T, typename O>
hipError_t expand(const ExpandArgs &a, const ExpandPlan &p, hipStream_t s) {
  const dim3 grid((uint32_t)p.workgroups);
  return p.row_tiles == 1 ? launch(reinterpret_cast<const void *>(&expand_kernel<T, O, 1>), grid, kExpandThreads, s, a)
                          : launch(reinterpret_cast<const void *>(&expand_kernel<T, O, 2>), grid, kExpandThreads, s, a);
}

template <typename T>
hipError_t grad(const AdapterGradArgs &a, hipStream_t s) {
  const int64_t tiles_k = a.da ? (a.k + kGradCols - 1) / kGradCols : 0;
  const int64_t tiles = tiles_k + (a.db ? (a.n + kGradCols - 1) / kGradCols : 0);
  const int64_t numbers = a.m / a.piece + a.count;
  if (tiles == 0) return hipSuccess;
  const int nr = a.rank <= 16 ? 1 : a.rank <= 32 ? 2 : 4;
  const dim3 grid((uint32_t)(numbers * tiles), (uint32_t)((a.rank + 16 * nr - 1) / (16 * nr)));
  const void *kernel = nr == 1   ? reinterpret_cast<const void *>(&adapter_grad_kernel<T, 1>)
                       : nr == 2 ? reinterpret_cast<const void *>(&adapter_grad_kernel<T, 2>)
                                 : reinterpret_cast<const void *>(&adapter_grad_kernel<T, 4>);
  const hipError_t e = launch(kernel, grid, kGradThreads, s, a, tiles_k, tiles);
  if (e != hipSuccess) return e;
  const int64_t values = (int64_t)a.rank * (a.k + a.n), most = 4096 / a.count + 1;
  const int64_t groups = std::min((values + kGradThreads - 1) / kGradThreads, most);
  return launch(reinterpret_cast<const void *>(&adapter_grad_sum_kernel), dim3((uint32_t)(groups * a.count)),
                kGradThreads, s, a, groups);
}

}  // namespace

ShrinkPlan shrink_plan(int64_t m, int64_t k, int64_t rank, int64_t count) {
  ShrinkPlan p{};
  p.row_tiles = m <= 4096 ? 1 : 2;
  const int64_t tiles = (m + 16 * p.row_tiles - 1) / (16 * p.row_tiles);
  // a tile's rows have 16 adapters at most
  const int64_t adapters = std::min<int64_t>(std::min<int64_t>(m, 16), count);
  p.slots = 1;
  while (p.slots < adapters && tiles * p.slots < 64) p.slots *= 2;
  const int64_t blocks = std::max<int64_t>(1, (k + kBlock - 1) / kBlock);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(16, 256 / (tiles * p.slots)));
  const int64_t most = (blocks + kShrinkWaves - 1) / kShrinkWaves;  // a block for each wave
  p.blocks_per_slice = (int)((blocks + std::min(want, most) - 1) / std::min(want, most));
  p.slices = (int)((blocks + p.blocks_per_slice - 1) / p.blocks_per_slice);
  return p;
}
hipError_t launch_shrink(const ShrinkArgs &a, const ShrinkPlan &p, int dtype, hipStream_t s) {
  return dtype == XPOSE_F32 ? shrink<float>(a, p, s) : dtype == XPOSE_F16 ? shrink<_Float16>(a, p, s) : shrink<__bf16>(a, p, s);
}

hipError_t launch_slices(const SlicesArgs &a, hipStream_t s) {
  const int64_t groups = (a.count + kSlicesThreads - 1) / kSlicesThreads;
  return launch(reinterpret_cast<const void *>(&slices_kernel), dim3((uint32_t)std::min<int64_t>(groups, 2048)),
                kSlicesThreads, s, a);
}

ExpandPlan expand_plan(int64_t m, int64_t n, int64_t count) {
  ExpandPlan p{};
  p.row_tiles = m <= 1024 ? 1 : 2;
  const int64_t tiles = (m + 16 * p.row_tiles - 1) / (16 * p.row_tiles) * ((n + kExpandCols - 1) / kExpandCols);
  const int64_t adapters = std::min<int64_t>(std::min<int64_t>(m, 16), count);
  p.slots = 1;
  while (p.slots < adapters && tiles * p.slots < 512) p.slots *= 2;
  p.workgroups = tiles * p.slots;
  return p;
}
hipError_t launch_expand(const ExpandArgs &a, const ExpandPlan &p, int dtype, int out_dtype, hipStream_t s) {
  if (dtype == XPOSE_F32) return expand<float, float>(a, p, s);
  if (dtype == XPOSE_F16)
    return out_dtype == XPOSE_F32 ? expand<_Float16, float>(a, p, s) : expand<_Float16, _Float16>(a, p, s);
  return out_dtype == XPOSE_F32 ? expand<__bf16, float>(a, p, s) : expand<__bf16, __bf16>(a, p, s);
}

hipError_t launch_adapter_prep(const AdapterPrepArgs &a, int dtype, hipStream_t s) {
  auto tiles = [&](int64_t len) { return (len + kPrepThreads - 1) / kPrepThreads * a.count; };
  const int64_t groups = (a.order ? a.count : 0) + (a.at ? tiles(a.k) : 0) + (a.bt ? tiles(a.n) : 0);
  if (groups == 0) return hipSuccess;
  const void *kernel = dtype == XPOSE_F32   ? reinterpret_cast<const void *>(&adapter_prep_kernel<float>)
                       : dtype == XPOSE_F16 ? reinterpret_cast<const void *>(&adapter_prep_kernel<_Float16>)
                                            : reinterpret_cast<const void *>(&adapter_prep_kernel<__bf16>);
  return launch(kernel, dim3((uint32_t)groups), kPrepThreads, s, a);
}

int adapter_grad_piece(int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = (n + kGradCols - 1) / kGradCols + (k + kGradCols - 1) / kGradCols;
  int piece = 64;
  while (piece < 4096 && m / piece * tiles > 1024) piece *= 2;
  return piece;
}
int64_t adapter_grad_slots(int64_t m, int piece) { return m > piece ? 2 * (m / piece + 1) : 0; }
hipError_t launch_adapter_grad(const AdapterGradArgs &a, int dtype, hipStream_t s) {
  return dtype == XPOSE_F32 ? grad<float>(a, s) : dtype == XPOSE_F16 ? grad<_Float16>(a, s) : grad<__bf16>(a, s);
}

template <typename T>
static hipError_t dropout(const DropoutArgs &a, dim3 grid, hipStream_t s) {
  return a.residual ? launch(reinterpret_cast<const void *>(&dropout_kernel<T, true>), grid, kDropThreads, s, a)
                    : launch(reinterpret_cast<const void *>(&dropout_kernel<T, false>), grid, kDropThreads, s, a);
}
hipError_t launch_dropout(const DropoutArgs &given, int dtype, hipStream_t s) {
  DropoutArgs a = given;
  const int64_t chunks = (a.cols + 7) / 8;
  a.lanes = kDropThreads;
  while (a.lanes / 2 >= chunks) a.lanes /= 2;
  const int64_t wide = (chunks + a.lanes - 1) / a.lanes, at_once = kDropThreads / a.lanes;
  const int64_t groups = std::min<int64_t>((a.rows + at_once - 1) / at_once, std::max<int64_t>(1, 4096 / wide));
  const dim3 grid((uint32_t)wide, (uint32_t)groups);
  return dtype == XPOSE_F32 ? dropout<float>(a, grid, s) : dtype == XPOSE_F16 ? dropout<_Float16>(a, grid, s) : dropout<__bf16>(a, grid, s);
}

}  // namespace xpose
