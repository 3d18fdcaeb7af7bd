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
#include <atomic>

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

// Chunks of 16 bytes: V of them from `col` on of a row of `len` elements.  As
// with load_row8, what lies beyond the row's end is loaded from before it, and
// settled into zeros later.
template <typename E> constexpr int kChunk = 16 / (int)sizeof(E);
typedef u32x4 u32x4_by2 __attribute__((aligned(2)));
typedef u32x4 u32x4_by4 __attribute__((aligned(4)));
// 16 bytes of elements E as they lie in memory; e4m3 rows have them aligned
template <typename E>
using Chunk = typename std::conditional<sizeof(E) == 1, u32x4,
                                        typename std::conditional<sizeof(E) == 2, u32x4_by2, u32x4_by4>::type>::type;
// Rows shorter than one (SHORT) are read by elements: a kernel of its own, as
// that path's waits would be in the way of the other one's loads.
template <bool SHORT, typename E>
__device__ inline u32x4 load_chunk(const E *row, int64_t len, int64_t col) {
  constexpr int V = kChunk<E>;
  if constexpr (!SHORT) return *reinterpret_cast<const Chunk<E> *>(row + (col < len - V ? col : len - V));
  E v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = col + e < len ? row[col + e] : (E)0.f;
  u32x4 w;
  __builtin_memcpy(&w, v, 16);
  return w;
}
template <typename E>
__device__ inline void settle_chunk(u32x4 &v, int64_t len, int64_t col) {
  constexpr int V = kChunk<E>;
  if (len < V || col <= len - V) return;
  const int64_t past = col + V - len;
  const int by = past < V ? (int)past : V, words = by * (int)sizeof(E) / 4;
  uint32_t w[5] = {v[0], v[1], v[2], v[3], 0};
#pragma unroll
  for (int d = 4; d; d /= 2)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (words & d) w[i] = i + d < 4 ? w[i + d] : 0;
  if constexpr (sizeof(E) == 2)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (by & 1) w[i] = w[i] >> 16 | w[i + 1] << 16;
  v = u32x4{w[0], w[1], w[2], w[3]};
}
template <typename E>
__device__ inline void store_chunk(E *row, int64_t len, int64_t col, const float (&f)[kChunk<E>]) {
  constexpr int V = kChunk<E>;
  typedef E any __attribute__((ext_vector_type(V), aligned(sizeof(E))));
  if (col + V <= len) {
    any r;
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = (E)f[e];
    *reinterpret_cast<any *>(row + col) = r;
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (col + e < len) row[col + e] = (E)f[e];
  }
}
template <typename E> __device__ inline float chunk_at(const u32x4 &v, int e) {
  if constexpr (sizeof(E) == 4) return __uint_as_float(v[e]);
  E r[8];
  __builtin_memcpy(r, &v, 16);
  return (float)r[e];
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

// What is the same in all lanes, in a scalar register: a quotient is not by itself.
__device__ inline int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The adapter of row t0 + lane in the lanes below `rows`, -1 for none and -2 for
// no row; the number itself is loaded before it is asked for.
__device__ inline int raw_id(const int32_t *ids, int64_t m, int64_t t0, int lane) {
  return ids[min(t0 + lane, m - 1)];
}
__device__ inline int tile_id(int raw, int64_t m, int count, int64_t t0, int rows, int lane) {
  if (lane >= rows || t0 + lane >= m) return -2;
  return (uint32_t)raw < (uint32_t)count ? raw : -1;
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
// waves of a workgroup share out the columns in steps of 128 bytes of x and add
// their sums up at the end.
//
// The instruction wants another row in each of 16 neighbouring lanes.  Loaded
// so, every lane is a memory request of its own, and a compute unit gets 16
// bytes a cycle (measured 36 GB/s, from the caches too).  So 8 lanes load 128
// bytes of a row (100 to 120 GB/s), two or four steps ahead, and the step goes
// through the wave's own piece of LDS: no barriers.  A row's 8 chunks there are
// permuted by an exclusive or with bits 1 to 3 of the row, which spreads the
// reads of 16 rows over all banks.  Weights that come with the rank along their
// rows (WT, B in the backward pass) are turned around by the reads.
//
// Reading x bounds it with many rows, the latency of a few steps with few: 4001 x
// 4096 bfloat16, rank 16, take 13.5 us (2.4 TB/s, of x and once a tile of A from
// the caches; 18 with the rows' own loads), 8192 x 4096 turned 23 us (2.9 TB/s),
// 16 tokens of 16 adapters 5.5 us.
template <typename T, bool Q> using ShrinkX = typename std::conditional<Q, uint8_t, T>::type;
constexpr int kShrinkWaves = 8, kShrinkThreads = 64 * kShrinkWaves;

__device__ inline int swizzle(int row) { return (row >> 1) & 7; }

// Steps whose loads are under way together, as registers allow.
template <typename T, bool Q, int NI, int NR> constexpr int shrink_depth() {
  return NI + NR * (Q ? (int)sizeof(T) : 1) <= 3 ? 4 : 2;
}

// A step of 128 bytes of x's rows and R times as many of w's, as loaded.
template <bool Q, int NI, int NW> struct ShrinkStep {
  u32x4 x[NI][2], w[NW][2];
  float scale[Q ? NI : 1];
};

// Four halves of a column of LDS: lane l of 16 gets those at place l of the
// four rows of 16 that lanes 4 j and on address, 8 bytes each.
__device__ inline u32x2 turn4(const uint8_t *p) {
  typedef short i16x4 __attribute__((ext_vector_type(4)));
  auto *lds = (__attribute__((address_space(3))) uint8_t *)p;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) i16x4 *)lds));
}

// The rows of adapter l, in order, behind those of all adapters before it, which
// are counted for that here too: ids are read by each adapter's workgroup, from
// the caches.  A wave has a stretch of rows, 512 of them under way.
__device__ inline void adapter_rows(const ShrinkArgs &a, int l, int32_t *lds) {
  constexpr int WAVES = kShrinkWaves;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int64_t stretch = (a.m + 64 * WAVES - 1) / (64 * WAVES) * 64;
  const int64_t begin = wave * stretch, end = min(begin + stretch, a.m);
  auto ids8 = [&](int64_t i0, int (&id)[8]) {  // -1 past the end
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int64_t i = i0 + 64 * s + lane;
      id[s] = i < end ? a.ids[i] : -1;
    }
  };
  int before = 0, mine = 0;
  for (int64_t i0 = begin; i0 < end; i0 += 512) {
    int id[8];
    ids8(i0, id);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      before += (uint32_t)id[s] < (uint32_t)l;
      mine += id[s] == l;
    }
  }
#pragma unroll
  for (int d = 32; d; d /= 2) {
    before += __shfl_xor(before, d);
    mine += __shfl_xor(mine, d);
  }
  if (lane == 0) {
    lds[wave] = before;
    lds[WAVES + wave] = mine;
  }
  __syncthreads();
  int at = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) at += lds[w];
  if (tid == 0) a.starts[l] = at;
  int place = at;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w < wave) place += lds[WAVES + w];
    at += lds[WAVES + w];
  }
  for (int64_t i0 = begin; i0 < end; i0 += 512) {
    int id[8];
    ids8(i0, id);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const uint64_t all = __ballot(id[s] == l);
      if (id[s] == l) a.order[place + __popcll(all & ((1ull << lane) - 1))] = (int32_t)(i0 + 64 * s + lane);
      place += __popcll(all);
    }
  }
  if (tid == 0 && l == a.count - 1) a.starts[a.count] = at;
}

template <typename T, bool Q, int NI, int NR, bool WT, bool SHORT>
__global__ __launch_bounds__(kShrinkThreads) void shrink_kernel(ShrinkArgs a) {
  using XT = ShrinkX<T, Q>;
  constexpr int WAVES = kShrinkWaves, THREADS = kShrinkThreads, DEPTH = shrink_depth<T, Q, NI, NR>();
  constexpr int ROWS = 16 * NI, R = Q ? (int)sizeof(T) : 1, NW = NR * R, UNITS = NI + NW;
  constexpr int kStep = 128 / (int)sizeof(XT);  // columns
  using Step = ShrinkStep<Q, NI, NW>;
  static_assert(UNITS * 2 >= NI * NR);  // the sums fit where the steps were
  __shared__ __align__(16) uint8_t lds[WAVES][UNITS * 2048];
  const int tid = threadIdx.x, lane = tid % 64, i16 = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  uint8_t *const mine = lds[wave];
  if (blockIdx.x >= a.tiles) {
    if (blockIdx.y == 0 && blockIdx.z == 0) adapter_rows(a, (int)(blockIdx.x - a.tiles), (int32_t *)lds[0]);
    return;
  }
  const int64_t t0 = (int64_t)blockIdx.x * ROWS;
  const int slice = scalar(blockIdx.y / a.slots), slot = scalar(blockIdx.y % a.slots);
  const int r0 = blockIdx.z * 16 * NR;
  const int id = tile_id(raw_id(a.ids, a.m, t0, lane), a.m, a.count, t0, ROWS, lane);
  float *h = a.h + slice * a.slice;
  const int steps = (int)((a.k + kStep - 1) / kStep), whole = (int)(a.k / kStep);
  const int first = scalar(slice * a.steps_per_slice);
  const int last = scalar(min(first + a.steps_per_slice, steps)), last_whole = scalar(min(last, whole));
  // what this lane loads: rows lane / 8 and 8 more, and their chunk
  const int row_in[2] = {lane / 8, lane / 8 + 8};
  const int chunk[2] = {lane % 8 ^ swizzle(row_in[0]), lane % 8 ^ swizzle(row_in[1])};
  const XT *x[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int o = 0; o < 2; ++o)
      x[i][o] = (const XT *)a.x + min(t0 + 16 * i + row_in[o], a.m - 1) * a.ldx + chunk[o] * kChunk<XT>;

  // WT: w's rows are its columns, 16 ranks of each are a row of a unit in LDS,
  // and this lane loads a chunk of ranks of one of the step's columns.
  auto turned_column = [&](int o) { return (64 * o + lane) / (int)sizeof(T); };
  auto turned_rank = [&](int o) { return (64 * o + lane) % (int)sizeof(T) * kChunk<T>; };

  auto load_x = [&](int step, Step &v, auto ragged) {
    constexpr bool RAGGED = decltype(ragged)::value;
    const int64_t c0 = (int64_t)step * kStep;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if constexpr (Q) v.scale[i] = a.scale_x[c0 / kStep * a.ld_scale_x + min(t0 + 16 * i + i16, a.m - 1)];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        if constexpr (!RAGGED) {
          v.x[i][o] = *reinterpret_cast<const Chunk<XT> *>(x[i][o] + c0);
        } else if constexpr (Q) {  // the 16 bytes that hold a row's end are all there
          const int64_t left = a.k - c0 - chunk[o] * 16;
          v.x[i][o] = *reinterpret_cast<const u32x4 *>(x[i][o] + (left > 0 ? c0 : -chunk[o] * 16));
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int64_t in = left - 4 * b;
            v.x[i][o][b] &= in >= 4 ? ~0u : in <= 0 ? 0u : (1u << (8 * (int)in)) - 1;
          }
        } else {
          const int64_t at = chunk[o] * kChunk<XT>;
          if (a.k < kChunk<XT>) {
            v.x[i][o] = load_chunk<true>(x[i][o] - at, a.k, c0 + at);
          } else {
            v.x[i][o] = load_chunk<false>(x[i][o] - at, a.k, c0 + at);
            settle_chunk<XT>(v.x[i][o], a.k, c0 + at);
          }
        }
      }
    }
  };
  if (slot == 0) {
    const uint64_t none = __ballot(id == -1);
    if (none)
      for (int i = tid; i < ROWS * 16 * NR; i += THREADS) {
        const int row = i / (16 * NR), r = r0 + i % (16 * NR);
        if ((none >> row & 1) && r < a.rank) h[(t0 + row) * a.rank + r] = 0.f;
      }
  }

  each_adapter(id, slot, a.slots, [&](int d, uint64_t match) {
    f32x4 sum[NI][NR];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < NR; ++q) sum[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    const T *w0 = (const T *)a.w + d * a.stride_w;
    const T *w[NR][2];
#pragma unroll
    for (int q = 0; q < NR; ++q)
#pragma unroll
      for (int o = 0; o < 2; ++o)
        w[q][o] = WT ? w0 + turned_column(o) * a.ldw
                     : w0 + min(r0 + 16 * q + row_in[o], a.rank - 1) * a.ldw + chunk[o] * kChunk<T>;

    auto load_w = [&](int step, Step &v, auto ragged) {
      constexpr bool RAGGED = decltype(ragged)::value;
      const int64_t c0 = (int64_t)step * kStep;
#pragma unroll
      for (int q = 0; q < NR; ++q)
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            u32x4 &to = v.w[q * R + j][o];
            if constexpr (WT) {
              const int64_t past = RAGGED ? max(c0 + turned_column(o) - (a.k - 1), (int64_t)0) : 0;  // the last column again
              to = load_chunk<SHORT>(w[q][o] + (c0 - past) * a.ldw, a.rank, r0 + 16 * q + turned_rank(o));
              if (RAGGED && past) to = u32x4{0, 0, 0, 0};
            } else {
              const int64_t c = c0 + 8 * j * kChunk<T>;
              if constexpr (!RAGGED) {
                to = *reinterpret_cast<const Chunk<T> *>(w[q][o] + c);
              } else {
                const int64_t at = chunk[o] * kChunk<T>;
                if (a.k < kChunk<T>) {
                  to = load_chunk<true>(w[q][o] - at, a.k, c + at);
                } else {
                  to = load_chunk<false>(w[q][o] - at, a.k, c + at);
                  settle_chunk<T>(to, a.k, c + at);
                }
              }
            }
          }
    };
    // chunk c of row i16 of a unit
    auto read = [&](int unit, int c) {
      return *reinterpret_cast<const u32x4 *>(mine + unit * 2048 + i16 * 128 + (c ^ swizzle(i16)) * 16);
    };
    // eight values along the columns, chunks g + 4 b and (float32) g + 4 b + 4 of x, of rank 16 q + i16
    auto read_w = [&](int q, int b) {
      Vec8<T> to;
      constexpr int C = (int)sizeof(Vec8<T>) / 16;
      if constexpr (!WT) {
        u32x4 c[C];
#pragma unroll
        for (int j = 0; j < C; ++j) c[j] = read(NI + q, g + 4 * (b * C + j));
        __builtin_memcpy(&to, c, sizeof to);
      } else if constexpr (C == 1) {
        u32x2 c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          c[h] = turn4(mine + (NI + q) * 2048 + ((g + 4 * b) * 8 + 4 * h + i16 / 4) * 32 + i16 % 4 * 8);
        __builtin_memcpy(&to, c, sizeof to);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          to.v[e / 4][e % 4] = *reinterpret_cast<const float *>(mine + (NI + q) * 2048 + ((g + e / 4 * 4) * 4 + e % 4) * 64 + i16 * 4);
      }
      return to;
    };
    auto multiply = [&](Step &v) {
      if constexpr (WT && !SHORT && NR < 4)  // four are for whole chunks of ranks alone
#pragma unroll
        for (int q = 0; q < NR; ++q)
#pragma unroll
          for (int o = 0; o < 2; ++o) settle_chunk<T>(v.w[q][o], a.rank, r0 + 16 * q + turned_rank(o));
#pragma unroll
      for (int o = 0; o < 2; ++o) {
#pragma unroll
        for (int i = 0; i < NI; ++i) *reinterpret_cast<u32x4 *>(mine + i * 2048 + o * 1024 + lane * 16) = v.x[i][o];
#pragma unroll
        for (int j = 0; j < NW; ++j)
          *reinterpret_cast<u32x4 *>(mine + (NI + j) * 2048 + o * 1024 + lane * 16) = v.w[j][o];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if constexpr (Q) {
        f32x4 part[NI][NR];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int q = 0; q < NR; ++q) part[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < 2; ++b) {  // chunks g and g + 4 of x: 16 values
          u32x4 xc[NI];
#pragma unroll
          for (int i = 0; i < NI; ++i) xc[i] = read(i, g + 4 * b);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            Vec8<T> xv[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) xv[i] = widen8<T>(xc[i][2 * half], xc[i][2 * half + 1]);
#pragma unroll
            for (int q = 0; q < NR; ++q) {
              Vec8<T> wv;
              u32x4 wc[R / 2];
#pragma unroll
              for (int j = 0; j < R / 2; ++j) {
                const int c = (g + 4 * b) * R + half * (R / 2) + j;  // of w's row
                wc[j] = read(NI + q * R + c / 8, c % 8);
              }
              __builtin_memcpy(&wv, wc, sizeof wv);
#pragma unroll
              for (int i = 0; i < NI; ++i) part[i][q] = multiply8<T>(wv, xv[i], part[i][q]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int q = 0; q < NR; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[i][q][e] = __builtin_fmaf(part[i][q][e], v.scale[i], sum[i][q][e]);
      } else {
        constexpr int C = (int)sizeof(Vec8<T>) / 16;  // chunks of eight values
#pragma unroll
        for (int b = 0; b < 2 / C; ++b) {
          Vec8<T> xv[NI], wv[NR];
          auto get = [&](int unit, Vec8<T> &to) {
            u32x4 c[C];
#pragma unroll
            for (int j = 0; j < C; ++j) c[j] = read(unit, g + 4 * (b * C + j));
            __builtin_memcpy(&to, c, sizeof to);
          };
#pragma unroll
          for (int i = 0; i < NI; ++i) get(i, xv[i]);
#pragma unroll
          for (int q = 0; q < NR; ++q) wv[q] = read_w(q, b);
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int q = 0; q < NR; ++q) sum[i][q] = multiply8<T>(wv[q], xv[i], sum[i][q]);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    // Where paths meet that have other loads under way, or in another order, all
    // of them are waited for: so one way through the main loop, no conditions in
    // it, and the last steps behind it.
    const int start = first + wave;
    if (start < last_whole) {
      Step v[DEPTH];
      auto fetch = [&](int step, Step &to) {
        load_x(step, to, std::false_type{});
        load_w(step, to, std::false_type{});
        __builtin_amdgcn_sched_barrier(0);
      };
      int step = start;
      if (start + (2 * DEPTH - 1) * WAVES < last_whole) {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) fetch(start + u * WAVES, v[u]);
        for (; step + (2 * DEPTH - 1) * WAVES < last_whole; step += DEPTH * WAVES)
#pragma unroll
          for (int u = 0; u < DEPTH; ++u) {
            multiply(v[u]);
            fetch(step + (DEPTH + u) * WAVES, v[u]);
          }
      } else {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u)
          if (start + u * WAVES < last_whole) fetch(start + u * WAVES, v[u]);
      }
#pragma unroll
      for (int u = 0; u < DEPTH; ++u) {
        if (step + u * WAVES < last_whole) multiply(v[u]);
        if (step + (DEPTH + u) * WAVES < last_whole) fetch(step + (DEPTH + u) * WAVES, v[u]);
      }
#pragma unroll
      for (int u = 0; u < DEPTH - 1; ++u)
        if (step + (DEPTH + u) * WAVES < last_whole) multiply(v[u]);
    }
    if (whole < last && wave == (whole - first) % WAVES) {
      Step end;
      load_x(whole, end, std::true_type{});
      load_w(whole, end, std::true_type{});
      multiply(end);
    }

    f32x4 *sums = reinterpret_cast<f32x4 *>(mine);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < NR; ++q) sums[(i * NR + q) * 64 + lane] = sum[i][q];
    __syncthreads();
    const float factor = a.scaled ? a.alpha * (a.scale ? a.scale[d] : 1.f) : 1.f;
    for (int f = wave; f < NI * NR; f += WAVES) {
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int o = 0; o < WAVES; ++o) v += reinterpret_cast<const f32x4 *>(lds[o])[f * 64 + lane];
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
    __syncthreads();  // before the next adapter's steps
  });
}

// ----- expand ------------------------------------------------------------------------
//
// out = base + h w^T, the rows of h as the first operand and the rows of w
// (columns of out) as the second: a lane has four rows of one column.  Which of
// the columns of eight instructions is which of their rows is chosen so that a
// lane has 16 bytes of each of its rows, and 16 lanes 256: with a row a lane
// instead, as in `shrink` above, 4001 x 8192 bfloat16 took 41 us, and so 32 (4.1
// TB/s of base and out, which bound it: copies reach 6.3).
//
// A workgroup has WR waves of 16 rows under each other and 4 / WR side by side,
// 128 columns each, and goes down the rows, the next tile's ids, base and h on
// their way.  Its columns of w lie in LDS as operands, 32 ranks at a time, until
// another adapter's are needed.
//
// h is float32 and stays it: for 16-bit weights it goes to the matrix cores as
// the sum of three bfloat16 numbers (24 bits; they have float32's range, which
// float16 has not), float16 weights as the sum of two.  Next to reading base
// and writing out, the products are free.
constexpr int kExpandWaves = 4, kExpandThreads = 64 * kExpandWaves;
constexpr int kExpandCols = 128;  // of a wave

// Eight float32 numbers as operands of multiply_split.  The first part is cut
// off, not rounded: the nearest bfloat16 of what lies over its largest number is
// infinite.  The other two are rounded, which leaves nothing of 24 bits.
template <typename T> struct Split8 {
  bf16x8 part[3];
  __device__ void set(const float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __bf16 first = __builtin_bit_cast(__bf16, (uint16_t)(__float_as_uint(f[e]) >> 16));
      // an infinity is one, and not one less itself; of a NaN the rest is one too
      float rest = __builtin_fabsf(f[e]) == __builtin_inff() ? 0.f : f[e] - (float)first;
      part[0][e] = first;
#pragma unroll
      for (int p = 1; p < 3; ++p) {
        part[p][e] = (__bf16)rest;
        rest -= (float)part[p][e];
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
  for (int p = 2; p >= 0; --p) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h.part[p], (bf16x8)w.v, sum, 0, 0, 0);
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
  for (int p = 1; p >= 0; --p) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h.part[p], lo, sum, 0, 0, 0);
#pragma unroll
  for (int p = 2; p >= 0; --p) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h.part[p], hi, sum, 0, 0, 0);
  return sum;
}
template <> __device__ inline f32x4 multiply_split<float>(const Vec8<float> &w, const Split8<float> &h, f32x4 sum) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    sum = __builtin_amdgcn_mfma_f32_16x16x4f32(h.v[e], w.v[e / 4][e % 4], sum, 0, 0, 0);
  return sum;
}

// An operand's 64 lanes follow each other, 16 bytes each (float32: twice), a
// bank group on from the previous operand's.
template <typename T> constexpr int kOperandBytes = 1024 * (int)sizeof(Vec8<T>) / 16 + 16;
template <typename T, int WR> constexpr int kExpandLds = kExpandCols * kExpandWaves / WR / 16 * kOperandBytes<T>;

template <typename T, typename O, int WR, bool WT, bool SHORT>
__device__ __forceinline__ void expand(const ExpandArgs &a, uint32_t block, uint8_t *lds) {
  constexpr int V = kChunk<O>, P = 8 / V, ROWS = 16 * WR, COLS = kExpandCols * kExpandWaves / WR;
  constexpr int C = (int)sizeof(Vec8<T>) / 16, kOperand = kOperandBytes<T>;
  const int tid = threadIdx.x, lane = tid % 64, i16 = lane % 16, g = lane / 16;
  const int wave = scalar(tid / 64);
  const int slot = scalar(block % a.slots), place = scalar(block / a.slots);
  const int first = scalar(place / a.strips) * a.tiles, last = scalar(min(first + a.tiles, (int)((a.m + ROWS - 1) / ROWS)));
  const int64_t n0 = (int64_t)scalar(place % a.strips) * COLS;
  const int side = wave / WR;      // of the waves side by side
  const int in0 = wave % WR * 16;  // this wave's rows of a tile
  auto column = [&](int p) { return n0 + side * kExpandCols + 16 * V * p + V * i16; };  // the first of V
  const bool has_columns = n0 + side * kExpandCols < a.n;

  struct Tile {
    int id;
    u32x4 base[4][P];
    Vec8<float> h;  // of the first 32 ranks, of all slices
  };
  auto load_h = [&](int64_t row0, int c) {
    const float *h = a.h + min(row0 + i16, a.m - 1) * a.rank;
    const int r = c + 8 * g;
    auto slice = [&](int s) {
      if constexpr (SHORT) return load_raw8(h + s * a.slice + r, valid8(a.rank - r));
      else return load_row8(h + s * a.slice, a.rank, r);
    };
    Vec8<float> f = slice(0);
    if (a.slices > 1) {
      Vec8<float> more[3];
#pragma unroll
      for (int s = 0; s < 3; ++s) more[s] = slice(min(s + 1, a.slices - 1));
#pragma unroll
      for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e / 4][e % 4] += s + 1 < a.slices ? more[s].v[e / 4][e % 4] : 0.f;
    }
    return f;
  };
  // without conditions, so that the loads stay together: what is out of the
  // tile, or no base, is read from elsewhere and not used
  const O *base = (const O *)(a.base ? a.base : a.out);
  const int64_t ld_base = a.base ? a.ld_base : a.ld_out;
  auto load = [&](int tile, Tile &to) {
    const int64_t t0 = (int64_t)tile * ROWS, row0 = t0 + in0;
    to.id = raw_id(a.ids, a.m, t0, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int p = 0; p < P; ++p)
        to.base[e][p] = load_chunk<SHORT>(base + min(row0 + 4 * g + e, a.m - 1) * ld_base, a.n, column(p));
    if (a.count) to.h = load_h(row0, 0);
  };

  Tile now;
  int has = -1;  // the adapter whose operands are in LDS
  load(first, now);
  // Here, where the adapter has to be waited for anyway: else the first tile's
  // loads count as under way in all turns, and each waits for the next tile's.
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  for (int tile = first; tile < last; ++tile) {
    const int64_t t0 = (int64_t)tile * ROWS, row0 = t0 + in0;
    const bool here = has_columns && row0 < a.m;
    const int id = tile_id(now.id, a.m, a.count, t0, ROWS, lane);
    Tile next;
    if (tile + 1 < last) load(tile + 1, next);
    auto store = [&](uint64_t match, const f32x4 (&sum)[8], auto add) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(match >> (in0 + 4 * g + e) & 1)) continue;
        O *to = (O *)a.out + (row0 + 4 * g + e) * a.ld_out;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float y[V];
          u32x4 b = now.base[e][p];
          if constexpr (!SHORT) settle_chunk<O>(b, a.n, column(p));
#pragma unroll
          for (int j = 0; j < V; ++j) {
            y[j] = a.base ? chunk_at<O>(b, j) : 0.f;
            if constexpr (decltype(add)::value) y[j] += sum[p * V + j][e];
          }
          store_chunk(to, a.n, column(p), y);
        }
      }
    };
    if (slot == 0 && a.base != a.out && here) {
      const uint64_t none = __ballot(id == -1);
      const f32x4 nothing[8] = {};
      if (none >> in0 & 0xffff) store(none, nothing, std::false_type{});
    }
    each_adapter(id, slot, a.slots, [&](int d, uint64_t match) {
      const bool mine = here && (match >> in0 & 0xffff) != 0;
      const float factor = a.alpha * (a.scale ? a.scale[d] : 1.f);
      const T *w0 = (const T *)a.w + d * a.stride_w;
      f32x4 sum[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < a.rank; c += 32) {
        if (a.rank > 32 || has != d) {
          constexpr int EACH = COLS * 4 / kExpandThreads;  // chunks of eight, of 32 ranks of each column
          Vec8<T> w[EACH];
          if constexpr (!WT) {
#pragma unroll
            for (int u = 0; u < EACH; ++u) {
              const int i = u * kExpandThreads + tid, r = c + i % 4 * 8;
              const T *from = w0 + min(n0 + i / 4, a.n - 1) * a.ldw;
              if constexpr (SHORT) w[u] = load_raw8(from + r, valid8(a.rank - r));
              else w[u] = load_row8(from, a.rank, r);
            }
          } else {
#pragma unroll
            for (int u = 0; u < EACH; ++u) {
              const int i = u * kExpandThreads + tid;
              const int64_t col = n0 + i % (COLS / 8) * 8;
              const T *from = w0 + min(c + i / (COLS / 8), a.rank - 1) * a.ldw;
              if constexpr (SHORT) w[u] = load_raw8(from + col, valid8(a.n - col));
              else w[u] = load_row8(from, a.n, col);
            }
          }
          __syncthreads();  // the operands before these are done with
#pragma unroll
          for (int u = 0; u < EACH; ++u) {
            const int i = u * kExpandThreads + tid;
            auto operand = [&](int col) {  // and its lane of ranks 0 to 7
              return lds + (col / kExpandCols * 8 + col % kExpandCols / (16 * V) * V + col % V) * kOperand + col / V % 16 * 16;
            };
            if constexpr (!WT) {
              if constexpr (!SHORT) settle8<T>(w[u], a.rank, c + i % 4 * 8);
              u32x4 v[C];
              __builtin_memcpy(v, &w[u], sizeof v);
              uint8_t *to = operand(i / 4) + i % 4 * 256;
#pragma unroll
              for (int q = 0; q < C; ++q) *reinterpret_cast<u32x4 *>(to + 1024 * q) = v[q];
            } else {
              const int col = i % (COLS / 8) * 8, r = i / (COLS / 8);
              if constexpr (!SHORT) settle8<T>(w[u], a.n, n0 + col);
              T v[8];
              __builtin_memcpy(v, &w[u], sizeof v);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                uint8_t *to = operand(col + e) + r / 8 * 256 + r % 8 * (int)sizeof(T) / 16 * 1024 + r % 8 * (int)sizeof(T) % 16;
                *reinterpret_cast<T *>(to) = c + r < a.rank ? v[e] : (T)0.f;
              }
            }
          }
          __syncthreads();
          has = d;
        }
        if (!mine) continue;
        Vec8<float> raw = c == 0 ? now.h : load_h(row0, c);
        // ranks past the last one stay zeros whatever the factor is
        const int ranks = SHORT ? valid8(a.rank - c - 8 * g) : 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) raw.v[e / 4][e % 4] = e < ranks ? raw.v[e / 4][e % 4] * factor : 0.f;
        if constexpr (!SHORT) settle8<float>(raw, a.rank, c + 8 * g);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = at8<float>(raw, e);
        Split8<T> h;
        h.set(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint8_t *p = lds + (side * 8 + j) * kOperand + lane * 16;
          u32x4 v[C];
#pragma unroll
          for (int q = 0; q < C; ++q) v[q] = *reinterpret_cast<const u32x4 *>(p + 1024 * q);
          Vec8<T> wj;
          __builtin_memcpy(&wj, v, sizeof v);
          sum[j] = multiply_split<T>(wj, h, sum[j]);
        }
      }
      if (mine) store(match, sum, std::true_type{});
    });
    now = next;
  }
}

template <typename T, typename O, int WR, bool WT, bool SHORT>
__global__ __launch_bounds__(kExpandThreads) void expand_kernel(ExpandArgs a) {
  __shared__ __align__(16) uint8_t lds[kExpandLds<T, WR>];
  expand<T, O, WR, WT, SHORT>(a, blockIdx.x, lds);
}

// ----- the adapters' gradients ----------------------------------------------------------
//
// G[r][c] = sum over rows u[row][r] v[row][c], u of r columns in float32, v as
// it is.  With bfloat16 v, u is the sum of three bfloat16 numbers, as in `expand`;
// a lane loads four columns of each of eight rows twice over and turns them around
// in registers, a byte permutation for two values.  Other types take the float32
// matrix cores, whose operands need no turning around, as a lane has one rank or
// eight neighbouring columns of one row in four; in bfloat16 that took 8192 rows,
// 4096 columns both ways, all gradients, with pieces of 1024 rows, 92 us for 84 at
// rank 16, 137 for 97 at 32, 281 for 158 at 64.  (Float16 v would have to be split
// too.)
//
// An adapter's rows are cut into pieces, a workgroup for 128 columns of each.
// An adapter of one piece, or none, is done with that; the pieces of larger ones go to
// the workspace and a second launch adds them up, in their order.  Adapter l's
// pieces are the numbers starts[l] / piece + l and on: there are enough
// numbers between one adapter's first and the next one's.  Workspace slots,
// which only adapters of over a piece need, are 2 (starts[l] / piece) and on: an
// adapter of p > 1 pieces has over (p - 1) piece rows, so the next one's first
// slot is 2 (p - 1) >= p further at least.
//
// Reading x and dout bounds it, once for each 64 ranks.
constexpr int kGradThreads = 256, kGradCols = 128, kGradWaves = 4;

__device__ inline int grad_pieces(int rows, int piece) { return (rows + piece - 1) / piece; }

template <typename T> constexpr bool kGradSplit = std::is_same_v<T, __bf16>;
template <typename T> constexpr int kGradRows = kGradSplit<T> ? 32 : 16;  // of a block

template <typename T, int NR> struct GradRows {
  Vec8<T> v[4];
  float u[4][NR];
};
template <int NR> struct GradRows<__bf16, NR> {
  u32x2 v[2][8];  // four columns of each half
  float u[8][NR];
};

typedef u32x2 u32x2_by2 __attribute__((aligned(2)));
// Four columns from `col` on, to be settled where they go past the end
template <bool SHORT>
__device__ inline u32x2 load_row4(const __bf16 *row, int64_t len, int64_t col) {
  if constexpr (!SHORT) return *reinterpret_cast<const u32x2_by2 *>(row + (col < len - 4 ? col : len - 4));
  __bf16 v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = col + e < len ? row[col + e] : (__bf16)0.f;
  u32x2 w;
  __builtin_memcpy(&w, v, 8);
  return w;
}

template <typename T, int NR, bool SHORT>
__device__ __forceinline__ void adapter_grad(const AdapterGradArgs &a, uint32_t block, f32x4 (*lds)[8][64]) {
  constexpr bool SPLIT = kGradSplit<T>;
  // blocks of rows under way, as registers allow
  constexpr int DEPTH = SPLIT ? (NR < 4 ? 2 : 1) : NR * (int)sizeof(T) <= 4 ? 3 : 2;
  constexpr int BLOCK = kGradRows<T>;
  const int tiles_k = a.tiles_k, tiles = a.tiles;
  const int tid = threadIdx.x, lane = tid % 64, i16 = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int number = scalar((int)(block / (uint32_t)tiles)), tile = scalar((int)(block % (uint32_t)tiles));
  const int r0 = blockIdx.y * 16 * NR;
  // the last adapter whose first number is no later, by 64 of them at a time
  int l = 0;
  for (int left = a.count; left > 1;) {
    const int step = (left + 63) / 64, probe = lane * step;
    const bool no_later = probe < left && a.starts[l + probe] / a.piece + l + probe <= number;
    const int p = __popcll(__ballot(no_later)) - 1;  // the first one's is 0
    l += p * step;
    left = min(step, left - p * step);
  }
  l = scalar(l);
  const int start = scalar(a.starts[l]), rows = scalar(a.starts[l + 1]) - start;
  const int j = number - (start / a.piece + l);
  const int pieces = grad_pieces(rows, a.piece);
  if (j >= max(pieces, 1)) return;  // the first one of an adapter of no rows stores zeros
  const int begin = start + j * a.piece, end = min(begin + a.piece, start + rows);

  const bool of_b = tile >= tiles_k;
  const int64_t cols = of_b ? a.n : a.k, c0 = (of_b ? tile - tiles_k : tile) * (int64_t)kGradCols;
  const T *v = (const T *)(of_b ? a.dout : a.x);
  const int64_t ldv = of_b ? a.lddout : a.ldx;
  const float *u = of_b ? a.h : a.dh;
  const float factor = of_b ? a.alpha * (a.scale ? a.scale[l] : 1.f) : 1.f;
  const int64_t col = c0 + (SPLIT ? 4 : 8) * i16;  // SPLIT: and 64 on

  f32x4 sum[NR][8];
#pragma unroll
  for (int q = 0; q < NR; ++q)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[q][e] = f32x4{0.f, 0.f, 0.f, 0.f};
  // BLOCK rows at a time, the next ones' loads under way and the numbers of those
  // after them; past the end the last row is read, for nothing
  GradRows<T, NR> rows_of[DEPTH];
  int numbers[DEPTH];
  auto number_of = [&](int p0) { return a.order[min(p0 + lane % BLOCK, end - 1)]; };
  // rows with these numbers; then numbers are those of p0
  auto load = [&](int &numbers, int p0, GradRows<T, NR> &to) {
    int64_t row[BLOCK / 4];
#pragma unroll
    for (int s = 0; s < BLOCK / 4; ++s) row[s] = __shfl(numbers, SPLIT ? 8 * g + s : 4 * s + g);
    __builtin_amdgcn_sched_barrier(0);
    numbers = number_of(p0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < BLOCK / 4; ++s) {
      const T *from = v + row[s] * ldv;
      if constexpr (SPLIT) {
        to.v[0][s] = load_row4<SHORT>(from, cols, col);
        to.v[1][s] = load_row4<SHORT>(from, cols, col + 64);
      } else if constexpr (SHORT) {
        to.v[s] = load_raw8(from + col, valid8(cols - col));
      } else {
        to.v[s] = load_row8(from, cols, col);
      }
#pragma unroll
      for (int q = 0; q < NR; ++q) to.u[s][q] = u[row[s] * a.rank + min(r0 + 16 * q + i16, a.rank - 1)];
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int p0, GradRows<T, NR> &rows) {
    if constexpr (SPLIT) {
      if (!SHORT && c0 + kGradCols > cols)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t past = col + 64 * h + 4 - cols;
          const int by = past < 0 ? 0 : past < 4 ? (int)past : 4;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            uint64_t w = (uint64_t)rows.v[h][s][1] << 32 | rows.v[h][s][0];
            w = by < 4 ? w >> (16 * by) : 0;
            rows.v[h][s] = u32x2{(uint32_t)w, (uint32_t)(w >> 32)};
          }
        }
      if (p0 + BLOCK > end)  // rows past the piece may hold anything
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const bool in = p0 + 8 * g + s < end;
#pragma unroll
          for (int q = 0; q < NR; ++q) rows.u[s][q] = in ? rows.u[s][q] : 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) rows.v[h][s][i] = in ? rows.v[h][s][i] : 0;
        }
      Split8<T> part[NR];
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        float f[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) f[s] = rows.u[s][q];
        part[q].set(f);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // a column: its rows two by two
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = __builtin_amdgcn_perm(rows.v[e / 4][2 * i + 1][e % 4 / 2], rows.v[e / 4][2 * i][e % 4 / 2],
                                       e % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int q = 0; q < NR; ++q)
#pragma unroll
          for (int p = 2; p >= 0; --p)
            sum[q][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(part[q].part[p], __builtin_bit_cast(bf16x8, w), sum[q][e], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool in = p0 + 4 * s + g < end;  // rows past the piece may hold anything
        if constexpr (!SHORT) settle8<T>(rows.v[s], cols, col);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = in ? at8<T>(rows.v[s], e) : 0.f;
#pragma unroll
          for (int q = 0; q < NR; ++q)
            sum[q][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(in ? rows.u[s][q] : 0.f, f, sum[q][e], 0, 0, 0);
        }
      }
    }
  };
  // as in shrink_kernel, one way through the loop
  constexpr int kApart = BLOCK * kGradWaves;
  const int start_at = begin + BLOCK * wave;
  if (start_at < end) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) numbers[d] = number_of(start_at + d * kApart);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(numbers[d], start_at + (DEPTH + d) * kApart, rows_of[d]);
    for (int p0 = start_at; p0 < end; p0 += DEPTH * kApart)
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const int at = p0 + d * kApart;
        multiply(at, rows_of[d]);
        load(numbers[d], at + 2 * DEPTH * kApart, rows_of[d]);
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
  // lds[q][e][lane] has ranks 16 q + 4 (lane / 16) and on of column 8 (lane % 16) + e,
  // or 64 (e / 4) + 4 (lane % 16) + e % 4
  const float *flat = (const float *)lds;
  auto value = [&](int r, int c) {
    const int e = SPLIT ? c / 64 * 4 + c % 4 : c % 8, of = SPLIT ? c % 64 / 4 : c / 8;
    return flat[(((r / 16) * 8 + e) * 64 + r % 16 / 4 * 16 + of) * 4 + r % 4] * factor;
  };
  const int ranks = min(a.rank - r0, 16 * NR), here = (int)min(cols - c0, (int64_t)kGradCols);
  const int64_t slot = 2 * (int64_t)(start / a.piece) + j, each = (int64_t)a.rank * (a.k + a.n);
  const bool done = pieces <= 1;
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

template <typename T, int NR, bool SHORT>
__global__ __launch_bounds__(kGradThreads) void adapter_grad_kernel(AdapterGradArgs a) {
  __shared__ f32x4 lds[NR][8][64];
  adapter_grad<T, NR, SHORT>(a, blockIdx.x, lds);
}

// dx and the adapters' gradients in one launch, which need nothing of each other,
// a workgroup of each in turn: 8192 rows, 4096 columns both ways, bfloat16 take
// 81 us a pass, some 5 more one after the other or in two launches, 300 rows 20 and
// 25.  For over 32 ranks they are two launches: more sums than let two workgroups
// of both kinds share a compute unit (rank 64, pieces of 1024 rows, 158 us, 171 and
// 242 here with 32 and 64 ranks a workgroup, float32 2048 rows 98 and 119).
template <typename T, typename O, int NR, bool SHORT>
__global__ __launch_bounds__(kGradThreads, sizeof(T) == 2 ? 2 : 1) void adapter_both_kernel(ExpandArgs e, AdapterGradArgs g, uint32_t expands) {
  constexpr int kBytes = kExpandLds<T, 4> > NR * 8192 ? kExpandLds<T, 4> : NR * 8192;
  __shared__ __align__(16) uint8_t lds[kBytes];
  const uint32_t grads = gridDim.x - expands, pairs = min(expands, grads), block = blockIdx.x;
  const bool grad = block < 2 * pairs ? block % 2 : grads > expands;
  const uint32_t number = block < 2 * pairs ? block / 2 : block - pairs;
  if (grad) adapter_grad<T, NR, SHORT>(g, number, reinterpret_cast<f32x4 (*)[8][64]>(lds));
  else expand<T, O, 4, true, SHORT>(e, number, lds);
}

// Adapters of several pieces get their sum.
__global__ __launch_bounds__(kGradThreads) void adapter_grad_sum_kernel(AdapterGradArgs a, int64_t groups) {
  const int l = (int)(blockIdx.x / groups);
  const int start = a.starts[l], pieces = grad_pieces(a.starts[l + 1] - start, a.piece);
  if (pieces <= 1) return;
  const int64_t of_a = (int64_t)a.rank * a.k, each = of_a + (int64_t)a.rank * a.n;
  const float *p = a.partial + 2 * (int64_t)(start / a.piece) * each;
  for (int64_t i = (int64_t)(blockIdx.x % groups) * kGradThreads + threadIdx.x; i < each; i += groups * kGradThreads) {
    float *to = i < of_a ? (a.da ? a.da + l * of_a + i : nullptr)
                         : (a.db ? a.db + l * (each - of_a) + (i - of_a) : nullptr);
    if (!to) continue;
    float s = 0.f;
#pragma unroll 8
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
      // -0 added to a residual leaves each as it is, a 0 loses a zero's sign
      y[e] = random.bits(e) >= a.threshold ? x[e] * a.factor : RES ? -0.f : 0.f;
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

template <typename T, bool Q, int NI, int NR, bool WT, bool SHORT>
hipError_t shrink(const ShrinkArgs &a, const ShrinkPlan &p, hipStream_t s) {
  const dim3 grid(a.tiles + (a.order ? (uint32_t)a.count : 0), (uint32_t)(p.slices * p.slots),
                  (uint32_t)((a.rank + 16 * NR - 1) / (16 * NR)));
  return launch(reinterpret_cast<const void *>(&shrink_kernel<T, Q, NI, NR, WT, SHORT>), grid, kShrinkThreads, s, a);
}
template <typename T, bool Q, int NI, bool WT>
hipError_t shrink_rank(const ShrinkArgs &a, const ShrinkPlan &p, hipStream_t s) {
  // weights take 8 registers for 16 ranks and a step, twice that next to e4m3, four
  // times in float32 next to e4m3: more would spill.  So would 64 turned ranks that
  // end inside a chunk; whole ones take 27 us for 8192 x 4096, 47 as twice 32.
  constexpr int most = Q ? (sizeof(T) == 2 && NI == 1 ? 2 : 1) : sizeof(T) == 2 ? 4 : 2;
  if constexpr (WT)
    if (a.rank < kChunk<T>) return shrink<T, Q, NI, 1, WT, true>(a, p, s);
  if (a.rank <= 16 || most == 1) return shrink<T, Q, NI, 1, WT, false>(a, p, s);
  return a.rank <= 32 || most == 2 || (WT && a.rank % 8) ? shrink<T, Q, NI, most < 2 ? 1 : 2, WT, false>(a, p, s)
                                   : shrink<T, Q, NI, most, WT, false>(a, p, s);
}
template <typename T, bool Q, bool WT>
hipError_t shrink(ShrinkArgs a, const ShrinkPlan &p, hipStream_t s) {
  constexpr int most = Q && sizeof(T) == 2 ? 2 : 1;
  const int64_t rows = 16 * std::min(p.row_tiles, most);
  a.tiles = a.h ? (uint32_t)((a.m + rows - 1) / rows) : 0;
  return p.row_tiles == 1 ? shrink_rank<T, Q, 1, WT>(a, p, s) : shrink_rank<T, Q, most, WT>(a, p, s);
}
template <typename T>
hipError_t shrink(const ShrinkArgs &a, const ShrinkPlan &p, hipStream_t s) {
  return a.turned ? shrink<T, false, true>(a, p, s) : a.scale_x ? shrink<T, true, false>(a, p, s) : shrink<T, false, false>(a, p, s);
}

// How many workgroups of a kernel run at once.
template <typename Tag>
int64_t groups_at_once(const void *kernel, int threads) {
  static std::atomic<int> at_once{0};  // of a compute unit; kept once it is known
  int n = at_once.load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) == hipSuccess && n > 0)
      at_once.store(n, std::memory_order_relaxed);
    else
      n = 1;
  }
  return 256 * (int64_t)n;
}
// Tiles of a workgroup, for as many workgroups as run at once (4001 x 8192
// bfloat16, two of a compute unit: 44 us with 8 tiles, 49 with 6, 54 with one);
// how many there are then.
uint32_t deal_out(ExpandArgs &a, const ExpandPlan &p, int64_t at_once) {
  const int64_t side = (int64_t)a.strips * a.slots, down = std::max<int64_t>(1, at_once / side);
  a.tiles = (int32_t)((p.tiles + down - 1) / down);
  return (uint32_t)((p.tiles + a.tiles - 1) / a.tiles * side);
}

template <typename T, typename O, int WR, bool WT, bool SHORT>
hipError_t expand(ExpandArgs a, const ExpandPlan &p, hipStream_t s) {
  struct Tag;
  const void *kernel = reinterpret_cast<const void *>(&expand_kernel<T, O, WR, WT, SHORT>);
  const uint32_t groups = deal_out(a, p, groups_at_once<Tag>(kernel, kExpandThreads));
  return launch(kernel, dim3(groups), kExpandThreads, s, a);
}
template <typename T, typename O, bool WT, bool SHORT>
hipError_t expand(const ExpandArgs &a, const ExpandPlan &p, hipStream_t s) {
  return p.waves_down == 4 ? expand<T, O, 4, WT, SHORT>(a, p, s) : expand<T, O, 2, WT, SHORT>(a, p, s);
}
template <typename T, typename O, bool WT>
hipError_t expand(const ExpandArgs &a, const ExpandPlan &p, hipStream_t s) {
  // shorter than a load: of base, of h and w's ranks or columns
  return a.n < 8 || a.rank < 8 ? expand<T, O, WT, true>(a, p, s) : expand<T, O, WT, false>(a, p, s);
}
template <typename T, typename O>
hipError_t expand(const ExpandArgs &a, const ExpandPlan &p, hipStream_t s) {
  return a.turned ? expand<T, O, true>(a, p, s) : expand<T, O, false>(a, p, s);
}

// The gradients' launch: its workgroups, columns of tiles and operands.
struct GradGrid {
  uint32_t groups, chunks;
  int nr;
  bool narrow;  // columns shorter than a load
};
GradGrid grad_grid(AdapterGradArgs &a, bool wide) {
  a.tiles_k = a.da ? (int)((a.k + kGradCols - 1) / kGradCols) : 0;
  a.tiles = a.tiles_k + (a.db ? (int)((a.n + kGradCols - 1) / kGradCols) : 0);
  GradGrid g{};
  g.nr = a.rank <= 16 ? 1 : a.rank <= 32 || !wide ? 2 : 4;
  g.groups = (uint32_t)((a.m / a.piece + a.count) * a.tiles);
  g.chunks = (uint32_t)((a.rank + 16 * g.nr - 1) / (16 * g.nr));
  g.narrow = (a.da && a.k < 8) || (a.db && a.n < 8);
  return g;
}
hipError_t grad_sum(const AdapterGradArgs &a, hipStream_t s) {
  if (a.m <= a.piece) return hipSuccess;  // no adapter has two pieces
  const int64_t values = (int64_t)a.rank * (a.k + a.n), most = 4096 / a.count + 1;
  const int64_t groups = std::min((values + kGradThreads - 1) / kGradThreads, most);
  return launch(reinterpret_cast<const void *>(&adapter_grad_sum_kernel), dim3((uint32_t)(groups * a.count)),
                kGradThreads, s, a, groups);
}
template <typename T, bool SHORT>
hipError_t grad(const AdapterGradArgs &a, const GradGrid &g, hipStream_t s) {
  constexpr int most = kGradSplit<T> ? 4 : 2;
  const void *kernel = g.nr == 1   ? reinterpret_cast<const void *>(&adapter_grad_kernel<T, 1, SHORT>)
                       : g.nr == 2 ? reinterpret_cast<const void *>(&adapter_grad_kernel<T, 2, SHORT>)
                                   : reinterpret_cast<const void *>(&adapter_grad_kernel<T, most, SHORT>);
  return launch(kernel, dim3(g.groups, g.chunks), kGradThreads, s, a);
}
template <typename T>
hipError_t grad(AdapterGradArgs a, hipStream_t s) {
  const GradGrid g = grad_grid(a, kGradSplit<T>);
  if (g.groups == 0) return hipSuccess;
  const hipError_t e = g.narrow ? grad<T, true>(a, g, s) : grad<T, false>(a, g, s);
  return e == hipSuccess ? grad_sum(a, s) : e;
}

template <typename T, typename O, int NR, bool SHORT>
hipError_t both(ExpandArgs e, const ExpandPlan &p, const AdapterGradArgs &a, const GradGrid &g, hipStream_t s) {
  struct Tag;
  const void *kernel = reinterpret_cast<const void *>(&adapter_both_kernel<T, O, NR, SHORT>);
  const uint32_t expands = deal_out(e, p, groups_at_once<Tag>(kernel, kGradThreads));
  return launch(kernel, dim3(expands + g.groups), kGradThreads, s, e, a, expands);  // all ranks in one chunk
}
template <typename T, typename O, bool SHORT>
hipError_t both(const ExpandArgs &e, const ExpandPlan &p, const AdapterGradArgs &a, const GradGrid &g, hipStream_t s) {
  return g.nr == 1 ? both<T, O, 1, SHORT>(e, p, a, g, s) : both<T, O, 2, SHORT>(e, p, a, g, s);
}
template <typename T, typename O>
hipError_t both(const ExpandArgs &e, const ExpandPlan &p, AdapterGradArgs a, hipStream_t s) {
  const GradGrid g = grad_grid(a, false);
  const hipError_t err = g.narrow || e.n < 8 || e.rank < 8 ? both<T, O, true>(e, p, a, g, s) : both<T, O, false>(e, p, a, g, s);
  return err == hipSuccess ? grad_sum(a, s) : err;
}

}  // namespace

ShrinkPlan shrink_plan(int64_t m, int64_t k, int64_t rank, int64_t count, int x_size, bool whole) {
  ShrinkPlan p{};
  // e4m3 rows take twice their bytes of weights: 32 of them a workgroup from where
  // those still fill the card (4096 columns, rank 16, 8192 rows 18.5 and 23 us,
  // 16384 rows 32 and 40; but bfloat16 25 and 24, 5000 rows 25 and 21).  Over 16
  // ranks, of which 16 rows take 32 at a time and read x half as often, it makes little
  // difference (both launches, 8192 rows, 4096 columns both ways, rank 32 54 us, 53
  // with 16 rows, rank 64 77 both, rank 128 125 and 128).
  p.row_tiles = x_size == 1 && m > 4096 ? 2 : 1;
  const int64_t tiles = (m + 16 * p.row_tiles - 1) / (16 * p.row_tiles);
  // Few tiles: their adapters (16 of a tile at most) side by side, up to a
  // workgroup each, and the columns in up to four slices, which `expand` adds up
  // (16 rows of 16 adapters, 4096 columns, both launches: 24 us with one slot, 14.5
  // with 4, 12 with 16; then 12.8 with one slice, 11.9 with 2, 11.7 with 4).
  const int64_t adapters = std::min<int64_t>(std::min<int64_t>(m, 16), count);
  p.slots = 1;
  while (p.slots < adapters && tiles * p.slots < 64) p.slots *= 2;
  const int64_t columns = 128 / x_size, steps = std::max<int64_t>(1, (k + columns - 1) / columns);
  const int64_t room = whole ? 1 : std::max<int64_t>(1, 256 / (tiles * p.slots));
  const int64_t slices = std::min(std::min<int64_t>(4, room), (steps + kShrinkWaves - 1) / kShrinkWaves);
  p.steps_per_slice = (int)((steps + slices - 1) / slices);
  p.slices = (int)((steps + p.steps_per_slice - 1) / p.steps_per_slice);
  return p;
}
hipError_t launch_shrink(const ShrinkArgs &a, const ShrinkPlan &p, int dtype, hipStream_t s) {
  return dtype == XPOSE_F32 ? shrink<float>(a, p, s) : dtype == XPOSE_F16 ? shrink<_Float16>(a, p, s) : shrink<__bf16>(a, p, s);
}

ExpandPlan expand_plan(int64_t m, int64_t n, int64_t count, bool beside) {
  ExpandPlan p{};
  // Few rows leave waves down without any, but share h among fewer workgroups: 16
  // tokens beside e4m3 10.6 us a call with 2, 11.1 with 1 and 11.3 with 4 (4096
  // columns both ways).  More rows share an adapter's operands among 4.  But of many
  // adapters a tile of 64 rows goes through more than one of 32 does (bfloat16, 2048 to
  // 4096 columns, rank 16: 32 adapters of 64 rows 14.3 us, 11.9 with 2, 64 rows with one
  // each 21.1 and 16.0, 256 of 512 rows 53.9 and 37.6; 16 of 64 rows in any order 11.8
  // and 12.2).  How many of them have rows is not known here: 512 rows of one take 10.5
  // us, 10.8 with 2, and so may prompts, which have more rows and few adapters (4000
  // rows of 8 in order 5% more with 2; 4000 of 32 in any order 8% less).
  p.waves_down = beside || (m > 16 && (m > 512 || count < 32)) ? 4 : 2;
  const int rows = 16 * p.waves_down, cols = kExpandCols * kExpandWaves / p.waves_down;
  p.strips = (n + cols - 1) / cols;
  p.tiles = (m + rows - 1) / rows;
  // side by side as in shrink_plan; a tile's rows have so many adapters at most
  const int64_t adapters = std::min(std::min(m, (int64_t)rows), count);
  p.slots = 1;
  while (p.slots < adapters && p.tiles * p.strips * p.slots < 256) p.slots *= 2;
  return p;
}
hipError_t launch_expand(const ExpandArgs &a, const ExpandPlan &p, int dtype, int out_dtype, hipStream_t s) {
  if (dtype == XPOSE_F32) return expand<float, float>(a, p, s);
  if (dtype == XPOSE_F16)
    return out_dtype == XPOSE_F32 ? expand<_Float16, float>(a, p, s) : expand<_Float16, _Float16>(a, p, s);
  return out_dtype == XPOSE_F32 ? expand<__bf16, float>(a, p, s) : expand<__bf16, __bf16>(a, p, s);
}

int adapter_grad_piece(int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = (n + kGradCols - 1) / kGradCols + (k + kGradCols - 1) / kGradCols;
  // One piece an adapter, no second launch: bfloat16, 4096 columns both ways, rank 12,
  // 200 to 512 rows 15 to 17.6 us a pass, 19 to 23 with pieces of 128 rows, rank 64 38
  // to 43 and 43 to 46; but one adapter of 400 float32 rows, 2999 and 1222, 27.3 and 24.4.
  if (m <= 512) return 512;
  // a workgroup a compute unit, next to the other kernel's (8192 rows, 4096 columns
  // both ways, bfloat16: 128 rows a piece 130 us, 256 101, 512 92, 1024 85, 2048 82,
  // 4096 83; 2048 rows in float32: 128 55 us, 512 45, 2048 44)
  int piece = 128;
  while (piece < 4096 && m / piece * tiles > 256) piece *= 2;
  return piece;
}
int64_t adapter_grad_slots(int64_t m, int piece) { return m > piece ? 2 * (m / piece + 1) : 0; }
hipError_t launch_adapter_both(const ExpandArgs &e, const ExpandPlan &p, const AdapterGradArgs &a, int dtype,
                               int dx_dtype, hipStream_t s) {
  if (dtype == XPOSE_F32) return both<float, float>(e, p, a, s);
  if (dtype == XPOSE_F16)
    return dx_dtype == XPOSE_F32 ? both<_Float16, float>(e, p, a, s) : both<_Float16, _Float16>(e, p, a, s);
  return dx_dtype == XPOSE_F32 ? both<__bf16, float>(e, p, a, s) : both<__bf16, __bf16>(e, p, a, s);
}
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
  // A row a lane and short workgroups, which go through memory in order: 8192 x
  // 8192 bfloat16 with the residual takes 71 us, 77 where 4096 workgroups stay,
  // float32 134 and 146 (100000 x 128 bfloat16 14.3 and 14.4).
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(65535, ((int64_t)1 << 24) / wide - 1));
  const int64_t groups = std::min((a.rows + at_once - 1) / at_once, most);
  const dim3 grid((uint32_t)wide, (uint32_t)groups);
  return dtype == XPOSE_F32 ? dropout<float>(a, grid, s) : dtype == XPOSE_F16 ? dropout<_Float16>(a, grid, s) : dropout<__bf16>(a, grid, s);
}

}  // namespace xpose
