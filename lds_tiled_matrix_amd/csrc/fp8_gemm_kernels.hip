// gfx950 kernels of the matrix product in 8-bit floating point with a scale
// for each block of 128, c = a b^T.
//
// v_mfma_f32_16x16x128_f8f6f4 takes one whole block of 128 products of 16 x
// 16 outputs: it starts from zero, and its float32 result is then scaled by
// scale_a scale_b into the sum (kFp8Rows, kFp8Tiles: one multiply-add an
// output and block; with a scale of b for each row a multiplication more).
// Scales that are powers of two go into the instruction itself, which adds
// straight to the sum (kFp8Pow2).
//
// Precision.  The 8-bit instructions sum each 8 neighbouring products with
// what lies under 2^-13 of the largest one's leading bit cut off (measured:
// 2^16 + 2^2 gives 2^16 with both among the 8, and is exact with the other 8
// or more away; 1.4e-5 of the result's norm on normal data, however long the
// sum; v_mfma_f32_16x16x32_fp8_fp8 does the same).  That is under 1% of the
// rounding of a 16-bit result, and taken there.  A float32 result would lose
// by it: there (EXACT) both operands are widened to bfloat16, which holds
// every e4m3 value, and v_mfma_f32_16x16x32_bf16 multiplies them at half the
// rate, with 4e-8 to 2e-7 of the norm on the same data.  Powers of two are
// then scaled by like other scales.
//
// b's rows are the instruction's first operand, so a lane's four results are
// neighbours in a row of c.  Which 128 bytes of a row are which of the
// instruction's 128 k does not matter, as long as both operands agree: a lane
// of group g = lane / 16 takes the 16-byte chunks g and g + 4.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/linear/xpose_linear.h"
#include "linear_device.h"
#include "linear_kernels.h"

namespace xpose {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;

// 32 of a row's 128 values, as the matrix cores take them.
template <bool EXACT> struct Lane32;
template <> struct Lane32<false> {
  i32x8 v;
  __device__ void set(u32x4 lo, u32x4 hi) {
    v = i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
              (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  }
};
template <> struct Lane32<true> {
  bf16x8 v[4];
  __device__ void set(u32x4 lo, u32x4 hi) {
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const uint32_t bytes = w < 4 ? lo[w % 4] : hi[w % 4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bf16x2 r = h ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 1.f, true)
                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 1.f, false);
        v[w / 2][w % 2 * 4 + 2 * h] = r[0];
        v[w / 2][w % 2 * 4 + 2 * h + 1] = r[1];
      }
    }
  }
};

// A float32 power of two as the 8 exponent bits that the instruction takes
// (inf and NaN become its NaN: blocks that have one hold no number but 0).
__device__ inline int exponent_of(float scale) {
  return (int)(__float_as_uint(scale) >> 23);
}

__device__ inline f32x4 multiply(const Lane32<false> &b, const Lane32<false> &a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      b.v, a.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ inline f32x4 multiply(const Lane32<true> &b, const Lane32<true> &a) {
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s)
    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[s], a.v[s], sum, 0, 0, 0);
  return sum;
}
__device__ inline f32x4 multiply(const Lane32<false> &b, const Lane32<false> &a, f32x4 sum,
                                 int exp_b, int exp_a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, sum, 0, 0, 0, exp_b, 0, exp_a);
}

// The 16 bytes at p of which `valid` (may be out of 0..16) exist; zeros else.
__device__ inline u32x4 load_chunk(const uint8_t *p, int64_t valid) {
  if (valid >= 16) return *reinterpret_cast<const u32x4 *>(p);
  u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e < valid) w[e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
  return w;
}

// COUNT neighbours of a row of c, of which the first `valid` exist.
template <typename T, int COUNT>
__device__ inline void store_run(T *p, int64_t valid, const float *f) {
  typedef T run_any __attribute__((ext_vector_type(COUNT), aligned(sizeof(T))));
  if (valid >= COUNT) {
    run_any r;
#pragma unroll
    for (int e = 0; e < COUNT; ++e) r[e] = (T)f[e];
    *reinterpret_cast<run_any *>(p) = r;
  } else {
#pragma unroll
    for (int e = 0; e < COUNT; ++e)
      if (e < valid) p[e] = (T)f[e];
  }
}
template <int COUNT>
__device__ inline void store_run(void *c, int out, int64_t at, int64_t valid, const float *f) {
  if (out == XPOSE_F32) {
#pragma unroll
    for (int e = 0; e < COUNT; e += 4) store_run<float, 4>((float *)c + at + e, valid - e, f + e);
  } else if (out == XPOSE_F16) {
#pragma unroll
    for (int e = 0; e < COUNT; e += 8)
      store_run<_Float16, COUNT < 8 ? COUNT : 8>((_Float16 *)c + at + e, valid - e, f + e);
  } else {
#pragma unroll
    for (int e = 0; e < COUNT; e += 8)
      store_run<__bf16, COUNT < 8 ? COUNT : 8>((__bf16 *)c + at + e, valid - e, f + e);
  }
}

__device__ inline void to_lds16(const uint8_t *from, uint8_t *to) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void *)from,
      (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}
__device__ inline void to_lds4(const float *from, float *to) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void *)from,
      (__attribute__((address_space(3))) void *)to, 4, 0, 0);
}

// ----- tiles -------------------------------------------------------------------
//
// A workgroup has TM x TN outputs, a wave WM x WN of them.  Blocks of 128 k go
// to LDS by direct 16-byte loads (8 lanes a row), two buffers in turn: the next
// block's loads are under way while this one is multiplied, one barrier a
// block.  A row's 8 chunks are permuted by an exclusive or with three bits of
// the row that differ among the 16 rows of one operand read (of a parity), so
// that those 16 lanes' 16-byte reads cover all 64 banks.
//
// b's rows of one operand: lane l has row 16 (l / 4) + 4 j + l % 4 of the
// wave's 64, so that over j a lane's results are 16 neighbours in c.
//
// Scales of a block go to LDS too: of a, a wave's in the order [l][i] (a lane
// reads its WM / 16 with few wide reads); of b in the rows' order, or for
// kFp8Pow2 in [l][j].
template <int TM, int TN, int WM>
struct Tile {
  static constexpr int WN = 64;
  static constexpr int NI = WM / 16, NJ = WN / 16;
  static constexpr int WAVES = (TM / WM) * (TN / WN), THREADS = 64 * WAVES;
  static constexpr int A = 0, B = TM * kBlock, SA = B + TN * kBlock,
                       SB = SA + 4 * TM, BYTES = SB + 4 * TN;
  static_assert(TM + TN <= THREADS && TM % 64 == 0 && TN % 64 == 0);
  static_assert(TM % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0);
};

__device__ inline int swizzle_a(int row) { return (row >> 1) & 7; }
__device__ inline int swizzle_b(int row) { return ((row >> 1) & 1) | ((row >> 3) & 6); }

template <int TM, int TN, int WM, Fp8GemmMode MODE, bool EXACT>
__global__ __launch_bounds__((Tile<TM, TN, WM>::THREADS)) void fp8_tile_kernel(Fp8GemmArgs p) {
  using T = Tile<TM, TN, WM>;
  __shared__ __align__(16) uint8_t lds[2][T::BYTES];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int l16 = lane % 16, g = lane / 16;
  const int wm = wave % (TM / WM) * WM, wn = wave / (TM / WM) * T::WN;

  uint32_t id = blockIdx.x;
  const uint32_t tiles = p.tiles_m * p.tiles_n;
  const int split = (int)(id / tiles);
  id %= tiles;
  const int64_t m0 = (int64_t)(id % p.tiles_m) * TM, n0 = (int64_t)(id / p.tiles_m) * TN;

  // this slice's blocks: whole ones from `first` on, and maybe the ragged last
  const int64_t whole = p.k / kBlock, tail = p.k % kBlock;
  const int64_t first = (int64_t)split * p.blocks_per_split;
  int64_t last = first + p.blocks_per_split;
  const bool ragged = tail && last > whole;
  if (last > whole) last = whole;
  const int steps = (int)(last - first) + ragged;

  // Every load is of a row that exists: rows beyond the matrix are its last
  // one again, and their results are not stored.
  const uint8_t *a0 = p.a + m0 * p.lda, *b0 = p.b + n0 * p.ldb;
  const int rows_a = (int)(p.m - m0 < TM ? p.m - m0 : TM) - 1;
  const int rows_b = (int)(p.n - n0 < TN ? p.n - n0 : TN) - 1;
  constexpr int LA = TM / (8 * T::WAVES), LB = TN / (8 * T::WAVES);
  uint32_t off_a[LA], off_b[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int row = (i * T::WAVES + wave) * 8 + lane / 8;
    off_a[i] = (uint32_t)min(row, rows_a) * (uint32_t)p.lda + ((lane % 8) ^ swizzle_a(row)) * 16;
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int row = (i * T::WAVES + wave) * 8 + lane / 8;
    off_b[i] = (uint32_t)min(row, rows_b) * (uint32_t)p.ldb + ((lane % 8) ^ swizzle_b(row)) * 16;
  }
  // The scale that this lane brings to LDS: threads below TM one of a's, the
  // next TN one of b's.
  const float *scale = nullptr;
  int64_t scale_step = 0;
  if (tid < TM) {
    const int strip = tid / WM, at = tid % WM;
    const int row = strip * WM + at % T::NI * 16 + at / T::NI;
    scale = p.scale_a + m0 + min(row, rows_a);
    scale_step = p.ld_scale_a;
  } else if (tid < TM + TN) {
    int row = tid - TM;
    if (MODE == kFp8Pow2) {
      const int l = row % 64 / 4, j = row % 4;
      row = row / 64 * 64 + l / 4 * 16 + j * 4 + l % 4;
    }
    scale = p.scale_b + ((n0 + min(row, rows_b)) >> p.b_shift);
    scale_step = p.ld_scale_b;
  }

  auto stage_scales = [&](int64_t kb, uint8_t *buf) {
    if (tid < TM + TN)  // whole waves
      to_lds4(scale + kb * scale_step, (float *)(buf + T::SA) + wave * 64);
  };
  auto stage = [&](int64_t kb, uint8_t *buf) {
    const uint8_t *a = a0 + kb * kBlock, *b = b0 + kb * kBlock;
#pragma unroll
    for (int i = 0; i < LA; ++i) to_lds16(a + off_a[i], buf + T::A + (i * T::WAVES + wave) * 1024);
#pragma unroll
    for (int i = 0; i < LB; ++i) to_lds16(b + off_b[i], buf + T::B + (i * T::WAVES + wave) * 1024);
    stage_scales(kb, buf);
  };
  // The last block of k with fewer than 128 columns, the rest as zeros: what
  // lies between k and the pitch may be anything, or no memory at all.
  auto stage_ragged = [&](uint8_t *buf) {
    const uint8_t *a = a0 + whole * kBlock, *b = b0 + whole * kBlock;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int row = (i * T::WAVES + wave) * 8 + lane / 8;
      const int at = ((lane % 8) ^ swizzle_a(row)) * 16;
      *reinterpret_cast<u32x4 *>(buf + T::A + (i * T::WAVES + wave) * 1024 + lane * 16) =
          load_chunk(a + off_a[i], tail - at);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int row = (i * T::WAVES + wave) * 8 + lane / 8;
      const int at = ((lane % 8) ^ swizzle_b(row)) * 16;
      *reinterpret_cast<u32x4 *>(buf + T::B + (i * T::WAVES + wave) * 1024 + lane * 16) =
          load_chunk(b + off_b[i], tail - at);
    }
    stage_scales(whole, buf);
  };

  f32x4 acc[T::NI][T::NJ];
#pragma unroll
  for (int i = 0; i < T::NI; ++i)
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int row_b = wn + l16 / 4 * 16 + l16 % 4;  // + 4 j
  auto chunk = [&](const uint8_t *base, int row, int swizzle) {
    const u32x4 *r = reinterpret_cast<const u32x4 *>(base + row * kBlock);
    Lane32<EXACT> v;
    v.set(r[g ^ swizzle], r[(g + 4) ^ swizzle]);
    return v;
  };
  auto compute = [&](const uint8_t *buf) {
    const float *sa = (const float *)(buf + T::SA) + wm + l16 * T::NI;
    const float *sb = (const float *)(buf + T::SB) + wn;
    Lane32<EXACT> b[T::NJ];
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) b[j] = chunk(buf + T::B, row_b + 4 * j, swizzle_b(row_b + 4 * j));
    f32x4 sbj[T::NJ];
    int eb[T::NJ];
    float sb1 = 0.f;
    if constexpr (MODE == kFp8Pow2) {
#pragma unroll
      for (int j = 0; j < T::NJ; ++j) eb[j] = exponent_of(sb[l16 * 4 + j]);
    } else if constexpr (MODE == kFp8Rows) {
#pragma unroll
      for (int j = 0; j < T::NJ; ++j) sbj[j] = *reinterpret_cast<const f32x4 *>(sb + g * 16 + 4 * j);
    } else {
      sb1 = sb[0];  // 64 columns of one 128-block
    }
#pragma unroll
    for (int i = 0; i < T::NI; ++i) {
      const int row = wm + 16 * i + l16;
      const Lane32<EXACT> a = chunk(buf + T::A, row, swizzle_a(row));
      if constexpr (MODE == kFp8Pow2) {
        const int ea = exponent_of(sa[i]);
#pragma unroll
        for (int j = 0; j < T::NJ; ++j) acc[i][j] = multiply(b[j], a, acc[i][j], eb[j], ea);
      } else {
        const float s1 = MODE == kFp8Tiles ? sa[i] * sb1 : sa[i];
#pragma unroll
        for (int j = 0; j < T::NJ; ++j) {
          const f32x4 v = multiply(b[j], a);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] = __builtin_fmaf(v[e], MODE == kFp8Rows ? s1 * sbj[j][e] : s1, acc[i][j][e]);
        }
      }
    }
  };

  // The ragged block goes first: nothing is under way yet that its loads
  // through registers would hold up.
  if (steps > 0) {
    if (ragged) stage_ragged(lds[0]); else stage(first, lds[0]);
  }
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    if (s + 1 < steps) stage(first + s + 1 - ragged, lds[(s + 1) & 1]);
    compute(lds[s & 1]);
    __syncthreads();
  }

  uint8_t *c = (uint8_t *)p.c + (int64_t)split * p.slice * 4;  // slices are float32
  const int64_t col = n0 + wn + 16 * g;
#pragma unroll
  for (int i = 0; i < T::NI; ++i) {
    const int64_t row = m0 + wm + 16 * i + l16;
    if (row >= p.m || col >= p.n) continue;
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = acc[i][e / 4][e % 4];
    store_run<16>(c, p.out, row * p.ldc + col, p.n - col, f);
  }
}

template <int TM, int TN, int WM, bool EXACT>
hipError_t launch_tile(const Fp8GemmArgs &a, Fp8GemmMode mode, hipStream_t s) {
  Fp8GemmArgs copy = a;
  void *args[] = {&copy};
  const void *kernel =
      mode == kFp8Rows ? reinterpret_cast<const void *>(&fp8_tile_kernel<TM, TN, WM, kFp8Rows, EXACT>)
                       : reinterpret_cast<const void *>(&fp8_tile_kernel<TM, TN, WM, kFp8Tiles, EXACT>);
  if constexpr (!EXACT)
    if (mode == kFp8Pow2)
      kernel = reinterpret_cast<const void *>(&fp8_tile_kernel<TM, TN, WM, kFp8Pow2, false>);
  return hipLaunchKernel(kernel, dim3(a.tiles_m * a.tiles_n * a.splits),
                         dim3(Tile<TM, TN, WM>::THREADS), args, 0, s);
}

// ----- few rows of a -------------------------------------------------------------
//
// Serving: reading b bounds it.  A workgroup has 16 rows of b and up to 16 MS
// of a; its waves take the blocks of k in turn, straight from memory into the
// instruction's registers, four at a time, and their sums are added through
// LDS in the waves' order.
constexpr int kSkinnyWaves = 8;

template <int MS, bool EXACT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void fp8_skinny_kernel(Fp8GemmArgs p) {
  constexpr int kDepth = MS > 2 ? 2 : 4;
  __shared__ __align__(16) float sums[kSkinnyWaves][MS][64][4];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int l16 = lane % 16, g = lane / 16;
  const int64_t n0 = (int64_t)(blockIdx.x % p.tiles_n) * 16;
  const int64_t m0 = (int64_t)(blockIdx.x / p.tiles_n) * 16 * MS;
  const int64_t blocks = (p.k + kBlock - 1) / kBlock;

  const int64_t brow = n0 + l16 < p.n ? n0 + l16 : p.n - 1;
  const uint8_t *b = p.b + brow * p.ldb + g * 16;
  const uint8_t *a[MS];
  const float *sa[MS];
  const float *sb[4];
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    const int64_t row = m0 + 16 * i + l16 < p.m ? m0 + 16 * i + l16 : p.m - 1;
    a[i] = p.a + row * p.lda + g * 16;
    sa[i] = p.scale_a + row;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t row = n0 + 4 * g + e < p.n ? n0 + 4 * g + e : p.n - 1;
    sb[e] = p.scale_b + (row >> p.b_shift);
  }

  f32x4 acc[MS];
#pragma unroll
  for (int i = 0; i < MS; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t kb0 = wave; kb0 < blocks; kb0 += kSkinnyWaves * kDepth) {
    u32x4 bv[kDepth][2], av[kDepth][MS][2];
    float sav[kDepth][MS], sbv[kDepth][4];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int64_t kb = kb0 + d * kSkinnyWaves;
      const int64_t left = kb < blocks ? p.k - kb * kBlock - g * 16 : 0;  // 0: zeros
      bv[d][0] = load_chunk(b + kb * kBlock, left);
      bv[d][1] = load_chunk(b + kb * kBlock + 64, left - 64);
      const int64_t ks = kb < blocks ? kb : blocks - 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) sbv[d][e] = sb[e][ks * p.ld_scale_b];
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        av[d][i][0] = load_chunk(a[i] + kb * kBlock, left);
        av[d][i][1] = load_chunk(a[i] + kb * kBlock + 64, left - 64);
        sav[d][i] = sa[i][ks * p.ld_scale_a];
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (kb0 + d * kSkinnyWaves >= blocks) break;
      Lane32<EXACT> bl;
      bl.set(bv[d][0], bv[d][1]);
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        Lane32<EXACT> al;
        al.set(av[d][i][0], av[d][i][1]);
        const f32x4 v = multiply(bl, al);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][e] = __builtin_fmaf(v[e], sav[d][i] * sbv[d][e], acc[i][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MS; ++i) *reinterpret_cast<f32x4 *>(sums[wave][i][lane]) = acc[i];
  __syncthreads();
  // MS * 64 lanes have four neighbours of a row each
  if (tid < MS * 64) {
    const int i = tid / 64;
    f32x4 s = *reinterpret_cast<const f32x4 *>(sums[0][i][lane]);
#pragma unroll
    for (int w = 1; w < kSkinnyWaves; ++w) s += *reinterpret_cast<const f32x4 *>(sums[w][i][lane]);
    const int64_t row = m0 + 16 * i + l16, col = n0 + 4 * g;
    if (row < p.m && col < p.n) {
      const float f[4] = {s[0], s[1], s[2], s[3]};
      store_run<4>(p.c, p.out, row * p.ldc + col, p.n - col, f);
    }
  }
}

template <int MS, bool EXACT>
hipError_t launch_skinny(const Fp8GemmArgs &a, Fp8GemmMode, hipStream_t s) {
  Fp8GemmArgs copy = a;
  void *args[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void *>(&fp8_skinny_kernel<MS, EXACT>),
                         dim3(a.tiles_m * a.tiles_n), dim3(64 * kSkinnyWaves), args, 0, s);
}

template <int TM, int TN, int WM, bool EXACT>
constexpr Fp8GemmKernel tile_kernel() {
  return {TM, TN, Tile<TM, TN, WM>::THREADS, false, EXACT, &launch_tile<TM, TN, WM, EXACT>};
}
template <int MS, bool EXACT>
constexpr Fp8GemmKernel skinny_kernel() {
  return {16 * MS, 16, 64 * kSkinnyWaves, true, EXACT, &launch_skinny<MS, EXACT>};
}
const Fp8GemmKernel kKernels[] = {
    skinny_kernel<1, false>(), skinny_kernel<2, false>(), skinny_kernel<4, false>(),
    skinny_kernel<1, true>(), skinny_kernel<2, true>(), skinny_kernel<4, true>(),
    tile_kernel<256, 256, 128, false>(), tile_kernel<128, 128, 64, false>(),
    tile_kernel<128, 128, 64, true>(),
};

// ----- the sum over slices of k ------------------------------------------------------

__global__ __launch_bounds__(256) void fp8_reduce_kernel(Fp8ReduceArgs r) {
  const int64_t per_row = (r.n + 3) / 4, plane = r.m * r.n;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < r.m * per_row; v += step) {
    const int64_t i = v / per_row, j = (v - i * per_row) * 4, valid = r.n - j;
    const float *p = r.partial + i * r.n + j;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (valid >= 4) {
#pragma unroll 4
      for (int z = 0; z < r.splits; ++z) {
        const f32x4 t = *reinterpret_cast<const f32x4_any *>(p + z * plane);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] += t[e];
      }
    } else {
      for (int z = 0; z < r.splits; ++z)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < valid) f[e] += p[z * plane + e];
    }
    store_run<4>(r.c, r.out, i * r.ldc + j, valid, f);
  }
}

}  // namespace

const Fp8GemmKernel *fp8_gemm_kernels(int *count) {
  *count = (int)(sizeof kKernels / sizeof kKernels[0]);
  return kKernels;
}

hipError_t launch_fp8_reduce(const Fp8ReduceArgs &r, hipStream_t s) {
  Fp8ReduceArgs copy = r;
  void *args[] = {&copy};
  int64_t grid = (r.m * ((r.n + 3) / 4) + 255) / 256;
  if (grid > 8192) grid = 8192;
  return hipLaunchKernel(reinterpret_cast<const void *>(&fp8_reduce_kernel),
                         dim3((uint32_t)grid), dim3(256), args, 0, s);
}

}  // namespace xpose
