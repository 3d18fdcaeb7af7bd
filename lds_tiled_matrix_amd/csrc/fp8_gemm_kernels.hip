// gfx950 kernels of the matrix product in 8-bit floating point with a scale
// for each block of 128, c = a b^T.
//
// v_mfma_f32_16x16x128_f8f6f4 takes one whole block of 128 products of 16 x
// 16 outputs: it starts from zero, and its float32 result is then scaled by
// scale_a scale_b into the sum (kFp8Tiles: one multiply-add an output and block;
// kFp8Rows, with a scale of b for each row: a multiplication more).
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
// Scales.  The product of two scales may leave float32's range where the result
// does not (2^-70 and 2^-70 next to sums of 2^20, or 2^70 and 2^70 next to a sum
// of 0), so it is not formed: a block's result takes one scale after the other.
// A scale of b that holds for all of a wave's columns (kFp8Tiles) has its power
// of two applied by the instruction, or in the widening, and the rest goes to
// a's scale, for one multiply-add an output still (with another multiplication
// 4096^3 took 73 instead of 68 us, 8192^3 531 instead of 487).
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
  __device__ void set(u32x4 lo, u32x4 hi, float = 1.f) {
    v = i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
              (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  }
};
template <> struct Lane32<true> {
  bf16x8 v[4];
  // `power`, of two, is multiplied by.
  __device__ void set(u32x4 lo, u32x4 hi, float power = 1.f) {
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const uint32_t bytes = w < 4 ? lo[w % 4] : hi[w % 4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bf16x2 r = h ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, power, true)
                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, power, false);
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

// A scale, the same in all lanes of a wave, as a power of two and the rest, of
// magnitude 1 to 2.  What has no such power (zeros and what lies under float32's
// normal numbers, inf, NaN) is rest.
struct SplitScale {
  float power, rest;
  __device__ explicit SplitScale(float scale) {
    const uint32_t bits = (uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(scale));
    const uint32_t exponent = bits & 0x7f800000u;
    const bool none = exponent == 0 || exponent == 0x7f800000u;
    power = none ? 1.f : __uint_as_float(exponent);
    rest = __uint_as_float(none ? bits : (bits & 0x807fffffu) | 0x3f800000u);
  }
};

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

// The 16 bytes at p of which `valid` (may be out of 0..16) exist, zeros for the
// rest, without a branch: what does not exist at all is read from `some`, 16
// bytes that do, and a chunk that holds a row's end is read whole (it lies
// within one 16-byte line of memory with that end) and cut by keep().  Byte by
// byte, the one ragged block of 1000 x 2999 x 12345 took 30 of 150 us.
__device__ inline u32x4 load_chunk(const uint8_t *p, int64_t valid, const uint8_t *some) {
  return *reinterpret_cast<const u32x4 *>(valid > 0 ? p : some);
}
__device__ inline u32x4 keep(u32x4 w, int64_t valid) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int64_t left = valid - 4 * d;
    const uint32_t mask = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * (int)left)) - 1;
    w[d] &= mask;
  }
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

// Direct loads to LDS: 16 (4) bytes a lane, from base + offset + step, to
// `to` and on, lane by lane; zeros where the offset is `bytes` or more.  The
// buffer descriptor and the step are scalars, so a lane keeps 32 bits of
// address for all of its loads of a tile.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ inline Buffer buffer(const void *base, int64_t bytes) {
  const int64_t most = 0xffffffff;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0,
                                           (int)(uint32_t)(bytes < 0 ? 0 : bytes < most ? bytes : most),
                                           0x00020000);
}
__device__ inline void to_lds16(Buffer from, uint32_t offset, uint32_t step, void *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16,
                                           (int)offset, (int)step, 0, 0);
}
__device__ inline void to_lds4(Buffer from, uint32_t offset, void *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 4,
                                           (int)offset, 0, 0, 0);
}

// Waits until no more than LATER of this wave's loads to LDS are under way (they
// end in their order) and its reads of LDS are done, then for all waves: what
// any of them loaded before those, and read, is in place or done with after.
template <int LATER>
__device__ inline void loads_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(LATER) : "memory");
}
// Only the reads: loads stay under way.
__device__ inline void reads_and_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

// ----- tiles -------------------------------------------------------------------
//
// A workgroup has TM x TN outputs, a wave WM x 64 of them.  Blocks of 128 k go
// to LDS by direct 16-byte loads (8 lanes a row), two buffers in turn.  A row's
// 8 chunks are permuted by an exclusive or with bits 1 to 3 of its place, so
// that the 16-byte reads of an operand's 16 rows cover all 64 banks.
//
// The matrix cores never wait for LDS: a wave holds the operands of a's rows
// for a whole block and takes b's 16 rows at a time, the next 16 on the way.
// Once all waves have a's operands, its half of the buffer begins to be loaded
// with the block after the next; b's half once they have b's last 16 rows, and
// then a's operands of the next block come in while the last products use up
// this one's.  So two barriers a block, and one to one and a half blocks' time
// for a load to arrive (with one barrier and one block's time, the loads that
// miss the L2 cache held up every block).
//
// What bounds it: at 256 x 256 a block of k reads 192 KiB of LDS and writes 64,
// which at 128 bytes a cycle are the 2,048 cycles of its products, so both are
// near full; 8192^3 takes 410 to 420 us with powers of two (2.6 PFLOP/s, the clock
// down to 1.7 to 2.0 GHz), 480 to 490 with tile scales and 530 to 550 with row scales,
// whose multiply-adds take turns with the products.  The exact kernels (128 x 128, two
// workgroups on a compute unit) spend as many cycles on widening and scaling as
// on products: 4096^3 takes 130 to 137 us (1.0 PFLOP/s).
//
// b's rows of one operand: lane l has row 32 (j / 2) + 8 (l / 4) + 4 (j % 2) +
// l % 4 of the wave's 64, so that over two j a lane's results are 8 neighbours
// in c, and four lanes' 32: a store writes whole 64-byte pieces of 16 rows
// (with 16 neighbours a lane, half a 32-byte sector a store, 4096 x 4096 x 1024
// took 24.0 instead of 23.3 us).  Its place in LDS
// is 16 j + l.
template <int TM, int TN, int WM>
struct Tile {
  static constexpr int WN = 64;
  static constexpr int NI = WM / 16, NJ = WN / 16;
  static constexpr int WAVES = (TM / WM) * (TN / WN), THREADS = 64 * WAVES;
  static constexpr int A = 0, B = TM * kBlock, SA = B + TN * kBlock,
                       SB = SA + 4 * TM, BYTES = SB + 4 * TN;
  static_assert(TM + TN <= THREADS && TM % 64 == 0 && TN % 64 == 0);
  static_assert(TM % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0 && (WAVES == 4 || WAVES == 8));
};

__device__ inline int swizzle(int place) { return (place >> 1) & 7; }

// Workgroups go to the 8 dies in turn, and each die has its own L2 cache: it
// gets one stretch of the tiles, in the order of columns of kGroup tiles, so
// that what runs on it at one time is nearly square and shares most rows.
constexpr uint32_t kGroup = 4;
struct Place {
  int split;
  uint32_t tile_m, tile_n;
};
__device__ inline Place place(const Fp8GemmArgs &p, uint32_t block, uint32_t grid) {
  const uint32_t die = block % 8, per = grid / 8, more = grid % 8;
  uint32_t id = die * per + min(die, more) + block / 8;
  const uint32_t tiles = p.tiles_m * p.tiles_n;
  Place at;
  at.split = (int)(id / tiles);
  id %= tiles;
  const uint32_t group = id / (kGroup * p.tiles_n), in = id % (kGroup * p.tiles_n);
  const uint32_t high = min(kGroup, p.tiles_m - group * kGroup);
  at.tile_m = group * kGroup + in % high;
  at.tile_n = in / high;
  return at;
}

template <int TM, int TN, int WM, Fp8GemmMode MODE, bool EXACT>
__global__ __launch_bounds__((Tile<TM, TN, WM>::THREADS), 2) void fp8_tile_kernel(Fp8GemmArgs p) {
  using T = Tile<TM, TN, WM>;
  __shared__ __align__(16) uint8_t lds[2][T::BYTES];
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);  // a scalar
  const int l16 = lane % 16, g = lane / 16;
  const int wm = wave % (TM / WM) * WM, wn = wave / (TM / WM) * T::WN;

  int split;
  int64_t m0, n0;
  {
    const Place at = place(p, blockIdx.x, gridDim.x);
    split = __builtin_amdgcn_readfirstlane(at.split);
    m0 = (int64_t)at.tile_m * TM;
    n0 = (int64_t)at.tile_n * TN;
  }

  // this slice's blocks: whole ones from `first` on, and maybe the ragged last
  const int whole = (int)(p.k / kBlock), tail = (int)(p.k % kBlock);
  const int first = split * p.blocks_per_split;
  const int last = min(first + p.blocks_per_split, whole);
  const bool ragged = tail && first + p.blocks_per_split > whole;
  const int steps = last - first + ragged;

  // A wave's load covers 8 rows, 16 bytes a lane; the workgroup's, `kRows`.
  // Rows beyond the matrix come as zeros.
  constexpr int kRows = 8 * T::WAVES, LA = TM / kRows, LB = TN / kRows;
  const uint8_t *a0 = p.a + m0 * p.lda, *b0 = p.b + n0 * p.ldb;
  const int64_t bytes_a = (p.m - m0 - 1) * p.lda + p.k, bytes_b = (p.n - n0 - 1) * p.ldb + p.k;
  const int row_in = wave * 8 + lane / 8;  // of kRows
  const int at = ((lane % 8) ^ swizzle(row_in)) * 16;
  const int row_in_b = row_in / 32 * 32 + row_in % 16 / 4 * 8 + row_in / 16 % 2 * 4 + row_in % 4;
  const uint32_t off_a = (uint32_t)row_in * (uint32_t)p.lda + at;
  const uint32_t off_b = (uint32_t)row_in_b * (uint32_t)p.ldb + at;
  const int rows_a = (int)(p.m - m0 < TM ? p.m - m0 : TM) - 1;
  const int rows_b = (int)(p.n - n0 < TN ? p.n - n0 : TN) - 1;
  // The scale that this lane brings to LDS: threads below TM one of a's, the
  // next TN one of b's; a wave's base and pitch are scalars.
  const bool scale_of_a = wave < TM / 64;
  const float *scale0 = scale_of_a ? p.scale_a + m0 : p.scale_b + (n0 >> p.b_shift);
  const int64_t scale_ld = scale_of_a ? p.ld_scale_a : p.ld_scale_b;
  const uint32_t off_scale =
      4 * (scale_of_a ? (uint32_t)min(tid, rows_a)
                      : (uint32_t)(((n0 + min(tid - TM, rows_b)) >> p.b_shift) - (n0 >> p.b_shift)));
  auto stage_scales = [&](int kb, uint8_t *buf) {
    if (TM + TN == T::THREADS || wave < (TM + TN) / 64)
      to_lds4(buffer(scale0 + kb * scale_ld, 4 * (TM + TN)), off_scale, buf + T::SA + wave * 256);
  };
  // Descriptors by the load: rows from the matrix's end on lie past its bytes.
  Buffer from_a[LA], from_b[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) from_a[i] = buffer(a0 + i * kRows * p.lda, bytes_a - i * kRows * p.lda);
#pragma unroll
  for (int i = 0; i < LB; ++i) from_b[i] = buffer(b0 + i * kRows * p.ldb, bytes_b - i * kRows * p.ldb);
  auto stage_a = [&](int kb, uint8_t *buf) {
#pragma unroll
    for (int i = 0; i < LA; ++i)
      to_lds16(from_a[i], off_a, kb * kBlock, buf + T::A + (i * T::WAVES + wave) * 1024);
  };
  auto stage_b = [&](int kb, uint8_t *buf) {
#pragma unroll
    for (int i = 0; i < LB; ++i)
      to_lds16(from_b[i], off_b, kb * kBlock, buf + T::B + (i * T::WAVES + wave) * 1024);
    stage_scales(kb, buf);
  };
  // The last block of k with fewer than 128 columns, the rest as zeros: what
  // lies between k and the pitch may be anything, or no memory at all.
  auto stage_ragged = [&](uint8_t *buf) {
    const uint8_t *a = a0 + (int64_t)whole * kBlock, *b = b0 + (int64_t)whole * kBlock;
    u32x4 from_a[LA], from_b[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const uint8_t *row = a + min(i * kRows + row_in, rows_a) * p.lda;
      from_a[i] = load_chunk(row + at, tail - at, row);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const uint8_t *row = b + min(i * kRows + row_in_b, rows_b) * p.ldb;
      from_b[i] = load_chunk(row + at, tail - at, row);
    }
#pragma unroll
    for (int i = 0; i < LA; ++i)
      *reinterpret_cast<u32x4 *>(buf + T::A + (i * T::WAVES + wave) * 1024 + lane * 16) =
          keep(from_a[i], tail - at);
#pragma unroll
    for (int i = 0; i < LB; ++i)
      *reinterpret_cast<u32x4 *>(buf + T::B + (i * T::WAVES + wave) * 1024 + lane * 16) =
          keep(from_b[i], tail - at);
    stage_scales(whole, buf);
  };

  f32x4 acc[T::NI][T::NJ];
#pragma unroll
  for (int i = 0; i < T::NI; ++i)
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // One operand read from LDS: 32 bytes, and the scales that go with them.
  struct Rows16 {
    u32x4 lo, hi;
    float scale;  // of the lane's row (kFp8Rows: not b's)
    f32x4 scales; // kFp8Rows: of the four rows of b whose results the lane has
  };
  // A lane's places, from a buffer's start and for i = j = 0: the others lie at
  // constant distances, which the reads hold themselves.
  const int x = swizzle(l16), lo = (g ^ x) * 16, hi = ((g + 4) ^ x) * 16;
  const int place_a = T::A + (wm + l16) * kBlock, place_b = T::B + (wn + l16) * kBlock;
  const int place_sa = T::SA + 4 * (wm + l16);
  const int place_sb = T::SB + 4 * (MODE == kFp8Pow2   ? wn + l16 / 4 * 8 + l16 % 4
                                    : MODE == kFp8Rows ? wn + 8 * g
                                                       : wn);  // 64 rows of one tile
  auto read_a = [&](const uint8_t *buf, int i) {
    Rows16 v;
    v.lo = *reinterpret_cast<const u32x4 *>(buf + (place_a + lo) + i * 16 * kBlock);
    v.hi = *reinterpret_cast<const u32x4 *>(buf + (place_a + hi) + i * 16 * kBlock);
    v.scale = *reinterpret_cast<const float *>(buf + place_sa + i * 64);
    return v;
  };
  auto read_b = [&](const uint8_t *buf, int j) {
    Rows16 v;
    v.lo = *reinterpret_cast<const u32x4 *>(buf + (place_b + lo) + j * 16 * kBlock);
    v.hi = *reinterpret_cast<const u32x4 *>(buf + (place_b + hi) + j * 16 * kBlock);
    if constexpr (MODE == kFp8Pow2) v.scale = *reinterpret_cast<const float *>(buf + place_sb + j / 2 * 128 + j % 2 * 16);
    if (MODE == kFp8Tiles && j == 0) v.scale = *reinterpret_cast<const float *>(buf + place_sb);
    if constexpr (MODE == kFp8Rows) v.scales = *reinterpret_cast<const f32x4 *>(buf + place_sb + j / 2 * 128 + j % 2 * 16);
    return v;
  };

  // The ragged block goes first: nothing is under way yet that its loads
  // through registers would hold up.
  if (steps > 0) {
    if (ragged) {
      stage_ragged(lds[0]);
    } else {
      stage_a(first, lds[0]);
      stage_b(first, lds[0]);
    }
  }
  loads_and_barrier<0>();
  if (steps > 1) {
    stage_a(first + 1 - ragged, lds[1]);
    stage_b(first + 1 - ragged, lds[1]);
  }
  Rows16 a[T::NI], b = read_b(lds[0], 0);
#pragma unroll
  for (int i = 0; i < T::NI; ++i) a[i] = read_a(lds[0], i);
  // One block.  MORE: there is a next one; STAGE: and one after that.  These
  // are constants so that a block is one stretch of code, without branches for
  // products to be moved across.
  auto block = [&](int s, auto stage_next, auto more) {
    constexpr bool STAGE = stage_next(), MORE = more();
    uint8_t *const buf = lds[s & 1], *const next = lds[(s + 1) & 1];
    f32x4 last, last_s2;
    float last_s1;
    auto add = [&](f32x4 &sum) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sum[e] = MODE == kFp8Rows ? __builtin_fmaf(last[e] * last_s1, last_s2[e], sum[e])
                                  : __builtin_fmaf(last[e], last_s1, sum[e]);
    };
    const SplitScale of_b(MODE == kFp8Tiles ? b.scale : 1.f);
    Lane32<EXACT> al[T::NI];
#pragma unroll
    for (int i = 0; i < T::NI; ++i) al[i].set(a[i].lo, a[i].hi);
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) {
      const Rows16 now = b;
      Lane32<EXACT> bl;
      bl.set(now.lo, now.hi, of_b.power);
      if (j + 1 < T::NJ) {
        b = read_b(buf, j + 1);
      } else if constexpr (MORE) {
        // every wave has all of this block, and the next has landed
        loads_and_barrier<STAGE ? LA : 0>();
        if constexpr (STAGE) stage_b(first + s + 2 - ragged, buf);
        b = read_b(next, 0);
      }
      if (STAGE && j == 1) {
        reads_and_barrier();  // every wave has a's operands of this block
        stage_a(first + s + 2 - ragged, buf);
      }
#pragma unroll
      for (int i = 0; i < T::NI; ++i) {
        if constexpr (MODE == kFp8Pow2) {
          acc[i][j] = multiply(bl, al[i], acc[i][j], exponent_of(now.scale), exponent_of(a[i].scale));
        } else {
          // Each product is added in behind the next one's start, not waited for.
          f32x4 v;
          if constexpr (MODE == kFp8Tiles && !EXACT)
            v = multiply(bl, al[i], f32x4{0.f, 0.f, 0.f, 0.f}, exponent_of(of_b.power), exponent_of(1.f));
          else
            v = multiply(bl, al[i]);
          if (i > 0) add(acc[i - 1][j]);
          else if (j > 0) add(acc[T::NI - 1][j - 1]);
          last = v;
          last_s1 = MODE == kFp8Tiles ? a[i].scale * of_b.rest : a[i].scale;
          last_s2 = now.scales;
        }
        if (MORE && j + 1 == T::NJ) {
          // in this order: the registers of a[i] are free from here on
          __builtin_amdgcn_sched_barrier(0);
          a[i] = read_a(next, i);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (MODE != kFp8Pow2) add(acc[T::NI - 1][T::NJ - 1]);
  };
  using std::bool_constant;
  int s = 0;
  for (; s + 2 < steps; ++s) block(s, bool_constant<true>{}, bool_constant<true>{});
  if (s + 1 < steps) block(s++, bool_constant<false>{}, bool_constant<true>{});
  if (s < steps) block(s, bool_constant<false>{}, bool_constant<false>{});

  uint8_t *c = (uint8_t *)p.c + (int64_t)split * p.slice * 4;  // slices are float32
#pragma unroll
  for (int i = 0; i < T::NI; ++i) {
    const int64_t row = m0 + wm + 16 * i + l16;
    if (row >= p.m) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t col = n0 + wn + 32 * h + 8 * g;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = acc[i][2 * h + e / 4][e % 4];
      if (col < p.n) store_run<8>(c, p.out, row * p.ldc + col, p.n - col, f);
    }
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
// instruction's registers, two or four at a time, and their sums are added through
// LDS in the waves' order.  One token through 4096 x 4096 takes 6.0 us (2.8 TB/s;
// the launch is over half of it), through 4096 x 8192 9 to 10 us.  A long k and few
// rows of b go in slices, as for the tiles.
constexpr int kSkinnyWaves = 8;

template <int MS, bool EXACT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void fp8_skinny_kernel(Fp8GemmArgs p) {
  constexpr int kDepth = MS > 1 ? 2 : 4;
  __shared__ __align__(16) float sums[kSkinnyWaves][MS][64][4];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int l16 = lane % 16, g = lane / 16;
  const uint32_t tiles = p.tiles_m * p.tiles_n, split = blockIdx.x / tiles, id = blockIdx.x % tiles;
  const int64_t n0 = (int64_t)(id % p.tiles_n) * 16;
  const int64_t m0 = (int64_t)(id / p.tiles_n) * 16 * MS;
  // this slice's blocks of k, from `first` to before `blocks`
  const int64_t first = (int64_t)split * p.blocks_per_split;
  const int64_t blocks = min((p.k + kBlock - 1) / kBlock, first + p.blocks_per_split);

  const int64_t brow = n0 + l16 < p.n ? n0 + l16 : p.n - 1;
  const uint8_t *b = p.b + brow * p.ldb;
  const uint8_t *a[MS];
  const float *sa[MS];
  const float *sb[4];
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    const int64_t row = m0 + 16 * i + l16 < p.m ? m0 + 16 * i + l16 : p.m - 1;
    a[i] = p.a + row * p.lda;
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
  for (int64_t kb0 = first + wave; kb0 < blocks; kb0 += kSkinnyWaves * kDepth) {
    u32x4 bv[kDepth][2], av[kDepth][MS][2];
    float sav[kDepth][MS], sbv[kDepth][4];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int64_t kb = kb0 + d * kSkinnyWaves;
      const int64_t ks = kb < blocks ? kb : blocks - 1, at = ks * kBlock;
      const int64_t left = p.k - at;  // of the row, from this block on
      bv[d][0] = load_chunk(b + at + g * 16, left - g * 16, b + at);
      bv[d][1] = load_chunk(b + at + g * 16 + 64, left - g * 16 - 64, b + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) sbv[d][e] = sb[e][ks * p.ld_scale_b];
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        av[d][i][0] = load_chunk(a[i] + at + g * 16, left - g * 16, a[i] + at);
        av[d][i][1] = load_chunk(a[i] + at + g * 16 + 64, left - g * 16 - 64, a[i] + at);
        sav[d][i] = sa[i][ks * p.ld_scale_a];
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (kb0 + d * kSkinnyWaves >= blocks) break;
      const int64_t left = p.k - (kb0 + d * kSkinnyWaves) * kBlock - g * 16;
      const bool cut = left < 128;  // only a row's last block can be
      Lane32<EXACT> bl;
      bl.set(cut ? keep(bv[d][0], left) : bv[d][0], cut ? keep(bv[d][1], left - 64) : bv[d][1]);
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        Lane32<EXACT> al;
        al.set(cut ? keep(av[d][i][0], left) : av[d][i][0], cut ? keep(av[d][i][1], left - 64) : av[d][i][1]);
        const f32x4 v = multiply(bl, al);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][e] = __builtin_fmaf(v[e] * sav[d][i], sbv[d][e], acc[i][e]);
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
      uint8_t *c = (uint8_t *)p.c + (int64_t)split * p.slice * 4;  // slices are float32
      store_run<4>(c, p.out, row * p.ldc + col, p.n - col, f);
    }
  }
}

template <int MS, bool EXACT>
hipError_t launch_skinny(const Fp8GemmArgs &a, Fp8GemmMode, hipStream_t s) {
  Fp8GemmArgs copy = a;
  void *args[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void *>(&fp8_skinny_kernel<MS, EXACT>),
                         dim3(a.tiles_m * a.tiles_n * a.splits), dim3(64 * kSkinnyWaves), args, 0, s);
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
