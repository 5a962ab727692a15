// qr_product.hpp -- gfx950 kernels of the products with 4-bit block weights
// (include/qr_ops.h): y = x W^T for one weight or one per group of rows.
//
// y[m][c] = sum over k of x[m][k] W[c][k], W[c][k] = d[c][k / group] (code - z)
// (FP4: d times the E2M1 value).  Three kernels, chosen by how often a weight is
// used once it is there:
//   row_kernel        1 or 2 rows of x: fp32 FMAs, bound by memory and the launch
//   few_rows_kernel   up to a few tens of rows a weight: matrix unit on the
//                     codes, scales applied to fp32 sums of a block; bound by
//                     vector instructions and the wait for each round of loads
//   many_rows_kernel  more: the same in large tiles; bound by the issue of
//                     instructions, mostly the vector unit's
// All of them use W as it stands, and only y is rounded to the dtype.  The matrix
// unit takes 16-bit operands, which hold a code (less its zero point) exactly
// but not its product with an fp16 scale; so the scale is applied to the fp32 sum
// of a block.  That is four FMAs of the vector unit for every product of 16 x 16
// x 32, which take as long to issue as the product takes the matrix unit.
//
// The matrix unit's product is 16 x 16 x 32: lane (r = lane & 15, g = lane >> 4)
// holds 8 consecutive k, 8 g .. 8 g + 7, of row r of A and of B, and gets rows
// 4 g .. 4 g + 3 of A's side in column r of B's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "qr.h"
#include "qr_codec.hpp"
#include "qr_ops.h"

namespace qr {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// 16- and 8-byte accesses at the alignment of a 2-byte value: rows of odd
// stride are read and written without a special case (gfx950 serves unaligned
// global accesses in hardware).
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;

// A launch holds fewer than 2^32 threads; a call of more is made of several
// launches.  (A small limit lets small calls run that way too.)
#ifndef QR_MAX_LAUNCH_THREADS
#define QR_MAX_LAUNCH_THREADS 0xffffffff
#endif
constexpr long long kMaxLaunchThreads = QR_MAX_LAUNCH_THREADS;

// The whole card.  In a partition of it the choices that count on them are less
// apt, the results the same.
constexpr int kCUs = 256, kXCDs = 8;

constexpr int kChunk = 128;        // values of k of the weights that the many-row kernel asks for at a time
constexpr int kChunkBlocks = kChunk / kBlockValues;

// Arguments of the product kernels.  Dense products have offsets == nullptr
// and one expert.
struct ProductArgs {
  const uint8_t* x;
  const uint8_t* w;
  uint8_t* y;
  const int32_t* offsets;
  const int32_t* rows;
  long long ldx, ldy;   // row strides in values
  long long xrows;      // rows of x
  int slots;            // rows of y
  int experts;
  int n;                // columns of y
  int k;
  int blocks;           // 32-value blocks of one (padded) weight row
  int ntiles;           // column tiles of the grid
  int tile0;            // row tile that the launch begins with
};

// ---------------------------------------------------------------------------
// which rows a workgroup computes
// ---------------------------------------------------------------------------

struct RowTile {
  int expert;
  int m0, m1;  // rows m0 .. m1 - 1 of y (m0 >= m1: nothing to do)
  bool zero;   // rows of no expert: set to zero
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Row tile `t` of the launch: experts in order, each cut into tiles of BM
// rows, and then the rows of no expert.  One wave finds it (every wave on its
// own, no exchange): a lane takes an expert, counts its tiles, and a scan over
// the lanes shows which expert's range holds t.  64 experts a step.  An offset
// below an earlier one counts as that one, so that no two groups share a row
// and the launch has a tile for every row.
template <int BM>
__device__ __forceinline__ RowTile find_rows(const ProductArgs& a, int t, int* first_of_group = nullptr, int* tiles_of_group = nullptr) {
  RowTile rt;
  rt.zero = false;
  if (!a.offsets) {
    rt.expert = 0;
    rt.m0 = t * BM;
    rt.m1 = a.slots < rt.m0 + BM ? a.slots : rt.m0 + BM;
    return rt;
  }
  const int lane = threadIdx.x & (kWave - 1);
  int before = 0;  // tiles of the experts of earlier steps
  int top = 0;     // where the last of them ends
  for (int e0 = 0; e0 <= a.experts; e0 += kWave) {
    const int e = e0 + lane;  // e == experts: the rows of no expert
    int lo = a.slots, hi = a.slots;
    if (e <= a.experts) {
      lo = clampi(a.offsets[e], 0, a.slots);
      hi = e < a.experts ? clampi(a.offsets[e + 1], 0, a.slots) : a.slots;
    }
    if (__any(lo < top || hi < lo)) {  // out of order: each becomes the largest up to it
      lo = lo > top ? lo : top;
#pragma unroll
      for (int s = 1; s < kWave; s <<= 1) {
        const int o = __shfl_up(lo, s);
        if (lane >= s && o > lo) lo = o;
      }
      hi = hi > lo ? hi : lo;
    }
    top = __builtin_amdgcn_readlane(hi, kWave - 1);
    const int mine = hi > lo ? (hi - lo + BM - 1) / BM : 0;
    int upto = mine;
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) {
      const int o = __shfl_up(upto, s);
      if (lane >= s) upto += o;
    }
    const unsigned long long found = __ballot(before + upto > t);
    if (found) {
      const int l = __ffsll(found) - 1;
      const int first = before + __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(mine, l);
      const int begin = __builtin_amdgcn_readlane(lo, l), end = __builtin_amdgcn_readlane(hi, l);
      rt.expert = e0 + l;
      rt.zero = rt.expert == a.experts;
      rt.m0 = begin + (t - first) * BM;
      rt.m1 = end < rt.m0 + BM ? end : rt.m0 + BM;
      if (first_of_group) {
        *first_of_group = first;
        *tiles_of_group = __builtin_amdgcn_readlane(mine, l);
      }
      return rt;
    }
    before += __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  rt.expert = a.experts;
  rt.m0 = rt.m1 = 0;
  return rt;
}

// Largest number of row tiles that find_rows() can hand out: the groups share no
// row, no more of them than there are rows are not empty, each of these has a tile
// that holds at least one row, and the other tiles are full.
inline long long row_tiles(long long slots, long long experts, bool dense, int bm) {
  if (dense) return (slots + bm - 1) / bm;
  const long long groups = experts + 1 < slots ? experts + 1 : slots;
  return groups + (slots - groups) / bm;
}

// Row of x that row m of y is computed from, -1 if none.
__device__ __forceinline__ long long source_row(const ProductArgs& a, int m) {
  if (!a.rows) return m;
  const int r = a.rows[m];
  return r >= 0 && r < a.xrows ? (long long)r : -1LL;
}

// ---------------------------------------------------------------------------
// weights: one 16-byte load of codes and its scale, and their decode
// ---------------------------------------------------------------------------

struct RawBlock {
  u32x4 codes;
  uint32_t scale;  // fp16 bits
  uint32_t zero;   // zero point (asymmetric format)
};

// Block `b` of the packed weight that starts at `w` (b counts 32-value blocks
// from a tile boundary).
template <int F>
__device__ __forceinline__ RawBlock load_raw(const uint8_t* w, uint32_t b) {
  constexpr uint32_t TB = Format<F>::kTileBytes;
  const uint32_t tile = (b >> 6) * TB, in = b & 63;
  RawBlock r;
  r.codes = *reinterpret_cast<const u32x4*>(w + (tile + in * 16));
  if constexpr (Format<F>::kAsym) {
    r.scale = *reinterpret_cast<const uint16_t*>(w + (tile + Format<F>::kScaleOffset + (in >> 2) * 2));
    r.zero = w[tile + Format<F>::kZeroOffset + (in >> 2)];
  } else {
    r.scale = *reinterpret_cast<const uint16_t*>(w + (tile + Format<F>::kScaleOffset + in * 2));
    r.zero = 0;
  }
  return r;
}

// ---------------------------------------------------------------------------
// x: 8 values of a row
// ---------------------------------------------------------------------------

// Values k0 .. k0 + 7 of a row of k; those from k on are zero and are not read.
// No branch but one that is the same for the whole launch, so that several such
// loads are in flight together: the last 8 values of the row are moved down.
__device__ __forceinline__ u32x4 load_x8_tail(const uint8_t* row, int k0, int k) {
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  if (k >= 8) {
    const int from = k0 < k - 8 ? k0 : k - 8;
    const u64x2 v = __builtin_bit_cast(u64x2, *reinterpret_cast<const u32x4_any*>(row + 2 * (size_t)from));
    const int drop = k0 - from < 8 ? k0 - from : 8;  // values
    const int low = 16 * (drop & 3);
    const unsigned long long down = low ? v.x >> low | v.y << (64 - low) : v.x;
    const unsigned long long high = v.y >> low;
    return __builtin_bit_cast(u32x4, drop >= 8 ? u64x2{0, 0} : drop >= 4 ? u64x2{high, 0} : u64x2{down, high});
  }
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 7; ++j) {
    const int at = k0 + j < k ? k0 + j : k - 1;
    const uint32_t h = *reinterpret_cast<const uint16_t*>(row + 2 * (size_t)at);
    if (k0 + j < k) v[j >> 1] |= (j & 1) ? h << 16 : h;
  }
  return v;
}

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 w, u32x4 x, f32x4 c) {
  if constexpr (DT == kFp16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0, 0,
                                                   0);
}

// bf16 has the range of fp32, so a sum of codes times x could overflow where the
// scaled sum does not (x of the type's lowest value).  There the products take
// 1 / kStep of the values: no sum over a block of 32 is then larger than the
// largest |x|, and kStep, a power of two, goes into the scale or into y.
template <int F, int DT>
constexpr float kStep = DT == kFp16 ? 1.0f : Format<F>::kFp4 ? 256.0f : 512.0f;

// silu(g) * u in fp32.
__device__ __forceinline__ float gate(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// ---------------------------------------------------------------------------
// one or two rows
// ---------------------------------------------------------------------------

// The 8 values of a unit in fp32, without the scale and in steps of 1 / kStep;
// INT4: 16 times the values.  `zero` is in the same steps.
template <int F, int DT>
__device__ __forceinline__ void unit_f32(uint32_t w, float zero, float (&v)[8]) {
  constexpr float step = 1.0f / kStep<F, DT>;
  if constexpr (Format<F>::kFp4) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, step, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, step, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, step, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, step, 3);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y; v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
  } else if constexpr (Format<F>::kAsym) {
    // the byte c as FP8 E4M3 is c / 512 for every 4-bit c
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;  // values 0 2 4 6 and 1 3 5 7
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.0f * step, false);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.0f * step, true);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.0f * step, false);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.0f * step, true);
    v[0] = a.x - zero; v[2] = a.y - zero; v[4] = b.x - zero; v[6] = b.y - zero;
    v[1] = c.x - zero; v[3] = c.y - zero; v[5] = d.x - zero; v[7] = d.y - zero;
  } else {
    // signed bytes 16 (c - 8); the 16 is taken out of the scale
    const uint32_t lo = ((w << 4) & 0xF0F0F0F0u) ^ 0x80808080u, hi = (w & 0xF0F0F0F0u) ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = sbyte(lo, i);
      v[2 * i + 1] = sbyte(hi, i);
    }
  }
}

// The sum over the wave's lanes, in lane 63: within each row of 16 lanes, and
// then from row to row.
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](auto ctrl) {
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF,
                                                               0xF, true));
  };
  add(std::integral_constant<int, 0x111>{});  // row_shr:1
  add(std::integral_constant<int, 0x112>{});  // row_shr:2
  add(std::integral_constant<int, 0x114>{});  // row_shr:4
  add(std::integral_constant<int, 0x118>{});  // row_shr:8
  add(std::integral_constant<int, 0x142>{});  // row_bcast:15
  add(std::integral_constant<int, 0x143>{});  // row_bcast:31
  return v;
}

// One workgroup multiplies MR rows of x by kRowsPerWave weight rows for each of
// its 8 / KS groups of KS waves; the waves of a group share the k axis in
// slices of 2048 values, one 32-value block a lane, so that a row's codes and
// scales are read in whole lines.  x goes through LDS once for the workgroup
// and stays in fp32 registers for the wave's weight rows; every product and
// sum is an fp32 FMA, so W is not rounded.  Bound by reading the weights, and in
// small calls by the launch and the one trip to memory: all of a slice's loads
// are in flight at once.  One row, int4, 4096 x 4096 (9.4 MB): 4.6 us on the
// device, 2.1 TB/s, where an empty kernel takes 2.5; two experts' gated 2048 x
// 4096 (18.9 MB): 8.2 us, 2.3 TB/s.
constexpr int kRowWaves = 8;
constexpr int kRowsPerWave = 4;
constexpr int kSlice = kWave * kBlockValues;

template <int F, int DT, bool GATED, int MR, int KS>
__global__ __launch_bounds__(kWave* kRowWaves) void row_kernel(ProductArgs a) {
  constexpr int HALVES = GATED ? 2 : 1, R = kRowsPerWave, GROUPS = kRowWaves / KS;
  constexpr int CW = R / HALVES, COLS = GROUPS * CW;  // columns of y of a wave, of the workgroup
  constexpr int XC = MR * KS * kSlice / 8;            // 16-byte pieces of x in a panel of KS slices
  __shared__ u32x4 lds_x[XC];
  __shared__ float sums[kRowWaves][MR][R];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int ks = wave % KS, c0 = (blockIdx.x % a.ntiles) * COLS;
  RowTile rt = find_rows<MR>(a, a.tile0 + blockIdx.x / a.ntiles);
  if (rt.m0 >= rt.m1) return;
  rt.zero |= a.xrows == 0;  // every row number is out of range then
  long long src[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) src[m] = rt.zero || rt.m0 + m >= rt.m1 ? -1 : source_row(a, rt.m0 + m);

  // weight rows as blocks from the tile that holds the workgroup's first of each half
  const uint8_t* w[HALVES];
  uint32_t first[R];
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    const long long b = (((long long)(rt.zero ? 0 : rt.expert) * HALVES + h) * a.n + c0) * a.blocks;
    w[h] = a.w + (b >> 6) * Format<F>::kTileBytes;
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      const int c = c0 + (wave / KS) * CW + i;  // columns past the last repeat it
      first[h * CW + i] = (uint32_t)(b & 63) + (uint32_t)((c < a.n ? c : a.n - 1) - c0) * (uint32_t)a.blocks;
    }
  }
  float acc[MR][R];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int i = 0; i < R; ++i) acc[m][i] = 0.0f;
  const int panels = rt.zero ? 0 : (a.blocks + KS * kWave - 1) / (KS * kWave);
  for (int p = 0; p < panels; ++p) {
    const int kb = (p * KS + ks) * kWave + lane;
    // past the row's last block: that block again, times zeros of x
    const uint32_t b = (uint32_t)(kb < a.blocks ? kb : a.blocks - 1);
    RawBlock raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) raw[i] = load_raw<F>(w[i / CW], first[i] + b);
    u32x4 xv[(XC + kWave * kRowWaves - 1) / (kWave * kRowWaves)];
    const int k0 = p * KS * kSlice;
#pragma unroll
    for (int t = 0; t < (int)(sizeof(xv) / sizeof(xv[0])); ++t) {
      const int q = tid + kWave * kRowWaves * t, m = MR == 1 ? 0 : q / (XC / MR), k = k0 + 8 * (q % (XC / MR));
      xv[t] = u32x4{0u, 0u, 0u, 0u};
      const long long s = MR > 1 && m ? src[MR - 1] : src[0];
      if (q < XC && s >= 0 && k < a.k) xv[t] = load_x8_tail(a.x + 2 * s * a.ldx, k, a.k);
    }
    if (p) __syncthreads();  // everyone is done with the last panel's x
    // lane l reads pieces 4 l .. 4 l + 3, which lie at places (piece ^ l / 4) of its 64 bytes:
    // 8 lanes that read one of them hit 8 groups of banks
#pragma unroll
    for (int t = 0; t < (int)(sizeof(xv) / sizeof(xv[0])); ++t) {
      const int q = tid + kWave * kRowWaves * t;
      if (q < XC) lds_x[q ^ ((q >> 4) & 3)] = xv[t];
    }
    __syncthreads();
    // INT4's bytes become fp32 as they are, so there x takes the step, and the bytes' 16
    constexpr bool kStepX = !Format<F>::kAsym && !Format<F>::kFp4 && DT == kBf16;
    constexpr float kX = kStepX ? 1.0f / (16.0f * kStep<F, DT>) : 1.0f;
    float x[MR][kBlockValues];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int q = (m * KS + ks) * (kSlice / 8) + 4 * lane + u;
        const u32x4 v = lds_x[q ^ ((q >> 4) & 3)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[m][8 * u + 2 * i] = lo_to_f32<DT>(v[i]) * kX;
          x[m][8 * u + 2 * i + 1] = hi_to_f32<DT>(v[i]) * kX;
        }
      }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float t[MR][2];
#pragma unroll
      for (int m = 0; m < MR; ++m) t[m][0] = t[m][1] = 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float v[8];
        unit_f32<F, DT>(raw[i].codes[u], (float)raw[i].zero * (1.0f / kStep<F, DT>), v);
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
          for (int j = 0; j < 8; ++j) t[m][j & 1] = __builtin_fmaf(v[j], x[m][8 * u + j], t[m][j & 1]);
      }
      float d = (float)__builtin_bit_cast(_Float16, (uint16_t)raw[i].scale) * kStep<F, DT>;
      if constexpr (!Format<F>::kAsym && !Format<F>::kFp4 && !kStepX) d *= 0.0625f;
#pragma unroll
      for (int m = 0; m < MR; ++m) acc[m][i] = __builtin_fmaf(d, t[m][0] + t[m][1], acc[m][i]);
    }
  }
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float v = wave_sum(acc[m][i]);
      if (lane == kWave - 1) sums[wave][m][i] = v;
    }
  __syncthreads();
  if (tid >= MR * COLS) return;
  const int m = tid / COLS, col = tid % COLS, grp = col / CW;
  if (rt.m0 + m >= rt.m1 || c0 + col >= a.n) return;
  float s[HALVES];
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    s[h] = sums[grp * KS][m][h * CW + col % CW];
#pragma unroll
    for (int k = 1; k < KS; ++k) s[h] += sums[grp * KS + k][m][h * CW + col % CW];
  }
  const float v = GATED ? gate(s[0], s[HALVES - 1]) : s[0];
  const bool real = MR > 1 && m ? src[MR - 1] >= 0 : src[0] >= 0;
  *reinterpret_cast<uint16_t*>(a.y + 2 * ((rt.m0 + m) * a.ldy + c0 + col)) = (uint16_t)pack2<DT>(real ? v : 0.0f, 0.0f);
}

// ---------------------------------------------------------------------------
// loads that go to LDS
// ---------------------------------------------------------------------------

// 16 bytes from each lane's address to lds + 16 lane, which is the same for the
// whole wave.  In assembly, because the compiler would wait for it before the
// next LDS read of any address, also of the buffer that is not being written;
// it has no result that a register waits for.  M0 holds the LDS address.  Who
// reads the bytes waits with loads_done() and a barrier.
__device__ __forceinline__ uint32_t lds_address(void* lds) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
}
__device__ __forceinline__ void load_to_lds(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory", "m0");
}
// One value of SIZE bytes (1 or 2, zero-extended) from each lane's address to lds + 4 lane.
template <int SIZE>
__device__ __forceinline__ void load_value_to_lds(const uint8_t* p, uint32_t lds) {
  if constexpr (SIZE == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, off" : : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off" : : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory", "m0");
}
// The same from a base of the whole wave plus each lane's offset.
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(base)
               : "memory", "m0");
}
template <int SIZE>
__device__ __forceinline__ void load_value_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
  if constexpr (SIZE == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(base)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(base)
                 : "memory", "m0");
}
// A barrier of the workgroup that leaves loads to LDS on their way, which
// __syncthreads() would wait for; each wave's LDS accesses are done before it.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// Waits until at most N of the wave's loads are still on their way (they arrive in order).
template <int N>
__device__ __forceinline__ void loads_done() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

// A weight block as the few-row kernel multiplies it: the values without the
// scale, exact in either dtype, and the scale applied to the fp32 sum over the
// block.  One product of the matrix unit then has to cover one block (k = 32),
// so the lanes (r, 0..3), which loaded blocks 0..3 of a chunk of row r whole,
// exchange units: afterwards lane (r, g) holds unit g of block i in codes[i].
// Four row swaps do it, two between the halves of the wave and two between
// its odd and even rows of 16 lanes.
__device__ __forceinline__ u32x4 exchange_units(u32x4 c) {
  auto a = __builtin_amdgcn_permlane32_swap(c.x, c.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(c.y, c.w, false, false);
  auto p = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto q = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{p[0], p[1], q[0], q[1]};
}

// The 8 values of a unit without the scale, in steps of 1 / kStep: E2M1 values;
// else the codes less `zero` (SIGNED; in the same steps) or the codes themselves.
template <int F, int DT, bool SIGNED>
__device__ __forceinline__ u32x4 unit_values(uint32_t w, float zero) {
  constexpr float step = 1.0f / kStep<F, DT>;
  u32x4 o;
  if constexpr (Format<F>::kFp4) {
    if constexpr (DT == kFp16) {
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
    } else {
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, step, 0));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, step, 1));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, step, 2));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, step, 3));
    }
  } else {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;  // values 0 2 4 6 and 1 3 5 7
    const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u), b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
    // the byte c as FP8 E4M3 is c / 512 for every 4-bit c
    if constexpr (SIGNED) {
      const f32x2 v01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(a, 512.0f * step, false);
      const f32x2 v23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(a, 512.0f * step, true);
      const f32x2 v45 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b, 512.0f * step, false);
      const f32x2 v67 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b, 512.0f * step, true);
      o.x = pack2<DT>(v01.x - zero, v01.y - zero);
      o.y = pack2<DT>(v23.x - zero, v23.y - zero);
      o.z = pack2<DT>(v45.x - zero, v45.y - zero);
      o.w = pack2<DT>(v67.x - zero, v67.y - zero);
    } else if constexpr (DT == kFp16) {
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.0f * step, false));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.0f * step, true));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.0f * step, false));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.0f * step, true));
    } else {
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f * step, false));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f * step, true));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f * step, false));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f * step, true));
    }
  }
  return o;
}

// One workgroup multiplies 16 MF rows of x by NW fragments of 16 weight rows
// (gated: NW / 2 of the gate rows and as many of the up rows).  Its KW x NW
// waves share the k axis in KW groups (group kw takes every KW-th segment of
// 256 values); a wave has one weight fragment, and the waves of a group share
// the segment's x.  The groups' sums are joined through LDS in their order.
//
// Requests are dear: a load takes the CU's address unit a cycle for every
// 64-byte piece it touches, 16 when four neighbouring lanes share one and 64
// when each lane reads a row of its own, as the fragments of the matrix unit
// want it.  So nothing is loaded in fragment order: codes, scales and x go to
// LDS in whole runs of a row, the next segment's while one is multiplied.
// There, 16-byte piece p of row r (a block of codes, a unit of x) lies at place
// p ^ (r & 7), so that lanes which read one piece of eight rows hit eight
// different groups of banks; the lanes that load it take their pieces in that
// order.  Rows r and r + 8 of x meet in one group; conflicts are 0.42 to 0.54 of the
// cycles in which LDS is active.
//
// x is the matrix unit's A here and the weight its B, so that a lane's results
// belong to one weight row, whose scales it applies to them: lane (r, g) has
// rows 4 g .. 4 g + 3 of x and weight row r.  It reads codes of blocks 2 g + j,
// j = 0, 1, of a segment; after exchange_units() product i of step j is block
// 2 i + j.
//
// sum_k x (c - z) is taken as sum_k x c - z sum_k x: the codes need no
// subtraction, and sum_k x comes from one more product.  An infinity in x
// would make that inf - inf, and x of the largest values may overflow before the
// difference; a wave whose sum is not finite computes it again with the values
// c - z themselves.
//
// 16 rows, asym4, gated, n = k = 8192 (71 MB): 20.5 us, 3.4 TB/s; 64 tokens, 8
// of 64 experts, gated, n 1024, k 2048 (143 MB): 49.3 us, 2.9 TB/s; 37 rows that
// begin on odd addresses, fp4, 5003 x 4129 (11.7 MB): 12.7 us, 0.9 TB/s.  No one
// part fills this time: of the cycles in which CUs are busy, the vector unit issues
// in 43, 62 and 46 %, LDS is active in 21, 26 and 40 % (conflicts 9, 11 and 21 %),
// the matrix unit is busy in 15, 18 and 8 %.  A CU holds two segments of at most
// 16 waves, 72 to 144 KB of LDS, half of it on its way, and each of a workgroup's
// rounds (8, 8 and 5) waits for all its loads.
constexpr int kSegment = 256;
constexpr int kSegBlocks = kSegment / kBlockValues;
constexpr int kSegUnits = kSegment / 8;

template <int F, int DT, int MF, int NW, int KW, bool ALIGNED>
struct FewRows {
  static constexpr bool kAsym = Format<F>::kAsym;
  static constexpr bool kZeros = !Format<F>::kFp4;  // codes have a zero point
  static constexpr int XL = MF * 8 / NW;            // loads of x of one wave in a segment: two rows each
  static_assert(XL * NW == MF * 8, "the waves of a group share the loads of x evenly");
  struct Wave {
    u32x4 codes[16][kSegBlocks];
    uint32_t scales[16][kSegBlocks];  // asymmetric: [row][group] scales and, 64 words on, zero points
  };
  struct Buffer {
    u32x4 x[KW][16 * MF][kSegUnits];
    Wave w[KW][NW];
  };
  union Stage {
    Buffer buffer[2];
    f32x4 sums[KW][NW][MF][kWave];  // when all is multiplied
  };

  const uint8_t* w;
  uint32_t cblock[2];  // first block of weight rows lane / 8 and 8 + lane / 8, from w
  uint32_t gblock;     // the same of row lane / 2 % 16 (asymmetric: scales)
  const uint8_t* xrow[ALIGNED ? 1 : XL];  // of each load: its row of x, at this lane's unit
  uint32_t xoff[XL];                      // ... from x
  u32x4 xv[ALIGNED ? 1 : XL];
  f32x4 acc[MF];

  __device__ __forceinline__ static int unit_of(int lane, int t, int nw) {
    return (lane & 31) ^ ((2 * (nw + NW * t) + (lane >> 5)) & 7);
  }

  __device__ __forceinline__ void fetch_weights(const ProductArgs& a, Buffer& to, int seg, int kw, int nw,
                                                int lane) const {
    constexpr uint32_t TB = Format<F>::kTileBytes;
    const int last = a.blocks - 1;
    // a block past the row's last: that block again, times zeros of x
    auto clamp = [&](int kb) { return (uint32_t)(kb < last ? kb : last); };
    const uint32_t codes = lds_address(&to.w[kw][nw].codes[0][0]), scales = lds_address(&to.w[kw][nw].scales[0][0]);
    const uint32_t kc = clamp(seg * kSegBlocks + ((lane & 7) ^ (lane >> 3)));
    const uint32_t ks = clamp(seg * kSegBlocks + (kAsym ? 4 * (lane & 1) : lane & 7));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t b = cblock[q] + kc;
      load_to_lds(w + ((b >> 6) * TB + (b & 63) * 16), codes + 1024 * q);
    }
    if constexpr (kAsym) {
      const uint32_t b = gblock + ks, tile = (b >> 6) * TB, in = (b & 63) >> 2;
      if (lane < 32) {  // the other half would ask for the same again
        load_value_to_lds<2>(w + (tile + Format<F>::kScaleOffset + in * 2), scales);
        load_value_to_lds<1>(w + (tile + Format<F>::kZeroOffset + in), scales + 256);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t b = cblock[q] + ks;
        load_value_to_lds<2>(w + ((b >> 6) * TB + Format<F>::kScaleOffset + (b & 63) * 2), scales + 256 * q);
      }
    }
  }

  __device__ __forceinline__ void fetch_x(const ProductArgs& a, Buffer& to, int seg, int kw, int nw, int lane) {
    const bool whole = kSegment * (seg + 1) <= a.k;
    if constexpr (ALIGNED) {
      const uint8_t* from = a.x + 2 * kSegment * (size_t)seg;
      const uint32_t x = lds_address(&to.x[kw][0][0]);
      if (whole) {
#pragma unroll
        for (int t = 0; t < XL; ++t) load_to_lds(from, xoff[t], x + 1024 * (nw + NW * t));
      } else {
#pragma unroll
        for (int t = 0; t < XL; ++t) {
          const int q = nw + NW * t;
          if (kSegment * seg + 8 * unit_of(lane, t, nw) < a.k)
            load_to_lds(from, xoff[t], x + 1024 * q);
          else
            to.x[kw][2 * q + (lane >> 5)][lane & 31] = u32x4{0u, 0u, 0u, 0u};
        }
      }
    } else {
      if (whole) {
#pragma unroll
        for (int t = 0; t < XL; ++t)
          xv[t] = *reinterpret_cast<const u32x4_any*>(xrow[t] + 2 * kSegment * (size_t)seg);
      } else {
#pragma unroll
        for (int t = 0; t < XL; ++t) {
          const int unit = unit_of(lane, t, nw);
          xv[t] = load_x8_tail(xrow[t] - 16 * unit, kSegment * seg + 8 * unit, a.k);
        }
      }
    }
  }

  // Asks for the first segment.  Its weights need not wait for the numbers of the
  // rows of x, which are a trip to memory of their own.
  template <typename ROWS>
  __device__ __forceinline__ void begin(const ProductArgs& a, Stage& stage, int kw, int nw, int lane, ROWS find) {
    if (kSegment * kw < a.k) fetch_weights(a, stage.buffer[0], kw, kw, nw, lane);
    find();
    if (kSegment * kw < a.k) fetch_x(a, stage.buffer[0], kw, kw, nw, lane);
  }

  // Adds this wave's share to acc, after begin().
  template <bool SIGNED>
  __device__ __forceinline__ void sum(const ProductArgs& a, Stage& stage, int kw, int nw, int lane) {
    const int r = lane & 15, g = lane >> 4;
    const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[m] = none;
    // the factor of sum_k x: the zero point where it is the same for all; in steps
    const uint32_t factor = kAsym ? (DT == kFp16 ? 0x3C003C00u : 0x3B003B00u)   // 1, 1 / 512
                                  : (DT == kFp16 ? 0xC800C800u : 0xBC80BC80u);  // -8, -8 / 512
    const u32x4 factors = {factor, factor, factor, factor};
    const int segments = (a.k + kSegment - 1) / kSegment;  // each has values of x
    // every wave goes through as many rounds as the first group
    for (int s0 = 0, buf = 0; s0 < segments; s0 += KW, buf = buf ? 0 : 1) {
      const int seg = s0 + kw;
      Buffer& now = stage.buffer[buf];
      loads_done<0>();
      if constexpr (!ALIGNED) {
        if (seg < segments) {
#pragma unroll
          for (int t = 0; t < XL; ++t) now.x[kw][2 * (nw + NW * t) + (lane >> 5)][lane & 31] = xv[t];
        }
      }
      stage_barrier();
      if (seg + KW < segments) {
        fetch_weights(a, stage.buffer[1 - buf], seg + KW, kw, nw, lane);
        fetch_x(a, stage.buffer[1 - buf], seg + KW, kw, nw, lane);
      }
      if (seg >= segments) continue;
      const Wave& mine = now.w[kw][nw];
      u32x4 codes[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) codes[j] = exchange_units(mine.codes[r][(2 * g + j) ^ (r & 7)]);
      uint32_t scale[kAsym ? 2 : 8], zero[2];
      if constexpr (kAsym) {
        const uint32_t* sc = &mine.scales[0][0];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          scale[h] = sc[2 * r + h];
          zero[h] = sc[64 + 2 * r + h];
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(&mine.scales[r][4 * h]);
          scale[4 * h] = v.x; scale[4 * h + 1] = v.y; scale[4 * h + 2] = v.z; scale[4 * h + 3] = v.w;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the asymmetric format's groups: blocks 4 h .. 4 h + 3
        f32x4 part[MF], sx[MF];
        const float z = kAsym ? (float)zero[h] : 8.0f, step = 1.0f / kStep<F, DT>;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int b = 4 * h + q, i = b >> 1, j = b & 1;
          const u32x4 wv = unit_values<F, DT, SIGNED>(codes[j][i], z * step);
          const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)scale[kAsym ? h : b]) * kStep<F, DT>;
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            const u32x4 x = now.x[kw][16 * m + r][(4 * b + g) ^ (r & 7)];
            if constexpr (kAsym && !SIGNED) {
              part[m] = mfma<DT>(x, wv, q ? part[m] : none);
              sx[m] = mfma<DT>(x, factors, q ? sx[m] : none);
            } else {
              f32x4 p = none;
              if constexpr (kZeros && !SIGNED) p = mfma<DT>(x, factors, none);
              p = mfma<DT>(x, wv, p);
#pragma unroll
              for (int t = 0; t < 4; ++t) acc[m][t] = __builtin_fmaf(d, p[t], acc[m][t]);
            }
          }
        }
        if constexpr (kAsym && !SIGNED) {
          const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)scale[h]) * kStep<F, DT>;
#pragma unroll
          for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t)
              acc[m][t] = __builtin_fmaf(d, __builtin_fmaf(-z, sx[m][t], part[m][t]), acc[m][t]);
        }
      }
    }
  }
};

template <int F, int DT, bool GATED, int MF, int NW, int KW, bool ALIGNED>
__global__ __launch_bounds__(kWave* NW* KW) void few_rows_kernel(ProductArgs a) {
  using T = FewRows<F, DT, MF, NW, KW, ALIGNED>;
  constexpr int HALVES = GATED ? 2 : 1;
  constexpr int NF = NW / HALVES;  // column fragments of y
  __shared__ typename T::Stage stage;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int kw = wave / NW, nw = wave % NW;
  const int r = lane & 15, g = lane >> 4;
  const int nt = blockIdx.x % a.ntiles;
  RowTile rt = find_rows<16 * MF>(a, a.tile0 + blockIdx.x / a.ntiles);
  if (rt.m0 >= rt.m1) return;
  rt.zero |= a.xrows == 0;  // every row number is out of range then
  const int n0 = nt * 16 * NF;

  if (!rt.zero) {
    T t;
    const int c0 = n0 + 16 * (nw % NF);  // first weight row of the wave, of the gate or the up rows
    const long long row0 = ((long long)rt.expert * HALVES + nw / NF) * a.n;
    const long long first = (row0 + n0) * a.blocks;
    t.w = a.w + (first >> 6) * Format<F>::kTileBytes;
    // columns past the last repeat it
    auto block_of = [&](int c) {
      return (uint32_t)(first & 63) + (uint32_t)((c < a.n ? c : a.n - 1) - n0) * (uint32_t)a.blocks;
    };
#pragma unroll
    for (int q = 0; q < 2; ++q) t.cblock[q] = block_of(c0 + 8 * q + (lane >> 3));
    t.gblock = block_of(c0 + (lane >> 1) % 16);
    t.begin(a, stage, kw, nw, lane, [&] {
#pragma unroll
      for (int i = 0; i < T::XL; ++i) {
        // rows past the end repeat the last, rows of no source the first of x
        const int m = rt.m0 + 2 * (nw + NW * i) + (lane >> 5);
        const long long s = source_row(a, m < rt.m1 ? m : rt.m1 - 1);
        const long long at = 2 * (s < 0 ? 0 : s) * a.ldx + 16 * T::unit_of(lane, i, nw);
        if constexpr (ALIGNED)
          t.xoff[i] = (uint32_t)at;
        else
          t.xrow[i] = a.x + at;
      }
    });
    t.template sum<false>(a, stage, kw, nw, lane);
    if constexpr (T::kZeros) {
      bool finite = true;
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) finite &= __builtin_fabsf(t.acc[i][j]) < __builtin_inff();
      // the waves share x, so they decide together
      if (__syncthreads_or(!finite)) {
        f32x4 was[MF];
#pragma unroll
        for (int i = 0; i < MF; ++i) was[i] = t.acc[i];
        t.begin(a, stage, kw, nw, lane, [] {});
        t.template sum<true>(a, stage, kw, nw, lane);
        // the finite ones stay as they are, so that no row depends on another
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (__builtin_fabsf(was[i][j]) < __builtin_inff()) t.acc[i][j] = was[i][j];
      }
    }
    __syncthreads();  // every wave is done with the segments
#pragma unroll
    for (int i = 0; i < MF; ++i) stage.sums[kw][nw][i][lane] = t.acc[i];
  }
  __syncthreads();
  // fragment (i, f) of y is joined and stored by wave (i NF + f) % (KW NW)
  for (int frag = wave; frag < MF * NF; frag += KW * NW) {
    const int i = frag / NF, f = frag % NF;
    f32x4 s[HALVES];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      s[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (!rt.zero) {
#pragma unroll
        for (int k = 0; k < KW; ++k) s[h] += stage.sums[k][h * NF + f][i][lane];
      }
    }
    const int c = n0 + 16 * f + r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = rt.m0 + 16 * i + 4 * g + j;
      if (m >= rt.m1 || c >= a.n) continue;
      const float v = GATED ? gate(s[0][j], s[HALVES - 1][j]) : s[0][j];
      const bool real = !rt.zero && source_row(a, m) >= 0;
      *reinterpret_cast<uint16_t*>(a.y + 2 * (m * a.ldy + c)) = (uint16_t)pack2<DT>(real ? v : 0.0f, 0.0f);
    }
  }
}

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

// The 8 values of a unit without the scale, four at a time: exact in either
// dtype, and in steps of 1 / kStep.
template <int F, int DT>
struct UnitHalves {
  static constexpr float kValue = 1.0f / kStep<F, DT>;
  uint32_t a, b;
  __device__ __forceinline__ void set(uint32_t w) {
    if constexpr (Format<F>::kFp4) {
      a = w;
    } else {
      const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;  // values 0 2 4 6 and 1 3 5 7
      a = DT == kFp16 ? __builtin_amdgcn_perm(hi, lo, 0x05010400u) : lo;
      b = DT == kFp16 ? __builtin_amdgcn_perm(hi, lo, 0x07030602u) : hi;
    }
  }
  // Values 4 J .. 4 J + 3.
  template <int J>
  __device__ __forceinline__ u32x2 four(uint32_t zero) const {
    if constexpr (Format<F>::kFp4) {
      if constexpr (DT == kFp16)
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(a, 1.0f, 2 * J)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(a, 1.0f, 2 * J + 1))};
      else
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, kValue, 2 * J)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, kValue, 2 * J + 1))};
    } else if constexpr (DT == kFp16) {
      // bytes c 0x64 are the fp16 value 1024 + c; 0xE400 + zero is -1024 - zero
      const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)(0xE400u + (Format<F>::kAsym ? zero : 8u)));
      auto pair = [&](uint32_t sel) {
        const uint32_t t = __builtin_amdgcn_perm(0x64646464u, J ? b : a, sel);
        return __builtin_bit_cast(uint32_t, (f16x2)(__builtin_bit_cast(f16x2, t) + f16x2{z, z}));
      };
      return u32x2{pair(0x04010400u), pair(0x04030402u)};
    } else {
      // the byte c as FP8 E4M3 is c / 512 for every 4-bit c
      const float z = (float)zero * kValue;
      const f32x2 v02 = __builtin_amdgcn_cvt_pk_f32_fp8((int)a, J != 0), v13 = __builtin_amdgcn_cvt_pk_f32_fp8((int)b, J != 0);
      return u32x2{pack2<DT>(v02.x - z, v13.x - z), pack2<DT>(v02.y - z, v13.y - z)};
    }
  }
};

// A workgroup of WM x WN waves computes a tile of WM MFR 16 rows of x by WN NFR
// 16 weight rows, each wave MFR x NFR fragments of it, in stages of 64 values
// of k.  A stage's x and a chunk's codes and scales (128 values: a load costs
// the address unit as much for 32 bytes of a row as for 64) go to LDS without a
// stop in registers, while the one before is multiplied.  Each wave decodes the
// weights it multiplies, codes less zero points, straight into the matrix unit's
// B: they pass LDS once, in 4 bits, and the work of a decode is shared by MFR
// products.  x is the unit's A, so that a lane's results belong to one weight
// row, whose scale it applies to them.
//
// LDS: row m of x is 8 units of 16 bytes, unit u at place u ^ (m & 7), so that
// 8 lanes that read one unit of 8 rows hit 8 groups of banks; the lanes that
// load it take their units in that order.
//
// A lane's results are 4 rows of x in one column.  The column fragments of a
// wave interleave (lane r of fragment f has column OUT r + f), so that a lane
// has OUT neighbours of a row and 16 lanes a run of it.  Gated: the first half of
// a wave's fragments are gate rows, the second the same columns' up rows.
//
// A wave goes through the weight fragments of a step of 32 values of k one
// after another, each by all rows of x: x stays in registers for the step, and
// only two decoded fragments do, the present and the next.
//
// Bound by the issue of instructions: a product takes 4 FMAs for the scale and
// (int4 bf16, MFR = 8) 2.4 instructions for its share of a decode, 8.6 with
// itself and the rest, of 4 cycles each, where it keeps the matrix unit busy for
// 16 (the vector unit issues in 87 % of the cycles, the matrix unit is busy in 40).  8192 tokens, 2 of 16 experts, gated, n = k = 4096, int4
// bf16: 1366 us, 805 TFLOP/s; of 1404 on another card, 1087 without the scale's
// FMAs, 1171 without the decode, 1236 without the loads, 975 without the last two.
// 1024 x 8192 x 8192 int4 bf16: 165 us, 830 TFLOP/s.  1000 tokens, 4 of 40
// experts, 1001 x 2080, fp4 fp16: 51 us, where a tile's 33 stages are too few to
// hide the trips to memory that begin it.
//
// Weights rounded to the dtype before the product need no FMAs for the scale:
// 1164, 135 and 49 us, with errors of 2.9e-3, 2.4e-3 and 2.7e-4 instead of the
// 1.7e-3, 1.7e-3 and 2.1e-4 that the rounding of y has.
//
// Slower here: branches around loads past the end (1452 us where this kernel was
// at 1363), two products between a product and its scale instead of three (1535
// and 1517, one 1554), tiles of 256 x 128 and of 128 x 256 for 8 waves in grouped
// products (1950 and 1920 where it was at 1480), tiles of 128 x 128 (1523; 2048
// rows, gated, of 4096 x 4096 int4 fp16 186 and 167).
constexpr int kStage = 64;
constexpr int kStageBlocks = kStage / kBlockValues;

// Tile of the launch's index space that workgroup `id` of `total` computes.
// Workgroups are dealt to the 8 XCDs in turn; each XCD takes a contiguous run
// of tiles, ordered in bands of kBand row tiles by all column tiles, so that
// the tiles that run on it at one time share rows of x and of the weight in
// its L2.
constexpr int kBand = 4;
struct TileIndex {
  int row, col;
};
__device__ __forceinline__ TileIndex tile_index(int id, int total, int ncols) {
  const int per = total / kXCDs, rest = total % kXCDs, xcd = id % kXCDs;
  const int t = xcd * per + (xcd < rest ? xcd : rest) + id / kXCDs;
  const int rows = total / ncols, band = t / (kBand * ncols), in = t - band * kBand * ncols;
  const int height = rows - band * kBand < kBand ? rows - band * kBand : kBand;
  return {band * kBand + in % height, in / height};
}

template <int F, int DT, bool GATED, int WM, int WN, int MFR, int NFR, bool ALIGNED>
__global__ __launch_bounds__(kWave* WM* WN, 2) void many_rows_kernel(ProductArgs a) {
  constexpr int WAVES = WM * WN, HALVES = GATED ? 2 : 1;
  constexpr int OUT = NFR / HALVES;               // column fragments of y of one wave
  static_assert(OUT * HALVES == NFR, "as many gate as up fragments");
  constexpr int BM = 16 * WM * MFR, BN = 16 * WN * NFR;
  constexpr int COLS = 16 * NFR / HALVES;         // columns of y of one wave
  constexpr int XI = BM / 8 / WAVES;              // loads of x of one wave in a stage: 8 rows each
  static_assert(XI * 8 * WAVES == BM, "the waves share the loads of x evenly");
  constexpr int WL = BN / 16 / WAVES;             // loads of codes of one wave in a chunk: a fragment's rows each
  static_assert(WL * 16 * WAVES == BN && WL <= MFR, "the waves share the loads of codes evenly");
  static_assert(XI <= MFR, "a load of x goes with each row of the first step's products");
  constexpr int kAhead = MFR >= 8 ? 1 : 2;        // fragments between the read of codes and their decode
  constexpr uint32_t TB = Format<F>::kTileBytes;
  constexpr bool kAsym = Format<F>::kAsym;
  struct Weights {
    u32x4 codes[BN][kChunkBlocks];
    uint32_t scales[BN][kChunkBlocks];              // asymmetric: the group's, four times
    uint32_t zeros[kAsym ? BN : 1][kChunkBlocks];
  };
  // The first fragment of a stage is decoded while the last of the one before it
  // is multiplied, and x of its first step read: a stage's x is asked for a stage
  // ahead, and a chunk's weights in the second stage of the one before it.
  __shared__ u32x4 lds_x[2][BM][8];
  __shared__ Weights lds_w[2];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int r = lane & 15, g = lane >> 4;
  const TileIndex ti = tile_index(blockIdx.x, gridDim.x, a.ntiles);
  RowTile rt = find_rows<BM>(a, a.tile0 + ti.row);
  if (rt.m0 >= rt.m1) return;
  rt.zero |= a.xrows == 0;  // every row number is out of range then
  const int n0 = ti.col * (BN / HALVES);

  f32x4 acc[MFR][NFR];
#pragma unroll
  for (int i = 0; i < MFR; ++i)
#pragma unroll
    for (int f = 0; f < NFR; ++f) acc[i][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (!rt.zero) {
    // weights: row R of the tile is a column of its half; columns past the last
    // repeat it.  Load l of this wave brings fragment WAVES l + wave, row lane / 4
    const long long row0 = (long long)rt.expert * HALVES * a.n + n0;
    const uint8_t* wbase[WL];
    uint32_t wblock[WL];  // first block of the lane's row, from wbase
#pragma unroll
    for (int l = 0; l < WL; ++l) {
      const int part = WAVES * l + wave, f = part % NFR, q = lane >> 2;
      const int half = f / OUT, ff = f % OUT;
      const int in = COLS * (part / NFR) + OUT * q + ff;
      const long long first = (row0 + (long long)half * a.n) * a.blocks;
      wbase[l] = a.w + (first >> 6) * TB;
      wblock[l] = (uint32_t)(first & 63) + (uint32_t)(n0 + in < a.n ? in : a.n - 1 - n0) * (uint32_t)a.blocks;
    }

    // x: load i of this wave brings rows 8 (XI wave + i) + lane / 8 of the tile,
    // unit (lane & 7) ^ (row & 7); rows past the end repeat the last, rows of no
    // source the first of x
    const int unit = (lane & 7) ^ (lane >> 3);
    const uint8_t* xrow[ALIGNED ? 1 : XI];
    uint32_t xoff[XI];
    const int last = a.blocks - 1;
    const int stages = (a.k + kStage - 1) / kStage;  // each has values of x
    u32x4 xv[ALIGNED ? 1 : XI];
    auto fetch_weights = [&](int chunk, int buf, int l) {
      const int kb = chunk * kChunkBlocks + ((lane & 3) ^ (lane >> 4));
      // past the last: that one, times zeros of x
      const uint32_t b = wblock[l] + (uint32_t)(kb < last ? kb : last), at = (b >> 6) * TB, in = b & 63;
      const uint32_t to = lds_address(&lds_w[0]) + (uint32_t)(sizeof(Weights) * buf);
      const int part = WAVES * l + wave;
      load_to_lds(wbase[l], at + in * 16, to + (uint32_t)(1024 * part));
      load_value_to_lds<2>(wbase[l], at + Format<F>::kScaleOffset + (kAsym ? in >> 2 : in) * 2,
                           to + (uint32_t)(offsetof(Weights, scales) + 256 * part));
      if constexpr (kAsym)
        load_value_to_lds<1>(wbase[l], at + Format<F>::kZeroOffset + (in >> 2),
                             to + (uint32_t)(offsetof(Weights, zeros) + 256 * part));
    };
    // Rows that begin on 16 bytes (ALIGNED) go to LDS directly, others pass through
    // registers.  Stages past the last repeat the row's end, for nobody.
    auto fetch_x = [&](int st, int buf, int i) {
      if constexpr (ALIGNED) {
        const uint32_t to = lds_address(&lds_x[0][0][0]) + (uint32_t)(BM * 128 * buf + 1024 * (XI * wave + i));
        const uint32_t in = (uint32_t)(kStage * st + 8 * unit), end = (uint32_t)a.k - 8;
        load_to_lds(a.x, xoff[i] + 2 * (in < end ? in : end), to);
      } else {
        if (kStage * (st + 1) <= a.k)
          xv[i] = *reinterpret_cast<const u32x4_any*>(xrow[i] + 2 * kStage * (size_t)st);
        else
          xv[i] = load_x8_tail(xrow[i] - 16 * unit, kStage * st + 8 * unit, a.k);
      }
    };
    // A step is 32 values of k, one block: fragment s = NFR b + f of a stage is
    // weight fragment f in step b.  While the products of one fragment are
    // issued, the next one is decoded and the codes of the kAhead-th next are
    // read from LDS.
    constexpr int kSteps = kStageBlocks * NFR;
    const int p0 = r >> 2;
    u32x4 wv[2], x[MFR];
    float d[2];
    uint32_t code[kAhead], scale[kAhead], zero[kAhead];
    auto read_codes = [&](const Weights& w, int block, int f, int slot) {
      const int R = 16 * (NFR * wn + f) + r, p = block ^ p0;
      code[slot] = reinterpret_cast<const uint32_t*>(&w.codes[R][p])[g];
      scale[slot] = w.scales[R][p];
      zero[slot] = kAsym ? w.zeros[kAsym ? R : 0][p] : 8u;
    };
    UnitHalves<F, DT> half;
    // Half j of a fragment's unit.
    auto decode = [&](u32x4& to, int slot, int j) {
      if (j == 0) {
        half.set(code[slot]);
        const u32x2 v = half.template four<0>(zero[slot]);
        to.x = v.x;
        to.y = v.y;
      } else {
        const u32x2 v = half.template four<1>(zero[slot]);
        to.z = v.x;
        to.w = v.y;
      }
    };
    auto scale_of = [&](int slot) {
      return (float)__builtin_bit_cast(_Float16, (uint16_t)scale[slot]);
    };
    // The block's scale is applied to a product's sums kLag products later, when they are there.
    constexpr int kLag = 3, kRing = 4;
    static_assert(MFR % kRing == 0 && NFR % 2 == 0, "rings begin anew with each fragment, and with each step");
    f32x4 part[kRing];
    auto add_part = [&](int q) {  // product q of a step, from -kLag on
      const int f = q < 0 ? NFR - 1 : q / MFR, i = (q + MFR) % MFR;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        acc[i][f][t] = __builtin_fmaf(d[f & 1], part[(q + kRing) % kRing][t], acc[i][f][t]);
      asm volatile("" : "+v"(acc[i][f]));  // here, not where the loop ends
    };

    // The first weights need not wait for the numbers of the rows of x, which are
    // a trip to memory of their own.
#pragma unroll
    for (int l = 0; l < WL; ++l) fetch_weights(0, 0, l);
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int m = rt.m0 + 8 * (XI * wave + i) + (lane >> 3);
      const long long s = source_row(a, m < rt.m1 ? m : rt.m1 - 1);
      const long long at = 2 * (s < 0 ? 0 : s) * a.ldx;
      if constexpr (ALIGNED)
        xoff[i] = (uint32_t)at;
      else
        xrow[i] = a.x + at + 16 * unit;
    }
#pragma unroll
    for (int i = 0; i < XI; ++i) fetch_x(0, 0, i);
    // Everything asked for is there, x of stage `st` in buffer `buf`, for every wave, and every
    // wave has read what lay in the buffers that are asked for next.
    auto arrived = [&](int st, int buf) {
      loads_done<0>();
      if constexpr (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < XI; ++i) lds_x[buf][8 * (XI * wave + i) + (lane >> 3)][lane & 7] = xv[i];
      } else if (kStage * (st + 1) > a.k) {  // zeros past the row's end
        if (kStage * st + 8 * unit >= a.k) {
#pragma unroll
          for (int i = 0; i < XI; ++i)
            lds_x[buf][8 * (XI * wave + i) + (lane >> 3)][lane & 7] = u32x4{0u, 0u, 0u, 0u};
        }
      }
      stage_barrier();
    };
    arrived(0, 0);
#pragma unroll
    for (int i = 0; i < XI; ++i) fetch_x(1, 1, i);
    auto read_x = [&](int buf, int b, int i) { x[i] = lds_x[buf][16 * (MFR * wm + i) + r][(4 * b + g) ^ (r & 7)]; };
#pragma unroll
    for (int s = 0; s < kAhead; ++s) read_codes(lds_w[0], 0, s, s);
#pragma unroll
    for (int i = 0; i < MFR; ++i) read_x(0, 0, i);
#pragma unroll
    for (int j = 0; j < 2; ++j) decode(wv[0], 0, j);
    d[0] = scale_of(0);
    d[1] = 0.0f;
#pragma unroll
    for (int q = 0; q < kRing; ++q) part[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // Stage st, the first (H = 0) or second of a chunk whose weights are in buffer wb.
    auto multiply = [&](auto H, int st, int wb) __attribute__((always_inline)) {
      constexpr int h = decltype(H)::value;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int b = s / NFR, f = s % NFR;
        // The next stage's x, and the next chunk's weights if it begins one, have to be
        // there kAhead fragments before the end, and the x of this one is in registers by then.
        if (s == kSteps - kAhead) arrived(st + 1, 1 - h);
        const int to = s + kAhead;  // whose codes are read
        if (to < kSteps)
          read_codes(lds_w[wb], kStageBlocks * h + to / NFR, to % NFR, to % kAhead);
        else
          read_codes(lds_w[h ? 1 - wb : wb], kStageBlocks * (1 - h), to % NFR, to % kAhead);
        __builtin_amdgcn_sched_barrier(0);
        // The matrix unit and the vector unit work side by side: a product, then the scaling
        // of an earlier one's sums and half of the next fragment's unit.  The compiler would
        // put them one after another; it is held to this order.
#pragma unroll
        for (int i = 0; i < MFR; ++i) {
          part[i % kRing] = mfma<DT>(x[i], wv[s & 1], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
          add_part(f * MFR + i - kLag);
          if (i % 2 == MFR / 8 && i >= MFR - 4) decode(wv[(s + 1) & 1], (s + 1) % kAhead, (i - (MFR - 4)) / 2);
          if (i == MFR - 1) {
            d[(s + 1) & 1] = scale_of((s + 1) % kAhead);
            asm volatile("" : "+v"(wv[(s + 1) & 1]), "+v"(d[(s + 1) & 1]));
          }
          if (f == NFR - 1) read_x(b ? 1 - h : h, 1 - b, i);
          __builtin_amdgcn_sched_barrier(0);
          if (s == kSteps - 1 && i < XI) {
            fetch_x(st + 2, h, i);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (s == 0 && i < WL && h) {
            fetch_weights((st >> 1) + 1, 1 - wb, i);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    };
    for (int st = 0; st < stages; st += 2) {
      multiply(std::integral_constant<int, 0>{}, st, (st >> 1) & 1);
      if (st + 1 < stages) multiply(std::integral_constant<int, 1>{}, st + 1, (st >> 1) & 1);
    }
    loads_done<0>();  // what was asked for past the end: LDS is the next workgroup's soon
#pragma unroll
    for (int q = -kLag; q < 0; ++q) add_part(q);
  }

  // which of the wave's rows have a source: bit m & 63 of word m / 64
  unsigned long long sources[MFR / 4];
#pragma unroll
  for (int q = 0; q < MFR / 4; ++q) {
    const int m = rt.m0 + 16 * MFR * wm + 64 * q + lane;
    sources[q] = __ballot(!rt.zero && m < rt.m1 && source_row(a, m) >= 0);
  }
#pragma unroll
  for (int i = 0; i < MFR; ++i) {
    const int in = 16 * (MFR * wm + i) + 4 * g, c = n0 + COLS * wn + OUT * r;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (rt.m0 + in + t >= rt.m1) continue;
      const bool real = (sources[i / 4] >> (16 * (i % 4) + 4 * g + t)) & 1;
      uint8_t* to = a.y + 2 * ((long long)(rt.m0 + in + t) * a.ldy + c);
      float v[OUT + 1];
#pragma unroll
      for (int p = 0; p < OUT; ++p) {
        const float h = acc[i][p][t] * kStep<F, DT>;
        v[p] = !real ? 0.0f : GATED ? gate(h, acc[i][p + (GATED ? OUT : 0)][t] * kStep<F, DT>) : h;
      }
      v[OUT] = 0.0f;
      uint16_t o[OUT + 1];
#pragma unroll
      for (int p = 0; p < OUT; p += 2) {
        const uint32_t two = pack2<DT>(v[p], v[p + 1]);
        o[p] = (uint16_t)two;
        o[p + 1] = (uint16_t)(two >> 16);
      }
      if (c + OUT <= a.n) {
        __builtin_memcpy(to, o, 2 * OUT);
      } else {
#pragma unroll
        for (int p = 0; p < OUT; ++p)
          if (c + p < a.n) reinterpret_cast<uint16_t*>(to)[p] = o[p];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------

// Launches `kernel` for row tiles of `bm` rows and column tiles of `bc` columns
// of y, as many row tiles at a time as a launch holds (one always fits: at most
// n / 4 column tiles of 512 threads).
template <typename ARGS>
qr_status launch_tiles(void (*kernel)(ARGS), ARGS a, int bm, int bc, int threads, hipStream_t st) {
  static_assert(QR_MAX_N / 4 * 512LL < 0xffffffffLL, "a row tile fits a launch");
  a.ntiles = (a.n + bc - 1) / bc;
  const long long tiles = row_tiles(a.slots, a.experts, !a.offsets, bm);
  const long long fit = kMaxLaunchThreads / ((long long)a.ntiles * threads), most = fit > 1 ? fit : 1;
  for (long long t = 0; t < tiles; t += most) {
    const long long now = tiles - t < most ? tiles - t : most;
    a.tile0 = (int)t;
    void* argv[] = {&a};
    if (hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)(now * a.ntiles)), dim3(threads), argv, 0,
                        st) != hipSuccess)
      return QR_ERR_HIP;
  }
  return QR_OK;
}

qr_status launch_product_int4(int dt, bool gated, const ProductArgs& a, hipStream_t st);
qr_status launch_product_asym4(int dt, bool gated, const ProductArgs& a, hipStream_t st);
qr_status launch_product_fp4(int dt, bool gated, const ProductArgs& a, hipStream_t st);

}  // namespace qr
