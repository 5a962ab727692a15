// qr_product.hpp -- gfx950 kernels of the products with 4-bit block weights
// (include/qr_ops.h): y = x W^T for one weight or one per group of rows.
//
// All products run on the matrix unit as v_mfma_f32_16x16x32: A is a fragment
// of 16 weight rows, B one of 16 rows of x, each lane (r = lane & 15, g = lane
// >> 4) holding 8 consecutive k of row r, and the result has, in that lane,
// four consecutive weight rows 4 g .. 4 g + 3 of x row r: a lane stores
// neighbouring values of one row of y.
//
// The order of k inside a product is free as long as both operands agree.  A
// lane loads 16 bytes of codes, one 32-value block (so one scale a load), and
// feeds them unit by unit: in step i of four, lane (r, g) supplies unit i of
// block g of a 128-value chunk, k = 32 g + 8 i .. + 7, of both operands.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qr.h"
#include "qr_codec.hpp"

namespace qr {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// 16- and 8-byte accesses at the alignment of a 2-byte value: rows of odd
// stride are read and written without a special case (gfx950 serves unaligned
// global accesses in hardware).
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;

constexpr int kChunk = 128;        // values of k that one 16-byte load per lane covers
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
// the lanes shows which expert's range holds t.  64 experts a step.
template <int BM>
__device__ __forceinline__ RowTile find_rows(const ProductArgs& a, int t) {
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
  for (int e0 = 0; e0 <= a.experts; e0 += kWave) {
    const int e = e0 + lane;  // e == experts: the rows of no expert
    int lo = 0, hi = 0;
    if (e <= a.experts) {
      lo = clampi(a.offsets[e], 0, a.slots);
      hi = e < a.experts ? clampi(a.offsets[e + 1], 0, a.slots) : a.slots;
    }
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
      return rt;
    }
    before += __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  rt.expert = a.experts;
  rt.m0 = rt.m1 = 0;
  return rt;
}

// Largest number of row tiles that find_rows() can hand out: every group ends
// in at most one partial tile, and no more groups than rows are not empty.
inline long long row_tiles(long long slots, long long experts, bool dense, int bm) {
  if (dense) return (slots + bm - 1) / bm;
  const long long groups = experts + 1 < slots ? experts + 1 : slots;
  return slots / bm + groups;
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

// What decode_unit() needs of a block's scale.  The decoded weight is
// dtype(value * d), the rounding of qr_decode.  For fp16, value is an exact
// fp16 and one packed multiply rounds the product; for bf16 the product is
// exact in fp32 and the conversion to bf16 rounds it.
template <int F, int DT>
struct BlockScale;
template <int F>
struct BlockScale<F, kFp16> {
  f16x2 d, off;  // off: what takes 1024 + code to the signed value
  __device__ __forceinline__ BlockScale() {}
  __device__ __forceinline__ explicit BlockScale(const RawBlock& r) {
    const _Float16 s = __builtin_bit_cast(_Float16, (uint16_t)r.scale);
    d = f16x2{s, s};
    if constexpr (Format<F>::kAsym) {
      // fp16 patterns of 1024 + z, negated
      const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)(0xE400u + r.zero));
      off = f16x2{z, z};
    } else {
      off = f16x2{(_Float16)-1032.0f, (_Float16)-1032.0f};
    }
  }
};
template <int F>
struct BlockScale<F, kBf16> {
  float d, off;  // value * d = (code / 512) * (512 d) + off, both products exact
  __device__ __forceinline__ BlockScale() {}
  __device__ __forceinline__ explicit BlockScale(const RawBlock& r) {
    const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)r.scale);
    if constexpr (Format<F>::kFp4) {
      d = s;
      off = 0.0f;
    } else if constexpr (Format<F>::kAsym) {
      d = s * 512.0f;
      off = (float)r.zero * -s;
    } else {
      d = s * 512.0f;
      off = s * -8.0f;
    }
  }
};

// The 8 values of one unit word as four packed pairs of the dtype.
template <int F, int DT>
__device__ __forceinline__ u32x4 decode_unit(uint32_t w, const BlockScale<F, DT>& s) {
  u32x4 o;
  if constexpr (Format<F>::kFp4) {
    if constexpr (DT == kFp16) {
      // the conversions' scale operand is a power of two: 1, and the block
      // scale is multiplied in afterwards
      o.x = __builtin_bit_cast(uint32_t, (f16x2)(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s.d));
      o.y = __builtin_bit_cast(uint32_t, (f16x2)(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s.d));
      o.z = __builtin_bit_cast(uint32_t, (f16x2)(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s.d));
      o.w = __builtin_bit_cast(uint32_t, (f16x2)(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s.d));
    } else {
      const f32x2 a = fp4_unpack<0>(w), b = fp4_unpack<1>(w), c = fp4_unpack<2>(w), d = fp4_unpack<3>(w);
      o.x = pack2<kBf16>(a.x * s.d, a.y * s.d);
      o.y = pack2<kBf16>(b.x * s.d, b.y * s.d);
      o.z = pack2<kBf16>(c.x * s.d, c.y * s.d);
      o.w = pack2<kBf16>(d.x * s.d, d.y * s.d);
    }
  } else {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;  // values 0 2 4 6 and 1 3 5 7
    if constexpr (DT == kFp16) {
      const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u), b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
      // bytes c 0x64: the fp16 value 1024 + c
      auto pair = [&](uint32_t v, uint32_t sel) {
        const uint32_t t = __builtin_amdgcn_perm(0x64646464u, v, sel);
        return __builtin_bit_cast(uint32_t, (f16x2)((__builtin_bit_cast(f16x2, t) + s.off) * s.d));
      };
      o.x = pair(a, 0x04010400u);
      o.y = pair(a, 0x04030402u);
      o.z = pair(b, 0x04010400u);
      o.w = pair(b, 0x04030402u);
    } else {
      // the byte c as FP8 E4M3 is c / 512 for every 4-bit c
      const f32x2 v02 = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo, false), v46 = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo, true);
      const f32x2 v13 = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi, false), v57 = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi, true);
      auto val = [&](float c) { return __builtin_fmaf(c, s.d, s.off); };
      o.x = pack2<kBf16>(val(v02.x), val(v13.x));
      o.y = pack2<kBf16>(val(v02.y), val(v13.y));
      o.z = pack2<kBf16>(val(v46.x), val(v57.x));
      o.w = pack2<kBf16>(val(v46.y), val(v57.y));
    }
  }
  return o;
}

// ---------------------------------------------------------------------------
// x: 8 values of a row
// ---------------------------------------------------------------------------

// Values k0 .. k0 + 7 of a row; those from k on are zero and are not read.
__device__ __forceinline__ u32x4 load_x8_tail(const uint8_t* row, int k0, int k) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k0 + 8 <= k) {
    v = *reinterpret_cast<const u32x4_any*>(row + 2 * (size_t)k0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k0 + j < k) {
        const uint32_t h = *reinterpret_cast<const uint16_t*>(row + 2 * ((size_t)k0 + j));
        v[j >> 1] |= (j & 1) ? h << 16 : h;
      }
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

// silu(g) * u in fp32.
__device__ __forceinline__ float gate(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// Four neighbouring values of a row of y, columns c .. c + 3 of n.
template <int DT>
__device__ __forceinline__ void store4(uint8_t* row, int c, int n, const float (&v)[4]) {
  const u32x2 p = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
  if (c + 4 <= n) {
    *reinterpret_cast<u32x2_any*>(row + 2 * (size_t)c) = p;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < n) *reinterpret_cast<uint16_t*>(row + 2 * (size_t)(c + i)) = (uint16_t)(p[i >> 1] >> (16 * (i & 1)));
  }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

// One workgroup computes 16 MF rows by 16 NF columns of y.  Its waves share
// the k axis (wave w takes every WAVES-th chunk of 128), each weight block is
// loaded and decoded once for all rows, and the waves' sums are joined through
// LDS in the order of the waves.  Bound by reading the weights; x (16 MF rows)
// comes from the caches.
template <int F, int DT, bool GATED, int MF, int NF, int WAVES>
__global__ __launch_bounds__(kWave * WAVES) void few_rows_kernel(ProductArgs a) {
  constexpr int HALVES = GATED ? 2 : 1;
  constexpr int WF = NF * HALVES;  // weight fragments: NF of the gate rows (or all), NF of the up rows
  __shared__ f32x4 sums[WAVES][MF * WF][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, g = lane >> 4;
  const int nt = blockIdx.x % a.ntiles;
  RowTile rt = find_rows<16 * MF>(a, blockIdx.x / a.ntiles);
  if (rt.m0 >= rt.m1) return;
  rt.zero |= a.xrows == 0;  // every row number is out of range then, and no row of x can stand in
  const int n0 = nt * 16 * NF;

  const uint8_t* xrow[MF];
  bool real[MF];
  if (!rt.zero) {
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int m = rt.m0 + 16 * f + r;
      // rows past the end repeat the last one, which is in the caches
      const long long s = source_row(a, m < rt.m1 ? m : rt.m1 - 1);
      real[f] = s >= 0;
      xrow[f] = a.x + 2 * (real[f] ? s : 0) * a.ldx;
    }
    // the weight rows of this lane, as blocks from the tile that holds the
    // first of them
    const uint8_t* wbase[HALVES];
    uint32_t wblock[WF];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      const long long row0 = ((long long)rt.expert * HALVES + h) * a.n;
      const long long first = (row0 + n0) * a.blocks;
      wbase[h] = a.w + (first >> 6) * Format<F>::kTileBytes;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int c = n0 + 16 * f + r;
        wblock[h * NF + f] = (uint32_t)(first & 63) + (uint32_t)((c < a.n ? c : a.n - 1) - n0) * (uint32_t)a.blocks;
      }
    }
    f32x4 acc[MF][WF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < WF; ++f) acc[i][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int chunks = (a.blocks + kChunkBlocks - 1) / kChunkBlocks;
    for (int c = wave; c < chunks; c += WAVES) {
      const int kb = c * kChunkBlocks + g;
      // past the row's last block: that block again, times zeros of x
      const uint32_t b = (uint32_t)(kb < a.blocks ? kb : a.blocks - 1);
      RawBlock raw[WF];
#pragma unroll
      for (int f = 0; f < WF; ++f) raw[f] = load_raw<F>(wbase[f / NF], wblock[f] + b);
      u32x4 xv[MF][4];
      const int k0 = kBlockValues * kb;
      if (kChunk * (c + 1) <= a.k) {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) xv[i][u] = *reinterpret_cast<const u32x4_any*>(xrow[i] + 2 * (size_t)(k0 + 8 * u));
      } else {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) xv[i][u] = load_x8_tail(xrow[i], k0 + 8 * u, a.k);
      }
#pragma unroll
      for (int f = 0; f < WF; ++f) {
        const BlockScale<F, DT> s(raw[f]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const u32x4 wv = decode_unit<F, DT>(raw[f].codes[u], s);
#pragma unroll
          for (int i = 0; i < MF; ++i) acc[i][f] = mfma<DT>(wv, xv[i][u], acc[i][f]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < WF; ++f) sums[wave][i * WF + f][lane] = acc[i][f];
  } else {
#pragma unroll
    for (int f = 0; f < MF; ++f) real[f] = false;
  }
  __syncthreads();
  // fragment (i, f) of y is joined and stored by wave (i NF + f) % WAVES
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      if ((i * NF + f) % WAVES != wave) continue;
      const int m = rt.m0 + 16 * i + r;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (real[i]) {
        f32x4 s[HALVES];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          s[h] = sums[0][i * WF + h * NF + f][lane];
#pragma unroll
          for (int w = 1; w < WAVES; ++w) s[h] += sums[w][i * WF + h * NF + f][lane];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = GATED ? gate(s[0][j], s[HALVES - 1][j]) : s[0][j];
      }
      if (m < rt.m1) store4<DT>(a.y + 2 * (long long)m * a.ldy, n0 + 16 * f + 4 * g, a.n, v);
    }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------

qr_status launch_product_int4(int dt, bool gated, const ProductArgs& a, hipStream_t st);
qr_status launch_product_asym4(int dt, bool gated, const ProductArgs& a, hipStream_t st);
qr_status launch_product_fp4(int dt, bool gated, const ProductArgs& a, hipStream_t st);

}  // namespace qr
