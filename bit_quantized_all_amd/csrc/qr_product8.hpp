// qr_product8.hpp -- gfx950 kernels of the products of 8-bit rows
// (include/qr_rows.h): y = x W^T for one weight or one per group of rows.
//
// y[m][c] = (sum over k of x[m][k] w[c][k]) xs[m] ws[c], codes of signed bytes.
// The sum is a whole number below 2^31 (k <= QR_MAX_ROW_K), which the matrix
// unit's 32-bit sums hold without rounding, in whatever order they are taken; so
// k may be shared out at will.  It is rounded once, to fp32, when it is scaled.
#pragma once

#include "qr_product.hpp"
#include "qr_rows.h"

namespace qr {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kRowRun = 128;  // bytes that a row of codes is padded to a multiple of

// Dense products have offsets == nullptr and one expert; `blocks` counts the
// runs of a row.
struct Product8Args : ProductArgs {
  const float* xs;
  const float* ws;
};

// A sum times the scales of its two rows.  |sum| < 2^31: 2^-24 of it times the
// first scale, the largest |x| over 127, stays in the range of fp32, where the sum
// times the scale might leave it though the result does not.
__device__ __forceinline__ float scaled(int sum, float xs, float ws) {
  return (float)sum * (xs * 0x1p-24f) * ws * 0x1p24f;
}

// ---------------------------------------------------------------------------
// fragments from memory
// ---------------------------------------------------------------------------

// One workgroup of KW waves multiplies 16 MF rows of x by 16 NF rows of the
// weight (gated: NF / 2 fragments of the gate rows and as many of the up rows),
// each wave a share of the runs of k.  The matrix unit's product is 16 x 16 x 64:
// lane (r = lane & 15, g = lane >> 4) holds 16 bytes of row r of either side, and
// which bytes of k they are does not matter as long as both sides have the same.
// The weight is the unit's A, so that a lane gets four neighbouring columns of
// one row of y.
template <int DT, bool GATED, int MF, int NF, int KW>
__global__ __launch_bounds__(kWave* KW) void fragments8_kernel(Product8Args a) {
  constexpr int HALVES = GATED ? 2 : 1, OUT = NF / HALVES;
  static_assert(OUT * HALVES == NF, "as many gate as up fragments");
  __shared__ i32x4 sums[KW > 1 ? KW : 1][MF][NF][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, g = lane >> 4;
  RowTile rt = find_rows<16 * MF>(a, a.tile0 + blockIdx.x / a.ntiles);
  if (rt.m0 >= rt.m1) return;
  rt.zero |= a.xrows == 0;  // every row number is out of range then
  const int n0 = (int)(blockIdx.x % a.ntiles) * 16 * OUT;
  const long long row_bytes = (long long)a.blocks * kRowRun;

  i32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[i][f] = i32x4{0, 0, 0, 0};
  if (!rt.zero) {
    // rows past the end repeat the last, rows of no source the first of x, columns past the last the last
    const uint8_t *x[MF], *w[NF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = rt.m0 + 16 * i + r;
      const long long s = source_row(a, m < rt.m1 ? m : rt.m1 - 1);
      x[i] = a.x + (s < 0 ? 0 : s) * row_bytes + 16 * g;
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int c = n0 + 16 * (f % OUT) + r;
      w[f] = a.w + (((long long)rt.expert * HALVES + f / OUT) * a.n + (c < a.n ? c : a.n - 1)) * row_bytes + 16 * g;
    }
    for (int b = wave; b < a.blocks; b += KW) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        i32x4 xv[MF], wv[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) wv[f] = *reinterpret_cast<const i32x4*>(w[f] + (size_t)b * kRowRun + 64 * h);
#pragma unroll
        for (int i = 0; i < MF; ++i) xv[i] = *reinterpret_cast<const i32x4*>(x[i] + (size_t)b * kRowRun + 64 * h);
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int f = 0; f < NF; ++f)
            acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[f], xv[i], acc[i][f], 0, 0, 0);
      }
    }
  }
  if constexpr (KW > 1) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f) sums[wave][i][f][lane] = acc[i][f];
    __syncthreads();
  }
  // fragment (i, f) of y is joined and stored by wave (i OUT + f) % KW
#pragma unroll
  for (int i = 0; i < MF; ++i) {
#pragma unroll
    for (int f = 0; f < OUT; ++f) {
      if (KW > 1 && (i * OUT + f) % KW != wave) continue;
      const int m = rt.m0 + 16 * i + r, c = n0 + 16 * f + 4 * g;
      if (m >= rt.m1 || c >= a.n) continue;
      i32x4 s[HALVES];
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        s[h] = KW > 1 ? sums[0][i][h * OUT + f][lane] : acc[i][h * OUT + f];
#pragma unroll
        for (int k = 1; k < KW; ++k) s[h] += sums[k][i][h * OUT + f][lane];
      }
      const long long src = rt.zero ? -1 : source_row(a, m);
      const float xs = src >= 0 ? a.xs[src] : 0.0f;
      const float* ws = a.ws + (long long)(rt.zero ? 0 : rt.expert) * HALVES * a.n + c;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int cj = c + j < a.n ? j : a.n - 1 - c;
        const float p = scaled(s[0][j], xs, ws[cj]);
        v[j] = GATED ? gate(p, scaled(s[HALVES - 1][j], xs, ws[(GATED ? a.n : 0) + cj])) : p;
        if (src < 0) v[j] = 0.0f;
      }
      uint8_t* to = a.y + 2 * (m * a.ldy + c);
      const u32x2 o = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
      if (c + 4 <= a.n) {
        *reinterpret_cast<u32x2_any*>(to) = o;
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (c + j < a.n) reinterpret_cast<uint16_t*>(to)[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

qr_status launch_product8(int dt, bool gated, const Product8Args& a, hipStream_t st);

}  // namespace qr
