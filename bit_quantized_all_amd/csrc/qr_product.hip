// qr_product.hip -- instantiations and launches of the product kernels for one
// weight format (QR_PRODUCT_FMT: 4 = INT4, 20 = ASYM4, 36 = FP4).
#include "qr_ops.h"
#include "qr_product.hpp"

namespace qr {

// Launches `kernel` for row tiles of `bm` rows and column tiles of `bc` columns
// of y, as many row tiles at a time as a launch holds (one always fits: at most
// n / 4 column tiles of 512 threads).
static qr_status launch_tiles(void (*kernel)(ProductArgs), ProductArgs a, int bm, int bc, int threads, hipStream_t st) {
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

template <int F, int DT, bool GATED, int MR, int KS>
static qr_status launch_row(const ProductArgs& a, hipStream_t st) {
  return launch_tiles(row_kernel<F, DT, GATED, MR, KS>, a, MR, kRowWaves / KS * kRowsPerWave / (GATED ? 2 : 1),
                      kWave * kRowWaves, st);
}

template <int F, int DT, bool GATED, int MR>
static qr_status launch_rows(const ProductArgs& a, hipStream_t st) {
  // Several waves share the k axis where there is more than a slice of it for
  // each, and where the workgroups would not fill the CUs otherwise: 4096 rows
  // of weights of k = 4096, 128 workgroups 6.4 us, 256 with two waves each 6.0;
  // 16384 rows of 8192, 512 workgroups 17.1 us, 2048 with four waves each 21.9.
  const long long groups = row_tiles(a.slots, a.experts, !a.offsets, MR) * a.n * (GATED ? 2 : 1) /
                           (kRowWaves * kRowsPerWave);  // of KS = 1
  if (a.blocks <= kWave || groups >= kCUs) return launch_row<F, DT, GATED, MR, 1>(a, st);
  if (a.blocks <= 2 * kWave || groups >= kCUs / 2) return launch_row<F, DT, GATED, MR, 2>(a, st);
  return launch_row<F, DT, GATED, MR, 4>(a, st);
}

template <int F, int DT, bool GATED, int MF, int NW, int KW, bool ALIGNED>
static qr_status launch_few(const ProductArgs& a, hipStream_t st) {
  return launch_tiles(few_rows_kernel<F, DT, GATED, MF, NW, KW, ALIGNED>, a, 16 * MF, 16 * NW / (GATED ? 2 : 1),
                      kWave * NW * KW, st);
}

// Workgroups of four weight fragments and 16 rows: `quads`.
template <int F, int DT, bool GATED, bool ALIGNED>
static qr_status launch_few_rows(int rows, const ProductArgs& a, hipStream_t st) {
  const long long quads = row_tiles(a.slots, a.experts, !a.offsets, 16) * ((a.n + 63) / 64) * (GATED ? 2 : 1);
  if (rows > 16 && quads > kCUs) {
    // two fragments of rows share a weight's decode: 64 experts with 25 rows
    // each 55 us instead of 74, 100 rows of 4096 x 4096 17 instead of 22; with
    // 8 rows an expert 52 instead of 46.  Two waves share the k axis where
    // there are few workgroups: 64 rows of 8192 x 8192 32 and 50 us, of 16384 x
    // 4096 33 and 31
    if (quads >= 600) return launch_few<F, DT, GATED, 2, 8, 1, ALIGNED>(a, st);
    return launch_few<F, DT, GATED, 2, 4, 2, ALIGNED>(a, st);
  }
  // As many waves share the k axis as it takes to have 4096 waves in all:
  // 16384 rows of 8192, 16 rows of x: 23 us with four, 30 with twice as many
  // workgroups of half the waves; 4096 x 4096 and 8 rows 7.6 us with one
  // fragment a workgroup, 8.6 with two, 13 with four
  if (quads >= 4 * kCUs) return launch_few<F, DT, GATED, 1, 4, 1, ALIGNED>(a, st);
  if (quads >= 192) return launch_few<F, DT, GATED, 1, 4, 4, ALIGNED>(a, st);
  // (one wave would need over 256 registers for rows that pass through them)
  if constexpr (ALIGNED && !GATED) return launch_few<F, DT, GATED, 1, 1, 4, ALIGNED>(a, st);
  return launch_few<F, DT, GATED, 1, 2, 4, ALIGNED>(a, st);
}

template <int F, int DT, bool GATED, int WM, int MFR, int NFR, bool ALIGNED>
static qr_status launch_many(const ProductArgs& a, hipStream_t st) {
  return launch_tiles(many_rows_kernel<F, DT, GATED, WM, 4, MFR, NFR, ALIGNED>, a, 16 * WM * MFR,
                      64 * NFR / (GATED ? 2 : 1), kWave * 4 * WM, st);
}

template <int F, int DT, bool GATED>
static qr_status launch_product(const ProductArgs& a, hipStream_t st) {
  const int rows = (int)((a.slots + (long long)a.experts - 1) / a.experts);  // of one expert, on average
  // groups of unknown sizes: few rows in all
  const int most = a.offsets ? a.slots / 4 : a.slots;
  if (most <= 1) return launch_rows<F, DT, GATED, 1>(a, st);
  if (most <= 2) return launch_rows<F, DT, GATED, 2>(a, st);
  // rows of x that begin on 16 bytes and hold whole 16-byte pieces go to LDS
  // directly, by 32-bit offsets
  const bool aligned = ((uintptr_t)a.x & 15) == 0 && a.ldx % 8 == 0 && a.k % 8 == 0 && a.xrows * a.ldx < (1LL << 31);
  const long long tiles = row_tiles(a.slots, a.experts, !a.offsets, 64) * ((a.n * (GATED ? 2LL : 1LL) + 127) / 128);
  // Few rows, or no more tiles of 64 x 128 than CUs, which one workgroup of
  // four waves would not keep busy: 64 rows of 8192 x 8192 33 us here and 86
  // tiled, 192 rows 82 and 84, 256 rows 82 and 84, 300 rows of 4096 x 4096 42 and
  // 45, 600 of 1024 x 4096 27 and 44, 40 experts with 50 rows of 1024 x 2048 42 and
  // 48; with more tiles, 320 rows of 8192 x 8192 125 and 111, 512 rows 166 and 113
  if (rows <= 64 || tiles <= kCUs)
    return aligned ? launch_few_rows<F, DT, GATED, true>(rows, a, st) : launch_few_rows<F, DT, GATED, false>(rows, a, st);
  if (!aligned) return launch_many<F, DT, GATED, 1, 4, 2, false>(a, st);
  // Tiles of 128 x 256 decode a weight half as often as those of 64 x 128, but
  // leave more of the last one of a group empty, and one of them on a CU is four
  // waves that wait alone.  Groups: 16 experts with 330 rows of 2048 x 4096 (464
  // tiles at most) 154 us and 172, with 256 rows (384 at most, 256 that hold
  // rows) 153 and 134, 8 with 200 rows of 4096 x 4096 (336 at most) 151 and 130, 64
  // with 160 of 1024 x 2048 120 and 94
  const long long large = row_tiles(a.slots, a.experts, !a.offsets, 128) * ((a.n * (GATED ? 2LL : 1LL) + 255) / 256);
  if (a.offsets ? large >= 420 && rows >= 192 : large >= 192) {
    // Up to one large tile a CU, 8 waves share one, of 256 x 128: each SIMD
    // then has two waves to alternate between.  1024 rows of 8192 x 8192 166 us
    // and 180 with 4 waves (205 with 64 x 128), 768 rows 158 and 179 (158); 1536
    // rows 312 and 286
    if (!a.offsets && large <= kCUs) return launch_many<F, DT, GATED, 2, 8, 2, true>(a, st);
    return launch_many<F, DT, GATED, 1, 8, 4, true>(a, st);
  }
  return launch_many<F, DT, GATED, 1, 4, 2, true>(a, st);
}

template <int F>
static qr_status launch_format(int dt, bool gated, const ProductArgs& a, hipStream_t st) {
  if (dt == kFp16) return gated ? launch_product<F, kFp16, true>(a, st) : launch_product<F, kFp16, false>(a, st);
  return gated ? launch_product<F, kBf16, true>(a, st) : launch_product<F, kBf16, false>(a, st);
}

#if QR_PRODUCT_FMT == 4
qr_status launch_product_int4(int dt, bool gated, const ProductArgs& a, hipStream_t st) {
  return launch_format<4>(dt, gated, a, st);
}
#elif QR_PRODUCT_FMT == 20
qr_status launch_product_asym4(int dt, bool gated, const ProductArgs& a, hipStream_t st) {
  return launch_format<20>(dt, gated, a, st);
}
#else
qr_status launch_product_fp4(int dt, bool gated, const ProductArgs& a, hipStream_t st) {
  return launch_format<36>(dt, gated, a, st);
}
#endif

}  // namespace qr
