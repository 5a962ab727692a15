// qr_product8.hip -- instantiations and launches of the products of 8-bit rows.
#include "qr_product8.hpp"

namespace qr {

template <int DT, bool GATED, int MF, int NF, int KW>
static qr_status launch_fragments(const Product8Args& a, hipStream_t st) {
  return launch_tiles(fragments8_kernel<DT, GATED, MF, NF, KW>, a, 16 * MF, 16 * NF / (GATED ? 2 : 1), kWave * KW, st);
}

template <int DT, bool GATED, int WM, int WN, int MI, int NI, int NB>
static qr_status launch_tiles8(const Product8Args& a, hipStream_t st) {
  return launch_tiles(tiles8_kernel<DT, GATED, WM, WN, MI, NI, NB>, a, 16 * WM * MI, 16 * WN * NI / (GATED ? 2 : 1),
                      kWave * WM * WN, st);
}

template <int DT, bool GATED, int MF, int NF>
static qr_status launch_fragments(const Product8Args& a, hipStream_t st) {
  // Eight waves share k where there is hardly more than a workgroup a CU: 137 rows of 5003 x 4129, 237
  // workgroups, 19.9 us and 20.8 with four; 64 experts with 8 rows of 1024 x 2048, gated, 2900
  // workgroups, 65 and 52.
  const long long groups = row_tiles(a.slots, a.experts, !a.offsets, 16 * MF) * ((a.n * (GATED ? 2LL : 1LL) + 16 * NF - 1) / (16 * NF));
  return groups <= 320 ? launch_fragments<DT, GATED, MF, NF, 8>(a, st) : launch_fragments<DT, GATED, MF, NF, 4>(a, st);
}

template <int DT, bool GATED>
static qr_status launch_few(int rows, const Product8Args& a, hipStream_t st) {
  // What a CU reads is the rows of x and of the weight of its tile, in all at most 12 to 14 TB/s from L2:
  // the tile is as large, and as square, as still gives most CUs one.
  const long long area = row_tiles(a.slots, a.experts, !a.offsets, 16) * ((a.n + 15) / 16) * (GATED ? 2 : 1);  // fragments
  if (rows <= 16) {
    if (area >= 704) return launch_fragments<DT, GATED, 1, 4>(a, st);
    if (GATED || area >= 352) return launch_fragments<DT, GATED, 1, 2>(a, st);
    if constexpr (!GATED) return launch_fragments<DT, GATED, 1, 1>(a, st);
  }
  if (area >= 2816) {
    // 48 rows a tile where that takes no more of them: 137 rows of 5003 x 4129 18.1 us and 20.0, 96 of 8192 x 8192
    // 28.8 and 32.4.  (At most 256 workgroups come here without groups: see launch_dtype.)
    if (!a.offsets && (a.slots + 47) / 48 == (a.slots + 63) / 64) return launch_fragments<DT, GATED, 3, 4, 8>(a, st);
    return launch_fragments<DT, GATED, 4, 4>(a, st);
  }
  if (area >= 1408) return launch_fragments<DT, GATED, 2, 4>(a, st);
  if (GATED || area >= 512) return launch_fragments<DT, GATED, 2, 2>(a, st);
  if constexpr (!GATED) return launch_fragments<DT, GATED, 2, 1>(a, st);
}

// Tiles of bm x bn rows that a call is cut into, whole ones and the ends of groups: `rows` of a group on
// average, of which some have more than others and every one ends within a tile.
static double tiles_of(const Product8Args& a, bool gated, int bm, int bn) {
  const double cols = (double)((a.n * (gated ? 2LL : 1LL) + bn - 1) / bn);
  if (!a.offsets) return cols * (double)((a.slots + bm - 1) / bm);
  const double each = (double)a.slots / a.experts / bm + 0.7;
  return cols * a.experts * (each > 1.0 ? each : 1.0);
}

template <int DT, bool GATED>
static qr_status launch_dtype(const Product8Args& a, hipStream_t st) {
  const int rows = (int)((a.slots + (long long)a.experts - 1) / a.experts);  // of one expert, on average
  if (rows <= 16) return launch_few<DT, GATED>(rows, a, st);
  // What a round of a tile on every CU costs for a run of k, in ns, measured at 4096 and 8192 (the first round of
  // fragments is 64 x 64 for eight waves): larger tiles take longer than smaller ones, but less for what they do.
  //   rows x n x k           fragments  128x128  128x256  256x256   us
  //   250 x 4096 x 4096           18.5     17.9     27.7     47
  //   512 x 4096 x 4096           33.6     18.1     27.8     47
  //   1024 x 8192 x 8192           236     69.7     59.6     87
  //   4096 x 4096 x 4096           242     76.3     65.3     60.9
  //   8192 x 8192 x 8192          1809                       416
  //   40 experts with 100 rows, 1001 x 2080
  //                               61.2     36.2     28.2     42.8
  //   16 with 1024, gated, 4096 x 4096
  //                               2030      870      679      610
  auto cost = [&](int bm, int bn, int first, int more) {
    const double rounds = __builtin_ceil(tiles_of(a, GATED, bm, bn) / kCUs);
    return rounds <= 1.0 ? (double)first : more * rounds;
  };
  const double few = cost(64, 64, 570, 500), small = cost(128, 128, 620, 620), middle = cost(128, 256, 1000, 1000),
               large = cost(256, 256, 1440, 1440);
  if (few <= small && few <= middle && few <= large) return launch_few<DT, GATED>(rows, a, st);
  if (small <= middle && small <= large) return launch_tiles8<DT, GATED, 2, 4, 4, 2, 4>(a, st);
  if (middle <= large) return launch_tiles8<DT, GATED, 2, 4, 4, 4, 3>(a, st);
  return launch_tiles8<DT, GATED, 2, 4, 8, 4, 2>(a, st);
}

qr_status launch_product8(int dt, bool gated, const Product8Args& a, hipStream_t st) {
  if (dt == kFp16) return gated ? launch_dtype<kFp16, true>(a, st) : launch_dtype<kFp16, false>(a, st);
  return gated ? launch_dtype<kBf16, true>(a, st) : launch_dtype<kBf16, false>(a, st);
}

}  // namespace qr
