// qr_product8.hip -- instantiations and launches of the products of 8-bit rows.
#include "qr_product8.hpp"

namespace qr {

template <int DT, bool GATED, int MF, int NF, int KW>
static qr_status launch_fragments(const Product8Args& a, hipStream_t st) {
  return launch_tiles(fragments8_kernel<DT, GATED, MF, NF, KW>, a, 16 * MF, 16 * NF / (GATED ? 2 : 1), kWave * KW, st);
}

template <int DT, bool GATED, int WM, int WN, int MI, int NI>
static qr_status launch_tiles8(const Product8Args& a, hipStream_t st) {
  return launch_tiles(tiles8_kernel<DT, GATED, WM, WN, MI, NI>, a, 16 * WM * MI, 16 * WN * NI / (GATED ? 2 : 1),
                      kWave * WM * WN, st);
}

template <int DT, bool GATED>
static qr_status launch_dtype(const Product8Args& a, hipStream_t st) {
  if (a.slots >= 256) return launch_tiles8<DT, GATED, 2, 4, 8, 4>(a, st);
  return launch_fragments<DT, GATED, 4, 4, 1>(a, st);
}

qr_status launch_product8(int dt, bool gated, const Product8Args& a, hipStream_t st) {
  if (dt == kFp16) return gated ? launch_dtype<kFp16, true>(a, st) : launch_dtype<kFp16, false>(a, st);
  return gated ? launch_dtype<kBf16, true>(a, st) : launch_dtype<kBf16, false>(a, st);
}

}  // namespace qr
