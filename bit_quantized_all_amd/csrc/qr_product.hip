// qr_product.hip -- instantiations and launches of the product kernels for one
// weight format (QR_PRODUCT_FMT: 4 = INT4, 20 = ASYM4, 36 = FP4).
#include "qr_product.hpp"

namespace qr {

template <int F, int DT, bool GATED>
static qr_status launch_product(const ProductArgs& args, hipStream_t st) {
  constexpr int MF = 1, NF = 1, WAVES = 8;
  ProductArgs a = args;
  a.ntiles = (a.n + 16 * NF - 1) / (16 * NF);
  const long long groups = row_tiles(a.slots, a.experts, !a.offsets, 16 * MF) * a.ntiles;
  if (groups > 0x7fffffffLL) return QR_ERR_SIZE;
  void* argv[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(few_rows_kernel<F, DT, GATED, MF, NF, WAVES>),
                         dim3((unsigned)groups), dim3(kWave * WAVES), argv, 0, st) == hipSuccess
             ? QR_OK
             : QR_ERR_HIP;
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
