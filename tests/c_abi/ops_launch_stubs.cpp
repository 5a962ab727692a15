// ops_launch_stubs.cpp -- stand-ins for the product launches, so that
// qr_ops.hip links on its own for the host-sanitizer build of the argument
// checks.  A product that passes every check reaches one of them and returns
// QR_ERR_HIP, the sign that the call was accepted; no GPU work is launched.
#include <hip/hip_runtime.h>

#include "qr.h"
#include "qr_product.hpp"

namespace qr {
qr_status launch_product_int4(int, bool, const ProductArgs&, hipStream_t) { return QR_ERR_HIP; }
qr_status launch_product_asym4(int, bool, const ProductArgs&, hipStream_t) { return QR_ERR_HIP; }
qr_status launch_product_fp4(int, bool, const ProductArgs&, hipStream_t) { return QR_ERR_HIP; }
}  // namespace qr
