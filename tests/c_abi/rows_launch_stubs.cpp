// rows_launch_stubs.cpp -- a stand-in for the launch of the 8-bit products and for the
// HIP launch, so that qr_rows.hip links on its own for the host-sanitizer build of the
// argument checks.  A call that passes every check reaches one of them and returns
// QR_ERR_HIP, the sign that it was accepted; no GPU work is launched.
#include <hip/hip_runtime.h>

#include "qr.h"
#include "qr_product8.hpp"

extern "C" hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) { return hipErrorUnknown; }

namespace qr {
qr_status launch_product8(int, bool, const Product8Args&, hipStream_t) { return QR_ERR_HIP; }
}  // namespace qr
