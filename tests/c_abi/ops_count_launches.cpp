// ops_count_launches.cpp -- a stand-in for the HIP launch that counts launches and
// threads, and a driver of qr_combine on sizes whose threads exceed one launch (see
// tests/test_ops_launches.py).  Addresses are never read; no GPU work is launched.
#include <hip/hip_runtime.h>

#include <cstdio>

#include "qr.h"
#include "qr_ops.h"
#include "qr_product.hpp"

static unsigned long long launches, threads, largest;

extern "C" hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
  const unsigned long long t = (unsigned long long)grid.x * grid.y * grid.z * block.x * block.y * block.z;
  ++launches;
  threads += t;
  largest = t > largest ? t : largest;
  return hipSuccess;
}

namespace qr {
qr_status launch_product_int4(int, bool, const ProductArgs&, hipStream_t) { return QR_ERR_HIP; }
qr_status launch_product_asym4(int, bool, const ProductArgs&, hipStream_t) { return QR_ERR_HIP; }
qr_status launch_product_fp4(int, bool, const ProductArgs&, hipStream_t) { return QR_ERR_HIP; }
}  // namespace qr

int main() {
  const size_t sizes[][3] = {{64, 8, 2048}, {(size_t)1 << 23, 2, 4096}, {((size_t)1 << 24) + 3, 63, 7}, {((size_t)1 << 20) + 1, 1, 1 << 16},
                             {300, 1, QR_MAX_N}, {(size_t)1 << 30, 1, 9}, {((size_t)1 << 22) + 1, 4, 16388}};
  for (const auto& s : sizes) {
    launches = threads = largest = 0;
    const int st = qr_combine(QR_BF16, (void*)0x100000000000, s[2], 1024, (const int32_t*)0x200000000000,
                              (const float*)0x280000000000, (void*)0x300000000000, s[2], s[0], s[1], s[2], nullptr);
    std::printf("%zu %zu %d %llu %llu %llu\n", s[0], s[2], st, launches, threads, largest);
  }
  return 0;
}
