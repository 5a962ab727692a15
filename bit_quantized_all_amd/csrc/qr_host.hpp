// qr_host.hpp -- what the entry points of the layer operators share on the host:
// argument checks (no HIP call), and the launch of a one-dimensional grid.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qr.h"

namespace qr {

static inline bool bad_dtype(int dt) { return dt != QR_FP16 && dt != QR_BF16; }
static inline bool misaligned(const void* p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

static inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return na && nb && a0 < b0 + nb && b0 < a0 + na;
}

// Bytes from the first to the last value of `rows` rows of `cols` 2-byte values.
static inline size_t span(size_t rows, size_t ld, size_t cols) { return rows ? 2 * ((rows - 1) * ld + cols) : 0; }

// Whether two matrices share a value.  Rows of one stride may lie beside each
// other in a larger matrix (columns of it): there the distance of the first rows,
// within a stride, tells.  A matrix of one row has the other's stride.
static inline bool overlap_rows(const void* a, size_t ra, size_t lda, size_t ca, const void* b, size_t rb, size_t ldb, size_t cb) {
  if (!overlap(a, span(ra, lda, ca), b, span(rb, ldb, cb))) return false;
  const size_t ld = 2 * (ra > 1 ? lda : ldb);
  if (ra > 1 && rb > 1 && lda != ldb) return true;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  const size_t from = b0 >= a0 ? (b0 - a0) % ld : (ld - (a0 - b0) % ld) % ld;  // of b's row, from a's
  return from < 2 * ca || from + 2 * cb > ld;
}

// Row strides up to 2^32 values keep every byte offset of 2^30 rows within 63 bits.
constexpr size_t kMaxStride = (size_t)1 << 32;

// (The caller sees to it that a launch holds fewer than 2^32 threads.)
template <typename... P>
static inline qr_status launch_1d(void (*kernel)(P...), long long groups, int threads, hipStream_t st, P... args) {
  void* argv[] = {static_cast<void*>(&args)...};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)groups), dim3(threads), argv, 0, st) ==
                 hipSuccess
             ? QR_OK
             : QR_ERR_HIP;
}

}  // namespace qr
