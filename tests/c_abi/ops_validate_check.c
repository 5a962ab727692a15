/* ops_validate_check.c -- drives the argument checks of include/qr_ops.h with
 * addresses that are never read (see tests/test_ops_host_sanitized.py). */
#include <stdint.h>
#include <stdio.h>

#include "qr_ops.h"

static int failures;
#define EXPECT(call, want)                                                            \
  do {                                                                                \
    long long got_ = (long long)(call);                                               \
    if (got_ != (long long)(want)) {                                                  \
      printf("line %d: %s = %lld, not %lld\n", __LINE__, #call, got_, (long long)(want)); \
      ++failures;                                                                     \
    }                                                                                 \
  } while (0)

int main(void) {
  void *x = (void *)0x100000000000, *w = (void *)0x200000000000, *y = (void *)0x300000000000;
  int32_t *o = (int32_t *)0x400000000000, *r = (int32_t *)0x500000000000, *p = (int32_t *)0x600000000000;
  float *g = (float *)0x700000000000;
  const size_t huge[] = {(size_t)-1, (size_t)1 << 63, (size_t)1 << 62, ((size_t)1 << 32) + 1};
  const qr_format fmts[] = {QR_INT4, QR_ASYM4, QR_FP4};
  for (int f = 0; f < 3; ++f) {
    /* accepted, up to the limits */
    EXPECT(qr_linear(fmts[f], QR_FP16, 0, x, 64, w, y, 32, 5, 32, 64, 0), QR_ERR_HIP);
    EXPECT(qr_linear(fmts[f], QR_BF16, 1, x, 1, w, y, 1, 1, 1, 1, 0), QR_ERR_HIP);
    EXPECT(qr_linear(fmts[f], QR_BF16, 0, x, 8, w, y, 1, QR_MAX_SLOTS / 1024, 1, 8, 0), QR_ERR_HIP);
    EXPECT(qr_experts(fmts[f], QR_FP16, 1, x, 128, 7, w, o, r, y, 40, 9, QR_MAX_EXPERTS, 40, 128, 0), QR_ERR_HIP);
    EXPECT(qr_linear(fmts[f], QR_FP16, 0, 0, 64, 0, 0, 32, 0, 32, 64, 0), QR_OK);
    for (int i = 0; i < 4; ++i) {
      const size_t h = huge[i];
      EXPECT(qr_linear(fmts[f], QR_FP16, 0, x, 64, w, y, 32, h, 32, 64, 0), QR_ERR_SIZE);
      EXPECT(qr_linear(fmts[f], QR_FP16, 0, x, h, w, y, 32, 5, 32, 64, 0), QR_ERR_SIZE);
      EXPECT(qr_linear(fmts[f], QR_FP16, 0, x, 64, w, y, h, 5, 32, 64, 0), QR_ERR_SIZE);
      EXPECT(qr_linear(fmts[f], QR_FP16, 0, x, 64, w, y, 32, 5, h, 64, 0), QR_ERR_SIZE);
      EXPECT(qr_linear(fmts[f], QR_FP16, 0, x, 64, w, y, 32, 5, 32, h, 0), QR_ERR_SIZE);
      EXPECT(qr_experts(fmts[f], QR_FP16, 0, x, 64, h, w, o, r, y, 32, 5, 4, 32, 64, 0), QR_ERR_SIZE);
      EXPECT(qr_experts(fmts[f], QR_FP16, 0, x, 64, 5, w, o, r, y, 32, 5, h, 32, 64, 0), QR_ERR_SIZE);
    }
    EXPECT(qr_weight_bytes(fmts[f], (size_t)-1, QR_MAX_K), 0);
    EXPECT(qr_weight_bytes(fmts[f], (size_t)1 << 41, 1), 0);
  }
  for (int i = 0; i < 4; ++i) {
    const size_t h = huge[i];
    EXPECT(qr_route(x, 4, o, r, p, h, 2, 8, 0, 0), QR_ERR_SIZE);
    EXPECT(qr_route(x, 4, o, r, p, 16, h, 8, 0, 0), QR_ERR_SIZE);
    EXPECT(qr_route(x, 4, o, r, p, 16, 2, h, 0, 0), QR_ERR_SIZE);
    EXPECT(qr_route_workspace(h, 2, 8), 0);
    EXPECT(qr_combine(QR_FP16, y, 64, h, p, g, x, 64, 8, 2, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_combine(QR_FP16, y, 64, 16, p, g, x, 64, h, 2, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_combine(QR_FP16, y, 64, 16, p, g, x, 64, 8, h, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_combine(QR_FP16, y, 64, 16, p, g, x, 64, 8, 2, h, 0), QR_ERR_SIZE);
  }
  EXPECT(qr_linear((qr_format)77, QR_FP16, 0, x, 64, w, y, 32, 5, 32, 64, 0), QR_ERR_UNSUPPORTED);
  EXPECT(qr_linear(QR_INT4, (qr_dtype)9, 0, x, 64, w, y, 32, 5, 32, 64, 0), QR_ERR_UNSUPPORTED);
  EXPECT(qr_linear(QR_INT4, QR_FP16, 0, 0, 64, w, y, 32, 5, 32, 64, 0), QR_ERR_ARG);
  EXPECT(qr_linear(QR_INT4, QR_FP16, 0, x, 64, (char *)w + 4, y, 32, 5, 32, 64, 0), QR_ERR_ALIGN);
  EXPECT(qr_linear(QR_INT4, QR_FP16, 0, x, 64, w, x, 32, 5, 32, 64, 0), QR_ERR_ALIAS);
  EXPECT(qr_linear(QR_INT4, QR_FP16, 0, x, (size_t)1 << 32, w, (char *)x + ((size_t)1 << 34), 32, 5, 32, 64, 0),
         QR_ERR_ALIAS);
  EXPECT(qr_route(x, 3, o, r, p, 16, 2, 8, 0, 0), QR_ERR_UNSUPPORTED);
  EXPECT(qr_route(x, 4, o, r, r, 16, 2, 8, 0, 0), QR_ERR_ALIAS);
  EXPECT(qr_route(x, 4, o, r, p, 1 << 20, 2, 8, 0, 0), QR_ERR_ARG);
  EXPECT(qr_combine(QR_FP16, y, 64, 16, p, g, y, 64, 8, 2, 64, 0), QR_ERR_ALIAS);
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
