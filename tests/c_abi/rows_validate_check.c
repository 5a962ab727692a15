/* rows_validate_check.c -- drives the argument checks of include/qr_rows.h with
 * addresses that are never read (see tests/test_rows_host_sanitized.py). */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "qr_rows.h"

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
  void *x = (void *)0x100000000000, *r = (void *)0x140000000000, *w = (void *)0x200000000000, *y = (void *)0x300000000000;
  void *t = (void *)0x340000000000;
  int8_t *c = (int8_t *)0x400000000000, *d = (int8_t *)0x480000000000;
  float *s = (float *)0x500000000000, *v = (float *)0x580000000000;
  int32_t *o = (int32_t *)0x600000000000, *p = (int32_t *)0x680000000000;
  const size_t huge[] = {(size_t)-1, (size_t)1 << 63, (size_t)1 << 62, ((size_t)1 << 32) + 1};
  /* accepted, up to the limits */
  EXPECT(qr_encode_rows(QR_FP16, x, 64, c, s, 8, 64, 0), QR_ERR_HIP);
  EXPECT(qr_encode_rows(QR_BF16, x, 1, c, s, QR_MAX_SLOTS, 1, 0), QR_ERR_HIP);
  EXPECT(qr_encode_rows(QR_BF16, x, QR_MAX_ROW_K, c, s, 1, QR_MAX_ROW_K, 0), QR_ERR_HIP);
  EXPECT(qr_decode_rows(QR_BF16, c, s, y, 70, 3, 64, 0), QR_ERR_HIP);
  EXPECT(qr_norm(QR_FP16, x, 64, r, 70, w, 0.0f, t, 80, y, 64, c, s, 8, 64, 0), QR_ERR_HIP);
  EXPECT(qr_norm(QR_FP16, x, 64, r, 64, w, 1.0f, r, 64, x, 64, 0, 0, 8, 64, 0), QR_ERR_HIP);
  EXPECT(qr_norm(QR_BF16, x, 64, 0, 0, w, 1.0f, 0, 0, 0, 0, c, s, 8, 64, 0), QR_ERR_HIP);
  EXPECT(qr_linear8(QR_FP16, 1, c, s, d, v, y, 1, 1, 1, 1, 0), QR_ERR_HIP);
  EXPECT(qr_experts8(QR_BF16, 1, c, s, 7, d, v, o, p, y, 40, 9, QR_MAX_EXPERTS, 40, 128, 0), QR_ERR_HIP);
  EXPECT(qr_choose(QR_FP32, QR_SIGMOID, x, 1024, v, 64, 64, 2, 1, -1.0f, s, o, 4, 1024, 64, 0), QR_ERR_HIP);
  EXPECT(qr_choose(QR_BF16, QR_SOFTMAX, x, 1, 0, 1, 1, 1, 0, 1.0f, s, o, QR_MAX_SLOTS, 1, 1, 0), QR_ERR_HIP);
  for (int i = 0; i < 4; ++i) {
    const size_t h = huge[i];
    EXPECT(qr_row_bytes(h, h), 0);
    EXPECT(qr_row_bytes(1, h), 0);
    EXPECT(qr_encode_rows(QR_FP16, x, h, c, s, 8, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_encode_rows(QR_FP16, x, 64, c, s, h, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_encode_rows(QR_FP16, x, h, c, s, 8, h, 0), QR_ERR_SIZE);
    EXPECT(qr_decode_rows(QR_FP16, c, s, y, h, 8, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_norm(QR_FP16, x, 64, r, h, w, 0.0f, t, 64, y, 64, c, s, 8, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_norm(QR_FP16, x, 64, r, 64, w, 0.0f, t, 64, y, h, c, s, 8, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_norm(QR_FP16, x, 64, r, 64, w, 0.0f, t, h, y, 64, c, s, h, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_linear8(QR_FP16, 0, c, s, d, v, y, 32, h, 32, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_linear8(QR_FP16, 0, c, s, d, v, y, h, 5, h, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_experts8(QR_FP16, 0, c, s, h, d, v, o, p, y, 32, 5, 4, 32, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_experts8(QR_FP16, 0, c, s, 5, d, v, o, p, y, 32, 5, h, 32, 64, 0), QR_ERR_SIZE);
    EXPECT(qr_choose(QR_FP32, QR_SOFTMAX, x, 64, v, 1, 1, 1, 1, 1.0f, s, o, h, 64, 8, 0), QR_ERR_SIZE);
    EXPECT(qr_choose(QR_FP32, QR_SOFTMAX, x, 64, v, h, 1, 1, 1, 1.0f, s, o, 4, 64, 8, 0), QR_ERR_SIZE);
    EXPECT(qr_choose(QR_FP32, QR_SOFTMAX, x, h, v, 1, 1, 1, 1, 1.0f, s, o, 4, h, h, 0), QR_ERR_SIZE);
  }
  EXPECT(qr_encode_rows((qr_dtype)9, x, 64, c, s, 8, 64, 0), QR_ERR_UNSUPPORTED);
  EXPECT(qr_encode_rows(QR_FP32, x, 64, c, s, 8, 64, 0), QR_ERR_UNSUPPORTED);
  EXPECT(qr_choose(QR_FP32, (qr_score)77, x, 64, v, 1, 1, 1, 1, 1.0f, s, o, 4, 64, 8, 0), QR_ERR_UNSUPPORTED);
  EXPECT(qr_choose(QR_FP32, QR_SOFTMAX, x, 64, v, 1, 1, 1, 1, (float)NAN, s, o, 4, 64, 8, 0), QR_ERR_ARG);
  EXPECT(qr_norm(QR_FP16, x, 64, r, 64, w, 1.0f, r, 64, r, 64, 0, 0, 8, 64, 0), QR_ERR_ALIAS);
  EXPECT(qr_norm(QR_FP16, x, (size_t)1 << 32, 0, 0, w, 1.0f, 0, 0, (char *)x + ((size_t)1 << 34), 64, 0, 0, 8, 64, 0), QR_ERR_ALIAS);
  EXPECT(qr_linear8(QR_FP16, 0, c, s, c, s, c, 32, 5, 32, 64, 0), QR_ERR_ALIAS);
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
