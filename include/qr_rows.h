/*
 * qr_rows.h -- C ABI of the operators of a layer whose activations and weights
 * are held in rows of 8 bits: the norm in front of it, the rows' codec, dense
 * and per-expert products, and the router's choice that qr_route (qr_ops.h)
 * sorts by expert and qr_combine weighs.
 *
 * 8-bit rows.  A row of k values is k signed bytes and one fp32 scale:
 *   scale  s = max|x| / 127 (fp32)
 *   code   q = clamp(round_half_even(x * e), -127, 127), e = fp32 127 / max|x|
 *          (0 if max|x| = 0)
 *   decode y = q * s in fp32, rounded to the dtype.
 * A row that holds a NaN or an infinity has scale NaN and codes 0, so that
 * everything computed from it is NaN.  Codes of `rows` rows lie one after
 * another, each padded with zero codes to a multiple of 128 bytes, 16-byte
 * aligned: qr_row_bytes(rows, k) bytes in all.  Products read the padding, so
 * codes that come from elsewhere have zeros there too; they may hold -128.
 *
 * Conventions beyond those of qr.h and qr_ops.h:
 *   - Matrices of the dtype are row-major with a row stride (ld*) in values and
 *     need the alignment of their values only.  fp32 and int32 arrays are 4-byte
 *     aligned.
 *   - Checks run on the host before any HIP call, in the order dtype
 *     (QR_ERR_UNSUPPORTED), sizes (QR_ERR_SIZE), null pointers and other
 *     arguments (QR_ERR_ARG), alignment (QR_ERR_ALIGN), overlap of an output
 *     with anything else (QR_ERR_ALIAS), except where a call allows it.
 *   - A call with no rows is complete as it is: QR_OK, null pointers accepted.
 *   - Equal calls have equal results: every sum of floating-point values has a
 *     fixed order, which depends on sizes and alignment only.
 */
#ifndef QR_ROWS_H_
#define QR_ROWS_H_

#include <stdint.h>

#include "qr.h"
#include "qr_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest k: the sum of k products of any two codes is below 2^31. */
#define QR_MAX_ROW_K 130944

/* Logits may be fp32 (qr_choose only). */
#define QR_FP32 ((qr_dtype)2)

typedef enum QR_ENUM_INT { QR_SOFTMAX = 0, QR_SIGMOID = 1 } qr_score;

/* Bytes of the codes of `rows` rows of k values; 0 for k outside
 * [1, QR_MAX_ROW_K] or rows outside [1, 2^40]. */
size_t qr_row_bytes(size_t rows, size_t k);

/* Codes and scales of the rows of x.
 *   x       device, `rows` rows of k values of `dtype`, row stride ldx >= k
 *   codes   device, qr_row_bytes(rows, k) bytes, written, padding included
 *   scales  device, `rows` fp32, written */
qr_status qr_encode_rows(qr_dtype dtype, const void *x, size_t ldx, int8_t *codes, float *scales, size_t rows,
                         size_t k, void *stream);

/* The values that codes and scales stand for.
 *   y  device, `rows` rows of k values of `dtype`, row stride ldy >= k, written */
qr_status qr_decode_rows(qr_dtype dtype, const int8_t *codes, const float *scales, void *y, size_t ldy, size_t rows,
                         size_t k, void *stream);

/* h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, by rows, in fp32 and
 * with h unrounded.
 *   x         device, `rows` rows of k values of `dtype`, row stride ldx
 *   residual  device, the same with row stride ldr; NULL: h = x
 *   weight    device, k values of `dtype`
 *   eps       >= 0 (QR_ERR_ARG otherwise, NaN included); with 0 a row of zeros is
 *             NaN, as 0 / 0 is
 *   total     device, row stride ldt, written: h rounded to the dtype, which the
 *             next norm takes as its residual; NULL to leave it (without a
 *             residual it has to be: QR_ERR_ARG).  May be x or residual itself,
 *             with its row stride.
 *   y         device, row stride ldy, written; NULL if only codes are wanted.  May
 *             be x or residual itself, with its row stride, if total is not it.
 *   codes, scales  device, written: the 8-bit rows of the unrounded y; both NULL
 *             if only y is wanted.  (Neither y nor codes: QR_ERR_ARG.)
 * Row strides of matrices that are NULL are not looked at.  Squares that leave the
 * range of fp32 on either side do not: h of any finite size has its norm. */
qr_status qr_norm(qr_dtype dtype, const void *x, size_t ldx, const void *residual, size_t ldr, const void *weight,
                  float eps, void *total, size_t ldt, void *y, size_t ldy, int8_t *codes, float *scales, size_t rows,
                  size_t k, void *stream);

/* y = x W^T of 8-bit rows, or with `gated` y = silu(x G^T) * (x U^T):
 * y[m][c] = (sum over k of x codes times w codes) * xs[m] * ws[c], the sum a
 * whole number without rounding, the rest in fp32, rounded once.
 *   x, xs  device, codes and scales of m rows of k values
 *   w, ws  device, codes and scales of n rows of k values; gated: 2 n rows, the n
 *          rows of G and then the n rows of U
 *   y      device, m rows of n values of `dtype`, row stride ldy >= n, written */
qr_status qr_linear8(qr_dtype dtype, int gated, const int8_t *x, const float *xs, const int8_t *w, const float *ws,
                     void *y, size_t ldy, size_t m, size_t n, size_t k, void *stream);

/* The same product with another weight for each group of rows; groups, row
 * numbers and what is out of range as for qr_experts.
 *   x, xs  device, codes and scales of `tokens` rows of k values
 *   w, ws  device, codes and scales of [experts * n, k] (gated: [experts * 2 n, k]) */
qr_status qr_experts8(qr_dtype dtype, int gated, const int8_t *x, const float *xs, size_t tokens, const int8_t *w,
                      const float *ws, const int32_t *offsets, const int32_t *rows, void *y, size_t ldy, size_t slots,
                      size_t experts, size_t n, size_t k, void *stream);

/* A router's choice of experts for each token.
 *   p     = softmax or sigmoid of the token's logits, over the experts that can be
 *           had: a logit of -inf or NaN takes its expert out (+inf counts as the
 *           largest finite value)
 *   rank  = p + bias (a bias of NaN or -inf takes its expert out of the choice,
 *           not of the softmax)
 *   The experts lie in `groups` groups of experts / groups neighbours; a group's
 *   value is the sum of the `group_best` (1 or 2) largest ranks in it, and the
 *   top_groups groups of largest value are kept (groups without any expert that
 *   can be had never are).
 *   ids   = the `top` experts of largest rank in the kept groups, largest first
 *   gates = factor * p of these; with `renormalise` p is divided by the sum of the
 *           chosen p, which is done so that p too small for fp32 do not vanish.
 *           Computed in fp32, within (d + 60) 2^-24 of a gate whose p is a normal
 *           fp32 number: d is how far its logit lies below the row's largest, with
 *           `renormalise` the largest chosen one (QR_SIGMOID: logits count up to 0,
 *           and without `renormalise` from 0)
 * Ranks and values are compared as they are in 64 bits (without a bias, ranks and
 * the groups' largest ones as the logits are, of which p is an increasing
 * function); ties go to the lower number.  Where fewer than `top` experts can be had, the last ids are -1 and
 * their gates 0, which qr_route and qr_combine leave out.
 *   logits  device, `tokens` rows of `experts` values of `dtype` (QR_FP16,
 *           QR_BF16 or QR_FP32), row stride ldl >= experts
 *   bias    device, `experts` fp32, or NULL for none
 *   score   QR_SOFTMAX or QR_SIGMOID (QR_ERR_UNSUPPORTED otherwise)
 *   groups  divides experts, at most 64; 1 <= top_groups <= groups; 1 <= top <=
 *           min(QR_MAX_TOP, experts); group_best 1 or 2, at most experts / groups
 *           (QR_ERR_SIZE otherwise)
 *   factor  finite (QR_ERR_ARG)
 *   gates   device, tokens x top fp32, written
 *   ids     device, tokens x top int32, written */
qr_status qr_choose(qr_dtype dtype, qr_score score, const void *logits, size_t ldl, const float *bias, size_t groups,
                    size_t top_groups, int group_best, int renormalise, float factor, float *gates, int32_t *ids,
                    size_t tokens, size_t experts, size_t top, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QR_ROWS_H_ */
