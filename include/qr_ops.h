/*
 * qr_ops.h -- C ABI of the layer operators over 4-bit block weights: what a
 * tensor-parallel rank runs to make the buffers that qr.h reduces.
 *
 * Weights.  A weight of `rows` x `k` values is held in one of the 4-bit
 * formats of qr.h (QR_INT4, QR_ASYM4, QR_FP4): its rows one after another,
 * each padded to whole blocks of 32 values (QR_INT4, QR_FP4) or groups of 128
 * (QR_ASYM4), the whole padded to a multiple of 2048 values and packed as
 * qr_encode packs it.  So the packed form of a [rows, k] matrix whose k is a
 * multiple of the block and whose size is a multiple of 2048 is exactly
 * qr_encode's of its rows * k values.  Padding values are zero.
 * The weight that a product uses is W = code value * scale, which is not
 * rounded to the call's dtype first; products are summed in fp32 and y is
 * rounded once.  The order of the sums depends on the call's sizes and on the
 * alignment and stride of x only, so equal calls have equal results.
 *
 * Conventions beyond those of qr.h:
 *   - x and y are row-major with a row stride (ldx, ldy) counted in values and
 *     need the alignment of their values only; the packed weight is 16-byte
 *     aligned (QR_ERR_ALIGN).  int32 and fp32 arrays are 4-byte aligned.
 *   - Checks run on the host before any HIP call, in the order format/dtype
 *     (QR_ERR_UNSUPPORTED), sizes (QR_ERR_SIZE), null pointers (QR_ERR_ARG),
 *     alignment (QR_ERR_ALIGN), overlap of an output with anything (QR_ERR_ALIAS;
 *     matrices of one row stride may be columns of one larger matrix, and what
 *     lies between the rows of other outputs counts as theirs).
 *   - A call with no rows (m, slots or tokens = 0) is complete as it is:
 *     QR_OK, and where nothing is written null pointers are accepted.
 *   - What the device arrays hold is not seen by the host: offsets that are out
 *     of order or range, row numbers and positions out of range never lead to
 *     an access outside the buffers (see each call).
 *   - NaN and infinity go through the sums as IEEE arithmetic has them; they
 *     stay within the row of y that they belong to.
 */
#ifndef QR_OPS_H_
#define QR_OPS_H_

#include <stdint.h>

#include "qr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QR_MAX_K (1 << 22)       /* largest k of a weight */
#define QR_MAX_N (1 << 24)       /* largest n of a product (rows of one expert's weight: 2 n if gated) */
#define QR_MAX_EXPERTS 1024
#define QR_MAX_TOP 64            /* expert slots of one token */
#define QR_MAX_SLOTS 1073741824  /* rows of a product, expert slots of a plan: 2^30 */

/* Bytes of the packed form of a [rows, k] weight; 0 for a format that is not
 * one of the three, k outside [1, QR_MAX_K], rows == 0 or more than
 * QR_MAX_TILES tiles. */
size_t qr_weight_bytes(qr_format fmt, size_t rows, size_t k);

/* y = x W^T, or with `gated` y = silu(x G^T) * (x U^T), silu(v) = v / (1 + exp(-v)).
 *   x  device, m rows of k values of `dtype`, row stride ldx >= k
 *   w  device, packed [n, k] weight; gated: [2 n, k], the n rows of G and then
 *      the n rows of U
 *   y  device, m rows of n values of `dtype`, row stride ldy >= n, written */
qr_status qr_linear(qr_format fmt, qr_dtype dtype, int gated, const void *x, size_t ldx, const void *w, void *y,
                    size_t ldy, size_t m, size_t n, size_t k, void *stream);

/* The same product with another weight for each group of rows.
 *   x        device, `tokens` rows of k values, row stride ldx
 *   w        device, packed [experts * n, k] weight (gated: [experts * 2 n, k])
 *   offsets  device, experts + 1 int32, ascending from 0: rows offsets[e] to
 *            offsets[e + 1] of y belong to expert e.  The rows from
 *            offsets[experts] on belong to none and are set to zero.
 *            (Offsets out of range or order: each is clamped to [0, slots], and
 *            one below an earlier one counts as that one, which leaves its
 *            expert's group empty.  Rows before offsets[0] are left as they are.)
 *   rows     device, `slots` int32: row s of y is computed from row rows[s] of
 *            x (a number outside [0, tokens): the row is set to zero); NULL: from
 *            row s, and tokens must be at least slots (QR_ERR_SIZE)
 *   y        device, `slots` rows of n values, row stride ldy, written */
qr_status qr_experts(qr_format fmt, qr_dtype dtype, int gated, const void *x, size_t ldx, size_t tokens,
                     const void *w, const int32_t *offsets, const int32_t *rows, void *y, size_t ldy, size_t slots,
                     size_t experts, size_t n, size_t k, void *stream);

/* Bytes of device scratch that qr_route needs (0 when it needs none). */
size_t qr_route_workspace(size_t tokens, size_t top, size_t experts);

/* The plan of a router's choice: a stable sort of the tokens' expert slots by
 * expert.
 *   ids      device, tokens x top expert numbers of id_bytes bytes (4: int32,
 *            8: int64; other widths are QR_ERR_UNSUPPORTED); a number outside
 *            [0, experts) drops the slot
 *   offsets  device, experts + 1 int32, written: where each expert's rows begin
 *   rows     device, tokens * top int32, written: the token of each sorted row,
 *            rows of one expert in the order of their slots; -1 from
 *            offsets[experts] on
 *   pos      device, tokens x top int32, written: the sorted row of each slot,
 *            -1 for a dropped one
 *   workspace  device, qr_route_workspace() bytes (NULL where that is 0); its
 *            contents need not be set, and are used within the call only */
qr_status qr_route(const void *ids, int id_bytes, int32_t *offsets, int32_t *rows, int32_t *pos, size_t tokens,
                   size_t top, size_t experts, void *workspace, void *stream);

/* out[t] = sum over j of gates[t, j] * y[pos[t, j]], in the order of j, in
 * fp32, rounded once.  A position outside [0, slots) contributes nothing,
 * whatever its gate; a token without any contribution gets zeros.
 *   y      device, `slots` rows of n values of `dtype`, row stride ldy
 *   pos    device, tokens x top int32
 *   gates  device, tokens x top fp32
 *   out    device, tokens rows of n values of `dtype`, row stride ldo, written */
qr_status qr_combine(qr_dtype dtype, const void *y, size_t ldy, size_t slots, const int32_t *pos, const float *gates,
                     void *out, size_t ldo, size_t tokens, size_t top, size_t n, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QR_OPS_H_ */
