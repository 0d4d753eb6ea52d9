/*
 * srm_rows.h -- C ABI of the token rows' way to the experts and back, as calls
 * of their own with their gradients, for NVIDIA B200 (sm_100a).  Same library
 * as srm_moe.h (libsrm_moe.so); status codes, the device error word and the
 * conventions are the ones srm_moe.h states, element types those of srm_q8.h.
 *
 * moe_permute's (offsets, sorted) say which row each expert-sorted position
 * holds: sorted[p] = t*K + slot for a routed row, T*K + t for the shared
 * expert's.  moe_rows_sort brings token rows into that order and records the
 * inverse, pos; moe_rows_unsort brings the experts' rows back with the routing
 * weights applied:
 *     sort:    xs[p] = x[token of sorted[p]],   pos[sorted[p]] = p
 *     unsort:  y[t] = (residual[t] +) sum_k gate[t][k] ys[pos[t*K+k]]
 *                     + ys[pos[T*K+t]]                      (shared expert)
 * and for training, from dxs and dy:
 *     sort's gradient:    dx[t] = sum_k dxs[pos[t*K+k]] + dxs[pos[T*K+t]]
 *     unsort's gradient:  dys[pos[t*K+k]] = gate[t][k] dy[t],
 *                         dys[pos[T*K+t]] = dy[t],
 *                         dgate[t][k] = sum_h dy[t][h] ys[pos[t*K+k]][h]
 * (the residual's gradient is dy itself).  Products and sums are fp32, in slot
 * order with the shared row last, and rounded once: deterministic.
 *
 * An assignment without a row (pos -1: moe_permute skips expert ids out of
 * range) adds nothing, gets no gradient row and dgate 0.  Positions past
 * offsets[E + 1] belong to no row; those rows of xs, xs_scale and dys are left
 * as they were.
 */
#ifndef SRM_ROWS_H
#define SRM_ROWS_H

#include <stddef.h>
#include <stdint.h>

#include "srm_moe.h"
#include "srm_q8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape: T tokens, rows of H elements, E experts, K per token, has_shared as
 * in moe_cfg_t; P = T*K + T*has_shared positions.  1 <= K <= 16,
 * K <= E <= 256 (K == 0 with E == 0 and has_shared == 1 is accepted too: one
 * group), 1 <= H <= 2^20, 0 <= T, T*(K+1) < 2^31; T == 0 is a no-op.
 *   dtype:      the tokens' rows (x, y, dy, dx, residual): BF16, FP16, FP32;
 *               moe_rows_sort also INT8
 *   slot_dtype: the experts' rows (ys, dys): BF16, FP16, FP32; not used by
 *               moe_rows_sort and moe_rows_sort_grad, whose xs and dxs are of
 *               dtype
 *   ld_token:   row stride of x, y, dy or dx, in elements, at least H
 *   ld_slot:    row stride of xs, ys or dxs
 *   ld_residual, ld_dys: those of residual and dys, where the call has them
 * Pointers: aligned to their element; 16-byte multiples at 16-byte addresses
 * run faster.  ws: a workspace of this library (its error word), or any 256
 * device bytes at a 256-byte address, zeroed once. */
typedef struct {
    int64_t T;
    int32_t H, E, K, has_shared;
    int32_t dtype, slot_dtype;
    int64_t ld_token, ld_slot, ld_residual, ld_dys;
} moe_rows_cfg_t;

/*   x: dtype [T][H];  x_scale: fp32 [T] or NULL (the scales of 8-bit rows)
 *   offsets: int32 [E + 2], sorted: int32 [P] from moe_permute
 *   pos: int32 [P] out, -1 where no position holds the row
 *   xs: dtype [P][H] out;  xs_scale: fp32 [P] out (with x_scale)
 * A row id out of range, or a total outside 0..P, is ignored and flagged
 * MOE_ERR_BAD_INDEX on the device.  So is a row id's second position: the last
 * one takes the row, the others' rows of xs are left as they were. */
moe_status_t moe_rows_sort(const moe_rows_cfg_t *cfg, const void *x, const float *x_scale,
                           const int32_t *offsets, const int32_t *sorted, int32_t *pos, void *xs,
                           float *xs_scale, void *ws, void *stream);

/*   ys: slot_dtype [P][H];  gate: fp32 [T][K] or NULL (weights 1)
 *   residual: dtype [T][H] or NULL; may be y itself;  y: dtype [T][H] out
 * A pos outside -1..P-1 counts as -1 and is flagged MOE_ERR_BAD_INDEX. */
moe_status_t moe_rows_unsort(const moe_rows_cfg_t *cfg, const void *ys, const float *gate,
                             const int32_t *pos, const void *residual, void *y, void *ws, void *stream);

/*   dxs: dtype [P][H];  dx: dtype [T][H] out */
moe_status_t moe_rows_sort_grad(const moe_rows_cfg_t *cfg, const void *dxs, const int32_t *pos, void *dx,
                                void *ws, void *stream);

/*   dy: dtype [T][H];  ys: slot_dtype [P][H];  gate: fp32 [T][K] or NULL
 *   dys: slot_dtype [P][H] out, or NULL (no row gradient); may be ys itself
 *   dgate: fp32 [T][K] out, or NULL (then ys is not read and may be NULL)
 * With dys == ys each element is read before it is overwritten.  pos holds no
 * position twice, as moe_rows_sort leaves it. */
moe_status_t moe_rows_unsort_grad(const moe_rows_cfg_t *cfg, const void *dy, const void *ys,
                                  const float *gate, const int32_t *pos, void *dys, float *dgate, void *ws,
                                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SRM_ROWS_H */
