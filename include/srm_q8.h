/*
 * srm_q8.h -- C ABI of the 8-bit path of the decoder block's FFN sublayer for
 * NVIDIA B200 (sm_100a): rows in 8 bits with one scale per row, and products
 * of 8-bit integers with one scale per row and per channel.  Same library as
 * srm_moe.h (libsrm_moe.so); status codes, the device error word and the
 * conventions (device pointers owned by the caller, no allocation,
 * asynchronous on `stream`, host-side validation before any launch) are the
 * ones srm_moe.h states.
 *
 * An 8-bit row stands for the values q[k] * scale, q in -127..127.
 *
 * Strides (ld_*) are in elements, at least the row length, and 64-bit; rows
 * themselves are contiguous.  Outputs must not overlap inputs unless a call
 * says so.
 */
#ifndef SRM_Q8_H
#define SRM_Q8_H

#include <stddef.h>
#include <stdint.h>

#include "srm_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the row calls (here and in srm_rows.h). */
typedef enum {
    MOE_DTYPE_BF16 = 0,
    MOE_DTYPE_FP16 = 1,
    MOE_DTYPE_FP32 = 2,
    MOE_DTYPE_INT8 = 3 /* only where a call says so */
} moe_dtype_t;

/* Shape of a row call: T rows of H elements of type dtype (BF16, FP16, FP32);
 * 1 <= H <= 2^20, 0 <= T < 2^31, T == 0 is a no-op. */
typedef struct {
    int64_t T;
    int32_t H;
    int32_t dtype;
    int64_t ld_x;     /* x (moe_q8_dequantize: not used) */
    int64_t ld_delta; /* delta; not used when delta is NULL */
    int64_t ld_sum;   /* x_sum; not used when x_sum is NULL */
    int64_t ld_y;     /* y; not used when y is NULL */
    int64_t ld_q;     /* q */
} moe_q8_rows_t;

/* RMSNorm with the residual's addition and an 8-bit output: per row
 *     x'    = round(x + delta)     to dtype (x' = x when delta is NULL),
 *     n     = x' * gamma / sqrt(mean(x'^2) + eps)      in fp32,
 *     scale = max |n| / 127,   q = n / scale rounded to nearest even
 * (q is formed from x' * gamma, the root cancelling: of bf16 and fp16 rows it is
 * the exact quotient's integer, but where products below 2^-126 lose bits).
 *   x, delta: dtype [T][H] (delta may be NULL);  gamma: dtype [H]
 *   x_sum: dtype [T][H] or NULL; out: x' (the residual stream).  May be x or
 *          delta itself (same pointer and stride).
 *   y:     dtype [T][H] or NULL; out: n rounded to dtype (what the router
 *          reads).  May be x or delta itself, if x_sum is not that buffer.
 *   q:     int8 [T][H];  scale: fp32 [T]
 * The mean holds for rows whose squares leave fp32's range (they are summed
 * again under a power of two).  A row of zeros (eps > 0) gets scale 0 and
 * q = 0.  A row whose n holds an infinity or NaN gets scale NaN and q = 0, so
 * it does not pass for a finite row further on.  Pointers: aligned to their
 * element; rows of 16-byte multiples at 16-byte addresses run faster.
 * Deterministic. */
moe_status_t moe_q8_add_rmsnorm(const moe_q8_rows_t *cfg, const void *x, const void *delta,
                                const void *gamma, float eps, void *x_sum, void *y, int8_t *q,
                                float *scale, void *stream);

/* Rows to 8 bits without the norm: n = x in the equations above. */
moe_status_t moe_q8_quantize(const moe_q8_rows_t *cfg, const void *x, int8_t *q, float *scale,
                             void *stream);

/* The values 8-bit rows stand for: y = q * scale in fp32, rounded to dtype. */
moe_status_t moe_q8_dequantize(const moe_q8_rows_t *cfg, const int8_t *q, const float *scale, void *y,
                               void *stream);

/* Expert weights to 8 bits with one scale per output channel, in the layout
 * the products below read (the 8-bit form of moe_pack_weights).
 *   w1, w3, w2, ws1, ws3, ws2: bf16, as in moe_pack_weights (also its dense
 *   form, E = K = 0);  G = E + has_shared groups
 *   w13_q: int8 [G * 2I][H], per group units of 32 rows: 16 rows of W1, then the
 *        matching 16 rows of W3;  w13_scale: fp32 [G * 2I]
 *   w2_q: int8 [G * H][I];  w2_scale: fp32 [G * H]
 * cfg->T is not used. */
moe_status_t moe_q8_pack_weights(const moe_cfg_t *cfg, const void *w1, const void *w3, const void *w2,
                                 const void *ws1, const void *ws3, const void *ws2, int8_t *w13_q,
                                 float *w13_scale, int8_t *w2_q, float *w2_scale, void *stream);

/* Shape of a product: R rows of K elements times `groups` weight matrices of N
 * channels.  0 <= R < 2^31 - 1024 (R == 0 is a no-op), 1 <= N, groups * N <= 2^31 - 256,
 * 16 <= K <= 65536 and K % 16 == 0, 1 <= groups <= 257.
 *   swiglu: 0, or 1: the channels are units of 16 gate and the 16 matching up
 *           channels (moe_q8_pack_weights' w13; N % 32 == 0) and the result is
 *           silu(gate) * up, N / 2 columns
 *   dtype:  of y and residual: BF16, FP16 (past +-65504 saturated and flagged
 *           MOE_ERR_RANGE on the device), FP32
 *   ld_x, ld_y, ld_residual: row strides in elements; ld_x % 16 == 0. */
typedef struct {
    int64_t R;
    int32_t N, K, groups, swiglu, dtype;
    int64_t ld_x, ld_y, ld_residual;
} moe_q8_matmul_t;

/* Bytes of device workspace for this shape; 0 for an invalid one.  A workspace
 * for R rows serves every product of no more rows, whatever its other sizes,
 * one call at a time (at most 20 MB on 148 SMs). */
size_t moe_q8_matmul_workspace_size(const moe_q8_matmul_t *cfg);

/* Sets a workspace's control words, once when it is allocated (asynchronous on
 * `stream`); from then on the library keeps them.  In one that was not
 * initialised (but whose first 256 bytes are zero), and in one whose call
 * reported MOE_ERR_TIMEOUT until it is initialised again, products are correct
 * but their work is not dealt out dynamically. */
moe_status_t moe_q8_workspace_init(void *ws, size_t ws_bytes, void *stream);

/* Matrix product of 8-bit integers with a scale per row and per channel:
 *     y[r][n] = x_scale[r] * w_scale[g][n] * sum_k x[r][k] w[g][n][k]
 *               (+ residual[r][n])
 * for the rows r in [offsets[g], offsets[g + 1]) of each group g.
 *   x: int8 [R][K], 16-byte aligned;  x_scale: fp32 [R]
 *   w: int8 [groups * N][K], 16-byte aligned;  w_scale: fp32 [groups * N]
 *   offsets: int32 [groups + 1] (moe_permute's), or NULL with one group: all
 *            rows.  Rows past offsets[groups] are left as they were.  A range
 *            that is none is skipped and flagged MOE_ERR_BAD_INDEX.
 *   residual: dtype [R][N] or NULL (not with swiglu); may be y itself
 *   y: dtype [R][N], with swiglu [R][N / 2]
 * The sum is exact; scales, silu and residual are fp32, rounded once.  A row
 * whose scale is NaN comes out NaN.  Deterministic.  With
 * SRM_MOE_INJECT_STALL=1 (failure-detection tests) it reports MOE_ERR_TIMEOUT
 * like moe_expert_up. */
moe_status_t moe_q8_matmul(const moe_q8_matmul_t *cfg, const int8_t *x, const float *x_scale,
                           const int8_t *w, const float *w_scale, const int32_t *offsets,
                           const void *residual, void *y, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SRM_Q8_H */
