/*
 * sq_w8a8.h -- the part of libsq's C ABI with the products of 8-bit integers: one
 * scale per token and one per channel, dense or grouped by expert, forward and
 * input gradient, on SQ_FMT_INT8_ROW weights.  The conventions are those of sq.h
 * (device pointers, streams, caller-owned workspaces, status codes, checks before
 * anything is enqueued).
 */
#ifndef SQ_W8A8_H
#define SQ_W8A8_H

#include "sq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a flag beside those of sq.h */
#define SQ_ZERO_UNGROUPED      0x20u /* sq_grouped_*: output rows of no expert become 0
                                        (without it they are left as they were)            */

/*
 * Forward in 8-bit integers, y = x W^T on a SQ_FMT_INT8_ROW weight (SquareQ
 * README, "v3.1 -- int8-residual mode": int8 codes and one scale per row of the
 * rotated residual, a rank-16 branch).  sq_linear_fwd dequantises that weight to
 * bf16; here the rows of x are quantised too, with one scale per token, and the
 * product runs on the 8-bit integer tensor cores (32-bit sums, exact):
 *   r = H256 x (per row m),  s_x = RN(max|r| / 127),
 *   q_x[k] = clamp(rint(RN(r_k RN(1 / s_x))), -127, 127),
 *   y[m, n] = fma(float(sum_k q_x[m, k] Q[n, k]), RN(s_x s_w[n]), t[m] . lora_up[n]),
 *   t[m] = x[m] lora_down (fp32 sums).
 * The codes are the same bits as this sequence of fp32 operations gives.  A
 * scale below 2^-120 counts as 0 (zero codes).  A row with a NaN or an infinity
 * in r gives a row of NaN; other rows are not affected.  y [M, N] fp32 (device),
 * or bf16 with SQ_OUT_BF16 (one more rounding); x [M, K] bf16 (device).
 * lora_up and lora_down are both NULL or both given.  Any M >= 1; few tokens run
 * on narrow tiles that read each weight byte once.  The codes, the scales and
 * the integer sums of a row are the same bits whatever M is and whichever rows
 * lie beside it; t is summed in an order fixed by K, M, the number of experts of
 * a grouped call and the device's number of SMs, so equal calls on equal devices
 * give equal bits.
 * flags: SQ_OUT_BF16, SQ_CHECK_FINITE (a row whose rotation holds a NaN or an
 * infinity sets SQ_ERR_NONFINITE in the status word).
 * ws: sq_workspace_bytes(SQ_OP_LINEAR_FWD_W8A8, M, N, K) bytes.
 */
SQ_API sq_status sq_linear_fwd_w8a8(const sq_weight *w, const uint16_t *x, int64_t M, void *y, uint32_t flags,
                                    void *ws, size_t ws_bytes, void *stream);

/*
 * Input gradient of the layer in 8-bit integers (the counterpart of
 * sq_linear_bwd_dx, which multiplies by the bf16 reconstruct of W), straight
 * through the rounding of x: dx = dy W with the rows of dy quantised,
 *   r[n] = RN(dy[m, n] s_w[n]),  s_g and q_g from r as in sq_linear_fwd_w8a8,
 *   dx[m, :] = H256( RN(float(sum_n q_g[m, n] Q[n, :]) s_g) ) + u[m] . lora_down[k],
 *   u[m] = dy[m] lora_up (fp32 sums; it enters the last product as three bf16 terms:
 *   24 bits, below 2^-110 with an absolute error of 2^-134);
 * the codes are read as they lie, no transposed or reconstructed copy of W is
 * made.  dy [M, N] bf16, dx [M, K] fp32 (bf16 with SQ_OUT_BF16), device.
 * N <= 131072 (the 32-bit sums stay exact).  NaN, infinities, flags and status
 * as in sq_linear_fwd_w8a8.
 * ws: sq_workspace_bytes(SQ_OP_LINEAR_BWD_DX_W8A8, M, N, K) bytes.
 */
SQ_API sq_status sq_linear_bwd_dx_w8a8(const sq_weight *w, const uint16_t *dy, int64_t M, void *dx, uint32_t flags,
                                       void *ws, size_t ws_bytes, void *stream);

/*
 * The two calls above for E layers of the same N and K at once (a mixture of
 * experts; 1 <= E <= 1024): rows offsets[e] .. offsets[e + 1] - 1 of x (dy)
 * belong to expert e.  w describes E weights in a row: codes [E, N, K], scales
 * [E, N], lora_up [E, N, 16], lora_down [E, K, 16].  offsets [E + 1] int32
 * (device), not decreasing, between 0 and M; an expert may have no rows.  Rows
 * before offsets[0] and from offsets[E] on belong to none: they are left as they
 * were, or become 0 with SQ_ZERO_UNGROUPED.  A row's result is what the dense call
 * gives with that expert's weight (the same codes and integer sums).  M may be 0
 * (nothing is enqueued).  Offsets outside these rules are clamped, so that no access leaves
 * the buffers; the rows' results are then unspecified, and
 * sq_check_device_status reports SQ_ERR_INDEX.
 * ws: sq_grouped_workspace_bytes(SQ_OP_GROUPED_FWD_W8A8 or _BWD_DX_W8A8, E, M, N, K).
 */
SQ_API sq_status sq_grouped_fwd_w8a8(const sq_weight *w, int64_t E, const uint16_t *x, int64_t M,
                                     const int32_t *offsets, void *y, uint32_t flags, void *ws, size_t ws_bytes,
                                     void *stream);
SQ_API sq_status sq_grouped_bwd_dx_w8a8(const sq_weight *w, int64_t E, const uint16_t *dy, int64_t M,
                                        const int32_t *offsets, void *dx, uint32_t flags, void *ws, size_t ws_bytes,
                                        void *stream);

/* Workspace bytes of the grouped calls (0 for another op or E outside 1 .. 1024). */
SQ_API size_t sq_grouped_workspace_bytes(int op, int64_t E, int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* SQ_W8A8_H */
