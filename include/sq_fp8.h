/*
 * sq_fp8.h -- the part of libsq's C ABI with the products of 8-bit floating point
 * (e4m3) that carry one scale for each block of 128, dense or grouped by expert,
 * forward and input gradient, and the gated feed-forward projections on them.  The
 * conventions are those of sq.h (device pointers, streams, caller-owned workspaces,
 * status codes, checks before anything is enqueued), with shapes of its own: N and K
 * are multiples of 16 and at most 2^20; the last blocks of an axis may be narrower
 * than 128.
 *
 * The weight, SQ_FMT_FP8_BLOCK in an sq_weight:
 *   codes      [N, K] e4m3
 *   scales     [ceil(N / 128), ceil(K / 128)] e8m0: byte b is the factor 2^(b - 127)
 *   g_w, lora_up, lora_down   NULL
 *   W[n, k] = 2^(scales[n / 128, k / 128] - 127) codes[n, k]
 * It is not rotated.  Codes of NaN (0x7f, 0xff) give NaN in the sums that they enter;
 * so does the scale byte 255.
 *
 * The rows that meet it (x, dy, and the two gradients of a gated pair) are rounded in
 * the call, in blocks of 128 along the summed axis:
 *   s = the least power of two >= 2^-127 with max|r| <= 448 s,   code = e4m3(r / s),
 * r / s is exact, the conversion rounds to nearest even.  The products of codes and
 * scales are exact in the tensor cores and summed there in fp32 (a sum whose parts
 * pass fp32's range is infinite or NaN).  Each step of 32 products cuts the sum that it
 * adds to towards zero, by at most 2^-22 of the magnitudes summed so far: measured 5e-7 of
 * a result's size for 6144 values, 2e-6 for 16384 and 5e-6 for 32768 and more; for bf16
 * results and the gated forward 3e-5 for 2^17 and 4e-4 for 2^20.  Equal calls on equal
 * devices give equal bits; a row among another number of rows may be summed in another
 * order.  A row with a NaN or an infinity gives a row of NaN; other rows are not affected.
 *
 * Few rows are rounded by the product itself: M <= 16, and M <= 32 where N K <= 2^24
 * or E > 1 (the gradient of a gated pair: M <= 8 and 16).  Such a call needs no
 * workspace: its size is 0 and ws may be NULL.  A workspace given all the same holds at
 * least 256 bytes.
 *
 * The status of a call is the first word of its workspace, as in sq.h.  Without a
 * workspace, or with SQ_STATUS_LIBRARY, it is the library's own word on the device
 * (sq_check_device_status(NULL, stream)), to which calls only add: what the calls on
 * all streams have found since it was last read.
 */
#ifndef SQ_FP8_H
#define SQ_FP8_H

#include "sq.h"
#include "sq_w8a8.h"    /* SQ_ZERO_UNGROUPED, sq_grouped_workspace_bytes() */

#ifdef __cplusplus
extern "C" {
#endif

#define SQ_FMT_FP8_BLOCK 5          /* a value of sq_weight.fmt */

/* operations for sq_workspace_bytes() and, grouped, sq_grouped_workspace_bytes() */
#define SQ_OP_LINEAR_FWD_FP8           15
#define SQ_OP_LINEAR_BWD_DX_FP8        16
#define SQ_OP_GATED_FWD_FP8            17
#define SQ_OP_GATED_BWD_DX_FP8         18
#define SQ_OP_GROUPED_FWD_FP8          19
#define SQ_OP_GROUPED_BWD_DX_FP8       20
#define SQ_OP_GROUPED_GATED_FWD_FP8    21
#define SQ_OP_GROUPED_GATED_BWD_DX_FP8 22

/* flags beside those of sq.h and sq_w8a8.h */
#define SQ_IN_BF16             0x40u /* sq_build_fp8: W is bf16 instead of fp32 */
#define SQ_STATUS_LIBRARY      0x100u /* the products: report to the library's status word,
                                         not to the workspace's (which may be gone when
                                         somebody asks) */

/* activations of the gated projections */
#define SQ_ACT_SILU            0     /* g / (1 + e^-g) */
#define SQ_ACT_GELU_TANH       1     /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */

/*
 * Builder: W [N, K] fp32 (bf16 with SQ_IN_BF16) -> codes and scales, with the rule
 * above for each block of 128 x 128 (the maximum over its finite values; a NaN or an
 * infinity becomes a NaN code).
 */
SQ_API sq_status sq_build_fp8(const void *W, int64_t N, int64_t K, uint32_t flags, uint8_t *codes, uint8_t *scales,
                              void *stream);

/*
 * y [M, N] = x W^T, x [M, K] bf16; y fp32, or bf16 with SQ_OUT_BF16 (one more
 * rounding).  M >= 1.  flags: SQ_OUT_BF16, SQ_CHECK_FINITE (a NaN or an infinity in x
 * sets SQ_ERR_NONFINITE in the status word), SQ_STATUS_LIBRARY.
 * ws: sq_workspace_bytes(SQ_OP_LINEAR_FWD_FP8, M, N, K) bytes.
 */
SQ_API sq_status sq_linear_fwd_fp8(const sq_weight *w, const uint16_t *x, int64_t M, void *y, uint32_t flags,
                                   void *ws, size_t ws_bytes, void *stream);

/*
 * Input gradient, straight through the rounding of x: dx [M, K] = dy W, dy [M, N]
 * bf16, its rows rounded in blocks along N.  The codes of W are read as they lie.
 * ws: sq_workspace_bytes(SQ_OP_LINEAR_BWD_DX_FP8, M, N, K) bytes.
 */
SQ_API sq_status sq_linear_bwd_dx_fp8(const sq_weight *w, const uint16_t *dy, int64_t M, void *dx, uint32_t flags,
                                      void *ws, size_t ws_bytes, void *stream);

/*
 * The gated projections in one product: g = x Wgate^T, u = x Wup^T (fp32 sums),
 * h = act(g) u [M, N] fp32 or bf16.  gate and up are weights of the same N and K.
 * g_out and u_out [M, N] bf16 (both or neither) keep g and u, rounded once, for the
 * backward pass.  act: SQ_ACT_SILU or SQ_ACT_GELU_TANH.
 * ws: sq_workspace_bytes(SQ_OP_GATED_FWD_FP8, M, N, K) bytes.
 */
SQ_API sq_status sq_gated_fwd_fp8(const sq_weight *gate, const sq_weight *up, const uint16_t *x, int64_t M,
                                  int32_t act, void *h, uint16_t *g_out, uint16_t *u_out, uint32_t flags, void *ws,
                                  size_t ws_bytes, void *stream);

/*
 * Its input gradient: dg = dh u act'(g), du = dh act(g) in fp32 from dh, g, u [M, N]
 * bf16, both rounded in blocks along N; dx [M, K] = dg Wgate + du Wup, one sum.
 * ws: sq_workspace_bytes(SQ_OP_GATED_BWD_DX_FP8, M, N, K) bytes.
 */
SQ_API sq_status sq_gated_bwd_dx_fp8(const sq_weight *gate, const sq_weight *up, const uint16_t *dh,
                                     const uint16_t *g, const uint16_t *u, int64_t M, int32_t act, void *dx,
                                     uint32_t flags, void *ws, size_t ws_bytes, void *stream);

/*
 * The four calls above for E layers of the same N and K at once (1 <= E <= 1024):
 * rows offsets[e] .. offsets[e + 1] - 1 belong to expert e, whose weight is the e-th of
 * codes [E, N, K] and scales [E, ceil(N / 128), ceil(K / 128)].  offsets, M = 0, rows of
 * no expert and SQ_ZERO_UNGROUPED as in sq_w8a8.h (g_out and u_out are cleared too).
 * ws: sq_grouped_workspace_bytes(SQ_OP_GROUPED_..._FP8, E, M, N, K) bytes.
 */
SQ_API sq_status sq_grouped_fwd_fp8(const sq_weight *w, int64_t E, const uint16_t *x, int64_t M,
                                    const int32_t *offsets, void *y, uint32_t flags, void *ws, size_t ws_bytes,
                                    void *stream);
SQ_API sq_status sq_grouped_bwd_dx_fp8(const sq_weight *w, int64_t E, const uint16_t *dy, int64_t M,
                                       const int32_t *offsets, void *dx, uint32_t flags, void *ws, size_t ws_bytes,
                                       void *stream);
SQ_API sq_status sq_grouped_gated_fwd_fp8(const sq_weight *gate, const sq_weight *up, int64_t E, const uint16_t *x,
                                          int64_t M, const int32_t *offsets, int32_t act, void *h, uint16_t *g_out,
                                          uint16_t *u_out, uint32_t flags, void *ws, size_t ws_bytes, void *stream);
SQ_API sq_status sq_grouped_gated_bwd_dx_fp8(const sq_weight *gate, const sq_weight *up, int64_t E,
                                             const uint16_t *dh, const uint16_t *g, const uint16_t *u, int64_t M,
                                             const int32_t *offsets, int32_t act, void *dx, uint32_t flags, void *ws,
                                             size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SQ_FP8_H */
