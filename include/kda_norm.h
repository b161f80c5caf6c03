/*
 * kda_norm.h -- RMS norms of a KDA layer (gfx950), with their gradients.
 *
 * A KDA layer has two of them next to the recurrence of kda.h: the norm of the
 * residual stream in front of the q/k/v/gate projections, which adds the
 * previous block's output to the stream on the way and may leave its result in
 * fp8 for those projections, and the norm of every head's 128 output channels
 * (the `out` rows of kda_decode, kda_verify_ucache_flush and kda_prefill_varlen
 * as they are), multiplied by a sigmoid gate, in front of the output projection.
 * Both are one operation over (row, head) vectors of `width` channels:
 *   z = x + residual                     (z = x without a residual)
 *   y = z / sqrt(mean(z^2) + eps) * weight [* sigmoid(gate)]
 *
 * Conventions are those of kda.h: device pointers, strides in elements of the
 * tensor's own type, bf16 as raw bits, nothing allocated or synchronised, work
 * enqueued on `stream` only, host-visible errors returned before a launch.
 * Element (r, h, c) of every tensor sits at r * row_stride + h * width + c. Any
 * 2-byte-aligned bf16 pointer and any stride is accepted (fp8 outputs: any byte).
 */
#ifndef KDA_NORM_H_
#define KDA_NORM_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  KDA_NORM_OUT_BF16 = 0, /* out_dtype: y in bf16 */
  KDA_NORM_OUT_FP8 = 1   /* out_dtype: y / scale in fp8 e4m3, with scales */
};

/* Largest width. */
#define KDA_NORM_MAX_WIDTH 16384

/*
 * kda_rmsnorm -- residual addition, RMS norm, optional gate, bf16 or fp8 out.
 *
 *  rows, heads, width  rows (>= 0; 0 is a no-op), vectors per row (>= 1), channels
 *                     per vector (1 .. KDA_NORM_MAX_WIDTH)
 *  x                  bf16
 *  residual           bf16, or NULL (z = x)
 *  residual_out       receives z rounded to bf16 (the residual stream's new
 *                     value); NULL: not stored. Needs a residual. May be
 *                     `residual` itself with the same stride (in place).
 *  gate               bf16 gate logits, or NULL (no gate)
 *  weight             fp32 [width], shared by all rows and heads
 *  eps                > 0, finite
 *  out_dtype          KDA_NORM_OUT_BF16 or KDA_NORM_OUT_FP8
 *  out                y; with bf16 it may be x itself with the same stride
 *  scale_group        fp8 only: channels that share a scale: width (or 0, the
 *                     same), or 128, which must divide width
 *  scales             fp8 only: fp32, scale of group j of (r, h) at
 *                     r * scales_row_stride + h * (width / scale_group) + j:
 *                     max|y| over the group / 448, or 1 where that maximum is
 *                     below 1e-30; out holds y / scale rounded to nearest even.
 *                     NaNs of y are stored as NaN and do not enter the scale.
 * The sum of squares, the norm and the gate are fp32, and y is formed from z
 * before z is rounded for residual_out. No other output may overlap an input or
 * another output.
 * KDA_ERR_BAD_SHAPE: rows < 0, heads < 1, width < 1. KDA_ERR_UNSUPPORTED: width
 * or heads * width too large (2^30 channels a row), eps, out_dtype, scale_group,
 * or residual_out without residual. KDA_ERR_BAD_STRIDE: a negative stride, or
 * output rows that overlap.
 */
kda_status kda_rmsnorm(int64_t rows, int32_t heads, int32_t width,
                       const void* x, int64_t x_row_stride,
                       const void* residual, int64_t residual_row_stride,
                       void* residual_out, int64_t residual_out_row_stride,
                       const void* gate, int64_t gate_row_stride,
                       const float* weight, float eps, int32_t out_dtype,
                       void* out, int64_t out_row_stride,
                       int32_t scale_group, float* scales, int64_t scales_row_stride,
                       hipStream_t stream);

/*
 * kda_rmsnorm_backward_workspace_size -- bytes kda_rmsnorm_backward needs for
 * these sizes (0 for invalid ones), never less for more rows. Pure host arithmetic.
 */
size_t kda_rmsnorm_backward_workspace_size(int64_t rows, int32_t heads, int32_t width);

/*
 * kda_rmsnorm_backward -- gradients of y = norm(z) * weight [* sigmoid(gate)].
 *
 *  z                  bf16: the norm's input (kda_rmsnorm's x, or its residual_out)
 *  dy                 bf16: the gradient at y
 *  gate               bf16 gate logits, or NULL where the norm had no gate
 *  d_residual         bf16: the gradient that reaches z past the norm (the
 *                     residual stream's), added to dz; or NULL
 *  dz                 bf16 out: the gradient at z, which is the one at x and at
 *                     residual. May be dy or d_residual itself with the same stride.
 *  dgate              bf16 out: required with a gate, else must be NULL. May be
 *                     gate itself with the same stride.
 *  dweight            fp32 [width] out: summed over all rows and heads in an order
 *                     that depends on the sizes only (the same bits every call);
 *                     zeros when rows = 0; NULL: not computed
 *  workspace          >= kda_rmsnorm_backward_workspace_size(...) bytes, 256-byte
 *                     aligned (may be NULL without dweight); meaningless afterwards
 * With a = dy * weight [* sigmoid(gate)], s = 1 / sqrt(mean(z^2) + eps), n = z s:
 * dz = s (a - n mean(a n)) + d_residual, dgate = dy n weight sig (1 - sig),
 * dweight = sum of dy n [sig]; fp32, rounded once on output. No other overlap.
 * Errors as for kda_rmsnorm; KDA_ERR_WORKSPACE_TOO_SMALL; KDA_ERR_UNSUPPORTED for
 * an unaligned workspace.
 */
kda_status kda_rmsnorm_backward(int64_t rows, int32_t heads, int32_t width,
                                const void* z, int64_t z_row_stride,
                                const void* dy, int64_t dy_row_stride,
                                const void* gate, int64_t gate_row_stride,
                                const void* d_residual, int64_t d_residual_row_stride,
                                const float* weight, float eps,
                                void* dz, int64_t dz_row_stride,
                                void* dgate, int64_t dgate_row_stride, float* dweight,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_NORM_H_ */
