/*
 * moe_norm.h - C ABI of the norms and rotations of a serving step that moe_paged.h does not have (libmoe.so,
 * GB300 / sm_103a).
 *
 *   moe_add_rms_norm    the residual's addition and the root-mean-square norm of a token's row, in bf16 or 8 bits
 *   moe_qk_norm_mrope   moe_qk_norm_rope with several position axes (time, height, width)
 *
 * Conventions: those of moe.h. No workspace.
 */
#ifndef MOE_NORM_H_
#define MOE_NORM_H_

#include <stdint.h>

#include "../moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * r = x + residual, and its norm y = r * rsqrt(mean(r^2) + eps) * weight: what stands in front of the router and the
 * experts, and in front of the attention's product.
 *   x            [N, H] bf16, rows x_stride elements apart (a multiple of 8, at least H), or null: r = residual
 *   residual     [N, H] bf16
 *   weight       [H] bf16, or null: ones
 *   residual_out [N, H] bf16 out: r, rounded to bf16 (the norm is taken of the rounded values); may be residual itself,
 *                or null
 *   y            [N, H] bf16 out, or null; may be x when x_stride = H
 *   q, scales    [N, H] int8 and [N, H / 128] f32 out, or both null: y in 8 bits, in the form of the experts' INT8
 *                weights: with t = r * weight and T the largest |t| of 128 consecutive dimensions,
 *                q = round(127 t / T), halves to even, and scale = T * rsqrt(mean(r^2) + eps) / 127; all q = 0 and
 *                scale = 1 where T = 0. At least one of y and q is given.
 * Squares are summed in fp32, and y rounded once. The codes are those of the exact quotient: r has 8 bits and t 16, so
 * nothing before the division is rounded, and a quotient that is not a half is far enough from one. That holds while |t|
 * is 0 or within 2^-110 .. 2^120. y is r * weight in fp32 times the factor, so it needs r * weight within fp32's range too. A
 * row whose squares sum past 2^128 comes out as 0 (an infinity, or an r * weight past fp32's range, as NaN); NaN gives NaN (in
 * 8 bits: a NaN scale, for the groups that hold one and, through the mean, for the whole row).
 * H is a multiple of 8 (of 128 with q) up to 32768. N = 0 is a no-op. All pointers 16-byte aligned, scales 4-byte.
 */
moe_status_t moe_add_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual, const uint16_t* weight,
                              float eps, int N, int H, uint16_t* residual_out, uint16_t* y, int8_t* q, float* scales,
                              moe_stream_t stream);

/*
 * moe_qk_norm_rope (moe_paged.h) for positions with several axes, as images and video have them.
 *   positions  [n_axes] rows of N int32, axis_stride elements apart
 *   pair_axis  [rot_dim / 2] int32: pair i of token n turns by positions[pair_axis[i], n] * inv_freq[i]; a pair
 *              whose axis is outside [0, n_axes) does not turn
 * 1 <= n_axes <= 16, axis_stride >= 0 (0: the axes share their positions). Everything else as in moe_qk_norm_rope; with one
 * axis the results are its results.
 */
moe_status_t moe_qk_norm_mrope(const uint16_t* qkv, int64_t row_stride, int N, int h_q, int h_kv, int d,
                               const uint16_t* q_weight, const uint16_t* k_weight, float eps, const float* inv_freq,
                               const int32_t* pair_axis, int rot_dim, int interleaved, const int32_t* positions,
                               int64_t axis_stride, int n_axes, const int32_t* slots, uint16_t* q_out,
                               uint16_t* k_cache, uint16_t* v_cache, int num_pages, int page_size,
                               moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_NORM_H_ */
