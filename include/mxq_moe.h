/*
 * mxq_moe.h -- C ABI of libmxq, the mixture-of-experts half of a decoder layer on GB300: the
 * residual's addition with RMSNorm and MXFP8 output, the routing to experts, and the experts'
 * products on MXFP8 activations and weights.
 *
 * The conventions, status codes, MXFP8 format and scale layouts are those of mxq.h: device
 * pointers owned by the caller, work enqueued on `stream`, argument errors detected on the host
 * before anything is launched, nothing allocated and nothing synchronized. Row strides are below 2^40;
 * that of a single row is not looked at.
 *
 * No page describes these operators; they extend the chain of mxq.h so that activations stay
 * MXFP8 through the experts as they do through _o_proj.
 */
#ifndef MXQ_MOE_H_
#define MXQ_MOE_H_

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mxq_float_type {
  MXQ_TYPE_BF16 = 0,
  MXQ_TYPE_FP32 = 1
} mxq_float_type;

typedef enum mxq_moe_scoring {
  MXQ_MOE_SIGMOID = 0,
  MXQ_MOE_SOFTMAX = 1
} mxq_moe_scoring;

/*
 * add_rmsnorm_dual_out -- one pass over the residual stream:
 *   h[t, j]  = RNE_st( x[t, j] + residual[t, j] )                 st: the stream's type
 *   y[t, j]  = RNE_bf16( (h[t, j] * r_t) * gamma[j] ),  r_t = 1 / sqrt(mean_j h[t, j]^2 + eps)
 *   (y_q, scales) = mxfp8_quantize(y)                             of that bf16 y, bit-identical
 * The sum is taken in fp32 and rounded once to the stream's type; the norm reads the rounded h. The
 * value of y is the formula's, rounded once to fp32 (the sum of squares, r and the products carry
 * their error terms), before it is rounded to bf16; rows whose sum of squares lies outside fp32 are
 * taken in fp64. An infinity in h makes its own y NaN and the row's other y 0, a NaN the whole row.
 *
 *   x_bf16       [T, H] bf16, row stride ldx elements.
 *   residual     [T, H] of residual_type (MXQ_TYPE_BF16 or MXQ_TYPE_FP32), row stride ldr elements.
 *   residual_out [T, H] of the same type, row stride ldro elements; may be `residual` itself with
 *                ldro == ldr (in place), must not overlap it otherwise, nor x. (Column ranges of one
 *                buffer do not overlap; with different row strides the whole spans count.)
 *   y_bf16       [T, H] bf16 out (row stride H), or NULL.
 *   y_q          [T, H] E4M3 out (row stride H bytes) and at least one scale output, or all NULL.
 * At least one of y_bf16 and y_q. Requires T >= 1, 32 <= H <= 16384, H % 32 == 0 (H % 128 == 0 for
 * packed scales).
 */
MXQ_API mxq_status add_rmsnorm_dual_out(const void* x_bf16, int64_t ldx, const void* residual, int32_t residual_type,
                                        int64_t ldr, const void* gamma_bf16, float eps, int64_t T, int64_t H,
                                        void* residual_out, int64_t ldro, void* y_bf16, void* y_q,
                                        void* y_sf_packed_i32, void* y_sf_rowmajor, void* y_sf_128x4, void* stream);

/*
 * moe_route -- the router of a mixture of experts, from the gate's logits to k expert ids and
 * weights per token:
 *   score  s_e = sigmoid(l_e), or softmax over the experts whose logit is not -inf or NaN
 *   choice c_e = s_e + bias_e; without a bias experts are ordered by their logits
 *   groups > 1: the E experts are `groups` runs of E / groups. A group's value is the sum of its
 *     `group_top` (1 or 2) largest choices; the topk_groups groups of largest value are kept.
 *   ids: the k experts of the kept groups with the largest choices, in falling order
 *   weights: scale * s_e, or scale * s_e / (sum of the chosen s + 1e-20) with renormalize
 * Ties go to the lowest index, among experts and among groups. The order of choices and of group
 * values is that of their exact values: where two fp32 values lie within their error bounds the
 * row is decided in fp64 (equal fp64 values are ties).
 *
 * An expert whose logit, or choice, is -inf or NaN is never chosen, and a group of such experts is
 * never kept; slots that cannot be filled hold id -1 and weight 0. Logits of +inf count as the
 * largest finite value.
 *
 *   logits   [T, E] of logits_type, row stride ldl elements (any alignment of the element).
 *   bias     [E] fp32, or NULL.
 *   ids      [T, k] int32 out; weights [T, k] fp32 out (contiguous).
 * Requires T >= 1, 1 <= E <= 1024, 1 <= k <= 32, k <= topk_groups * (E / groups),
 * 1 <= topk_groups <= groups <= 32, E % groups == 0.
 */
MXQ_API mxq_status moe_route(const void* logits, int32_t logits_type, int64_t ldl, const void* bias_f32, int64_t T,
                             int32_t E, int32_t k, int32_t scoring, int32_t groups, int32_t topk_groups,
                             int32_t group_top, int32_t renormalize, float scale, void* ids_i32, void* weights_f32,
                             void* stream);

/*
 * moe_experts_mxfp8 -- the experts' products:
 *   (g, u)    = W13_e x_t                       fp32 accumulation, e = ids[t, j]
 *   a         = MXFP8( RNE_bf16( silu(g) * u ) )  the rule of mxfp8_quantize
 *   out[t]    = RNE_bf16( sum_j weights[t, j] * (W2_e a) )        fp32 throughout, j ascending
 * An id outside [0, E) takes no part; a token without any gives zeros. The same id may appear
 * more than once in a row.
 *
 *   x    [T, H] MXFP8, scales MXQ_SF_ROWMAJOR_U8 or MXQ_SF_TILED_128X4.
 *   ids  [T, k] int32, weights [T, k] fp32 (contiguous).
 *   w13  [E * 2 I, H] MXFP8, scales F8_128x4: expert e's rows start at e * 2 I and alternate, row
 *        2 i the gate of feature i and row 2 i + 1 its up projection (so that a tensor-core tile
 *        holds both).
 *   w2   [E * H, I] MXFP8, scales F8_128x4.
 *   out_bf16 [T, H], row stride ldo elements.
 *   workspace: required, mxq_moe_workspace_bytes(T, k, E, H, I) bytes, 16-byte aligned. Its
 *        contents need no clearing; calls that overlap in time need separate workspaces.
 *   status: optional device status word (mxq_status_bytes()).
 * Requires T >= 1, 1 <= k <= 64, 1 <= E <= 1024, H % 128 == 0, I % 128 == 0, T * k <= 2^24.
 * Four launches (plan, two grouped GEMMs, combine), five with many pairs (the scales' copies apart);
 * the results do not depend on timing.
 */
MXQ_API int64_t mxq_moe_workspace_bytes(int64_t T, int32_t k, int32_t E, int64_t H, int64_t I);

MXQ_API mxq_status moe_experts_mxfp8(const mxq_mx_tensor* x, const void* ids_i32, const void* weights_f32, int64_t T,
                                     int32_t k, const mxq_mx_tensor* w13, const mxq_mx_tensor* w2, int32_t E, int64_t H,
                                     int64_t I, void* out_bf16, int64_t ldo, void* workspace, int64_t workspace_bytes,
                                     void* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_MOE_H_ */
