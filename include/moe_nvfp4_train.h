/*
 * moe_nvfp4_train.h — the training operators of a MoE block, part of
 * libmoe_nvfp4.so (sm_103a): experts chosen from logits, routes sorted by
 * expert, token rows to their experts and back, the experts' BF16 matrix
 * products, layer norm, RMS norm with the residual's addition, the global
 * gradient norm with clipping, each with its gradient, and AdamW.
 *
 * The conventions of moe_nvfp4.h hold: data pointers are device pointers
 * owned by the caller, nothing is allocated or synchronized, arguments are
 * checked on the host before anything is launched, `stream` is a
 * cudaStream_t (NULL = legacy default stream).  Also:
 *   - No output may overlap an input or another output unless its comment
 *     says so (MOE_ERR_INVALID_ARG).  Token rows of one stride may lie side by
 *     side in one buffer; other ranges that cross count as overlapping.
 *   - An empty call (T = 0, rows = 0, no elements) is valid; operands of no
 *     elements may be NULL.
 *   - Sums, statistics and accumulators are FP32; each output is rounded
 *     once, to nearest even.  No atomics on data, fixed orders: results are
 *     bit-reproducible on the same device.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_WORKSPACE, MOE_ERR_UNSUPPORTED,
 * MOE_ERR_CUDA.
 */
#ifndef MOE_NVFP4_TRAIN_H
#define MOE_NVFP4_TRAIN_H

#include "moe_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the operators below. */
#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_F32 1

/* ---- experts chosen from logits ----------------------------------------------
 * For each token t, from its row of logits l [T][E] (MOE_DTYPE_*, rows
 * logits_stride elements apart):
 *   score   s = softmax of l over the E experts, or sigmoid(l)
 *   choice  c = s + bias, or l where bias is NULL (the same order)
 *   groups  experts [g E/groups, (g+1) E/groups) are group g; a group's score
 *           is the largest c of its experts, or the sum of the two largest s
 *           (+ bias); only experts of the topk_groups best groups are chosen
 *   topk_ids [T][K] the K largest c, from the largest down
 *   topk_w   [T][K] scale * s of the chosen, divided by their sum with
 *           renormalize; the bias does not enter
 * Ties go to the lower expert, or group.  c and the groups' scores compare as
 * if computed in 64 bits: where FP32 cannot tell two apart, they are computed
 * in FP64.  An expert whose logit or bias is -infinity or NaN is not chosen (a
 * logit's also has the score 0) and does not count for its group; a logit of
 * +infinity counts as the largest FP32 number (a bias of it is ahead of all).
 * Slots beyond the experts that can be chosen get id -1 and weight 0: dropped
 * routes of the calls below.
 * Renormalized weights do not underflow together: they come from l, relative to
 * the largest chosen.
 * Backward, dlogits [T][E] of the logits' type from dw [T][K], with the same
 * rule and the forward's ids (the choice itself has no gradient, nor the bias):
 * every element is written.  Ids outside [0, E) add nothing; slots of one
 * expert add up, in the slots' order.
 * 1 <= E <= 1024, 1 <= groups <= 32, E a multiple of groups, 1 <= topk_groups
 * <= groups, 1 <= K <= min(32, topk_groups * E / groups), 0 <= T <= 2^22;
 * scale finite.  bias FP32 [E]; topk_ids int32, topk_w and dw FP32; pointers
 * aligned to their element.  dlogits may be logits itself (same pointer and
 * stride). */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
#define MOE_GROUP_MAX 0
#define MOE_GROUP_TOP2 1
typedef struct {
    int32_t score;        /* MOE_SCORE_*                                      */
    int32_t groups;       /* 1: no groups                                     */
    int32_t topk_groups;
    int32_t group_score;  /* MOE_GROUP_*                                      */
    int32_t renormalize;  /* 0 or 1                                           */
    float scale;
} moe_route_rule;
MOE_API moe_status moe_nvfp4_route_topk(int T, int E, int K, int dtype,
                                        const void* logits, int64_t logits_stride,
                                        const float* bias, moe_route_rule rule,
                                        int32_t* topk_ids, float* topk_w, void* stream);
MOE_API moe_status moe_nvfp4_route_topk_backward(int T, int E, int K, int dtype,
                                                 const void* logits, int64_t logits_stride,
                                                 const int32_t* topk_ids, const float* dw,
                                                 moe_route_rule rule,
                                                 void* dlogits, int64_t dlogits_stride,
                                                 void* stream);

/* ---- routes sorted by expert ------------------------------------------------
 * Stable counting sort of the T*K routes r = t*K + k by their expert:
 *   topk_ids      [T][K] int32.  An id outside [0, E) is a dropped route.
 *                 Repeated experts of one token are kept as routes of their
 *                 own.
 *   count         [E]    routes of each expert
 *   offsets       [E+1]  exclusive prefix of count; offsets[E] = kept routes
 *   row_of_route  [T*K]  position of route r in the order, -1 if dropped
 *   route_of_row  [T*K]  route at a position; -1 from offsets[E] on
 * All int32, 4-byte aligned.  1 <= E <= 1024, 1 <= K <= 32, 0 <= T <= 2^22,
 * T*K <= 2^26.  workspace: moe_nvfp4_sort_workspace_bytes(T, E, K) (0 if the
 * sizes are invalid), 256-byte aligned. */
MOE_API size_t moe_nvfp4_sort_workspace_bytes(int T, int E, int K);
MOE_API moe_status moe_nvfp4_sort_routes(int T, int E, int K, const int32_t* topk_ids,
                                         int32_t* count, int32_t* offsets,
                                         int32_t* row_of_route, int32_t* route_of_row,
                                         void* workspace, size_t workspace_bytes,
                                         void* stream);

/* ---- token rows to their experts and back -------------------------------------
 * `rows` is the number of rows that the expert-ordered buffers hold and
 * row_of_route [T][K] int32 the row of each route: the output of
 * moe_nvfp4_sort_routes (rows >= T*K) or the tile-padded rows of
 * moe_nvfp4_route_noalloc.  No two routes share a row.  A route whose row is
 * outside [0, rows) is dropped: it is neither read nor written and
 * contributes nothing, whatever its weight.  Expert-ordered buffers are
 * contiguous [rows][H]; token buffers [T][H] have rows `*_stride` elements
 * apart (>= H).  dtype: MOE_DTYPE_*; 1 <= H <= 65536, 1 <= K <= 32,
 * 0 <= T <= 2^22, 0 <= rows <= 2^27; pointers aligned to their element
 * (16-byte aligned rows are copied 16 bytes at a time).
 *
 * dispatch:          x_rows[row(t,k)] = x[t]
 * combine:           y[t] = sum_k topk_w[t][k] * o_rows[row(t,k)], k ascending
 * dispatch_backward: dx[t] = sum_k dx_rows[row(t,k)], k ascending
 * combine_backward:  do_rows[row(t,k)] = topk_w[t][k] * dy[t]
 *                    dw[t][k] = sum_h dy[t][h] * o_rows[row(t,k)][h]; 0 if dropped
 * topk_w and dw are FP32 [T][K].  rows_used: device int32, rows [rows_used,
 * rows) of x_rows / do_rows are set to zero (offsets + E of the sort), by a
 * dispatch of T = 0 tokens those alone; NULL leaves every row that no route
 * owns as it was. */
MOE_API moe_status moe_nvfp4_dispatch(int T, int H, int K, int64_t rows, int dtype,
                                      const void* x, int64_t x_stride,
                                      const int32_t* row_of_route, const int32_t* rows_used,
                                      void* x_rows, void* stream);
MOE_API moe_status moe_nvfp4_dispatch_backward(int T, int H, int K, int64_t rows, int dtype,
                                               const void* dx_rows, const int32_t* row_of_route,
                                               void* dx, int64_t dx_stride, void* stream);
MOE_API moe_status moe_nvfp4_combine(int T, int H, int K, int64_t rows, int dtype,
                                     const void* o_rows, const int32_t* row_of_route,
                                     const float* topk_w, void* y, int64_t y_stride,
                                     void* stream);
MOE_API moe_status moe_nvfp4_combine_backward(int T, int H, int K, int64_t rows, int dtype,
                                              const void* dy, int64_t dy_stride,
                                              const void* o_rows, const int32_t* row_of_route,
                                              const float* topk_w, const int32_t* rows_used,
                                              void* do_rows, float* dw, void* stream);

/* ---- the experts' matrix products ------------------------------------------------
 * BF16 operands and outputs, FP32 accumulation on the tensor cores.  Expert e
 * owns the rows [offsets[e], offsets[e] + count[e]) (int32, device, [E]; the
 * entry offsets[E] of the sort is not read); w is [E][N][K].
 *   expert_linear        y_rows[r]  = x_rows[r] w[e]^T        [rows][N]
 *   expert_linear_dgrad  dx_rows[r] = dy_rows[r] w[e]         [rows][K]
 *   expert_linear_wgrad  dw[e] = sum over e's rows of dy_rows[r]^T x_rows[r]
 *                        [E][N][K], zero for an expert without rows
 * Rows of no expert are neither read into a result nor written.  A segment
 * that does not lie in [0, rows) counts as empty and, where `status` (device
 * uint32, NULL allowed) is given, sets a bit there that
 * moe_nvfp4_last_device_status reports as MOE_ERR_INVALID_ARG; a bounded
 * wait that gives up sets another (MOE_ERR_TIMEOUT; the output is then
 * undefined).  The caller clears the word.  Segments may not overlap.
 * 1 <= E <= 1024; N and K multiples of 8 in 8..65536; 0 <= rows <= 2^27;
 * E*N and E*K < 2^31; row buffers and w contiguous and 16-byte aligned. */
MOE_API moe_status moe_nvfp4_expert_linear(int64_t rows, int N, int K, int E,
                                           const void* x_rows, const void* w,
                                           const int32_t* count, const int32_t* offsets,
                                           void* y_rows, uint32_t* status, void* stream);
MOE_API moe_status moe_nvfp4_expert_linear_dgrad(int64_t rows, int N, int K, int E,
                                                 const void* dy_rows, const void* w,
                                                 const int32_t* count, const int32_t* offsets,
                                                 void* dx_rows, uint32_t* status, void* stream);
MOE_API moe_status moe_nvfp4_expert_linear_wgrad(int64_t rows, int N, int K, int E,
                                                 const void* dy_rows, const void* x_rows,
                                                 const int32_t* count, const int32_t* offsets,
                                                 void* dw, uint32_t* status, void* stream);

/* ---- layer norm ---------------------------------------------------------------------
 * Over the last dimension of x [T][H] (rows x_stride elements apart):
 *   mean[t] = sum_h x / H,  rstd[t] = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
 *   y = (x - mean) * rstd * gamma + beta
 * gamma and beta are FP32 [H] (beta may be NULL: 0); mean and rstd FP32 [T]
 * (both may be NULL for inference).  eps >= 0, finite.
 * 1 <= H <= 65536, 0 <= T <= 2^22.  y may be x itself (same pointer and
 * stride).
 * Backward, from the forward's mean and rstd, with xhat = (x - mean) * rstd
 * and g = dy * gamma:
 *   dx     = rstd * (g - sum_h g / H - xhat * sum_h (g * xhat) / H)
 *   dgamma = sum_t dy * xhat,  dbeta = sum_t dy   (FP32 [H]; dbeta may be NULL)
 * dx may be dy or x itself (same pointer and stride).  workspace:
 * moe_nvfp4_layer_norm_workspace_bytes(T, H) (0 if invalid), 256-byte
 * aligned.  With T = 0, dgamma and dbeta are zero.
 * Rows that are copied ahead (calls of many tokens) are waited for 1 s at most:
 * a row whose copy does not land, and the later rows of its block, leave NaN in
 * y or dx and in the statistics, and dgamma and dbeta become NaN.
 * MOE_DEBUG_NORM_SKIP_COPY, added to dtype, is a test hook: the copy of row
 * T / 2 is left out where rows are copied ahead. */
#define MOE_DEBUG_NORM_SKIP_COPY 0x100
MOE_API moe_status moe_nvfp4_layer_norm(int T, int H, int dtype, const void* x, int64_t x_stride,
                                        const float* gamma, const float* beta, float eps,
                                        void* y, int64_t y_stride, float* mean, float* rstd,
                                        void* stream);
MOE_API size_t moe_nvfp4_layer_norm_workspace_bytes(int T, int H);
MOE_API moe_status moe_nvfp4_layer_norm_backward(int T, int H, int dtype,
                                                 const void* dy, int64_t dy_stride,
                                                 const void* x, int64_t x_stride,
                                                 const float* gamma, const float* mean,
                                                 const float* rstd, void* dx, int64_t dx_stride,
                                                 float* dgamma, float* dbeta,
                                                 void* workspace, size_t workspace_bytes,
                                                 void* stream);

/* ---- RMS norm with the residual's addition -------------------------------------------
 * Over the last dimension of x [T][H] (rows x_stride elements apart), with a
 * residual of the same shape or NULL:
 *   h[t]    = x[t] + residual[t], rounded to the rows' type (x without a residual)
 *   rstd[t] = 1 / sqrt(sum_h h^2 / H + eps), from h as rounded
 *   y       = h * rstd * gamma
 * Outputs, each of which may be NULL, but not both y and q:
 *   h      [T][H] (only with a residual); may be x or the residual itself (same
 *          pointer and stride)
 *   y      [T][H] of x's type; may be x or the residual itself, if h is not
 *   q      [T][H] E4M3, contiguous: y before its rounding, divided by its scale
 *          and rounded to nearest even, at most 448 in magnitude
 *   scales of q, with scale_mode: MOE_SCALE_ROW FP32 [T], the row's largest
 *          |y| / 448 (1 for a row of zeros); MOE_SCALE_BLOCK128 FP32
 *          [T][ceil(H/128)], the same for each 128 elements (the last block may
 *          be shorter); MOE_SCALE_MX E8M0 bytes [T][ceil(H/32)], for each 32
 *          elements 2^(floor(log2 of the largest |y|) - 8) as in
 *          MOE_W8A8_MXFP8 (2^-127 for zeros).  NULL exactly if q is.
 *   rstd   [T] FP32
 * A NaN of y is a NaN of q, and does not enter the scales.  gamma FP32 [H];
 * eps >= 0, finite.  The squares and their sum are FP32: a row whose sum of
 * squares passes 3.4e38 has rstd 0, and y 0 where h is finite; with eps = 0 one
 * whose sum is zero has an infinite rstd, and y is not finite.  By row h * gamma
 * has to be within FP32, unless rstd is 0.  1 <= H <= 65536, 0 <= T <= 2^22; pointers
 * aligned to their element.
 * Backward, from the forward's h and rstd, with hhat = h * rstd and g = dy * gamma:
 *   dx     = dh + rstd * (g - hhat * sum_h (g * hhat) / H)     (dh NULL: 0)
 *   dgamma = sum_t dy * hhat   (FP32 [H])
 * dx is the gradient of x and of the residual; dh is the gradient that reaches
 * h from elsewhere.  dx may be dy, dh or h itself (same pointer and stride).
 * workspace: moe_nvfp4_rms_norm_workspace_bytes(T, H) (0 if invalid), 256-byte
 * aligned.  With T = 0, dgamma is zero. */
#define MOE_SCALE_ROW 0
#define MOE_SCALE_BLOCK128 1
#define MOE_SCALE_MX 2
MOE_API moe_status moe_nvfp4_rms_norm(int T, int H, int dtype, const void* x, int64_t x_stride,
                                      const void* residual, int64_t residual_stride,
                                      const float* gamma, float eps,
                                      void* h, int64_t h_stride, void* y, int64_t y_stride,
                                      void* q, void* scales, int scale_mode, float* rstd,
                                      void* stream);
MOE_API size_t moe_nvfp4_rms_norm_workspace_bytes(int T, int H);
MOE_API moe_status moe_nvfp4_rms_norm_backward(int T, int H, int dtype,
                                               const void* dy, int64_t dy_stride,
                                               const void* dh, int64_t dh_stride,
                                               const void* h, int64_t h_stride,
                                               const float* gamma, const float* rstd,
                                               void* dx, int64_t dx_stride, float* dgamma,
                                               void* workspace, size_t workspace_bytes,
                                               void* stream);

/* ---- global gradient norm and clipping ---------------------------------------------
 * Over a list of n tensors (host arrays of device pointers, element counts
 * and MOE_DTYPE_* types; read during the call, not kept):
 *   grad_norm: norm[0] = sqrt(sum over every element g^2)   (device FP32)
 *   grad_clip: out_i = g_i * s,  s = max_norm / (norm[0] + eps), at most 1;
 *              NaN if the quotient is
 * Two calls, so that norms of several devices can be joined between them.
 * out[i] has grads[i]'s type and may be grads[i] itself; in place with s = 1
 * nothing is written.  The squares and their sum are FP32: a norm above 1.8e19
 * is infinite, although every element may be smaller (s is 0 then), elements
 * below 1e-19 in magnitude lose digits and those below 1e-23 add nothing.  The
 * tensors are on the current device.
 * 0 <= n <= 65536, 0 <= numel < 2^40, each pointer aligned to its element;
 * a tensor of no elements may be NULL.  Sizes and pointers are not compared
 * for overlaps: the outputs must not overlap each other or another input.
 * max_norm >= 0 and eps >= 0, finite.  workspace:
 * moe_nvfp4_grad_norm_workspace_bytes(n) (0 if invalid), 256-byte aligned. */
MOE_API size_t moe_nvfp4_grad_norm_workspace_bytes(int n);
MOE_API moe_status moe_nvfp4_grad_norm(int n, const void* const* grads, const int64_t* numels,
                                       const int32_t* dtypes, float* norm,
                                       void* workspace, size_t workspace_bytes, void* stream);
MOE_API moe_status moe_nvfp4_grad_clip(int n, const void* const* grads, void* const* out,
                                       const int64_t* numels, const int32_t* dtypes,
                                       const float* norm, float max_norm, float eps,
                                       void* stream);

/* ---- AdamW -----------------------------------------------------------------------------
 * One step over a list of n tensors (a host array, read during the call, not
 * kept), in place.  With c the clipping factor (1 without a norm, else that of
 * grad_clip: max_norm / (norm[0] + clip_eps), at most 1, NaN if the quotient
 * is) and t the step's number, from 1:
 *   g = c * grad
 *   m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 * A tensor has numel elements, contiguous:
 *   param    BF16 or FP32 (param_dtype), the rounded p
 *   master   FP32 p, for a BF16 param, or NULL: the param is p
 *   grad     BF16 or FP32 (grad_dtype); read only
 *   exp_avg, exp_avg_sq   m and v, by state_bits:
 *     32: FP32, the scales NULL
 *      8: E4M3 bytes of m and of sqrt(v), each block of MOE_ADAMW_BLOCK elements
 *         (the last may be shorter) with an FP32 scale, [ceil(numel / block)] in
 *         exp_avg_scale and exp_avg_sq_scale: value = byte * scale.  Written
 *         with the scale largest magnitude * (1 / 448), rounded to nearest even; a
 *         block whose largest magnitude is below 2^-100 becomes zeros with
 *         scale 0, and no other sqrt(v) > 0 rounds to zero (its byte is 1 at
 *         least).  A block with a value that is not finite becomes NaN.  The
 *         step itself uses m and v before that rounding.  Zeros, bytes and
 *         scales, are the start.
 * Arithmetic is FP32, the bias corrections FP64 on the host; sqrt and the
 * division within 2 units of FP32's last place.  With lr_step (device FP32
 * [2]: lr and t, a whole number up to 2^24) these replace rule.lr and rule.step,
 * so that a captured graph can be replayed with other ones; the corrections
 * are FP32 then.
 * Squares and v are FP32; v below 2^-126 counts as zero, and so does a rate lr /
 * (1 - beta1^t) below 1e-30.  eps counts as 2^-126 times the rate at least, and an
 * element whose denominator passes 2^126 times the rate takes no step.  The rate is
 * 2^126 at most (one of lr_step that is not makes the parameters NaN).
 * 0 <= n <= 65536, 0 <= numel < 2^40; pointers aligned to their element; a
 * tensor of no elements may have NULL pointers.  lr and weight_decay >= 0,
 * 0 <= beta < 1, eps >= 2^-126, max_norm and clip_eps >= 0, all finite; step >= 1
 * (not looked at with lr_step).  The tensors are on the current device; no
 * buffer may overlap another one of the call (not compared). */
#define MOE_ADAMW_BLOCK 256
typedef struct {
    void* param;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    float* exp_avg_scale;
    float* exp_avg_sq_scale;
    float* master;
    int64_t numel;
    int32_t param_dtype;
    int32_t grad_dtype;
    int32_t state_bits;
    int32_t reserved;     /* 0 */
} moe_adamw_tensor;
typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    double max_norm, clip_eps;   /* of the clipping, where norm is given */
    int64_t step;
} moe_adamw_rule;
MOE_API moe_status moe_nvfp4_adamw(int n, const moe_adamw_tensor* tensors, moe_adamw_rule rule,
                                   const float* norm, const float* lr_step, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_NVFP4_TRAIN_H */
