/*
 * moe_nvfp4_train.h — the training operators of a MoE block, part of
 * libmoe_nvfp4.so (sm_103a): routes sorted by expert, token rows to their
 * experts and back, the experts' BF16 matrix products, layer norm, and the
 * global gradient norm with clipping, each with its gradient.
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

#ifdef __cplusplus
}
#endif
#endif /* MOE_NVFP4_TRAIN_H */
