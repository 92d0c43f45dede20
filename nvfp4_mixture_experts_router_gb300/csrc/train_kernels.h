// Kernel launchers (host side) of the training operators, used by
// train_api.cu.  `elem`: bytes of an element, 2 (BF16) or 4 (FP32).
#pragma once
#include "../../include/moe_nvfp4_train.h"
#include "kernels.h"

namespace moe {

// route_rows.cu
size_t sort_workspace_bytes(int T, int E, int K);
cudaError_t setup_sort_kernels();
cudaError_t launch_sort_routes(const LaunchCtx& c, int T, int E, int K, const int* ids, int* count, int* offsets,
                               int* row_of_route, int* route_of_row, int* workspace);
cudaError_t launch_dispatch(const LaunchCtx& c, int T, int H, int K, int64_t rows, int elem, const void* x,
                            int64_t x_stride, const int* row_of_route, const int* rows_used, void* x_rows);
// w == nullptr: weight 1
cudaError_t launch_combine(const LaunchCtx& c, int T, int H, int K, int64_t rows, int elem, const void* o,
                           const int* row_of_route, const float* w, void* y, int64_t y_stride);
cudaError_t launch_combine_backward(const LaunchCtx& c, int T, int H, int K, int64_t rows, int elem, const void* dy,
                                    int64_t dy_stride, const void* o, const int* row_of_route, const float* w,
                                    const int* rows_used, void* d_o, float* dw);

// layer_norm.cu (x and y may be the same rows; workspace of layer_norm_workspace_bytes;
// skip_row: a row that a ring kernel never copies, for tests, or -1)
cudaError_t launch_layer_norm(const LaunchCtx& c, int T, int H, int elem, const void* x, int64_t x_stride,
                              const float* gamma, const float* beta, float eps, void* y, int64_t y_stride, float* mean,
                              float* rstd, int skip_row);
cudaError_t setup_layer_norm_kernels();
size_t layer_norm_workspace_bytes(int T, int H);
cudaError_t launch_layer_norm_backward(const LaunchCtx& c, int T, int H, int elem, const void* dy, int64_t dy_stride,
                                       const void* x, int64_t x_stride, const float* gamma, const float* mean,
                                       const float* rstd, void* dx, int64_t dx_stride, float* dgamma, float* dbeta,
                                       float* workspace, int skip_row);

// grad_clip.cu
size_t grad_norm_workspace_bytes(int n);
cudaError_t launch_grad_norm(const LaunchCtx& c, int n, const void* const* grads, const int64_t* numels,
                             const int32_t* dtypes, float* norm, float* workspace);
cudaError_t launch_grad_clip(const LaunchCtx& c, int sms, int n, const void* const* grads, void* const* out,
                             const int64_t* numels, const int32_t* dtypes, const float* norm, float max_norm,
                             float eps);

// expert_linear.cu
enum ExpertProduct : int { kExpertForward = 0, kExpertDgrad = 1, kExpertWgrad = 2 };
struct ExpertArgs {
    int64_t rows;
    int N, K, E;
    const void* a;         // x_rows (forward), dy_rows (dgrad, wgrad)
    const void* b;         // w (forward, dgrad), x_rows (wgrad)
    void* out;
    const int* count;      // [E]
    const int* offsets;    // [E]
    unsigned int* status;  // may be null
};
cudaError_t setup_expert_linear_kernels(int device, int num_sms);
cudaError_t launch_expert_linear(const LaunchCtx& c, int product, int device, const ExpertArgs& a);

}  // namespace moe
