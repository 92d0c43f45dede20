// Layer norm over the rows of x, forward and backward.
//
//   mean = sum x / H,  var = sum (x - mean)^2 / H,  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd gamma + beta
//   g = dy gamma,  xhat = (x - mean) rstd
//   dx = rstd (g - sum g / H - xhat sum(g xhat) / H)
//   dgamma = sum_t dy xhat,  dbeta = sum_t dy
//
// The variance is the second pass's sum of squared differences, not
// E[x^2] - mean^2: a row whose mean is far larger than its spread would lose
// the difference of the two.  HBM is the bound: x and dy in, y or dx out.
#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormParts = 64;     // row groups of the dgamma / dbeta partial sums

// Sum over the block; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) r += s[i];
    return r;
}

template <typename T_, int VEC>
__global__ void __launch_bounds__(kNormThreads) layer_norm_kernel(int H, const typename RowVec<T_, VEC>::Raw* x,
                                                                  int64_t x_stride, const float* gamma,
                                                                  const float* beta, float eps,
                                                                  typename RowVec<T_, VEC>::Raw* y, int64_t y_stride,
                                                                  float* mean_out, float* rstd_out) {
    using RV = RowVec<T_, VEC>;
    __shared__ float s[kNormThreads / 32];
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int n = H / VEC;
    float sum = 0.0f;
    for (int c = threadIdx.x; c < n; c += kNormThreads) {
        float v[VEC];
        RV::unpack(x[t * x_stride + c], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum += v[j];
    }
    const float mean = block_sum(sum, s) / (float)H;
    float sq = 0.0f;
    for (int c = threadIdx.x; c < n; c += kNormThreads) {
        float v[VEC];
        RV::unpack(x[t * x_stride + c], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sq = fmaf(v[j] - mean, v[j] - mean, sq);
    }
    const float rstd = 1.0f / sqrtf(block_sum(sq, s) / (float)H + eps);
    for (int c = threadIdx.x; c < n; c += kNormThreads) {
        float v[VEC];
        RV::unpack(x[t * x_stride + c], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int h = c * VEC + j;
            v[j] = fmaf((v[j] - mean) * rstd, gamma[h], beta ? beta[h] : 0.0f);
        }
        y[t * y_stride + c] = RV::pack(v);
    }
    if (threadIdx.x == 0 && mean_out) {
        mean_out[t] = mean;
        rstd_out[t] = rstd;
    }
}

// Partial sums of dgamma and dbeta: a thread per column, a group of rows per
// blockIdx.y.
template <typename T_>
__global__ void __launch_bounds__(kNormThreads) layer_norm_partial_kernel(int T, int H,
                                                                          const typename RowVec<T_, 1>::Raw* dy,
                                                                          int64_t dy_stride,
                                                                          const typename RowVec<T_, 1>::Raw* x,
                                                                          int64_t x_stride, const float* mean,
                                                                          const float* rstd, float* part) {
    using RV = RowVec<T_, 1>;
    pdl_wait();
    const int h = blockIdx.x * kNormThreads + threadIdx.x;
    if (h >= H) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t t = blockIdx.y; t < T; t += kNormParts) {
        float g[1], v[1];
        RV::unpack(dy[t * dy_stride + h], g);
        RV::unpack(x[t * x_stride + h], v);
        dg = fmaf(g[0], (v[0] - mean[t]) * rstd[t], dg);
        db += g[0];
    }
    part[(size_t)blockIdx.y * 2 * H + h] = dg;
    part[(size_t)blockIdx.y * 2 * H + H + h] = db;
}

__global__ void __launch_bounds__(kNormThreads) layer_norm_reduce_kernel(int H, const float* part, float* dgamma,
                                                                         float* dbeta) {
    pdl_wait();
    const int h = blockIdx.x * kNormThreads + threadIdx.x;
    if (h >= H) return;
    float dg = 0.0f, db = 0.0f;
    for (int p = 0; p < kNormParts; ++p) {
        dg += part[(size_t)p * 2 * H + h];
        db += part[(size_t)p * 2 * H + H + h];
    }
    dgamma[h] = dg;
    if (dbeta) dbeta[h] = db;
}

template <typename T_, int VEC>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dx_kernel(int H, const typename RowVec<T_, VEC>::Raw* dy, int64_t dy_stride,
                         const typename RowVec<T_, VEC>::Raw* x, int64_t x_stride, const float* gamma,
                         const float* mean_in, const float* rstd_in, typename RowVec<T_, VEC>::Raw* dx,
                         int64_t dx_stride) {
    using RV = RowVec<T_, VEC>;
    __shared__ float s[kNormThreads / 32];
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int n = H / VEC;
    const float mean = mean_in[t], rstd = rstd_in[t];
    float sg = 0.0f, sgx = 0.0f;
    for (int c = threadIdx.x; c < n; c += kNormThreads) {
        float g[VEC], v[VEC];
        RV::unpack(dy[t * dy_stride + c], g);
        RV::unpack(x[t * x_stride + c], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            g[j] *= gamma[c * VEC + j];
            sg += g[j];
            sgx = fmaf(g[j], (v[j] - mean) * rstd, sgx);
        }
    }
    sg = block_sum(sg, s) / (float)H;
    sgx = block_sum(sgx, s) / (float)H;
    for (int c = threadIdx.x; c < n; c += kNormThreads) {
        float g[VEC], v[VEC];
        RV::unpack(dy[t * dy_stride + c], g);
        RV::unpack(x[t * x_stride + c], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            v[j] = rstd * (g[j] * gamma[c * VEC + j] - sg - (v[j] - mean) * rstd * sgx);
        dx[t * dx_stride + c] = RV::pack(v);
    }
}

bool vec16(const void* p, int64_t stride, int elem) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * elem % 16 == 0;
}

template <typename T_, int VEC>
cudaError_t forward_any(const LaunchCtx& c, int T, int H, const void* x, int64_t x_stride, const float* gamma,
                        const float* beta, float eps, void* y, int64_t y_stride, float* mean, float* rstd) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    return c.launch(layer_norm_kernel<T_, VEC>, dim3(T), dim3(kNormThreads), 0, H, static_cast<const Raw*>(x),
                    x_stride / VEC, gamma, beta, eps, static_cast<Raw*>(y), y_stride / VEC, mean, rstd);
}

template <typename T_, int VEC>
cudaError_t dx_any(const LaunchCtx& c, int T, int H, const void* dy, int64_t dy_stride, const void* x,
                   int64_t x_stride, const float* gamma, const float* mean, const float* rstd, void* dx,
                   int64_t dx_stride) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    return c.launch(layer_norm_dx_kernel<T_, VEC>, dim3(T), dim3(kNormThreads), 0, H, static_cast<const Raw*>(dy),
                    dy_stride / VEC, static_cast<const Raw*>(x), x_stride / VEC, gamma, mean, rstd,
                    static_cast<Raw*>(dx), dx_stride / VEC);
}

}  // namespace

cudaError_t launch_layer_norm(const LaunchCtx& c, int T, int H, int elem, const void* x, int64_t x_stride,
                              const float* gamma, const float* beta, float eps, void* y, int64_t y_stride, float* mean,
                              float* rstd) {
    const bool wide = (int64_t)H * elem % 16 == 0 && vec16(x, x_stride, elem) && vec16(y, y_stride, elem);
    if (elem == 2)
        return wide ? forward_any<__nv_bfloat16, 8>(c, T, H, x, x_stride, gamma, beta, eps, y, y_stride, mean, rstd)
                    : forward_any<__nv_bfloat16, 1>(c, T, H, x, x_stride, gamma, beta, eps, y, y_stride, mean, rstd);
    return wide ? forward_any<float, 4>(c, T, H, x, x_stride, gamma, beta, eps, y, y_stride, mean, rstd)
                : forward_any<float, 1>(c, T, H, x, x_stride, gamma, beta, eps, y, y_stride, mean, rstd);
}

size_t layer_norm_workspace_bytes(int T, int H) {
    (void)T;
    return align_up((uint64_t)kNormParts * 2 * H * 4, 256);
}

cudaError_t launch_layer_norm_backward(const LaunchCtx& c, int T, int H, int elem, const void* dy, int64_t dy_stride,
                                       const void* x, int64_t x_stride, const float* gamma, const float* mean,
                                       const float* rstd, void* dx, int64_t dx_stride, float* dgamma, float* dbeta,
                                       float* workspace) {
    // the column sums first: dx may overwrite dy or x
    const dim3 cols((unsigned)((H + kNormThreads - 1) / kNormThreads));
    const dim3 parts(cols.x, kNormParts);
    cudaError_t e;
    if (elem == 2)
        e = c.launch(layer_norm_partial_kernel<__nv_bfloat16>, parts, dim3(kNormThreads), 0, T, H,
                     static_cast<const uint16_t*>(dy), dy_stride, static_cast<const uint16_t*>(x), x_stride, mean,
                     rstd, workspace);
    else
        e = c.launch(layer_norm_partial_kernel<float>, parts, dim3(kNormThreads), 0, T, H,
                     static_cast<const uint32_t*>(dy), dy_stride, static_cast<const uint32_t*>(x), x_stride, mean,
                     rstd, workspace);
    if (e != cudaSuccess) return e;
    e = c.launch(layer_norm_reduce_kernel, cols, dim3(kNormThreads), 0, H, (const float*)workspace, dgamma, dbeta);
    if (e != cudaSuccess || T == 0) return e;
    const bool wide = (int64_t)H * elem % 16 == 0 && vec16(x, x_stride, elem) && vec16(dy, dy_stride, elem) &&
                      vec16(dx, dx_stride, elem);
    if (elem == 2)
        return wide ? dx_any<__nv_bfloat16, 8>(c, T, H, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx, dx_stride)
                    : dx_any<__nv_bfloat16, 1>(c, T, H, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx, dx_stride);
    return wide ? dx_any<float, 4>(c, T, H, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx, dx_stride)
                : dx_any<float, 1>(c, T, H, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx, dx_stride);
}

}  // namespace moe
