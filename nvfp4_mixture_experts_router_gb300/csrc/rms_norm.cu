// RMS norm with the residual's addition, forward and backward.
//
//   h = x + residual, rounded;  rstd = 1 / sqrt(sum h^2 / H + eps)
//   y = h rstd gamma;  q = E4M3(y / scale), the scale from the largest |y| of a
//   row, of 128 elements or (a power of two) of 32
//   hhat = h rstd,  g = dy gamma
//   dx = dh + rstd (g - hhat sum(g hhat) / H),  dgamma = sum_t dy hhat
//
// HBM is the bound: every input read once, every output written once.
#include <math.h>

#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr float kE4M3Max = 448.0f;

// A row's scale from the largest |y|, and what y is multiplied by.  At least
// 2^-126: the reciprocal stays finite.
__device__ __forceinline__ float linear_scale(float amax) {
    return amax == 0.0f ? 1.0f : fmaxf(amax / kE4M3Max, 1.17549435e-38f);
}

constexpr int kRmsThreads = 512;
constexpr int kRmsParts = 152;      // row groups of dgamma

// Sum (or maximum) over the block; every thread gets it.
template <bool MAX>
__device__ __forceinline__ float block_join(float v, float* s) {
    v = MAX ? warp_max(v) : warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < (int)(blockDim.x >> 5) ? s[lane] : 0.0f;
    return MAX ? warp_max(v) : warp_sum(v);
}

template <typename T_, int VEC>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&v)[VEC], float inv) {
    if constexpr (VEC == 1) {
        *q = (uint8_t)f32x2_to_e4m3x2(v[0] * inv, 0.0f);
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint16_t*>(q) = (uint16_t)f32x2_to_e4m3x2(v[0] * inv, v[1] * inv);
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k)
            w[k] = f32x2_to_e4m3x2(v[4 * k] * inv, v[4 * k + 1] * inv) |
                   f32x2_to_e4m3x2(v[4 * k + 2] * inv, v[4 * k + 3] * inv) << 16;
        if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(q) = w[0];
    }
}

// A block a row, which is walked once for each of its results.
template <typename T_, int VEC>
__global__ void __launch_bounds__(kRmsThreads)
    rms_norm_kernel(const RmsArgs a) {
    using RV = RowVec<T_, VEC>;
    using Raw = typename RV::Raw;
    __shared__ float s[32];
    extern __shared__ float s_block[];      // the largest |y| of each 32 elements
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int n = a.H / VEC, n32 = (a.H + 31) / 32;
    const Raw* x = static_cast<const Raw*>(a.x) + t * (a.x_stride / VEC);
    const Raw* res = a.residual ? static_cast<const Raw*>(a.residual) + t * (a.residual_stride / VEC) : nullptr;
    Raw* h = a.h ? static_cast<Raw*>(a.h) + t * (a.h_stride / VEC) : nullptr;
    auto row = [&](int c, bool again, float (&v)[VEC]) {
        if (again && h) {                   // x or the residual may be h
            RV::unpack(h[c], v);
            return;
        }
        RV::unpack(x[c], v);
        if (res) {
            float u[VEC];
            RV::unpack(res[c], u);
#pragma unroll
            for (int k = 0; k < VEC; ++k) u[k] += v[k];
            const Raw sum = RV::pack(u);
            if (h) h[c] = sum;
            RV::unpack(sum, v);
        }
    };
    float sq = 0.0f;
    for (int c = threadIdx.x; c < n; c += kRmsThreads) {
        float v[VEC];
        row(c, false, v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) sq = fmaf(v[k], v[k], sq);
    }
    const float rstd = 1.0f / sqrtf(block_join<false>(sq, s) / (float)a.H + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[t] = rstd;
    float scale = 1.0f;
    if (a.q) {
        float amax = 0.0f;
        if (a.scale_mode != MOE_SCALE_ROW) {
            for (int b = threadIdx.x; b < n32; b += kRmsThreads) s_block[b] = 0.0f;
            __syncthreads();
        }
        for (int c = threadIdx.x; c < n; c += kRmsThreads) {
            float v[VEC], m = 0.0f;
            row(c, true, v);
#pragma unroll
            for (int k = 0; k < VEC; ++k) m = fmaxf(m, fabsf(v[k] * rstd * a.gamma[c * VEC + k]));
            amax = fmaxf(amax, m);
            // of non-negative floats the order of the bits is that of the values
            if (a.scale_mode != MOE_SCALE_ROW)
                atomicMax(reinterpret_cast<int*>(s_block) + c * VEC / 32, __float_as_int(m));
        }
        if (a.scale_mode == MOE_SCALE_ROW) {
            scale = linear_scale(block_join<true>(amax, s));
            if (threadIdx.x == 0) static_cast<float*>(a.scales)[t] = scale;
        } else {
            __syncthreads();
            if (a.scale_mode == MOE_SCALE_MX) {
                for (int b = threadIdx.x; b < n32; b += kRmsThreads) {
                    const int e = mx_block_exp(s_block[b]);
                    static_cast<uint8_t*>(a.scales)[t * n32 + b] = (uint8_t)(e + 127);
                    s_block[b] = pow2f(-e);
                }
            } else {
                const int n128 = (a.H + 127) / 128;
                for (int b = threadIdx.x; b < n128; b += kRmsThreads) {
                    float m = 0.0f;
                    for (int k = 4 * b; k < 4 * b + 4 && k < n32; ++k) m = fmaxf(m, s_block[k]);
                    const float sc = linear_scale(m);
                    static_cast<float*>(a.scales)[t * n128 + b] = sc;
                    for (int k = 4 * b; k < 4 * b + 4 && k < n32; ++k) s_block[k] = 1.0f / sc;
                }
            }
            __syncthreads();
        }
    }
    Raw* y = a.y ? static_cast<Raw*>(a.y) + t * (a.y_stride / VEC) : nullptr;
    uint8_t* q = a.q ? static_cast<uint8_t*>(a.q) + t * a.H : nullptr;
    const float inv = 1.0f / scale;
    for (int c = threadIdx.x; c < n; c += kRmsThreads) {
        float v[VEC];
        row(c, true, v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = v[k] * rstd * a.gamma[c * VEC + k];
        if (y) y[c] = RV::pack(v);
        if (q) store_codes<T_, VEC>(q + c * VEC, v, a.scale_mode == MOE_SCALE_ROW ? inv : s_block[c * VEC / 32]);
    }
    pdl_launch_dependents();
}

// ---- backward -----------------------------------------------------------------------

// Partial sums of dgamma: a thread per column, a group of rows per blockIdx.y.
template <typename T_>
__global__ void __launch_bounds__(256) rms_partial_kernel(const RmsGradArgs a) {
    using RV = RowVec<T_, 1>;
    using Raw = typename RV::Raw;
    pdl_wait();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.H) return;
    float sum = 0.0f;
    for (int64_t t = blockIdx.y; t < a.T; t += kRmsParts) {
        float g[1], v[1];
        RV::unpack(static_cast<const Raw*>(a.dy)[t * a.dy_stride + c], g);
        RV::unpack(static_cast<const Raw*>(a.h)[t * a.h_stride + c], v);
        sum = fmaf(g[0], v[0] * a.rstd[t], sum);
    }
    a.part[(size_t)blockIdx.y * a.H + c] = sum;
}

__global__ void __launch_bounds__(256) rms_reduce_kernel(int H, int parts, const float* part, float* dgamma) {
    pdl_wait();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= H) return;
    float sum = 0.0f;
    for (int p = 0; p < parts; ++p) sum += part[(size_t)p * H + c];
    dgamma[c] = sum;
}

template <typename T_, int VEC>
__global__ void __launch_bounds__(kRmsThreads) rms_dx_kernel(const RmsGradArgs a) {
    using RV = RowVec<T_, VEC>;
    using Raw = typename RV::Raw;
    __shared__ float s[32];
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int n = a.H / VEC;
    const Raw* dy = static_cast<const Raw*>(a.dy) + t * (a.dy_stride / VEC);
    const Raw* h = static_cast<const Raw*>(a.h) + t * (a.h_stride / VEC);
    const Raw* dh = a.dh ? static_cast<const Raw*>(a.dh) + t * (a.dh_stride / VEC) : nullptr;
    Raw* dx = static_cast<Raw*>(a.dx) + t * (a.dx_stride / VEC);
    const float rstd = a.rstd[t];
    float sum = 0.0f;
    for (int c = threadIdx.x; c < n; c += kRmsThreads) {
        float g[VEC], v[VEC];
        RV::unpack(dy[c], g);
        RV::unpack(h[c], v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum = fmaf(g[k] * a.gamma[c * VEC + k], v[k] * rstd, sum);
    }
    const float mean = block_join<false>(sum, s) / (float)a.H;
    for (int c = threadIdx.x; c < n; c += kRmsThreads) {
        float g[VEC], v[VEC], u[VEC];
        RV::unpack(dy[c], g);
        RV::unpack(h[c], v);
        if (dh) RV::unpack(dh[c], u);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float d = rstd * (g[k] * a.gamma[c * VEC + k] - v[k] * rstd * mean);
            v[k] = dh ? u[k] + d : d;
        }
        dx[c] = RV::pack(v);
    }
}

template <typename T_, int VEC>
cudaError_t forward_any(const LaunchCtx& c, const RmsArgs& a) {
    const size_t smem = a.q && a.scale_mode != MOE_SCALE_ROW ? (size_t)(a.H + 31) / 32 * 4 : 0;
    return c.launch(rms_norm_kernel<T_, VEC>, dim3((unsigned)a.T), dim3(kRmsThreads), smem, a);
}
template <typename T_, int VEC>
cudaError_t dx_any(const LaunchCtx& c, const RmsGradArgs& a) {
    return c.launch(rms_dx_kernel<T_, VEC>, dim3((unsigned)a.T), dim3(kRmsThreads), 0, a);
}
cudaError_t launch_dx(const LaunchCtx& c, int elem, int bytes, const RmsGradArgs& a) {
    MOE_ROW_VEC(elem, bytes, dx_any, c, a);
}

}  // namespace

cudaError_t launch_rms_norm(const LaunchCtx& c, int elem, const RmsArgs& a) {
    const int bytes = row_vec_bytes(a.H, elem,
                                    row_at(a.x, a.x_stride, elem) | row_at(a.residual, a.residual ? a.residual_stride : 0, elem) |
                                        row_at(a.h, a.h ? a.h_stride : 0, elem) | row_at(a.y, a.y ? a.y_stride : 0, elem) |
                                        row_at(a.q) * elem);
    MOE_ROW_VEC(elem, bytes, forward_any, c, a);
}

size_t rms_norm_workspace_bytes(int T, int H) { return align_up((uint64_t)kRmsParts * H * 4, 256); }

cudaError_t launch_rms_norm_backward(const LaunchCtx& c, int elem, const RmsGradArgs& a) {
    // the column sums first: dx may overwrite dy or h
    const dim3 parts((unsigned)((a.H + 255) / 256), kRmsParts);
    cudaError_t e = c.launch(elem == 2 ? rms_partial_kernel<__nv_bfloat16> : rms_partial_kernel<float>, parts, dim3(256),
                             0, a);
    if (e != cudaSuccess) return e;
    e = c.launch(rms_reduce_kernel, dim3((unsigned)((a.H + 255) / 256)), dim3(256), 0, a.H, kRmsParts,
                 (const float*)a.part, a.dgamma);
    if (e != cudaSuccess || a.T == 0) return e;
    const int bytes = row_vec_bytes(a.H, elem,
                                    row_at(a.dy, a.dy_stride, elem) | row_at(a.dh, a.dh ? a.dh_stride : 0, elem) |
                                        row_at(a.h, a.h_stride, elem) | row_at(a.dx, a.dx_stride, elem));
    return launch_dx(c, elem, bytes, a);
}

}  // namespace moe
