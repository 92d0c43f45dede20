// The experts' BF16 matrix products over rows ordered by expert, with FP32
// accumulation:
//   forward  y[r]  = x[r] w[e]^T              (sum over K)
//   dgrad    dx[r] = dy[r] w[e]               (sum over N)
//   wgrad    dw[e] = sum over e's rows dy[r]^T x[r]
#include "common.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kTile = 64, kDepth = 16;

// Rows of expert e; a segment outside [0, rows) is empty and raises a bit.
__device__ __forceinline__ int2 segment(const ExpertArgs& a, int e) {
    const int64_t first = a.offsets[e], n = a.count[e];
    if (n < 0 || first < 0 || first + n > a.rows) {
        if (a.status && threadIdx.x == 0) atomicOr(a.status, kStatusBadRow);
        return make_int2(0, 0);
    }
    return make_int2((int)first, (int)n);
}

// A block per 64 x 64 tile of one expert's product C[m][n] = sum_k A(m,k) B(n,k).
template <int PRODUCT>
__global__ void __launch_bounds__(256) expert_tile_kernel(const ExpertArgs a) {
    __shared__ float s_a[kDepth][kTile + 1], s_b[kDepth][kTile + 1];
    pdl_wait();
    const int e = blockIdx.z;
    const int2 seg = segment(a, e);
    const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(a.a);
    const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(a.b);
    __nv_bfloat16* C = static_cast<__nv_bfloat16*>(a.out);
    const int M = PRODUCT == kExpertWgrad ? a.N : seg.y;
    const int Nc = PRODUCT == kExpertForward ? a.N : a.K;
    const int D = PRODUCT == kExpertForward ? a.K : PRODUCT == kExpertDgrad ? a.N : seg.y;
    const size_t w0 = (size_t)e * a.N * a.K;
    for (int m0 = blockIdx.y * kTile; m0 < M; m0 += gridDim.y * kTile) {
        const int n0 = blockIdx.x * kTile;
        float acc[4][4] = {};
        const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
        for (int d0 = 0; d0 < D; d0 += kDepth) {
            for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
                const int r = i / kDepth, d = i % kDepth;
                const int m = m0 + r, n = n0 + r, k = d0 + d;
                float va = 0.0f, vb = 0.0f;
                if (k < D) {
                    if (m < M)
                        va = PRODUCT == kExpertWgrad ? (float)A[(size_t)(seg.x + k) * a.N + m]
                                                     : (float)A[(size_t)(seg.x + m) * D + k];
                    if (n < Nc)
                        vb = PRODUCT == kExpertForward ? (float)B[w0 + (size_t)n * a.K + k]
                             : PRODUCT == kExpertDgrad ? (float)B[w0 + (size_t)k * a.K + n]
                                                       : (float)B[(size_t)(seg.x + k) * a.K + n];
                }
                s_a[d][r] = va;
                s_b[d][r] = vb;
            }
            __syncthreads();
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                float x[4], w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = s_a[d][ty * 4 + i];
                    w[i] = s_b[d][tx * 4 + i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], w[j], acc[i][j]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
                if (m >= M || n >= Nc) continue;
                const size_t at = PRODUCT == kExpertWgrad ? w0 + (size_t)m * a.K + n : (size_t)(seg.x + m) * Nc + n;
                C[at] = __float2bfloat16_rn(acc[i][j]);
            }
    }
}

}  // namespace

cudaError_t launch_expert_linear(const LaunchCtx& c, int product, const ExpertArgs& a) {
    const int cols = product == kExpertForward ? a.N : a.K;
    const int64_t most = product == kExpertWgrad ? a.N : a.rows;
    const int64_t mt = (most + kTile - 1) / kTile;
    const dim3 grid((unsigned)((cols + kTile - 1) / kTile), (unsigned)(mt < 256 ? mt : 256), (unsigned)a.E);
    if (product == kExpertForward) return c.launch(expert_tile_kernel<kExpertForward>, grid, dim3(256), 0, a);
    if (product == kExpertDgrad) return c.launch(expert_tile_kernel<kExpertDgrad>, grid, dim3(256), 0, a);
    return c.launch(expert_tile_kernel<kExpertWgrad>, grid, dim3(256), 0, a);
}

}  // namespace moe
