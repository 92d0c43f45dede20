// Routes sorted by expert, and token rows copied to their experts' segments
// and back: the data movement around the experts' products, with gradients.
//
//   sort              stable counting sort of the routes r = t*K + k by expert
//   dispatch          x_rows[row(r)] = x[t]
//   combine           y[t] = sum_k w[t,k] o_rows[row(t,k)]
//   combine_backward  do_rows[row(r)] = w_r dy[t],  dw_r = <dy[t], o_rows[row(r)]>
//   dispatch_backward dx[t] = sum_k dx_rows[row(t,k)]   (combine with weight 1)
//
// All of them are bound by HBM.  The row kernels go token by token: a token's
// row is read (or written) once and its K expert rows once each, so that the
// bytes moved are the algorithmic ones, and every sum has one owner and a
// fixed order.
#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

// ---- sort -------------------------------------------------------------------

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMinChunk = 1024;   // routes per block
constexpr int kSortMaxBlocks = 128;   // every block reads every block's counts

struct SortPlan {
    int chunk, blocks;
};
inline SortPlan sort_plan(int64_t routes) {
    int64_t chunk = (routes + kSortMaxBlocks - 1) / kSortMaxBlocks;
    chunk = (chunk + kSortThreads - 1) / kSortThreads * kSortThreads;
    if (chunk < kSortMinChunk) chunk = kSortMinChunk;
    int64_t blocks = (routes + chunk - 1) / chunk;
    return SortPlan{(int)chunk, (int)(blocks < 1 ? 1 : blocks)};
}

// Per-block expert counts [blocks][E].
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(int64_t routes, int E, int chunk,
                                                                  const int* __restrict__ ids,
                                                                  int* __restrict__ block_count) {
    extern __shared__ int s_count[];
    pdl_wait();
    for (int e = threadIdx.x; e < E; e += kSortThreads) s_count[e] = 0;
    __syncthreads();
    const int64_t r0 = (int64_t)blockIdx.x * chunk;
    const int64_t r1 = min(routes, r0 + chunk);
    for (int64_t r = r0 + threadIdx.x; r < r1; r += kSortThreads) {
        const int e = ids[r];
        if ((unsigned)e < (unsigned)E) atomicAdd(&s_count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) block_count[(size_t)blockIdx.x * E + e] = s_count[e];
    pdl_launch_dependents();
}

// Positions.  A block owns `chunk` consecutive routes, a warp an eighth of
// them.  First row of expert e for the block: (routes of earlier experts) +
// (routes of e in earlier blocks), from the block counts; the block's warps
// then divide it by their own counts, and a route's rank among the 32 of its
// warp step is the number of lower lanes with the same expert.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(int64_t routes, int E, int chunk, int blocks,
                                                                  const int* __restrict__ ids,
                                                                  const int* __restrict__ block_count,
                                                                  int* __restrict__ count, int* __restrict__ offsets,
                                                                  int* __restrict__ row_of_route,
                                                                  int* __restrict__ route_of_row) {
    extern __shared__ int smem[];
    int* s_warp = smem;                       // [kSortWarps][E] counts, then next rows
    int* s_base = smem + kSortWarps * E;      // [E]
    __shared__ int s_scan[kSortWarps + 1];
    __shared__ int s_used;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    for (int i = tid; i < kSortWarps * E; i += kSortThreads) s_warp[i] = 0;
    __syncthreads();
    const int64_t r0 = (int64_t)blockIdx.x * chunk;
    const int64_t r1 = min(routes, r0 + chunk);
    const int sub = chunk / kSortWarps;       // a multiple of 32
    const int64_t w0 = min(r1, r0 + (int64_t)warp * sub), w1 = min(r1, w0 + sub);
    for (int64_t r = w0 + lane; r < w1; r += 32) {
        const int e = ids[r];
        if ((unsigned)e < (unsigned)E) atomicAdd(&s_warp[warp * E + e], 1);
    }
    __syncthreads();
    // totals of all blocks, routes of earlier blocks; scan of the totals in
    // runs of 256 experts
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += kSortThreads) {
        const int e = e0 + tid;
        int total = 0, before = 0;
        if (e < E) {
            if (blocks == 1) {
                for (int w = 0; w < kSortWarps; ++w) total += s_warp[w * E + e];
            } else {
                for (int b = 0; b < blocks; ++b) {
                    const int c = block_count[(size_t)b * E + e];
                    before += b < (int)blockIdx.x ? c : 0;
                    total += c;
                }
            }
        }
        int incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += a;
        }
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        int below = carry, all = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            below += w < warp ? s_scan[w] : 0;
            all += s_scan[w];
        }
        const int first = below + incl - total;
        if (e < E) {
            s_base[e] = first + before;
            if (blockIdx.x == 0) {
                count[e] = total;
                offsets[e] = first;
            }
        }
        carry += all;
        __syncthreads();
    }
    if (tid == 0) {
        s_used = carry;
        if (blockIdx.x == 0) offsets[E] = carry;
    }
    for (int e = tid; e < E; e += kSortThreads) {
        int run = s_base[e];
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = s_warp[w * E + e];
            s_warp[w * E + e] = run;
            run += c;
        }
    }
    __syncthreads();
    for (int64_t b = w0; b < w1; b += 32) {
        const int64_t r = b + lane;
        int e = r < w1 ? ids[r] : -1;
        if ((unsigned)e >= (unsigned)E) e = -1;
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        int row = -1;
        if (e >= 0) row = s_warp[warp * E + e] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) s_warp[warp * E + e] += __popc(peers);
        __syncwarp();
        if (r < w1) {
            row_of_route[r] = row;
            if (row >= 0) route_of_row[row] = (int)r;
            if (r >= s_used) route_of_row[r] = -1;
        }
    }
    pdl_launch_dependents();
}

// ---- rows -------------------------------------------------------------------

constexpr int kRowThreads = 256;

// Threads per token: a power of two in 32..kRowThreads, about `per` vectors
// each.
inline int lanes_for(int vectors, int per) {
    int lanes = 32;
    while (lanes < kRowThreads && lanes * per < vectors) lanes *= 2;
    return lanes;
}

// V vectors of a token's row in registers, then a store per route.  The grid's
// y splits the row.
template <typename Raw, int V>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(int T, int n, int K, int64_t rows,
                                                               const Raw* __restrict__ x, int64_t x_stride,
                                                               const int* __restrict__ row_of_route,
                                                               const int* __restrict__ rows_used,
                                                               Raw* __restrict__ x_rows, int lanes) {
    pdl_wait();
    const int t = blockIdx.x * (kRowThreads / lanes) + threadIdx.x / lanes;
    const int c0 = blockIdx.y * lanes * V + threadIdx.x % lanes;
    if (c0 >= n) return;
    if (t < T) {
        Raw v[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c0 + i * lanes < n) v[i] = x[(int64_t)t * x_stride + c0 + i * lanes];
        for (int k = 0; k < K; ++k) {
            const int64_t row = row_of_route[(int64_t)t * K + k];
            if (row < 0 || row >= rows) continue;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c0 + i * lanes < n) x_rows[row * n + c0 + i * lanes] = v[i];
        }
    }
    if (rows_used) {
        const Raw zero = {};
        const int groups = gridDim.x * (kRowThreads / lanes);
        for (int64_t row = (int64_t)max(0, *rows_used) + t; row < rows; row += groups)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c0 + i * lanes < n) x_rows[row * n + c0 + i * lanes] = zero;
    }
}

// One vector of a token's row per thread: the weighted sum over its routes,
// k ascending, four rows in flight.
template <typename T_, int VEC, bool WEIGHTED>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(int T, int n, int K, int64_t rows,
                                                              const typename RowVec<T_, VEC>::Raw* __restrict__ o,
                                                              const int* __restrict__ row_of_route,
                                                              const float* __restrict__ topk_w,
                                                              typename RowVec<T_, VEC>::Raw* __restrict__ y,
                                                              int64_t y_stride, int lanes) {
    using RV = RowVec<T_, VEC>;
    pdl_wait();
    const int t = blockIdx.x * (kRowThreads / lanes) + threadIdx.x / lanes;
    if (t >= T) return;
    const int c = blockIdx.y * lanes + threadIdx.x % lanes;
    if (c >= n) return;
    float acc[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += 4) {
        typename RV::Raw v[4];
        float w[4];
        bool there[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = k0 + i < K ? row_of_route[(int64_t)t * K + k0 + i] : -1;
            there[i] = row >= 0 && row < rows;
            if (there[i]) {
                v[i] = o[row * n + c];
                w[i] = WEIGHTED ? topk_w[(int64_t)t * K + k0 + i] : 1.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!there[i]) continue;
            float f[VEC];
            RV::unpack(v[i], f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) acc[j] = WEIGHTED ? fmaf(w[i], f[j], acc[j]) : acc[j] + f[j];
        }
    }
    y[(int64_t)t * y_stride + c] = RV::pack(acc);
}

// A token's row of dy against its routes' rows of o, eight routes at a time.
template <typename T_, int VEC>
__global__ void __launch_bounds__(kRowThreads)
    combine_backward_kernel(int T, int n, int K, int64_t rows, const typename RowVec<T_, VEC>::Raw* __restrict__ dy,
                            int64_t dy_stride, const typename RowVec<T_, VEC>::Raw* __restrict__ o,
                            const int* __restrict__ row_of_route, const float* __restrict__ topk_w,
                            const int* __restrict__ rows_used, typename RowVec<T_, VEC>::Raw* __restrict__ d_o,
                            float* __restrict__ dw, int lanes) {
    using RV = RowVec<T_, VEC>;
    constexpr int kK = 8;
    __shared__ float s_part[kRowThreads / 32][kK];
    pdl_wait();
    const int t = blockIdx.x * (kRowThreads / lanes) + threadIdx.x / lanes;
    const int tl = threadIdx.x % lanes, warp = threadIdx.x >> 5;
    const bool live = t < T;
    for (int k0 = 0; k0 < K; k0 += kK) {
        int64_t row[kK];
        float w[kK], acc[kK];
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            row[i] = live && k0 + i < K ? row_of_route[(int64_t)t * K + k0 + i] : -1;
            if (row[i] >= rows) row[i] = -1;
            w[i] = row[i] >= 0 ? topk_w[(int64_t)t * K + k0 + i] : 0.0f;
            acc[i] = 0.0f;
        }
        if (live) {
            for (int c = tl; c < n; c += lanes) {
                float g[VEC];
                RV::unpack(dy[(int64_t)t * dy_stride + c], g);
#pragma unroll
                for (int i = 0; i < kK; ++i) {
                    if (row[i] < 0) continue;
                    float f[VEC], d[VEC];
                    RV::unpack(o[row[i] * n + c], f);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        acc[i] = fmaf(g[j], f[j], acc[i]);
                        d[j] = w[i] * g[j];
                    }
                    d_o[row[i] * n + c] = RV::pack(d);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const float s = warp_sum(acc[i]);
            if ((threadIdx.x & 31) == 0) s_part[warp][i] = s;
        }
        __syncthreads();
        if (live && tl < kK && k0 + tl < K) {
            float s = 0.0f;
            for (int v = 0; v < lanes / 32; ++v) s += s_part[threadIdx.x / lanes * (lanes / 32) + v][tl];
            dw[(int64_t)t * K + k0 + tl] = s;
        }
        __syncthreads();
    }
    if (rows_used) {
        const int groups = gridDim.x * (kRowThreads / lanes);
        for (int64_t r = (int64_t)max(0, *rows_used) + t; r < rows; r += groups)
            for (int c = tl; c < n; c += lanes) d_o[r * n + c] = RV::zero();
    }
}

bool vec16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Blocks for T tokens, `lanes` threads each (one for none: rows to clear).
unsigned token_blocks(int T, int lanes) {
    const int per = kRowThreads / lanes;
    return (unsigned)(T < 1 ? 1 : (T + per - 1) / per);
}

// Rows of H elements, `stride` apart, that all start on 16-byte boundaries.
bool vec16_rows(const void* p, int64_t stride, int elem) { return vec16(p) && stride * elem % 16 == 0; }

}  // namespace

size_t sort_workspace_bytes(int T, int E, int K) {
    const SortPlan p = sort_plan((int64_t)T * K);
    return align_up(p.blocks > 1 ? (uint64_t)p.blocks * E * 4 : 4, 256);
}

cudaError_t launch_sort_routes(const LaunchCtx& c, int T, int E, int K, const int* ids, int* count, int* offsets,
                               int* row_of_route, int* route_of_row, int* workspace) {
    const int64_t routes = (int64_t)T * K;
    const SortPlan p = sort_plan(routes);
    LaunchCtx next = c;
    if (p.blocks > 1) {
        const cudaError_t e = c.launch(sort_count_kernel, dim3(p.blocks), dim3(kSortThreads), (size_t)E * 4, routes, E,
                                       p.chunk, ids, workspace);
        if (e != cudaSuccess) return e;
        next.pdl = true;
    }
    return next.launch(sort_place_kernel, dim3(p.blocks), dim3(kSortThreads), (size_t)(kSortWarps + 1) * E * 4, routes,
                       E, p.chunk, p.blocks, ids, (const int*)workspace, count, offsets, row_of_route, route_of_row);
}

cudaError_t launch_dispatch(const LaunchCtx& c, int T, int H, int K, int64_t rows, int elem, const void* x,
                            int64_t x_stride, const int* row_of_route, const int* rows_used, void* x_rows) {
    const bool wide = H * elem % 16 == 0 && vec16_rows(x, x_stride, elem) && vec16(x_rows);
    const int per = wide ? 16 / elem : 1;
    const int n = H / per;
    constexpr int V = 4;
    const int lanes = lanes_for(n, V);
    const dim3 grid(token_blocks(T, lanes),
                    (unsigned)((n + lanes * V - 1) / (lanes * V)));
#define MOE_DISPATCH(RAW)                                                                                      \
    c.launch(dispatch_kernel<RAW, V>, grid, dim3(kRowThreads), 0, T, n, K, rows, static_cast<const RAW*>(x),    \
             x_stride / per, row_of_route, rows_used, static_cast<RAW*>(x_rows), lanes)
    if (wide) return MOE_DISPATCH(uint4);
    if (elem == 4) return MOE_DISPATCH(uint32_t);
    return MOE_DISPATCH(uint16_t);
#undef MOE_DISPATCH
}

template <typename T_, int VEC>
static cudaError_t combine_any(const LaunchCtx& c, int T, int H, int K, int64_t rows, const void* o,
                               const int* row_of_route, const float* w, void* y, int64_t y_stride) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    const int n = H / VEC;
    const int lanes = lanes_for(n, 1);
    const dim3 grid(token_blocks(T, lanes),
                    (unsigned)((n + lanes - 1) / lanes));
    if (w)
        return c.launch(combine_kernel<T_, VEC, true>, grid, dim3(kRowThreads), 0, T, n, K, rows,
                        static_cast<const Raw*>(o), row_of_route, w, static_cast<Raw*>(y), y_stride / VEC, lanes);
    return c.launch(combine_kernel<T_, VEC, false>, grid, dim3(kRowThreads), 0, T, n, K, rows,
                    static_cast<const Raw*>(o), row_of_route, w, static_cast<Raw*>(y), y_stride / VEC, lanes);
}

cudaError_t launch_combine(const LaunchCtx& c, int T, int H, int K, int64_t rows, int elem, const void* o,
                           const int* row_of_route, const float* w, void* y, int64_t y_stride) {
    const bool wide = H * elem % 16 == 0 && vec16(o) && vec16_rows(y, y_stride, elem);
    if (elem == 2)
        return wide ? combine_any<__nv_bfloat16, 8>(c, T, H, K, rows, o, row_of_route, w, y, y_stride)
                    : combine_any<__nv_bfloat16, 1>(c, T, H, K, rows, o, row_of_route, w, y, y_stride);
    return wide ? combine_any<float, 4>(c, T, H, K, rows, o, row_of_route, w, y, y_stride)
                : combine_any<float, 1>(c, T, H, K, rows, o, row_of_route, w, y, y_stride);
}

template <typename T_, int VEC>
static cudaError_t combine_backward_any(const LaunchCtx& c, int T, int H, int K, int64_t rows, const void* dy,
                                        int64_t dy_stride, const void* o, const int* row_of_route, const float* w,
                                        const int* rows_used, void* d_o, float* dw) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    const int n = H / VEC;
    const int lanes = lanes_for(n, 2);
    return c.launch(combine_backward_kernel<T_, VEC>,
                    dim3(token_blocks(T, lanes)), dim3(kRowThreads), 0, T, n,
                    K, rows, static_cast<const Raw*>(dy), dy_stride / VEC, static_cast<const Raw*>(o), row_of_route, w,
                    rows_used, static_cast<Raw*>(d_o), dw, lanes);
}

cudaError_t launch_combine_backward(const LaunchCtx& c, int T, int H, int K, int64_t rows, int elem, const void* dy,
                                    int64_t dy_stride, const void* o, const int* row_of_route, const float* w,
                                    const int* rows_used, void* d_o, float* dw) {
    const bool wide = H * elem % 16 == 0 && vec16(o) && vec16(d_o) && vec16_rows(dy, dy_stride, elem);
    if (elem == 2)
        return wide ? combine_backward_any<__nv_bfloat16, 8>(c, T, H, K, rows, dy, dy_stride, o, row_of_route, w,
                                                             rows_used, d_o, dw)
                    : combine_backward_any<__nv_bfloat16, 1>(c, T, H, K, rows, dy, dy_stride, o, row_of_route, w,
                                                             rows_used, d_o, dw);
    return wide ? combine_backward_any<float, 4>(c, T, H, K, rows, dy, dy_stride, o, row_of_route, w, rows_used, d_o,
                                                 dw)
                : combine_backward_any<float, 1>(c, T, H, K, rows, dy, dy_stride, o, row_of_route, w, rows_used, d_o,
                                                 dw);
}

}  // namespace moe
