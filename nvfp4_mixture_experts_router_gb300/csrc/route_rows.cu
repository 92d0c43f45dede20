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
// fixed order.  Measured on GB300 (16384 tokens, top-8, H = 7168, BF16; copy
// rate 6.8 TB/s): dispatch 320 us (6.6 TB/s), combine 313 (6.7), its gradient
// 582 (6.8), dispatch_backward 305 (6.9); the sort of the 131072 routes 12.
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

// Per-block expert counts [blocks][E] (more routes than one launch sorts).
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
#pragma unroll 16
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

// The same order in one launch, for up to two routes a thread of a block of
// 1024, or of a cluster of eight of them (`nc` blocks).  A warp counts its routes expert by expert as it ranks
// them (the rank stays in a register); a thread per expert turns the warps'
// counts into starts within the block; the blocks read each other's totals
// through distributed shared memory.
constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterThreads / 32;
constexpr int kClusterBlocks = 8;

template <int S>
__global__ void __launch_bounds__(kClusterThreads, 1)
    sort_cluster_kernel(int routes, int E, int nc, const int* __restrict__ ids, int* __restrict__ count,
                        int* __restrict__ offsets, int* __restrict__ row_of_route, int* __restrict__ route_of_row) {
    extern __shared__ int smem[];
    int* s_warp = smem;                            // [kClusterWarps][E] counts, then starts within the block
    int* s_total = smem + kClusterWarps * E;       // [E] this block's routes of an expert
    __shared__ int s_scan[kClusterWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = nc > 1 ? (int)cluster_cta_rank() : 0;
    for (int i = tid; i < kClusterWarps * E; i += kClusterThreads) s_warp[i] = 0;
    pdl_wait();
    const int r0 = (rank * kClusterThreads + warp * 32) * S + lane;      // S steps of 32 routes a warp
    int id[S], place[S];
#pragma unroll
    for (int i = 0; i < S; ++i) id[i] = r0 + 32 * i < routes ? ids[r0 + 32 * i] : -1;
    __syncthreads();
    int* mine = s_warp + warp * E;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if ((unsigned)id[i] >= (unsigned)E) id[i] = -1;
        const unsigned peers = __match_any_sync(0xffffffffu, id[i]);
        place[i] = 0;
        if (id[i] >= 0) place[i] = mine[id[i]] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (id[i] >= 0 && lane == __ffs(peers) - 1) mine[id[i]] = place[i] + __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    int total = 0;                                 // expert tid's (E <= 1024 threads)
    if (tid < E) {
#pragma unroll 8
        for (int w = 0; w < kClusterWarps; ++w) {
            const int c = s_warp[w * E + tid];
            s_warp[w * E + tid] = total;
            total += c;
        }
        s_total[tid] = total;
    }
    int before = 0;                                // its routes in earlier blocks
    if (nc > 1) {
        cluster_sync_all();
        if (tid < E) {
            int all = 0;
#pragma unroll
            for (int b = 0; b < kClusterBlocks; ++b) {
                int c = 0;
                if (b < nc)
                    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(cluster_map(s_total + tid, b)));
                before += b < rank ? c : 0;
                all += c;
            }
            total = all;
        }
    }
    // exclusive scan of the totals over the experts
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += a;
    }
    if (lane == 31) s_scan[warp] = incl;
    if (nc > 1) cluster_sync_all();                // the totals have been read: their place may be reused
    else __syncthreads();
    const int sum = s_scan[lane];
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += a;
    }
    const int used = __shfl_sync(0xffffffffu, run, 31);
    const int first = __shfl_sync(0xffffffffu, run - sum, warp) + incl - total;
    if (tid < E) {
        s_total[tid] = first + before;             // the block's first row of the expert
        if (rank == 0) {
            count[tid] = total;
            offsets[tid] = first;
        }
    }
    if (rank == 0 && tid == 0) offsets[E] = used;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int r = r0 + 32 * i;
        if (r >= routes) continue;
        const int row = id[i] >= 0 ? s_total[id[i]] + mine[id[i]] + place[i] : -1;
        row_of_route[r] = row;
        if (row >= 0) route_of_row[row] = r;
        if (r >= used) route_of_row[r] = -1;
    }
    pdl_launch_dependents();
}

// ---- rows -------------------------------------------------------------------

constexpr int kRowThreads = 256;

// A route's row, or -1: lane k of every warp of the token loads route k (at
// most 32 a token) in one access, instead of one dependent load per route.
__device__ __forceinline__ int token_route_row(const int* row_of_route, int t, int T, int K, int64_t rows) {
    const int lane = threadIdx.x & 31;
    const int row = t < T && lane < K ? row_of_route[(int64_t)t * K + lane] : -1;
    return row < rows ? row : -1;
}

// Route k's weight in lane k (a dropped route's weight is never used).
__device__ __forceinline__ float token_route_weight(const float* topk_w, int t, int T, int K) {
    const int lane = threadIdx.x & 31;
    return t < T && lane < K ? topk_w[(int64_t)t * K + lane] : 0.0f;
}

// V vectors of a token's row in registers, then a store per route.  The grid's
// y splits the row.  Bound by the stores (K bytes written per byte read).
template <typename Raw, int V>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(int T, int n, int K, int64_t rows,
                                                               const Raw* __restrict__ x, int64_t x_stride,
                                                               const int* __restrict__ row_of_route,
                                                               const int* __restrict__ rows_used,
                                                               Raw* __restrict__ x_rows, int lanes) {
    pdl_wait();
    const int t = blockIdx.x * (kRowThreads / lanes) + threadIdx.x / lanes;
    const int c0 = blockIdx.y * lanes * V + threadIdx.x % lanes;
    const int my_row = token_route_row(row_of_route, t, T, K, rows);
    if (t < T) {                             // warp-uniform: a warp holds one token
        Raw v[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c0 + i * lanes < n) v[i] = x[(int64_t)t * x_stride + c0 + i * lanes];
#pragma unroll 4
        for (int k = 0; k < K; ++k) {
            const int row = __shfl_sync(0xffffffffu, my_row, k);
            if (row < 0) continue;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c0 + i * lanes < n) x_rows[(int64_t)row * n + c0 + i * lanes] = v[i];
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
    pdl_launch_dependents();
}

// V vectors of a token's row per thread: the weighted sum over its routes, k
// ascending, KB rows in flight.
template <typename T_, int VEC, int V, int KB, bool WEIGHTED>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(int T, int n, int K, int64_t rows,
                                                              const typename RowVec<T_, VEC>::Raw* __restrict__ o,
                                                              const int* __restrict__ row_of_route,
                                                              const float* __restrict__ topk_w,
                                                              typename RowVec<T_, VEC>::Raw* __restrict__ y,
                                                              int64_t y_stride, int lanes) {
    using RV = RowVec<T_, VEC>;
    pdl_wait();
    const int t = blockIdx.x * (kRowThreads / lanes) + threadIdx.x / lanes;
    const int c0 = blockIdx.y * lanes * V + threadIdx.x % lanes;
    const int my_row = token_route_row(row_of_route, t, T, K, rows);
    const float my_w = WEIGHTED ? token_route_weight(topk_w, t, T, K) : 1.0f;
    if (t >= T) return;
    float acc[V][VEC];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[i][j] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += KB) {
        typename RV::Raw v[KB][V];
        int row[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            row[k] = __shfl_sync(0xffffffffu, my_row, k0 + k);
            if (k0 + k >= K) row[k] = -1;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (row[k] >= 0 && c0 + i * lanes < n) v[k][i] = o[(int64_t)row[k] * n + c0 + i * lanes];
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const float w = WEIGHTED ? __shfl_sync(0xffffffffu, my_w, k0 + k) : 1.0f;
            if (row[k] < 0) continue;              // warp-uniform
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[VEC];
                RV::unpack(v[k][i], f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[i][j] = WEIGHTED ? fmaf(w, f[j], acc[i][j]) : acc[i][j] + f[j];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (c0 + i * lanes < n) y[(int64_t)t * y_stride + c0 + i * lanes] = RV::pack(acc[i]);
    pdl_launch_dependents();
}

// A token's row of dy against its routes' rows of o, kK routes at a time.
template <typename T_, int VEC, int V, int kK>
__global__ void __launch_bounds__(kRowThreads)
    combine_backward_kernel(int T, int n, int K, int64_t rows, const typename RowVec<T_, VEC>::Raw* __restrict__ dy,
                            int64_t dy_stride, const typename RowVec<T_, VEC>::Raw* __restrict__ o,
                            const int* __restrict__ row_of_route, const float* __restrict__ topk_w,
                            const int* __restrict__ rows_used, typename RowVec<T_, VEC>::Raw* __restrict__ d_o,
                            float* __restrict__ dw, int lanes) {
    using RV = RowVec<T_, VEC>;
    __shared__ float s_part[kRowThreads / 32][kK];
    pdl_wait();
    const int t = blockIdx.x * (kRowThreads / lanes) + threadIdx.x / lanes;
    const int tl = threadIdx.x % lanes, warp = threadIdx.x >> 5;
    const bool live = t < T;
    const int my_row = token_route_row(row_of_route, t, T, K, rows);
    const float my_w = token_route_weight(topk_w, t, T, K);
    for (int k0 = 0; k0 < K; k0 += kK) {
        int row[kK];
        float w[kK], acc[kK];
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            row[k] = __shfl_sync(0xffffffffu, my_row, k0 + k);
            w[k] = __shfl_sync(0xffffffffu, my_w, k0 + k);
            if (k0 + k >= K) row[k] = -1;
            acc[k] = 0.0f;
        }
        if (live) {
            for (int c = tl; c < n; c += lanes * V) {
                typename RV::Raw gr[V], fr[kK][V];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i * lanes < n) gr[i] = dy[(int64_t)t * dy_stride + c + i * lanes];
#pragma unroll
                for (int k = 0; k < kK; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (row[k] >= 0 && c + i * lanes < n) fr[k][i] = o[(int64_t)row[k] * n + c + i * lanes];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (c + i * lanes >= n) continue;
                    float g[VEC];
                    RV::unpack(gr[i], g);
#pragma unroll
                    for (int k = 0; k < kK; ++k) {
                        if (row[k] < 0) continue;
                        float f[VEC], d[VEC];
                        RV::unpack(fr[k][i], f);
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            acc[k] = fmaf(g[j], f[j], acc[k]);
                            d[j] = w[k] * g[j];
                        }
                        d_o[(int64_t)row[k] * n + c + i * lanes] = RV::pack(d);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const float s = warp_sum(acc[k]);
            if ((threadIdx.x & 31) == 0) s_part[warp][k] = s;
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
        const typename RV::Raw zero = {};
        const int groups = gridDim.x * (kRowThreads / lanes);
        for (int64_t r = (int64_t)max(0, *rows_used) + t; r < rows; r += groups)
            for (int c = tl; c < n; c += lanes) d_o[r * n + c] = zero;
    }
    pdl_launch_dependents();
}

// Blocks for T tokens, `lanes` threads each (one for none: rows to clear).
unsigned token_blocks(int T, int lanes) {
    const int per = kRowThreads / lanes;
    return (unsigned)(T < 1 ? 1 : (T + per - 1) / per);
}

// Threads per token (a power of two in 32..kRowThreads) for rows of n items,
// an item a thread at a time: the most threads among the counts that leave
// the fewest idle in the last step.
int lanes_for(int n) {
    int best = 32, best_cost = 1 << 30;
    for (int lanes = 32; lanes <= kRowThreads; lanes *= 2) {
        const int cost = (n + lanes - 1) / lanes * lanes;
        if (cost <= best_cost) {
            best = lanes;
            best_cost = cost;
        }
    }
    return best;
}

// The same where a token's threads walk its whole row: with few tokens as many
// threads as there are items (23 FP32 tokens of 2688, top-8: 19 -> 5 us).
constexpr int kFewTokens = 608;
int walk_lanes(int n, int T) {
    if (T > kFewTokens) return lanes_for(n);
    int lanes = 32;
    while (lanes < kRowThreads && lanes < n) lanes *= 2;
    return lanes;
}

}  // namespace

size_t sort_workspace_bytes(int T, int E, int K) {
    const SortPlan p = sort_plan((int64_t)T * K);
    return align_up(p.blocks > 1 ? (uint64_t)p.blocks * E * 4 : 4, 256);
}

cudaError_t setup_sort_kernels() {
    constexpr int most = (kClusterWarps + 1) * 1024 * 4;
    const cudaError_t e = cudaFuncSetAttribute(sort_cluster_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(sort_cluster_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

// Up to 1024 routes: one block of sort_place_kernel, which counts for itself.
// Up to 16384: one launch of one block or a cluster of eight.  More: a block
// per 1024 routes and a launch before it for their counts (the match of equal
// experts takes about 1 us a step of 32 warps on an SM: eight SMs are too few).
// Measured on GB300 (top-8, 64 experts; us cluster, two launches): 1600 routes
// 3.6 5.4;  4096 5.1 5.6;  8192 5.2 7.0;  32768 7.6 7.0;  131072 22 10.5.
cudaError_t launch_sort_routes(const LaunchCtx& c, int T, int E, int K, const int* ids, int* count, int* offsets,
                               int* row_of_route, int* route_of_row, int* workspace) {
    const int64_t routes = (int64_t)T * K;
    const SortPlan p = sort_plan(routes);
    if (p.blocks > 1 && routes <= 2 * kClusterBlocks * kClusterThreads) {
        LaunchCtx one = c;
        one.cluster = routes <= 2 * kClusterThreads ? 1 : kClusterBlocks;
        auto kernel = routes <= one.cluster * kClusterThreads ? sort_cluster_kernel<1> : sort_cluster_kernel<2>;
        return one.launch(kernel, dim3(one.cluster), dim3(kClusterThreads), (size_t)(kClusterWarps + 1) * E * 4,
                          (int)routes, E, one.cluster, ids, count, offsets, row_of_route, route_of_row);
    }
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
    const int bytes = row_vec_bytes(H, elem, row_at(x, x_stride, elem) | row_at(x_rows));
    const int per = bytes / elem;
    const int n = H / per;
    // groups of threads: a token each, and of the rows to clear 32 each at most
    // (as many as a token has routes: more groups than tokens only where the
    // buffer is larger than the routes, as in a call that clears and copies none:
    // half of 131072 rows of 7168 BF16 2037 us with one group, 134 so)
    const int groups = rows_used && T < rows / 32 ? (int)(rows / 32) : T;
    // few tokens: a vector a thread over more blocks; else four, so that a
    // thread has four loads in flight
    const bool few = groups < 64;
    const int lanes = lanes_for(few ? n : (n + 3) / 4);
    const int slice = lanes * (few ? 1 : 4);
    const dim3 grid(token_blocks(groups, lanes), (unsigned)((n + slice - 1) / slice));
#define MOE_DISPATCH(RAW, V)                                                                                   \
    c.launch(dispatch_kernel<RAW, V>, grid, dim3(kRowThreads), 0, T, n, K, rows, static_cast<const RAW*>(x),    \
             x_stride / per, row_of_route, rows_used, static_cast<RAW*>(x_rows), lanes)
    switch (bytes) {
        case 16: return few ? MOE_DISPATCH(uint4, 1) : MOE_DISPATCH(uint4, 4);
        case 8: return few ? MOE_DISPATCH(uint2, 1) : MOE_DISPATCH(uint2, 4);
        case 4: return few ? MOE_DISPATCH(uint32_t, 1) : MOE_DISPATCH(uint32_t, 4);
        default: return few ? MOE_DISPATCH(uint16_t, 1) : MOE_DISPATCH(uint16_t, 4);
    }
#undef MOE_DISPATCH
}

template <typename T_, int VEC, int V, int KB>
static cudaError_t combine_shape(const LaunchCtx& c, int T, int H, int K, int64_t rows, const void* o,
                                 const int* row_of_route, const float* w, void* y, int64_t y_stride) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    const int n = H / VEC;
    const int lanes = lanes_for((n + V - 1) / V);
    const dim3 grid(token_blocks(T, lanes), (unsigned)((n + lanes * V - 1) / (lanes * V)));
    auto kernel = w ? combine_kernel<T_, VEC, V, KB, true> : combine_kernel<T_, VEC, V, KB, false>;
    return c.launch(kernel, grid, dim3(kRowThreads), 0, T, n, K, rows, static_cast<const Raw*>(o), row_of_route, w,
                    static_cast<Raw*>(y), y_stride / VEC, lanes);
}

// Loads in flight: of 16-byte vectors one of eight routes, or two of four
// (11639 FP32 tokens, top-3, 1392: 59 -> 42 us; top-6 is faster with eight: 74
// against 77); of narrower ones four of four, of single BF16 elements eight of
// two (4096 tokens, top-4, 7167: 91.6 -> 84.5 us; 36 tokens of 393, top-4: no).
template <typename T_, int VEC>
static cudaError_t combine_any(const LaunchCtx& c, int T, int H, int K, int64_t rows, const void* o,
                               const int* row_of_route, const float* w, void* y, int64_t y_stride) {
    if (K == 1) return combine_shape<T_, VEC, 4, 1>(c, T, H, K, rows, o, row_of_route, w, y, y_stride);
    if (K == 2) return combine_shape<T_, VEC, 4, 2>(c, T, H, K, rows, o, row_of_route, w, y, y_stride);
    if constexpr (sizeof(typename RowVec<T_, VEC>::Raw) == 16) {
        return K <= 4 ? combine_shape<T_, VEC, 2, 4>(c, T, H, K, rows, o, row_of_route, w, y, y_stride)
                      : combine_shape<T_, VEC, 1, 8>(c, T, H, K, rows, o, row_of_route, w, y, y_stride);
    } else {
        if constexpr (sizeof(typename RowVec<T_, VEC>::Raw) == 2)
            if (T >= 64) return combine_shape<T_, VEC, 8, 2>(c, T, H, K, rows, o, row_of_route, w, y, y_stride);
        return combine_shape<T_, VEC, 4, 4>(c, T, H, K, rows, o, row_of_route, w, y, y_stride);
    }
}

cudaError_t launch_combine(const LaunchCtx& c, int T, int H, int K, int64_t rows, int elem, const void* o,
                           const int* row_of_route, const float* w, void* y, int64_t y_stride) {
    const int bytes = row_vec_bytes(H, elem, row_at(o) | row_at(y, y_stride, elem));
    MOE_ROW_VEC(elem, bytes, combine_any, c, T, H, K, rows, o, row_of_route, w, y, y_stride);
}

template <typename T_, int VEC, int V, int kK>
static cudaError_t combine_backward_shape(const LaunchCtx& c, int T, int H, int K, int64_t rows, const void* dy,
                                          int64_t dy_stride, const void* o, const int* row_of_route, const float* w,
                                          const int* rows_used, void* d_o, float* dw) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    const int n = H / VEC;
    const int lanes = walk_lanes((n + V - 1) / V, T);
    return c.launch(combine_backward_kernel<T_, VEC, V, kK>, dim3(token_blocks(T, lanes)), dim3(kRowThreads), 0, T, n, K,
                    rows, static_cast<const Raw*>(dy), dy_stride / VEC, static_cast<const Raw*>(o), row_of_route, w,
                    rows_used, static_cast<Raw*>(d_o), dw, lanes);
}

// Routes at a time: eight, or four with few of them (11639 FP32 tokens, top-3,
// 1392: 78 -> 72 us; two narrower vectors each: 1001 BF16, 27.9 -> 27.3).
template <typename T_, int VEC>
static cudaError_t combine_backward_any(const LaunchCtx& c, int T, int H, int K, int64_t rows, const void* dy,
                                        int64_t dy_stride, const void* o, const int* row_of_route, const float* w,
                                        const int* rows_used, void* d_o, float* dw) {
    constexpr int V = sizeof(typename RowVec<T_, VEC>::Raw) == 16 ? 1 : 2;
    if (K == 1)
        return combine_backward_shape<T_, VEC, 4, 1>(c, T, H, K, rows, dy, dy_stride, o, row_of_route, w, rows_used, d_o,
                                                     dw);
    if (K == 2)
        return combine_backward_shape<T_, VEC, 2, 2>(c, T, H, K, rows, dy, dy_stride, o, row_of_route, w, rows_used, d_o,
                                                     dw);
    return K <= 4 ? combine_backward_shape<T_, VEC, V, 4>(c, T, H, K, rows, dy, dy_stride, o, row_of_route, w, rows_used,
                                                          d_o, dw)
                  : combine_backward_shape<T_, VEC, 1, 8>(c, T, H, K, rows, dy, dy_stride, o, row_of_route, w, rows_used,
                                                          d_o, dw);
}

cudaError_t launch_combine_backward(const LaunchCtx& c, int T, int H, int K, int64_t rows, int elem, const void* dy,
                                    int64_t dy_stride, const void* o, const int* row_of_route, const float* w,
                                    const int* rows_used, void* d_o, float* dw) {
    const int bytes = row_vec_bytes(H, elem, row_at(o) | row_at(d_o) | row_at(dy, dy_stride, elem));
    MOE_ROW_VEC(elem, bytes, combine_backward_any, c, T, H, K, rows, dy, dy_stride, o, row_of_route, w, rows_used, d_o,
                dw);
}

}  // namespace moe
