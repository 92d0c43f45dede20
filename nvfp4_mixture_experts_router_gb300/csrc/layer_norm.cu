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
//
// Up to 8192 columns a row lies in registers and is read once.  The backward
// kernels are persistent: a block walks rows with the next ones in flight, and
// each thread keeps the dgamma / dbeta sums of its columns in registers until
// the end, so that dy and x are read once for both gradients; the blocks' sums
// go through the workspace to a reduction in a fixed order.  Rows of up to 1024
// columns and calls of few rows go through registers (row kernels), the others
// through a ring of bulk copies in shared memory (ring kernels).  Longer rows
// are walked three times (forward) or twice (dx), the re-reads served by the
// caches, and the column sums are a pass of their own: 3.9 and 4.4 times the
// bytes' time in BF16, 1.9 and 2.8 in FP32.
//
// Measured on GB300 (BF16, 8191 rows; copy rate 6.8 TB/s): 7168 columns
// forward 46 us (5.1 TB/s), backward 67 (5.3); 7167 (rows off 16-byte blocks,
// single elements in and out of the ring) 72 and 123, in registers 202 and 222;
// 256 columns 4.0 and 6.5; 1001 13.6 and 21; 2000 rows of 16384 75 and 130.
// FP32, 7168: forward 72 (6.5 TB/s), backward 107 (6.6); 7167 100 and 120; 2000
// rows of 16384 72 and 161.  One
// row of 7168 BF16: 3.1.
#include <math.h>

#include "f32x2.cuh"
#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormParts = 64;      // row groups of the column sums, long rows
// The persistent kernels' grids are multiples of this.  A constant: the backward's
// workspace, a partial sum a block, is sized without a device
constexpr int kNormSms = 152;
constexpr int kCols = 8;            // columns per thread of the row kernels
constexpr int kRowColumns = 32 * 32 * kCols;
constexpr int kRingCols = 16;       // columns per thread of the ring kernel
// Columns of a row from which the ring kernels take it; rows off 16-byte
// boundaries go there earlier (forward, 8191 rows of 1001 BF16: 21.9 -> 13.6 us,
// of 601 14.8 -> 12.7, of 300 7.2 against 8.3; backward 21 against 25)
constexpr int kRingMin = 1024, kRingMinOdd = 512;
constexpr int kRingMax = 4;         // stages in flight in shared memory (at most)
constexpr int kRingBytes = 200 * 1024;

// The row kernels' shape: W warps a row, G rows a block (256 threads at least).
struct NormShape {
    int W, G;
    int threads() const { return W * G * 32; }
};
NormShape norm_shape(int H, int cols = kCols) {
    const int W = (H + 32 * cols - 1) / (32 * cols);
    return NormShape{W, W >= 8 ? 1 : 8 / W};
}

// Sums of (a, b) over the W warps of a row; every thread gets them.  `turn`
// alternates between calls: one barrier a call suffices.
__device__ __forceinline__ float2 row_sum2(float a, float b, int W, int turn, float2 (*s)[32]) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (W > 1) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) s[turn][warp] = make_float2(a, b);
        __syncthreads();
        const float2 v = lane < W ? s[turn][warp / W * W + lane] : make_float2(0.0f, 0.0f);
        a = warp_sum(v.x);
        b = warp_sum(v.y);
    }
    return make_float2(a, b);
}

constexpr int kPairs = kCols / 2;     // of the row kernels

// A thread's C columns: C / VEC vectors, `lanes` vectors apart.
template <typename T_, int VEC, int C>
__device__ __forceinline__ void unpack_cols(const typename RowVec<T_, VEC>::Raw (&r)[C / VEC], float2 (&v)[C / 2]) {
    float f[C];
#pragma unroll
    for (int i = 0; i < C / VEC; ++i) {
        float u[VEC];
        RowVec<T_, VEC>::unpack(r[i], u);
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[i * VEC + k] = u[k];
    }
#pragma unroll
    for (int q = 0; q < C / 2; ++q) v[q] = make_float2(f[2 * q], f[2 * q + 1]);
}
template <typename T_, int VEC, int C>
__device__ __forceinline__ typename RowVec<T_, VEC>::Raw pack_cols(const float2 (&v)[C / 2], int i) {
    float u[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const int q = i * VEC + k;
        u[k] = q & 1 ? v[q >> 1].y : v[q >> 1].x;
    }
    return RowVec<T_, VEC>::pack(u);
}

// The parameters of the thread's C columns (0 past the row's end).
template <int VEC, int C>
__device__ __forceinline__ void load_params(const float* p, int j, int lanes, int n, bool wide, float2 (&v)[C / 2]) {
#pragma unroll
    for (int i = 0; i < C / VEC; ++i) {
        float2 u[(VEC + 1) / 2];
#pragma unroll
        for (int q = 0; q < (VEC + 1) / 2; ++q) u[q] = both(0.0f);
        if (j + i * lanes < n) load_vector<VEC>(p, j + i * lanes, wide, u);
        if constexpr (VEC == 1) {
            if (i & 1) v[i >> 1].y = u[0].x;
            else v[i >> 1].x = u[0].x;
        } else {
#pragma unroll
            for (int q = 0; q < VEC / 2; ++q) v[i * (VEC / 2) + q] = u[q];
        }
    }
}

// C columns a thread.  The row stays packed in registers and is unpacked for
// each of the three passes.
template <typename T_, int VEC, int C, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_rows_kernel(int T, int H, int W, const typename RowVec<T_, VEC>::Raw* x,
                                                         int64_t x_stride, const float* gamma, const float* beta,
                                                         float eps, typename RowVec<T_, VEC>::Raw* y, int64_t y_stride,
                                                         float* mean_out, float* rstd_out, bool wide_params) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    constexpr int V = C / VEC;
    __shared__ float2 s_red[2][32];
    pdl_wait();
    const int lanes = W * 32, j = threadIdx.x % lanes;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / lanes) + threadIdx.x / lanes;
    const bool live = t < T;
    const int n = H / VEC;
    Raw r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = live && j + i * lanes < n ? x[t * x_stride + j + i * lanes] : Raw{};
    float2 sum = both(0.0f), sq = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float u[VEC];
        RowVec<T_, VEC>::unpack(r[i], u);
#pragma unroll
        for (int k = 0; k < VEC; ++k) (k & 1 ? sum.y : sum.x) += u[k];
    }
    const float mean = row_sum2(sum.x + sum.y, 0.0f, W, 0, s_red).x / (float)H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float u[VEC];
        RowVec<T_, VEC>::unpack(r[i], u);
        if (j + i * lanes < n)                    // columns past the row's end do not count
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float c = u[k] - mean;
                float& s = k & 1 ? sq.y : sq.x;
                s = fmaf(c, c, s);
            }
    }
    const float rstd = 1.0f / sqrtf(row_sum2(sq.x + sq.y, 0.0f, W, 1, s_red).x / (float)H + eps);
    if (live) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = j + i * lanes;
            if (c >= n) continue;
            float2 ga[(VEC + 1) / 2], be[(VEC + 1) / 2];
            float u[VEC];
            RowVec<T_, VEC>::unpack(r[i], u);
            load_vector<VEC>(gamma, c, wide_params, ga);
            if (beta) {
                load_vector<VEC>(beta, c, wide_params, be);
            } else {
#pragma unroll
                for (int q = 0; q < (VEC + 1) / 2; ++q) be[q] = both(0.0f);
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                u[k] = fmaf((u[k] - mean) * rstd, k & 1 ? ga[k >> 1].y : ga[k >> 1].x, k & 1 ? be[k >> 1].y : be[k >> 1].x);
            y[t * y_stride + c] = RowVec<T_, VEC>::pack(u);
        }
        if (j == 0 && mean_out) {
            mean_out[t] = mean;
            rstd_out[t] = rstd;
        }
    }
    pdl_launch_dependents();
}

// A row of the rings below in shared memory.  Rows of whole 16-byte vectors are
// one bulk copy.  Other rows keep their place within 16 bytes: a copy of the
// whole 16-byte blocks inside the row, and the elements before and after it (a
// lane of half a warp each) through a register, stored a turn later, before that
// turn's barrier: a turn ahead of their use at least, as S >= 2.
template <typename T_, bool WHOLE>
struct RingRow {
    static constexpr uint32_t kElem = sizeof(T_);
    using One = typename RowVec<T_, 1>::Raw;
    static __host__ __device__ uint32_t slot(uint32_t bytes) { return WHOLE ? bytes : (bytes + 31) & ~15u; }
    static __device__ __forceinline__ uint32_t offset(const void* row) {
        return WHOLE ? 0u : (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u;
    }
    // [lead, lead + copied(...)) of the row lies in whole blocks
    static __device__ __forceinline__ uint32_t lead(const void* row) {
        return WHOLE ? 0u : (16u - offset(row)) & 15u;
    }
    static __device__ __forceinline__ uint32_t copied(const void* row, uint32_t bytes) {
        return WHOLE ? bytes : (bytes - lead(row)) & ~15u;
    }
    static __device__ __forceinline__ void copy(uint8_t* slot, const void* row, uint32_t bytes, uint64_t* bar,
                                                uint64_t policy) {
        const uint32_t l = lead(row);
        bulk_load(slot + offset(row) + l, static_cast<const uint8_t*>(row) + l, copied(row, bytes), bar, policy);
    }
    One value;
    uint8_t* to = nullptr;
    // lane k of sixteen: an element before the copy (k < 8) or after it
    __device__ __forceinline__ void load(uint8_t* slot, const void* row, uint32_t bytes, int k) {
        const uint32_t l = lead(row);
        const uint32_t at = k < 8 ? k * kElem : l + copied(row, bytes) + (k - 8) * kElem;
        if (at < (k < 8 ? l : bytes)) {
            value = *reinterpret_cast<const One*>(static_cast<const uint8_t*>(row) + at);
            to = slot + offset(row) + at;
        }
    }
    __device__ __forceinline__ void store() {
        if (to) {
            *reinterpret_cast<One*>(to) = value;
            to = nullptr;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // a later copy may write here
        }
    }
};

// NaN in the vectors of a row from `at` on, `lanes` apart; thread j's is the j-th of n.
template <typename T_, int VEC>
__device__ __forceinline__ void put_nan_row(typename RowVec<T_, VEC>::Raw* at, int j, int lanes, int n) {
    float u[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) u[k] = NAN;
    const typename RowVec<T_, VEC>::Raw nan = RowVec<T_, VEC>::pack(u);
#pragma unroll 1
    for (int i = 0; j + i < n; i += lanes) at[i] = nan;
}

// The same for many rows of more than kRingMin columns:
// persistent blocks of up to 512 threads, two an SM where their shared memory
// allows, with gamma and beta in shared memory and the rows ahead in a ring of
// bulk copies, so that a row's two reductions overlap the copies of the next
// rows and the other block's arithmetic.  A stage is free once the first
// reduction has passed its barrier.  Waits as in the backward ring below.
// skip_row: a row whose copy is left out (tests of the wait's limit), or -1.
template <typename T_, int VEC>
__global__ void __launch_bounds__(512, 2)
    norm_ring_kernel(int T, int H, int S, const typename RowVec<T_, VEC>::Raw* x, int64_t x_stride,
                     const float* gamma, const float* beta, float eps, typename RowVec<T_, VEC>::Raw* y,
                     int64_t y_stride, float* mean_out, float* rstd_out, bool wide_params, int skip_row) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    constexpr int C = kRingCols, V = C / VEC, P = C / 2;
    constexpr bool kWhole = sizeof(Raw) == 16;
    using Row = RingRow<T_, kWhole>;
    __shared__ float s_red[2][16];
    __shared__ uint64_t s_full[kRingMax];
    extern __shared__ __align__(16) uint8_t s_ring[];      // gamma, beta [P][threads] float2 each, then [S][n] vectors
    pdl_wait();
    const int lanes = blockDim.x, j = threadIdx.x, lane = j & 31, warp = j >> 5, W = lanes >> 5;
    const int n = H / VEC;
    float2* s_gamma = reinterpret_cast<float2*>(s_ring);
    float2* s_beta = s_gamma + P * lanes;
    uint8_t* s_rows = s_ring + (size_t)lanes * C * 8;
    const uint32_t row_bytes = (uint32_t)n * (uint32_t)sizeof(Raw), slot = Row::slot(row_bytes);
    const int64_t step = gridDim.x, first = blockIdx.x;
    uint64_t policy = 0;
    auto fetch = [&](int64_t t, int stage) {               // thread 0
        if (t == skip_row) return;
        const Raw* row = x + t * x_stride;
        mbar_arrive_expect_tx(&s_full[stage], Row::copied(row, row_bytes));
        Row::copy(s_rows + stage * slot, row, row_bytes, &s_full[stage], policy);
    };
    Row edge;
    if (j == 0) {
        policy = policy_evict_first();                     // x is read once
        for (int q = 0; q < S; ++q) mbar_init(&s_full[q], 1);
        fence_mbar_init();
        for (int q = 0; q < S; ++q)
            if (first + q * step < T) fetch(first + q * step, q);
    }
    if (!kWhole && j < 16)
        for (int q = 0; q < S; ++q)
            if (first + q * step < T) {
                edge.load(s_rows + q * slot, x + (first + q * step) * x_stride, row_bytes, j);
                edge.store();
            }
    {
        float2 p[P];
        load_params<VEC, C>(gamma, j, lanes, n, wide_params, p);
#pragma unroll
        for (int q = 0; q < P; ++q) s_gamma[q * lanes + j] = p[q];     // read by this thread alone, as beta
#pragma unroll
        for (int q = 0; q < P; ++q) p[q] = both(0.0f);
        if (beta) load_params<VEC, C>(beta, j, lanes, n, wide_params, p);
#pragma unroll
        for (int q = 0; q < P; ++q) s_beta[q * lanes + j] = p[q];
    }
    __syncthreads();
    const float inv = 1.0f / (float)H;
    int stage = 0;
    uint32_t parity = 0;
    y += first * y_stride + j;
    const int64_t y_step = step * y_stride;
    volatile int never = 0;
    int64_t t = first;
    for (; t < T; t += step) {
        const bool landed = mbar_wait(&s_full[stage], parity, &never, nullptr, 0);
        float2 v[P];
        {
            const Raw* at = reinterpret_cast<const Raw*>(s_rows + stage * slot + Row::offset(x + t * x_stride)) + j;
            Raw r[V];
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = j + i * lanes < n ? at[i * lanes] : Raw{};
            unpack_cols<T_, VEC, C>(r, v);
        }
        float2 sum = v[0];
#pragma unroll
        for (int q = 1; q < P; ++q) sum = add2(sum, v[q]);
        const float a = warp_sum(sum.x + sum.y);
        if (lane == 0) s_red[0][warp] = a;
        if (!kWhole) edge.store();
        if (__syncthreads_or(!landed)) {
            for (int i = 0; i < 100; ++i) __nanosleep(10000);   // copies in flight land before the block leaves
            break;
        }
        if (t + S * step < T) {
            if (j == 0) fetch(t + S * step, stage);
            if (!kWhole && j < 16) edge.load(s_rows + stage * slot, x + (t + S * step) * x_stride, row_bytes, j);
        }
        const float mean = warp_sum(lane < W ? s_red[0][lane & 15] : 0.0f) * inv;
        float2 sq = both(0.0f);
#pragma unroll
        for (int q = 0; q < P; ++q) {
            v[q] = add2(v[q], both(-mean));
            // columns past the row's end do not count (a pair is of one vector, or of two of one element)
            if (VEC == 1 && j + (2 * q + 1) * lanes >= n) v[q].y = 0.0f;
            if (j + 2 * q / VEC * lanes < n) sq = fma2(v[q], v[q], sq);
        }
        const float b = warp_sum(sq.x + sq.y);
        if (lane == 0) s_red[1][warp] = b;
        __syncthreads();
        const float rstd = 1.0f / sqrtf(warp_sum(lane < W ? s_red[1][lane & 15] : 0.0f) * inv + eps);
#pragma unroll
        for (int q = 0; q < P; ++q) v[q] = fma2(mul2(v[q], both(rstd)), s_gamma[q * lanes + j], s_beta[q * lanes + j]);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (j + i * lanes < n) y[i * lanes] = pack_cols<T_, VEC, C>(v, i);
        if (j == 0 && mean_out) {
            mean_out[t] = mean;
            rstd_out[t] = rstd;
        }
        y += y_step;
        if (++stage == S) { stage = 0; parity ^= 1u; }
    }
    // gave up: no result for row t and the block's later ones
    for (; t < T; t += step) {
        put_nan_row<T_, VEC>(y, j, lanes, n);
        if (j == 0 && mean_out) mean_out[t] = rstd_out[t] = NAN;
        y += y_step;
    }
    pdl_launch_dependents();
}

// A row of dy and x in flight.
template <typename Raw, int V>
struct NormRow {
    Raw dy[V], x[V];
    float mean, rstd;
};

// Rows of up to kRingMin columns: four warps a row at most, two rows or more a
// block, and kAhead of each group's rows in flight beyond the current one, in
// registers.  Bound by the loads in flight and, a row, the two reductions'
// latency.  FULL: the threads' columns are the row's, no guards.  Columns past
// the row's end have dy = 0 and so add nothing to any sum.
constexpr int kAhead = 2;
template <typename T_, int VEC, bool FULL>
__global__ void __launch_bounds__(kNormThreads)
    norm_rows_backward_kernel(int T, int H, int W, const typename RowVec<T_, VEC>::Raw* dy, int64_t dy_stride,
                              const typename RowVec<T_, VEC>::Raw* x, int64_t x_stride, const float* gamma,
                              const float* mean, const float* rstd, typename RowVec<T_, VEC>::Raw* dx,
                              int64_t dx_stride, float* part, bool wide_params) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    constexpr int V = kCols / VEC, D = kAhead;
    __shared__ float2 s_red[2][32];
    extern __shared__ float2 s_dyn[];        // [G][2][W * 128] sums
    pdl_wait();
    const int lanes = W * 32, j = threadIdx.x % lanes, G = blockDim.x / lanes, g = threadIdx.x / lanes;
    const int n = H / VEC;
    const int64_t step = (int64_t)gridDim.x * G;
    float2 ga[kPairs], dg[kPairs], db[kPairs];
    load_params<VEC, kCols>(gamma, j, lanes, n, wide_params, ga);
#pragma unroll
    for (int q = 0; q < kPairs; ++q) dg[q] = db[q] = both(0.0f);
    const int64_t first = (int64_t)blockIdx.x * G + g;
    dy += first * dy_stride + j;
    x += first * x_stride + j;
    dx += first * dx_stride + j;
    const int64_t dy_step = step * dy_stride, x_step = step * x_stride, dx_step = step * dx_stride;
    auto load = [&](int64_t t) {             // the next row in turn
        NormRow<Raw, V> r;
        const bool live = t < T;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool there = live && (FULL || j + i * lanes < n);
            r.dy[i] = there ? dy[i * lanes] : Raw{};
            r.x[i] = there ? x[i * lanes] : Raw{};
        }
        r.mean = live ? mean[t] : 0.0f;
        r.rstd = live ? rstd[t] : 0.0f;
        dy += dy_step;
        x += x_step;
        return r;
    };
    NormRow<Raw, V> ahead[D];
#pragma unroll
    for (int q = 0; q < D; ++q) ahead[q] = load(first + q * step);
    const float inv = 1.0f / (float)H;
    int turn = 0;
    for (int64_t tb = first; tb - g < T; tb += D * step) {   // uniform over the block
        // unrolled over the D buffers: a buffer moved to another register
        // would wait for its load
#pragma unroll
        for (int u = 0; u < D; ++u) {
            const int64_t t = tb + u * step;
            if (t - g >= T) break;
            const float2 m = both(-ahead[u].mean), r = both(ahead[u].rstd);
            float2 d[kPairs], hat[kPairs];
            unpack_cols<T_, VEC, kCols>(ahead[u].dy, d);
            unpack_cols<T_, VEC, kCols>(ahead[u].x, hat);
            ahead[u] = load(t + D * step);
            float2 sg = both(0.0f), sgx = both(0.0f);
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                hat[q] = mul2(add2(hat[q], m), r);
                dg[q] = fma2(d[q], hat[q], dg[q]);
                db[q] = add2(db[q], d[q]);
                d[q] = mul2(d[q], ga[q]);
                sg = add2(sg, d[q]);
                sgx = fma2(d[q], hat[q], sgx);
            }
            const float2 s = row_sum2(sg.x + sg.y, sgx.x + sgx.y, W, turn, s_red);
            turn ^= 1;
            if (t < T) {
                const float2 a = both(-(s.x * inv)), b = both(-(s.y * inv));
#pragma unroll
                for (int q = 0; q < kPairs; ++q) d[q] = mul2(fma2(hat[q], b, add2(d[q], a)), r);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (FULL || j + i * lanes < n) dx[i * lanes] = pack_cols<T_, VEC, kCols>(d, i);
            }
            dx += dx_step;
        }
    }
    // this block's sums: its rows' groups in order.  Column of pair q's first
    // element: eight columns in V vectors
    float* out = part + (size_t)blockIdx.x * 2 * H;
    float* sums = reinterpret_cast<float*>(s_dyn);
    const int cols = lanes * kCols;
#pragma unroll
    for (int q = 0; q < kCols; ++q) {
        const int h = (j + q / VEC * lanes) * VEC + q % VEC;
        sums[(g * 2) * cols + h] = q & 1 ? dg[q >> 1].y : dg[q >> 1].x;
        sums[(g * 2 + 1) * cols + h] = q & 1 ? db[q >> 1].y : db[q >> 1].x;
    }
    __syncthreads();
    for (int h = threadIdx.x; h < H; h += blockDim.x) {
        float a = 0.0f, b = 0.0f;
        for (int q = 0; q < G; ++q) {
            a += sums[(q * 2) * cols + h];
            b += sums[(q * 2 + 1) * cols + h];
        }
        out[h] = a;
        out[H + h] = b;
    }
    pdl_launch_dependents();
}

// The same for rows of more than kRingMin columns: sixteen
// columns a thread, 512 threads an SM (one block of 512 or up to four of 128).  The rows ahead
// wait in shared memory (the copy engine's bulk copies, a ring of S rows of dy
// and x) instead of registers, which the column sums and the row at hand fill.
// A stage is free once the row's reduction has passed its barrier: every
// thread has read its columns by then.  The wait for a copy is bounded (1 s);
// a block that gave up stops at the barrier, all its threads together, and
// leaves NaN where its results belong.
template <typename T_, int VEC>
__global__ void __launch_bounds__(512, 1)
    norm_ring_backward_kernel(int T, int H, int S, const typename RowVec<T_, VEC>::Raw* dy, int64_t dy_stride,
                              const typename RowVec<T_, VEC>::Raw* x, int64_t x_stride, const float* gamma,
                              const float* mean, const float* rstd, typename RowVec<T_, VEC>::Raw* dx,
                              int64_t dx_stride, float* part, bool wide_params, int skip_row) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    constexpr int C = kRingCols, V = C / VEC, P = C / 2;
    constexpr bool kWhole = sizeof(Raw) == 16;
    using Row = RingRow<T_, kWhole>;
    __shared__ float2 s_red[2][16];
    __shared__ uint64_t s_full[kRingMax];
    extern __shared__ __align__(16) uint8_t s_ring[];      // gamma [P][threads] float2, then [S][dy, x][n] vectors
    pdl_wait();
    const int lanes = blockDim.x, j = threadIdx.x, lane = j & 31, warp = j >> 5, W = lanes >> 5;
    const int n = H / VEC;
    float2* s_gamma = reinterpret_cast<float2*>(s_ring);
    uint8_t* s_rows = s_ring + (size_t)lanes * C * 4;
    const uint32_t row_bytes = (uint32_t)n * (uint32_t)sizeof(Raw), slot = Row::slot(row_bytes);
    const int64_t step = gridDim.x, first = blockIdx.x;
    uint64_t policy = 0;
    auto fetch = [&](int64_t t, int stage) {               // thread 0
        if (t == skip_row) return;
        uint8_t* to = s_rows + stage * 2 * slot;
        const Raw *row_d = dy + t * dy_stride, *row_x = x + t * x_stride;
        mbar_arrive_expect_tx(&s_full[stage], Row::copied(row_d, row_bytes) + Row::copied(row_x, row_bytes));
        Row::copy(to, row_d, row_bytes, &s_full[stage], policy);
        Row::copy(to + slot, row_x, row_bytes, &s_full[stage], policy);
    };
    Row edge;
    auto load_edge = [&](int64_t t, int stage) {           // the first 32 threads
        const Raw* row = j < 16 ? dy + t * dy_stride : x + t * x_stride;
        edge.load(s_rows + (stage * 2 + (j >> 4)) * slot, row, row_bytes, j & 15);
    };
    if (j == 0) {
        policy = policy_evict_first();                     // dy and x are read once
        for (int q = 0; q < S; ++q) mbar_init(&s_full[q], 1);
        fence_mbar_init();
        for (int q = 0; q < S; ++q)
            if (first + q * step < T) fetch(first + q * step, q);
    }
    if (!kWhole && j < 32)
        for (int q = 0; q < S; ++q)
            if (first + q * step < T) {
                load_edge(first + q * step, q);
                edge.store();
            }
    float2 dg[P], db[P];
    {
        float2 ga[P];
        load_params<VEC, C>(gamma, j, lanes, n, wide_params, ga);
#pragma unroll
        for (int q = 0; q < P; ++q) {
            s_gamma[q * lanes + j] = ga[q];                // read by this thread alone
            dg[q] = db[q] = both(0.0f);
        }
    }
    __syncthreads();
    const float inv = 1.0f / (float)H;
    int stage = 0, turn = 0;
    uint32_t parity = 0;
    float next_mean = first < T ? mean[first] : 0.0f, next_rstd = first < T ? rstd[first] : 0.0f;
    dx += first * dx_stride + j;
    const int64_t dx_step = step * dx_stride;
    volatile int never = 0;
    int64_t t = first;
    for (; t < T; t += step) {
        const float2 m = both(-next_mean), r = both(next_rstd);
        if (t + step < T) {
            next_mean = mean[t + step];
            next_rstd = rstd[t + step];
        }
        const bool landed = mbar_wait(&s_full[stage], parity, &never, nullptr, 0);
        float2 d[P], hat[P];
        {
            const uint8_t* at = s_rows + stage * 2 * slot;
            const Raw* at_d = reinterpret_cast<const Raw*>(at + Row::offset(dy + t * dy_stride)) + j;
            const Raw* at_x = reinterpret_cast<const Raw*>(at + slot + Row::offset(x + t * x_stride)) + j;
            Raw rd[V], rx[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool there = j + v * lanes < n;
                rd[v] = there ? at_d[v * lanes] : Raw{};
                rx[v] = there ? at_x[v * lanes] : Raw{};
            }
            unpack_cols<T_, VEC, C>(rd, d);
            unpack_cols<T_, VEC, C>(rx, hat);
        }
        float2 sg = both(0.0f), sgx = both(0.0f);
#pragma unroll
        for (int q = 0; q < P; ++q) {
            hat[q] = mul2(add2(hat[q], m), r);
            dg[q] = fma2(d[q], hat[q], dg[q]);
            db[q] = add2(db[q], d[q]);
            d[q] = mul2(d[q], s_gamma[q * lanes + j]);
            sg = add2(sg, d[q]);
            sgx = fma2(d[q], hat[q], sgx);
        }
        const float wa = warp_sum(sg.x + sg.y), wb = warp_sum(sgx.x + sgx.y);
        if (lane == 0) s_red[turn][warp] = make_float2(wa, wb);
        if (!kWhole) edge.store();
        if (__syncthreads_or(!landed)) {
            for (int i = 0; i < 100; ++i) __nanosleep(10000);   // copies in flight land before the block leaves
            break;
        }
        if (t + S * step < T) {
            if (j == 0) fetch(t + S * step, stage);
            if (!kWhole && j < 32) load_edge(t + S * step, stage);
        }
        const float2 w = lane < W ? s_red[turn][lane & 15] : both(0.0f);
        const float2 a = both(-(warp_sum(w.x) * inv)), b = both(-(warp_sum(w.y) * inv));
#pragma unroll
        for (int q = 0; q < P; ++q) d[q] = mul2(fma2(hat[q], b, add2(d[q], a)), r);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (j + v * lanes < n) dx[v * lanes] = pack_cols<T_, VEC, C>(d, v);
        turn ^= 1;
        dx += dx_step;
        if (++stage == S) { stage = 0; parity ^= 1u; }
    }
    if (t < T) {      // gave up: no result for row t and the block's later ones, nor for the column sums
#pragma unroll
        for (int q = 0; q < P; ++q) dg[q] = db[q] = both(NAN);
        for (; t < T; t += step, dx += dx_step) put_nan_row<T_, VEC>(dx, j, lanes, n);
    }
    float* out = part + (size_t)blockIdx.x * 2 * H;
    if constexpr (VEC % 4 == 0) {
        // 16-byte stores: H is a multiple of VEC, part 256-byte aligned
#pragma unroll
        for (int q = 0; q < P; q += 2) {
            const int v = j + 2 * q / VEC * lanes, h = v * VEC + 2 * q % VEC;
            if (v < n) {
                *reinterpret_cast<float4*>(out + h) = make_float4(dg[q].x, dg[q].y, dg[q + 1].x, dg[q + 1].y);
                *reinterpret_cast<float4*>(out + H + h) = make_float4(db[q].x, db[q].y, db[q + 1].x, db[q + 1].y);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < C; ++q) {
            const int v = j + q / VEC * lanes, h = v * VEC + q % VEC;
            if (v < n) {
                out[h] = q & 1 ? dg[q >> 1].y : dg[q >> 1].x;
                out[H + h] = q & 1 ? db[q >> 1].y : db[q >> 1].x;
            }
        }
    }
    pdl_launch_dependents();
}

// dgamma and dbeta from `parts` partial sums [parts][2][H]: 32 VEC columns a
// block, a 32nd of the parts a warp, then the warps' sums in order.
template <int VEC, int UNROLL>
__global__ void __launch_bounds__(1024) norm_reduce_kernel(int H, int parts, const float* part, float* dgamma,
                                                                   float* dbeta) {
    using RV = RowVec<float, VEC>;
    constexpr int kWarps = 32;
    __shared__ float s[kWarps][32 * VEC];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = H / VEC, c = blockIdx.x * 32 + lane;
    float v[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = 0.0f;
    if (c < n) {
        const typename RV::Raw* p = reinterpret_cast<const typename RV::Raw*>(part) + (blockIdx.y ? n : 0) + c;
#pragma unroll UNROLL
        for (int q = warp; q < parts; q += kWarps) {
            float u[VEC];
            RV::unpack(p[(size_t)q * 2 * n], u);
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] += u[k];
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[warp][lane * VEC + k] = v[k];
    __syncthreads();
    const int h = blockIdx.x * 32 * VEC + (int)threadIdx.x;
    if (threadIdx.x < 32 * VEC && h < H) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s[w][threadIdx.x];
        (blockIdx.y ? dbeta : dgamma)[h] = sum;
    }
    pdl_launch_dependents();
}

cudaError_t launch_reduce(const LaunchCtx& c, int H, int parts, const float* part, float* dgamma, float* dbeta) {
    // short rows: more blocks and more loads in flight (5453 rows of 1624,
    // backward, us for vectors of 4, 2 and 1: 19.0 17.8 17.1; 8191 of 7168: 67.4
    // 67.1 69.5)
    const int wide = H % 2 == 0 && H > 2048 ? 2 : 1;
    const dim3 grid((unsigned)((H / wide + 31) / 32), dbeta ? 2 : 1);
    return c.launch(wide == 2 ? norm_reduce_kernel<2, 4> : norm_reduce_kernel<1, 8>, grid, dim3(1024), 0, H, parts,
                    part, dgamma, dbeta);
}

// ---- rows of more than kRowColumns columns -------------------------------------

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

// Resident blocks of the ring kernel on an SM (its shared memory leaves two
// stages to each: the longest FP32 rows of a share take 16 KB of gamma and 64
// KB a stage, or a quarter of it).
int ring_blocks(int H) {
    const int share = (H + 32 * kRingCols - 1) / (32 * kRingCols);   // warps, of 16
    return share <= 4 ? 4 : share <= 8 ? 2 : 1;
}

template <typename T_, int VEC>
cudaError_t forward_any(const LaunchCtx& c, int T, int H, const void* x, int64_t x_stride, const float* gamma,
                        const float* beta, float eps, void* y, int64_t y_stride, float* mean, float* rstd,
                        int skip_row) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    const Raw* xv = static_cast<const Raw*>(x);
    Raw* yv = static_cast<Raw*>(y);
    if (H > kRowColumns)
        return c.launch(layer_norm_kernel<T_, VEC>, dim3(T), dim3(kNormThreads), 0, H, xv, x_stride / VEC, gamma, beta,
                        eps, yv, y_stride / VEC, mean, rstd);
    const bool wide_params = (row_at(gamma) | row_at(beta)) % 16 == 0;
    constexpr bool kWhole = sizeof(Raw) == 16;
    if (H > (kWhole ? kRingMin : kRingMinOdd) && T > 4 * kNormSms) {
        const int threads = (H + 32 * kRingCols - 1) / (32 * kRingCols) * 32;
        const int held = threads * kRingCols * 8, row = (int)RingRow<T_, kWhole>::slot(H * sizeof(T_));
        int per_sm = threads <= 64 ? 12 : ring_blocks(H) < 2 ? 2 : ring_blocks(H);
        if (kRingBytes / per_sm < held + 2 * row) per_sm = 1;
        const int fit = (kRingBytes / per_sm - held) / row;
        const int S = fit > kRingMax ? kRingMax : fit;
        return c.launch(norm_ring_kernel<T_, VEC>, dim3(per_sm * kNormSms), dim3(threads),
                        (size_t)held + (size_t)S * row, T, H, S, xv, x_stride / VEC, gamma, beta, eps, yv,
                        y_stride / VEC, mean, rstd, wide_params, skip_row);
    }
    // long rows, enough of them to fill the SMs: 32 columns a thread, so that
    // several rows share an SM and overlap their loads with their reductions
    const bool many = H > 32 * 8 * kCols && T > 152;
    const NormShape s = norm_shape(H, many ? 32 : kCols);
    const dim3 grid((unsigned)((T + s.G - 1) / s.G)), block(s.threads());
    auto kernel = many                 ? norm_rows_kernel<T_, VEC, 32, 256>
                  : s.threads() <= 256 ? norm_rows_kernel<T_, VEC, kCols, 256>
                                       : norm_rows_kernel<T_, VEC, kCols, 1024>;
    return c.launch(kernel, grid, block, 0, T, H, s.W, xv, x_stride / VEC, gamma, beta, eps, yv, y_stride / VEC, mean,
                    rstd, wide_params);
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

// Blocks of a persistent backward kernel with `rows` rows at a time: the
// resident ones, or as many as there are rows for.
int backward_blocks(int T, int rows, int resident) {
    const int64_t most = ((int64_t)T + rows - 1) / rows;
    return (int)(most < 1 ? 1 : most < resident ? most : resident);
}

template <typename T_, int VEC>
cudaError_t backward_rows_any(const LaunchCtx& c, int T, int H, const void* dy, int64_t dy_stride, const void* x,
                              int64_t x_stride, const float* gamma, const float* mean, const float* rstd, void* dx,
                              int64_t dx_stride, float* part, int* blocks, int skip_row) {
    using Raw = typename RowVec<T_, VEC>::Raw;
    const bool wide_params = row_at(gamma) % 16 == 0;
    const NormShape s = norm_shape(H);
    if (H > kRingMin) {
        const int threads = (H + 32 * kRingCols - 1) / (32 * kRingCols) * 32;
        const int per_sm = ring_blocks(H);
        const int held = threads * kRingCols * 4;
        const int stage = 2 * (int)RingRow<T_, sizeof(Raw) == 16>::slot(H * sizeof(T_));
        const int fit = (kRingBytes / per_sm - held) / stage;
        const int S = fit > kRingMax ? kRingMax : fit;
        *blocks = backward_blocks(T, 1, per_sm * kNormSms);
        return c.launch(norm_ring_backward_kernel<T_, VEC>, dim3(*blocks), dim3(threads),
                        (size_t)held + (size_t)S * stage, T, H, S, static_cast<const Raw*>(dy), dy_stride / VEC,
                        static_cast<const Raw*>(x), x_stride / VEC, gamma, mean, rstd, static_cast<Raw*>(dx),
                        dx_stride / VEC, part, wide_params, skip_row);
    }
    const bool full = s.W * 32 * kCols == H;
    auto kernel = full ? norm_rows_backward_kernel<T_, VEC, true> : norm_rows_backward_kernel<T_, VEC, false>;
    const size_t smem = (size_t)s.G * 2 * s.W * 32 * kCols * 4;
    *blocks = backward_blocks(T, s.G, 2 * kNormSms);
    return c.launch(kernel, dim3(*blocks), dim3(s.threads()), smem, T, H, s.W, static_cast<const Raw*>(dy),
                    dy_stride / VEC, static_cast<const Raw*>(x), x_stride / VEC, gamma, mean, rstd,
                    static_cast<Raw*>(dx), dx_stride / VEC, part, wide_params);
}

}  // namespace

cudaError_t launch_layer_norm(const LaunchCtx& c, int T, int H, int elem, const void* x, int64_t x_stride,
                              const float* gamma, const float* beta, float eps, void* y, int64_t y_stride, float* mean,
                              float* rstd, int skip_row) {
    const int bytes = row_vec_bytes(H, elem, row_at(x, x_stride, elem) | row_at(y, y_stride, elem));
    MOE_ROW_VEC(elem, bytes, forward_any, c, T, H, x, x_stride, gamma, beta, eps, y, y_stride, mean, rstd, skip_row);
}

cudaError_t setup_layer_norm_kernels() {
    static_assert(512 * kRingCols * 8 + 2 * (kRowColumns * 4 + 32) <= kRingBytes &&
                      512 * kRingCols * 4 + 2 * 2 * (kRowColumns * 4 + 32) <= kRingBytes,
                  "two stages of the longest rows");
    cudaError_t e = cudaSuccess;
    auto allow = [&](auto kernel) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    };
    allow(norm_ring_kernel<__nv_bfloat16, 8>);
    allow(norm_ring_kernel<__nv_bfloat16, 4>);
    allow(norm_ring_kernel<__nv_bfloat16, 2>);
    allow(norm_ring_kernel<__nv_bfloat16, 1>);
    allow(norm_ring_kernel<float, 4>);
    allow(norm_ring_kernel<float, 2>);
    allow(norm_ring_kernel<float, 1>);
    allow(norm_ring_backward_kernel<__nv_bfloat16, 8>);
    allow(norm_ring_backward_kernel<__nv_bfloat16, 4>);
    allow(norm_ring_backward_kernel<__nv_bfloat16, 2>);
    allow(norm_ring_backward_kernel<__nv_bfloat16, 1>);
    allow(norm_ring_backward_kernel<float, 4>);
    allow(norm_ring_backward_kernel<float, 2>);
    allow(norm_ring_backward_kernel<float, 1>);
    return e;
}

size_t layer_norm_workspace_bytes(int T, int H) {
    // a block has a row at least
    const int most = H > kRowColumns ? kNormParts : H > kRingMin && H <= 2048 ? 4 * kNormSms : 2 * kNormSms;
    return align_up((uint64_t)(H > kRowColumns || T > most ? most : T < 1 ? 1 : T) * 2 * H * 4, 256);
}

static cudaError_t launch_dx(const LaunchCtx& c, int bytes, int T, int H, int elem, const void* dy, int64_t dy_stride,
                             const void* x, int64_t x_stride, const float* gamma, const float* mean, const float* rstd,
                             void* dx, int64_t dx_stride) {
    MOE_ROW_VEC(elem, bytes, dx_any, c, T, H, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx, dx_stride);
}

static cudaError_t launch_backward_rows(const LaunchCtx& c, int bytes, int T, int H, int elem, const void* dy,
                                        int64_t dy_stride, const void* x, int64_t x_stride, const float* gamma,
                                        const float* mean, const float* rstd, void* dx, int64_t dx_stride,
                                        float* part, int* blocks, int skip_row) {
    MOE_ROW_VEC(elem, bytes, backward_rows_any, c, T, H, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx, dx_stride,
                part, blocks, skip_row);
}

cudaError_t launch_layer_norm_backward(const LaunchCtx& c, int T, int H, int elem, const void* dy, int64_t dy_stride,
                                       const void* x, int64_t x_stride, const float* gamma, const float* mean,
                                       const float* rstd, void* dx, int64_t dx_stride, float* dgamma, float* dbeta,
                                       float* workspace, int skip_row) {
    const int bytes = row_vec_bytes(
        H, elem, row_at(x, x_stride, elem) | row_at(dy, dy_stride, elem) | row_at(dx, dx_stride, elem));
    cudaError_t e;
    if (H <= kRowColumns) {
        int blocks = 0;
        e = launch_backward_rows(c, bytes, T, H, elem, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx, dx_stride,
                                 workspace, &blocks, skip_row);
        if (e != cudaSuccess) return e;
        return launch_reduce(c, H, blocks, workspace, dgamma, dbeta);
    }
    // the column sums first: dx may overwrite dy or x
    const dim3 parts((unsigned)((H + kNormThreads - 1) / kNormThreads), kNormParts);
    if (elem == 2)
        e = c.launch(layer_norm_partial_kernel<__nv_bfloat16>, parts, dim3(kNormThreads), 0, T, H,
                     static_cast<const uint16_t*>(dy), dy_stride, static_cast<const uint16_t*>(x), x_stride, mean,
                     rstd, workspace);
    else
        e = c.launch(layer_norm_partial_kernel<float>, parts, dim3(kNormThreads), 0, T, H,
                     static_cast<const uint32_t*>(dy), dy_stride, static_cast<const uint32_t*>(x), x_stride, mean,
                     rstd, workspace);
    if (e != cudaSuccess) return e;
    e = launch_reduce(c, H, kNormParts, workspace, dgamma, dbeta);
    if (e != cudaSuccess || T == 0) return e;
    return launch_dx(c, bytes, T, H, elem, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx, dx_stride);
}

}  // namespace moe
