// Global norm of a list of gradients, and the list scaled down to a largest
// norm.
//
//   norm = sqrt(sum_i sum_j g_ij^2)
//   out_ij = g_ij s,  s = min(1, max_norm / (norm + eps)), NaN if it is one
//
// The list travels as a kernel argument (pointers, sizes, types), a launch per
// 960 tensors: nothing is copied to the device beforehand, and a captured graph
// replays it.  Shorter lists take a smaller argument.  Tensors are cut into
// chunks of kChunkMost elements, or of fewer where the whole list fits one round
// of the blocks, that the blocks take in turn; the argument names the entry of
// each block's first chunk, so that a short call does not wait for a search of
// cold constants (249 tensors, 5 million BF16: norm and scaling 16.6 -> 7.8 us).
// HBM is the bound: one read for the norm, one read and one write for the
// scaling.  Measured on GB300 (302 million BF16 in 131 tensors): norm 93 us (6.5
// TB/s), scaling 182 (6.6); 0.77 million FP32 in 19 tensors 3.3 and 2.3.
#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kClipThreads = 512;
constexpr int kListMax = 960;         // tensors of a launch: 30 KB of its 32 KB of arguments
constexpr int kChunkMost = 16384;     // elements: a thread's kInFlight loads of BF16
constexpr int kChunkLeast = 4096;
constexpr int kChunkStep = 2048;
constexpr int kInFlight = 4;          // 16-byte loads of a thread
// Partial sums per launch, four blocks on each of 152 SMs: a constant, as the
// workspace's size is asked for without a device and the sums' order follows it
constexpr int kNormBlocks = 608;

struct GradEntry {
    const void* in;
    void* out;
    int64_t numel;
    int32_t last_chunk;   // one past this tensor's last chunk in the launch
    int32_t elem;         // bytes of an element
};
template <int MAX>
struct GradTable {
    static constexpr bool kStart = MAX > 32;
    int n;
    int chunks;
    int chunk;            // elements of a chunk
    // entry of a block's first chunk (a short list is searched: five steps)
    uint16_t start[kStart ? kNormBlocks : 1];
    GradEntry e[MAX];
};

// A chunk [at, at + count) of a tensor as vectors of VEC, kInFlight of them
// loaded by a thread before the first is used; f(vector's values, its index),
// then f1(element's index) for the elements past the last vector.
template <typename T_, int VEC, typename F, typename F1>
__device__ __forceinline__ void for_chunk(const void* base, int64_t at, int count, F f, F1 f1) {
    using RV = RowVec<T_, VEC>;
    const typename RV::Raw* p = reinterpret_cast<const typename RV::Raw*>(static_cast<const T_*>(base) + at);
    const int n = count / VEC;
    for (int i0 = threadIdx.x; i0 < n; i0 += kClipThreads * kInFlight) {
        typename RV::Raw r[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (i0 + u * kClipThreads < n) r[u] = p[i0 + u * kClipThreads];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (i0 + u * kClipThreads < n) {
                float v[VEC];
                RV::unpack(r[u], v);
                f(v, i0 + u * kClipThreads);
            }
    }
    if ((int)threadIdx.x < count - n * VEC) f1(n * VEC + (int)threadIdx.x);
}

// Sum of squares of a chunk's part of this thread.
template <typename T_, int VEC>
__device__ __forceinline__ float square_part(const void* base, int64_t at, int count) {
    float s = 0.0f;
    for_chunk<T_, VEC>(
        base, at, count,
        [&](const float (&v)[VEC], int) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) s = fmaf(v[j], v[j], s);
        },
        [&](int i) {
            const float v = (float)static_cast<const T_*>(base)[at + i];
            s = fmaf(v, v, s);
        });
    return s;
}

// `in` and `out` may be the same tensor: a thread writes what it has read.
template <typename T_, int VEC>
__device__ __forceinline__ void scale_part(const void* in, void* out, int64_t at, int count, float scale) {
    using RV = RowVec<T_, VEC>;
    typename RV::Raw* q = reinterpret_cast<typename RV::Raw*>(static_cast<T_*>(out) + at);
    for_chunk<T_, VEC>(
        in, at, count,
        [&](const float (&v)[VEC], int i) {
            float w[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[j] = v[j] * scale;
            q[i] = RV::pack(w);
        },
        [&](int i) { static_cast<T_*>(out)[at + i] = (T_)((float)static_cast<const T_*>(in)[at + i] * scale); });
}

// First chunk of entry i.
template <int MAX>
__device__ __forceinline__ int first_chunk(const GradTable<MAX>& t, int i) {
    return i ? t.e[i - 1].last_chunk : 0;
}

// The entry of chunk c, which lies in entries lo..hi.
template <int MAX>
__device__ __forceinline__ int entry_of(const GradTable<MAX>& t, int c, int lo, int hi) {
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (c < t.e[mid].last_chunk) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// The entry of this block's first chunk c.
template <int MAX>
__device__ __forceinline__ int first_entry(const GradTable<MAX>& t, int c) {
    if (GradTable<MAX>::kStart && blockIdx.x < kNormBlocks) return t.start[blockIdx.x];
    return c < t.e[0].last_chunk ? 0 : entry_of(t, c, 1, t.n - 1);
}

template <int MAX>
__global__ void __launch_bounds__(kClipThreads) grad_square_kernel(const __grid_constant__ GradTable<MAX> t,
                                                                   float* part) {
    __shared__ float s_part[kClipThreads / 32];
    int i = first_entry(t, blockIdx.x);
    pdl_wait();
    float sum = 0.0f;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        if (c >= t.e[i].last_chunk) i = entry_of(t, c, i + 1, t.n - 1);
        const GradEntry& e = t.e[i];
        const int64_t at = (int64_t)(c - first_chunk(t, i)) * t.chunk;
        const int count = (int)min((int64_t)t.chunk, e.numel - at);
        const bool wide = reinterpret_cast<uintptr_t>(e.in) % 16 == 0;
        if (e.elem == 2)
            sum += wide ? square_part<__nv_bfloat16, 8>(e.in, at, count) : square_part<__nv_bfloat16, 1>(e.in, at, count);
        else
            sum += wide ? square_part<float, 4>(e.in, at, count) : square_part<float, 1>(e.in, at, count);
    }
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        const float v = warp_sum(threadIdx.x < kClipThreads / 32 ? s_part[threadIdx.x] : 0.0f);
        if (threadIdx.x == 0) part[blockIdx.x] = v;
    }
    pdl_launch_dependents();
}

__global__ void __launch_bounds__(1024) grad_norm_kernel(int n, const float* part, float* norm) {
    __shared__ float s_part[32];
    pdl_wait();
    float s = 0.0f;
    for (int i = threadIdx.x; i < n; i += 1024) s += part[i];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = warp_sum(s_part[threadIdx.x]);
        if (threadIdx.x == 0) norm[0] = sqrtf(s);
    }
    pdl_launch_dependents();
}

template <int MAX>
__global__ void __launch_bounds__(kClipThreads) grad_scale_kernel(const __grid_constant__ GradTable<MAX> t,
                                                                  const float* norm, float max_norm, float eps) {
    // from the list's end: what the norm's pass has read last may still be in L2
    int i = first_entry(t, t.chunks - 1 - (int)blockIdx.x);
    pdl_wait();
    const float q = max_norm / (norm[0] + eps);
    const float scale = q > 1.0f ? 1.0f : q;      // NaN stays NaN
    for (int c = t.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        if (c < first_chunk(t, i)) i = entry_of(t, c, 0, i - 1);
        const GradEntry& e = t.e[i];
        if (scale == 1.0f && e.in == e.out) continue;
        const int64_t at = (int64_t)(c - first_chunk(t, i)) * t.chunk;
        const int count = (int)min((int64_t)t.chunk, e.numel - at);
        const bool wide = (reinterpret_cast<uintptr_t>(e.in) | reinterpret_cast<uintptr_t>(e.out)) % 16 == 0;
        if (e.elem == 2) {
            if (wide) scale_part<__nv_bfloat16, 8>(e.in, e.out, at, count, scale);
            else scale_part<__nv_bfloat16, 1>(e.in, e.out, at, count, scale);
        } else {
            if (wide) scale_part<float, 4>(e.in, e.out, at, count, scale);
            else scale_part<float, 1>(e.in, e.out, at, count, scale);
        }
    }
}

// Launches a kernel on a table without copying it on the way.
template <typename... KArgs>
cudaError_t launch_table(const LaunchCtx& c, void (*kernel)(KArgs...), int blocks, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kClipThreads);
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = c.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args);
}

// Calls f(table) for every launch's share of the list: at most MAX tensors and
// 2^30 chunks; tensors without elements are left out.  `backward`: the blocks
// take the chunks from the last one on.
template <int MAX, typename F>
cudaError_t for_tables_of(int n, const void* const* in, void* const* out, const int64_t* numels, const int32_t* dtypes,
                          bool backward, F f) {
    GradTable<MAX> t;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) total += numels[i];
    // a chunk for every block, in one round: total / chunk + n chunks at most
    const int64_t share = total / (n < kNormBlocks / 2 ? kNormBlocks - n : kNormBlocks / 2);
    // (0.77 million FP32 elements: chunks of 4096 6.0 us, of 16384 6.9, of 2048 7.7)
    t.chunk = share >= kChunkMost    ? kChunkMost
              : share <= kChunkLeast ? kChunkLeast
                                     : (int)((share + kChunkStep) / kChunkStep * kChunkStep);
    int64_t chunks = 0;
    t.n = 0;
    auto flush = [&]() {
        if (t.n == 0) return cudaSuccess;
        t.chunks = (int)chunks;
        if constexpr (GradTable<MAX>::kStart) {
            const int blocks = chunks < kNormBlocks ? (int)chunks : kNormBlocks;
            for (int b = 0, k = backward ? t.n - 1 : 0; b < blocks; ++b) {
                while (backward && k > 0 && chunks - 1 - b < t.e[k - 1].last_chunk) --k;
                while (!backward && b >= t.e[k].last_chunk) ++k;
                t.start[b] = (uint16_t)k;
            }
        }
        const cudaError_t e = f(t);
        t.n = 0;
        chunks = 0;
        return e;
    };
    for (int i = 0; i < n; ++i) {
        if (numels[i] == 0) continue;
        const int64_t c = (numels[i] + t.chunk - 1) / t.chunk;
        if (t.n == MAX || chunks + c > (1 << 30)) {
            const cudaError_t e = flush();
            if (e != cudaSuccess) return e;
        }
        chunks += c;
        t.e[t.n++] = GradEntry{in[i], out ? out[i] : nullptr, numels[i], (int32_t)chunks,
                               dtypes[i] == MOE_DTYPE_F32 ? 4 : 2};
    }
    return flush();
}

// With the smallest table that holds the list.
template <typename F>
cudaError_t for_tables(int n, const void* const* in, void* const* out, const int64_t* numels, const int32_t* dtypes,
                       bool backward, F f) {
    if (n <= 32) return for_tables_of<32>(n, in, out, numels, dtypes, backward, f);
    if (n <= 160) return for_tables_of<160>(n, in, out, numels, dtypes, backward, f);
    return for_tables_of<kListMax>(n, in, out, numels, dtypes, backward, f);
}

}  // namespace

// Partial sums of every launch: a launch takes kListMax tensors, or fewer if
// they fill its 2^30 chunks (sixteen tensors of the largest size do).
size_t grad_norm_workspace_bytes(int n) {
    const uint64_t launches = (uint64_t)n / kListMax + (uint64_t)n / 16 + 2;
    return align_up(launches * kNormBlocks * 4, 256);
}

cudaError_t launch_grad_norm(const LaunchCtx& c, int n, const void* const* grads, const int64_t* numels,
                             const int32_t* dtypes, float* norm, float* workspace) {
    int used = 0;
    cudaError_t e = for_tables(n, grads, nullptr, numels, dtypes, false, [&](auto& t) {
        const int blocks = t.chunks < kNormBlocks ? t.chunks : kNormBlocks;
        float* part = workspace + used;
        used += blocks;
        void* args[] = {&t, &part};
        return launch_table(c, grad_square_kernel<sizeof(t.e) / sizeof(GradEntry)>, blocks, args);
    });
    if (e != cudaSuccess) return e;
    return c.launch(grad_norm_kernel, dim3(1), dim3(1024), 0, used, (const float*)workspace, norm);
}

cudaError_t launch_grad_clip(const LaunchCtx& c, int sms, int n, const void* const* grads, void* const* out,
                             const int64_t* numels, const int32_t* dtypes, const float* norm, float max_norm,
                             float eps) {
    return for_tables(n, grads, out, numels, dtypes, true, [&](auto& t) {
        const int blocks = t.chunks < 8 * sms ? t.chunks : 8 * sms;
        void* args[] = {&t, &norm, &max_norm, &eps};
        return launch_table(c, grad_scale_kernel<sizeof(t.e) / sizeof(GradEntry)>, blocks, args);
    });
}

}  // namespace moe
