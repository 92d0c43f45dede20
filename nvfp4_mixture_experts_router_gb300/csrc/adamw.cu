// One AdamW step over a list of tensors.
//
//   g = clip grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// The list travels as a kernel argument, a launch per kAdamMax tensors of one
// kind of states; nothing is copied to the device beforehand, and a captured
// graph replays it.  A warp takes 256 consecutive elements, eight a lane: a
// block of the states in 8 bits, whose largest magnitude is one warp-wide
// maximum.  HBM is the bound: every buffer read and written once.
#include <math.h>

#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamMax = 384;           // tensors of a launch: 27.6 KB of its 32 KB of arguments
constexpr int kAdamBlocks = 152 * 8;
constexpr int kChunk = 8192;            // elements

struct AdamEntry {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    float* w;
    int64_t numel;
    int32_t last_chunk;     // one past this tensor's last chunk in the launch
    uint8_t p_bf16, g_bf16, wide, pad;
};
struct AdamNumbers {
    float b1, one_b1, b2, one_b2, eps, wd;
    float lr;               // the rest of this line: with lr on the host
    float keep, rate, root; // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    float log_b1, log_b2;   // for t on the device
    float max_norm, clip_eps;
};
template <int MAX>
struct AdamTable {
    int n;
    int chunks;
    AdamNumbers k;
    const float* norm;
    const float* lr_step;
    AdamEntry e[MAX];
};

__device__ __forceinline__ float sqrt_fast(float v) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// What a thread needs of the numbers.
struct AdamStep {
    float clip, b1, one_b1, b2, one_b2, eps, keep, rate, root;
};
__device__ __forceinline__ AdamStep step_of(const AdamNumbers& k, const float* norm, const float* lr_step) {
    AdamStep s{1.0f, k.b1, k.one_b1, k.b2, k.one_b2, k.eps, k.keep, k.rate, k.root};
    if (norm) {
        const float q = k.max_norm / (norm[0] + k.clip_eps);
        s.clip = q > 1.0f ? 1.0f : q;       // NaN stays NaN
    }
    if (lr_step) {
        const float lr = lr_step[0], t = lr_step[1];
        s.keep = 1.0f - lr * k.wd;
        s.rate = lr / -expm1f(t * k.log_b1);
        s.root = 1.0f / sqrtf(-expm1f(t * k.log_b2));
    }
    return s;
}

__device__ __forceinline__ void update(const AdamStep& s, float grad, float& m, float& v, float& p) {
    const float g = grad * s.clip;
    m = fmaf(s.b1, m, s.one_b1 * g);
    v = fmaf(s.b2, v, s.one_b2 * (g * g));
    p = fmaf(-s.rate, __fdividef(m, fmaf(sqrt_fast(v), s.root, s.eps)), p * s.keep);
}

// Eight elements of type T_ from p on, or the first `count` of them.
template <typename T_>
__device__ __forceinline__ void load8(const void* at, int64_t i, int count, bool wide, float (&v)[8]) {
    const T_* p = static_cast<const T_*>(at) + i;
    constexpr int VEC = 16 / sizeof(T_);
    if (wide && count == 8) {
#pragma unroll
        for (int k = 0; k < 8; k += VEC) {
            float u[VEC];
            RowVec<T_, VEC>::unpack(reinterpret_cast<const uint4*>(p)[k / VEC], u);
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[k + j] = u[j];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < count ? (float)p[k] : 0.0f;
    }
}
template <typename T_>
__device__ __forceinline__ void store8(void* at, int64_t i, int count, bool wide, const float (&v)[8]) {
    T_* p = static_cast<T_*>(at) + i;
    constexpr int VEC = 16 / sizeof(T_);
    if (wide && count == 8) {
#pragma unroll
        for (int k = 0; k < 8; k += VEC) {
            float u[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[j] = v[k + j];
            reinterpret_cast<uint4*>(p)[k / VEC] = RowVec<T_, VEC>::pack(u);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) p[k] = (T_)v[k];
    }
}

// Eight E4M3 bytes times a scale.
__device__ __forceinline__ void load_codes(const void* at, int64_t i, int count, bool wide, float scale, float (&v)[8]) {
    const uint8_t* p = static_cast<const uint8_t*>(at) + i;
    uint64_t w = 0;
    if (wide && count == 8) {
        w = *reinterpret_cast<const uint64_t*>(p);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) w |= (uint64_t)p[k] << (8 * k);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = e4m3_to_f32((uint32_t)(w >> (8 * k))) * scale;
}
// A warp's 256 values as E4M3 with a scale, which lane 0 stores.  ROOT: values
// that are not negative, of which none but zero becomes zero.
template <bool ROOT>
__device__ __forceinline__ void store_codes(void* at, float* scale_at, int64_t i, int count, bool wide,
                                            const float (&v)[8]) {
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) most = max(most, __float_as_uint(v[k]) & 0x7fffffffu);    // a NaN is above infinity
    const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, most));
    const bool flush = amax < 7.88860905e-31f;      // 2^-100
    const bool bad = !(amax < INFINITY);
    const float scale = flush ? 0.0f : bad ? NAN : amax / 448.0f;
    const float inv = flush ? 0.0f : 448.0f / amax;
    const float least = flush ? 0.0f : 0x1p-9f;
    uint64_t w = 0;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        float a = v[k] * inv, b = v[k + 1] * inv;
        if (ROOT) {
            a = v[k] > 0.0f ? fmaxf(a, least) : a;
            b = v[k + 1] > 0.0f ? fmaxf(b, least) : b;
        }
        w |= (uint64_t)f32x2_to_e4m3x2(a, b) << (8 * k);
    }
    uint8_t* p = static_cast<uint8_t*>(at) + i;
    if (wide && count == 8) {
        *reinterpret_cast<uint64_t*>(p) = w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) p[k] = (uint8_t)(w >> (8 * k));
    }
    if ((threadIdx.x & 31) == 0) *scale_at = scale;
}

template <int BITS, int MAX>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamTable<MAX> t) {
    pdl_wait();
    const AdamStep s = step_of(t.k, t.norm, t.lr_step);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int i = 0;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        while (c >= t.e[i].last_chunk) ++i;
        const AdamEntry& e = t.e[i];
        const int64_t first = (int64_t)(c - (i ? t.e[i - 1].last_chunk : 0)) * kChunk;
        const int64_t end = min(first + kChunk, e.numel);
        for (int64_t b = first + warp * 256; b < end; b += kAdamThreads * 8) {
            const int64_t at = b + lane * 8;
            const int count = (int)max((int64_t)0, min((int64_t)8, end - at));
            float p[8], g[8], m[8], v[8];
            if (e.w) load8<float>(e.w, at, count, e.wide, p);
            else if (e.p_bf16) load8<__nv_bfloat16>(e.p, at, count, e.wide, p);
            else load8<float>(e.p, at, count, e.wide, p);
            if (e.g_bf16) load8<__nv_bfloat16>(e.g, at, count, e.wide, g);
            else load8<float>(e.g, at, count, e.wide, g);
            if (BITS == 32) {
                load8<float>(e.m, at, count, e.wide, m);
                load8<float>(e.v, at, count, e.wide, v);
            } else {
                load_codes(e.m, at, count, e.wide, e.ms[b / 256], m);
                load_codes(e.v, at, count, e.wide, e.vs[b / 256], v);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= v[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) update(s, g[k], m[k], v[k], p[k]);
            if (e.w) store8<float>(e.w, at, count, e.wide, p);
            if (e.p_bf16) store8<__nv_bfloat16>(e.p, at, count, e.wide, p);
            else store8<float>(e.p, at, count, e.wide, p);
            if (BITS == 32) {
                store8<float>(e.m, at, count, e.wide, m);
                store8<float>(e.v, at, count, e.wide, v);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = sqrt_fast(v[k]);
                // (past the end g and the states are zeros, and stay zeros)
                store_codes<false>(e.m, e.ms + b / 256, at, count, e.wide, m);
                store_codes<true>(e.v, e.vs + b / 256, at, count, e.wide, v);
            }
        }
    }
    pdl_launch_dependents();
}

template <int BITS, int MAX>
cudaError_t launch_kind(const LaunchCtx& c, int n, const moe_adamw_tensor* tensors, const AdamNumbers& k,
                        const float* norm, const float* lr_step) {
    AdamTable<MAX> t;
    t.k = k;
    t.norm = norm;
    t.lr_step = lr_step;
    t.n = 0;
    int64_t chunks = 0;
    auto flush = [&]() {
        if (t.n == 0) return cudaSuccess;
        t.chunks = (int)chunks;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(chunks < kAdamBlocks ? chunks : kAdamBlocks));
        cfg.blockDim = dim3(kAdamThreads);
        cfg.stream = c.stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = c.pdl ? 1 : 0;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        void* args[] = {&t};
        const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(adamw_kernel<BITS, MAX>), args);
        t.n = 0;
        chunks = 0;
        return e;
    };
    for (int i = 0; i < n; ++i) {
        const moe_adamw_tensor& x = tensors[i];
        if (x.numel == 0 || x.state_bits != BITS) continue;
        const int64_t its = (x.numel + kChunk - 1) / kChunk;
        if (t.n == MAX || chunks + its > (1 << 30)) {
            const cudaError_t e = flush();
            if (e != cudaSuccess) return e;
        }
        chunks += its;
        const uint64_t where = row_at(x.param) | row_at(x.grad) | row_at(x.master) |
                               (BITS == 32 ? row_at(x.exp_avg) | row_at(x.exp_avg_sq)
                                           : (row_at(x.exp_avg) | row_at(x.exp_avg_sq)) * 2);
        t.e[t.n++] = AdamEntry{x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.exp_avg_scale, x.exp_avg_sq_scale, x.master,
                               x.numel, (int32_t)chunks, (uint8_t)(x.param_dtype == MOE_DTYPE_BF16),
                               (uint8_t)(x.grad_dtype == MOE_DTYPE_BF16), (uint8_t)(where % 16 == 0), 0};
    }
    return flush();
}

template <int BITS>
cudaError_t launch_bits(const LaunchCtx& c, int n, const moe_adamw_tensor* tensors, const AdamNumbers& k,
                        const float* norm, const float* lr_step) {
    if (n <= 32) return launch_kind<BITS, 32>(c, n, tensors, k, norm, lr_step);
    return launch_kind<BITS, kAdamMax>(c, n, tensors, k, norm, lr_step);
}

}  // namespace

cudaError_t launch_adamw(const LaunchCtx& c, int n, const moe_adamw_tensor* tensors, const moe_adamw_rule& r,
                         const float* norm, const float* lr_step) {
    AdamNumbers k{};
    k.b1 = (float)r.beta1;
    k.one_b1 = (float)(1.0 - r.beta1);
    k.b2 = (float)r.beta2;
    k.one_b2 = (float)(1.0 - r.beta2);
    k.eps = (float)r.eps;
    k.wd = (float)r.weight_decay;
    k.lr = (float)r.lr;
    if (!lr_step) {
        k.keep = (float)(1.0 - r.lr * r.weight_decay);
        k.rate = (float)(r.lr / (1.0 - pow(r.beta1, (double)r.step)));
        k.root = (float)(1.0 / sqrt(1.0 - pow(r.beta2, (double)r.step)));
    }
    k.log_b1 = (float)log(r.beta1);
    k.log_b2 = (float)log(r.beta2);
    k.max_norm = (float)r.max_norm;
    k.clip_eps = (float)r.clip_eps;
    const cudaError_t e = launch_bits<32>(c, n, tensors, k, norm, lr_step);
    return e != cudaSuccess ? e : launch_bits<8>(c, n, tensors, k, norm, lr_step);
}

}  // namespace moe
