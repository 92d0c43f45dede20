// One AdamW step over a list of tensors.
//
//   g = clip grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// The list travels as a kernel argument, a launch per kAdamMax tensors of one
// kind of states; nothing is copied to the device beforehand, and a captured
// graph replays it.  A warp takes 256 consecutive elements, eight a lane: a
// block of the states in 8 bits, whose largest magnitude is one warp-wide
// maximum.  HBM is the bound: every buffer read and written once; with states in 8
// bits the instructions are near it (39 an element).  Measured on GB300 (copy rate
// 6.8 TB/s), 302 million BF16 in 130 tensors: with FP32 master values and states
// 1204 us (7.0 TB/s), with states in 8 bits and no master 540 (5.6); 67 million
// FP32 269 (7.0) and 186 (5.7); 0.77 million FP32 in 18 tensors 4.9.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "f32x2.cuh"
#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamMax = 384;           // tensors of a launch: 27.6 KB of its 32 KB of arguments
// Blocks: states in 32 bits, one for each chunk, so that the SMs sweep the buffers
// in step (1207 us against 1428 with as many blocks as are resident, 302 million
// BF16 with master values); in 8 bits the resident ones, as a block's start weighs
// more beside the fewer bytes of a chunk (541 us against 597).
constexpr int kResident = 152 * 3;
constexpr int kStarts = 152 * 6;        // blocks whose first entry travels with the list
constexpr int kChunkMost = 4096, kChunkLeast = 2048;    // elements
constexpr int kGroup = MOE_ADAMW_BLOCK;                 // a warp's elements at a time

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
    uint8_t kind;           // of AdamKind
    uint8_t wide;           // every buffer in vectors
};
// Where the parameter's value is, and the type of the gradient.
enum AdamKind : uint8_t { kF32 = 0, kBf16 = 1, kMaster = 2, kBf16Grad = 4 };

struct AdamNumbers {
    float b1, one_b1, b2, one_b2, eps, wd;
    float keep, rate, root; // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    float log_b1, log_b2;   // for t on the device
    float max_norm, clip_eps;
};
template <int MAX>
struct AdamTable {
    static constexpr bool kStart = MAX > 32;
    int n;
    int chunks;
    int chunk;              // elements of a chunk
    AdamNumbers k;
    const float* norm;
    const float* lr_step;
    // entry of a block's first chunk (a short list is searched)
    uint16_t start[kStart ? kStarts : 1];
    AdamEntry e[MAX];
};

// What a thread needs of the numbers: with the rate -lr / (1 - b1^t) divided into
// the denominator's terms, p' = p keep + m / (sqrt(v) root + eps).  The denominator
// stays from 2^-126 on, below which its reciprocal would be infinite (and 0 times that
// NaN): eps counts as 2^-126 times the rate at least.
struct AdamStep {
    float clip, b1, one_b1, minus_b2, minus_one_b2, keep, root, eps;
};
__device__ __forceinline__ AdamStep step_of(const AdamNumbers& k, const float* norm, const float* lr_step) {
    AdamStep s{1.0f, k.b1, k.one_b1, -k.b2, -k.one_b2, k.keep, k.root, k.eps};
    float rate = k.rate;
    if (norm) {
        const float q = k.max_norm / (norm[0] + k.clip_eps);
        s.clip = q > 1.0f ? 1.0f : q;       // NaN stays NaN
    }
    if (lr_step) {
        const float lr = lr_step[0], t = lr_step[1];
        s.keep = 1.0f - lr * k.wd;
        rate = lr / -expm1f(t * k.log_b1);
        s.root = 1.0f / sqrtf(-expm1f(t * k.log_b2));
    }
    // (a rate that is zero, or too small to divide by: a denominator whose reciprocal is zero)
    s.root = rate >= 1e-30f ? -s.root / rate : -1.0f;
    s.eps = rate >= 1e-30f ? fminf(-s.eps / rate, -0x1p-126f) : -FLT_MAX;
    if (rate > 0x1p126f) s.eps = NAN;       // (of lr_step; the host's is refused)
    return s;
}

__device__ __forceinline__ float rsqrt_fast(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// The largest of values that are not negative, NaN if one is.
__device__ __forceinline__ float max3(float a, float2 v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float min3(float a, float2 v) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(v.x), "f"(v.y));
    return r;
}

// fma2 whose results below 2^-126 are zeros.
__device__ __forceinline__ float2 fma2_flush(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}

// The moments and the parameter of two elements, the moments in the order of the
// formula (codes are those of its FP32 values, and a code more or less is 6 % of
// a value; an added rounding changes one in a million).  nv: minus v, which what
// follows takes without further operations.  Returns sqrt(v), the nearest but for
// one in some thousands: r = v y with y = rsqrt(v), and Newton's correction by the
// residual r^2 - v that an FMA has exactly (Markstein 1990).  Of v = 0, y is taken
// down to a number; an infinite v comes out as NaN and is seen to by the caller.
__device__ __forceinline__ float2 update(const AdamStep& s, float2 grad, float2& m, float2 v, float2& nv, float2& p) {
    const float2 g = mul2(grad, both(s.clip));
    m = fma2(both(s.one_b1), g, mul2(both(s.b1), m));
    nv = fma2_flush(both(s.minus_one_b2), mul2(g, g), mul2(both(s.minus_b2), v));
    const float2 minus_y = make_float2(fmaxf(-rsqrt_fast(-nv.x), -3.0e38f), fmaxf(-rsqrt_fast(-nv.y), -3.0e38f));
    const float2 r = mul2(nv, minus_y);
    const float2 root = fma2(fma2(r, r, nv), mul2(minus_y, both(0.5f)), r);
    const float2 over = fma2(root, both(s.root), both(s.eps));
    p = fma2(m, make_float2(rcp_fast(over.x), rcp_fast(over.y)), mul2(p, both(s.keep)));
    return root;
}
// The root and the parameter where a v is not finite.
__device__ __noinline__ float2 update_any(float root_factor, float eps, float keep, float m, float v, float p) {
    const float root = sqrtf(v);
    return make_float2(root, p * keep + m / fmaf(root, root_factor, eps));
}

// Eight elements of type T_: packed in vectors, or the first `count` of them.
template <typename T_>
struct Eight {
    static constexpr int VEC = 16 / sizeof(T_), N = 8 / VEC;
    uint4 r[N];
    __device__ __forceinline__ void load(const void* base, uint32_t i) {
#pragma unroll
        for (int k = 0; k < N; ++k) r[k] = reinterpret_cast<const uint4*>(static_cast<const T_*>(base) + i)[k];
    }
    __device__ __forceinline__ void load_some(const void* base, uint32_t i, int count) {
        T_ u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = k < count ? static_cast<const T_*>(base)[i + k] : T_(0.0f);
        float2 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = make_float2((float)u[2 * k], (float)u[2 * k + 1]);
        put(v);
    }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float u[VEC];
            RowVec<T_, VEC>::unpack(r[k], u);
#pragma unroll
            for (int j = 0; j < VEC; j += 2) v[(k * VEC + j) / 2] = make_float2(u[j], u[j + 1]);
        }
    }
    __device__ __forceinline__ void put(const float2 (&v)[4]) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float u[VEC];
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                u[j] = v[(k * VEC + j) / 2].x;
                u[j + 1] = v[(k * VEC + j) / 2].y;
            }
            r[k] = RowVec<T_, VEC>::pack(u);
        }
    }
    __device__ __forceinline__ void store(void* base, uint32_t i) const {
#pragma unroll
        for (int k = 0; k < N; ++k) reinterpret_cast<uint4*>(static_cast<T_*>(base) + i)[k] = r[k];
    }
    __device__ __forceinline__ void store_some(void* base, uint32_t i, int count) const {
        float2 v[4];
        get(v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) static_cast<T_*>(base)[i + k] = T_(k & 1 ? v[k >> 1].y : v[k >> 1].x);
    }
};

// Eight E4M3 bytes with their block's scale.
struct EightCodes {
    uint2 r;
    float scale;
    __device__ __forceinline__ void load(const void* base, uint32_t i) {
        r = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + i);
    }
    __device__ __forceinline__ void load_some(const void* base, uint32_t i, int count) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) w[k >> 2] |= (uint32_t)static_cast<const uint8_t*>(base)[i + k] << (8 * (k & 3));
        r = make_uint2(w[0], w[1]);
    }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        const uint32_t w[2] = {r.x, r.y};
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(e4m3x2_to_f32x2(w[k >> 1] >> (16 * (k & 1))), both(scale));
    }
    // The codes of a warp's 256 values, of which `most` is the lane's largest
    // magnitude: each value / scale rounded to FP32 and then to E4M3.  The quotients
    // are products with the reciprocal and the same correction.  ROOT: of values
    // that are not negative none but zero becomes zero.
    template <bool ROOT>
    __device__ __forceinline__ void put(const float2 (&v)[4], float most) {
        const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));   // (NaN's bits are above infinity's)
        const bool flush = amax < 7.88860905e-31f;      // 2^-100
        scale = flush ? 0.0f : amax * (1.0f / 448.0f);
        const float2 inv = both(flush ? 0.0f : rcp_fast(scale)), by = both(-scale);
        float2 q[4];
        float least = 1.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            q[k] = mul2(v[k], inv);
            q[k] = fma2(fma2(q[k], by, v[k]), inv, q[k]);
            if (ROOT) least = min3(least, q[k]);
        }
        if (ROOT && least < 0x1p-9f && !flush) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (v[k].x > 0.0f) q[k].x = fmaxf(q[k].x, 0x1p-9f);
                if (v[k].y > 0.0f) q[k].y = fmaxf(q[k].y, 0x1p-9f);
            }
        }
        r = make_uint2(f32x2_to_e4m3x2(q[0].x, q[0].y) | f32x2_to_e4m3x2(q[1].x, q[1].y) << 16,
                       f32x2_to_e4m3x2(q[2].x, q[2].y) | f32x2_to_e4m3x2(q[3].x, q[3].y) << 16);
    }
    __device__ __forceinline__ void store(void* base, uint32_t i) const {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + i) = r;
    }
    __device__ __forceinline__ void store_some(void* base, uint32_t i, int count) const {
        const uint32_t w[2] = {r.x, r.y};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) static_cast<uint8_t*>(base)[i + k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
    }
};

// A chunk's part of each buffer of its tensor.
struct AdamChunk {
    uint8_t *at;            // where the parameter is read: the master values, or itself
    uint8_t *p, *m, *v;
    const uint8_t* g;
    float *ms, *vs;
};
__device__ __forceinline__ AdamChunk chunk_of(const AdamEntry& e, int64_t first, int pb, int gb, int sb) {
    AdamChunk c;
    c.p = static_cast<uint8_t*>(e.p) + first * pb;
    c.at = e.w ? reinterpret_cast<uint8_t*>(e.w + first) : c.p;
    c.g = static_cast<const uint8_t*>(e.g) + first * gb;
    c.m = static_cast<uint8_t*>(e.m) + first * sb;
    c.v = static_cast<uint8_t*>(e.v) + first * sb;
    c.ms = e.ms + first / kGroup;
    c.vs = e.vs + first / kGroup;
    return c;
}

// A warp's 256 elements, eight of them a lane, from `at` in the chunk.
template <int BITS, int KIND>
struct AdamGroup {
    using P = typename std::conditional<(KIND & 3) == kBf16, __nv_bfloat16, float>::type;     // where p is read
    using G = typename std::conditional<(KIND & kBf16Grad) != 0, __nv_bfloat16, float>::type;
    using S = typename std::conditional<BITS == 32, Eight<float>, EightCodes>::type;
    Eight<P> p;
    Eight<G> g;
    S m, v;
    __device__ __forceinline__ void load(const AdamChunk& c, uint32_t at) {
        p.load(c.at, at);
        g.load(c.g, at);
        m.load(c.m, at);
        v.load(c.v, at);
        load_scales(c, at);
    }
    __device__ __forceinline__ void load_some(const AdamChunk& c, uint32_t at, int count) {
        p.load_some(c.at, at, count);
        g.load_some(c.g, at, count);
        m.load_some(c.m, at, count);
        v.load_some(c.v, at, count);
        load_scales(c, at);
    }
    __device__ __forceinline__ void load_scales(const AdamChunk& c, uint32_t at) {
        if constexpr (BITS == 8) {
            m.scale = c.ms[at / kGroup];
            v.scale = c.vs[at / kGroup];
        }
    }
    __device__ __forceinline__ void compute(const AdamStep& s, float2 (&fp)[4]) {
        float2 fg[4], fm[4], fv[4], root[4];
        p.get(fp);
        g.get(fg);
        m.get(fm);
        v.get(fv);
        float most = 0.0f, most_m = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (BITS == 8) fv[k] = mul2(fv[k], fv[k]);
            root[k] = update(s, fg[k], fm[k], fv[k], fv[k], fp[k]);
            most = max3(most, root[k]);
            if constexpr (BITS == 8) most_m = fmaxf(most_m, fmaxf(fabsf(fm[k].x), fabsf(fm[k].y)));
        }
        if (!(most < INFINITY)) {
            p.get(fp);
            most = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = update_any(s.root, s.eps, s.keep, fm[k].x, -fv[k].x, fp[k].x);
                const float2 y = update_any(s.root, s.eps, s.keep, fm[k].y, -fv[k].y, fp[k].y);
                root[k] = make_float2(x.x, y.x);
                fp[k] = make_float2(x.y, y.y);
                most = max3(most, root[k]);
            }
        }
        p.put(fp);
        if constexpr (BITS == 32) {
            m.put(fm);
#pragma unroll
            for (int k = 0; k < 4; ++k) fv[k] = make_float2(-fv[k].x, -fv[k].y);
            v.put(fv);
        } else {
            v.template put<true>(root, most);
            m.template put<false>(fm, v.scale == v.scale ? most_m : NAN);
        }
    }
    __device__ __forceinline__ void store(const AdamChunk& c, uint32_t at, const float2 (&fp)[4]) const {
        p.store(c.at, at);
        if constexpr ((KIND & 3) == kMaster) rounded(fp).store(c.p, at);
        m.store(c.m, at);
        v.store(c.v, at);
        store_scales(c, at);
    }
    __device__ __forceinline__ void store_some(const AdamChunk& c, uint32_t at, int count, const float2 (&fp)[4]) const {
        p.store_some(c.at, at, count);
        if constexpr ((KIND & 3) == kMaster) rounded(fp).store_some(c.p, at, count);
        m.store_some(c.m, at, count);
        v.store_some(c.v, at, count);
        store_scales(c, at);
    }
    __device__ __forceinline__ void store_scales(const AdamChunk& c, uint32_t at) const {
        if constexpr (BITS == 8)
            if ((threadIdx.x & 31) == 0) {
                c.ms[at / kGroup] = m.scale;
                c.vs[at / kGroup] = v.scale;
            }
    }
    static __device__ __forceinline__ Eight<__nv_bfloat16> rounded(const float2 (&fp)[4]) {
        Eight<__nv_bfloat16> b;
        b.put(fp);
        return b;
    }
};

// The `count` elements of a tensor from `first` on: the block's warps take
// groups in turn, U of them in flight.
template <int BITS, int KIND>
__device__ __forceinline__ void adam_chunk(const AdamStep& s, const AdamEntry& e, int64_t first, int count) {
    constexpr int kStep = kAdamThreads * 8, U = BITS == 32 ? 1 : 2;
    const AdamChunk c = chunk_of(e, first, (KIND & 3) == kF32 ? 4 : 2, KIND & kBf16Grad ? 2 : 4, BITS / 8);
    const int lane = threadIdx.x & 31;
    int at = (threadIdx.x >> 5) * kGroup + lane * 8;
    if (e.wide) {
        for (; at - lane * 8 + (U - 1) * kStep + kGroup <= count; at += U * kStep) {
            AdamGroup<BITS, KIND> x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u].load(c, at + u * kStep);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 p[4];
                x[u].compute(s, p);
                x[u].store(c, at + u * kStep, p);
            }
        }
    }
    // the last groups, and buffers off their vectors.  Past the end all is zero and
    // stays zero (or NaN, where the clipping factor is)
#pragma unroll 1
    for (; at - lane * 8 < count; at += kStep) {
        const int some = max(0, min(8, count - at));
        const bool full = e.wide && some == 8;
        AdamGroup<BITS, KIND> x;
        float2 p[4];
        if (full) x.load(c, at);
        else x.load_some(c, at, some);
        x.compute(s, p);
        if (full) x.store(c, at, p);
        else x.store_some(c, at, some, p);
    }
}

template <int BITS, int MAX>
__global__ void __launch_bounds__(kAdamThreads, kResident / 152) adamw_kernel(const __grid_constant__ AdamTable<MAX> t) {
    int i = 0;
    if (AdamTable<MAX>::kStart && blockIdx.x < kStarts) {
        i = t.start[blockIdx.x];
    } else if (MAX > 32) {
        for (int hi = t.n - 1; i < hi;) {
            const int mid = (i + hi) >> 1;
            if ((int)blockIdx.x < t.e[mid].last_chunk) hi = mid;
            else i = mid + 1;
        }
    }
    pdl_wait();
    const AdamStep s = step_of(t.k, t.norm, t.lr_step);
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        while (c >= t.e[i].last_chunk) ++i;
        const AdamEntry& e = t.e[i];
        const int64_t first = (int64_t)(c - (i ? t.e[i - 1].last_chunk : 0)) * t.chunk;
        const int count = (int)min((int64_t)t.chunk, e.numel - first);
        switch (e.kind) {
            case kF32: adam_chunk<BITS, kF32>(s, e, first, count); break;
            case kBf16: adam_chunk<BITS, kBf16>(s, e, first, count); break;
            case kMaster: adam_chunk<BITS, kMaster>(s, e, first, count); break;
            case kF32 | kBf16Grad: adam_chunk<BITS, kF32 | kBf16Grad>(s, e, first, count); break;
            case kBf16 | kBf16Grad: adam_chunk<BITS, kBf16 | kBf16Grad>(s, e, first, count); break;
            default: adam_chunk<BITS, kMaster | kBf16Grad>(s, e, first, count);
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
    int64_t total = 0;
    for (int i = 0; i < n; ++i)
        if (tensors[i].state_bits == BITS) total += tensors[i].numel;
    t.chunk = kChunkLeast;
    while (t.chunk < kChunkMost && total > (int64_t)t.chunk * kStarts) t.chunk *= 2;
    int64_t chunks = 0;
    auto flush = [&]() {
        if (t.n == 0) return cudaSuccess;
        t.chunks = (int)chunks;
        const int blocks = BITS == 8 && chunks > kResident ? kResident : (int)chunks;
        if constexpr (AdamTable<MAX>::kStart) {
            for (int b = 0, at = 0; b < blocks && b < kStarts; ++b) {
                while (b >= t.e[at].last_chunk) ++at;
                t.start[b] = (uint16_t)at;
            }
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)blocks);
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
        const int64_t its = (x.numel + t.chunk - 1) / t.chunk;
        if (t.n == MAX || chunks + its > (1 << 30)) {
            const cudaError_t e = flush();
            if (e != cudaSuccess) return e;
        }
        chunks += its;
        const uint64_t where = row_at(x.param) | row_at(x.grad) | row_at(x.master) |
                               (BITS == 32 ? row_at(x.exp_avg) | row_at(x.exp_avg_sq)
                                           : (row_at(x.exp_avg) | row_at(x.exp_avg_sq)) * 2);
        const int kind = (x.master ? kMaster : x.param_dtype == MOE_DTYPE_BF16 ? kBf16 : kF32) |
                         (x.grad_dtype == MOE_DTYPE_BF16 ? kBf16Grad : 0);
        t.e[t.n++] = AdamEntry{x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.exp_avg_scale, x.exp_avg_sq_scale, x.master,
                               x.numel, (int32_t)chunks, (uint8_t)kind, (uint8_t)(where % 16 == 0)};
    }
    return flush();
}

template <int BITS>
cudaError_t launch_bits(const LaunchCtx& c, int n, const moe_adamw_tensor* tensors, const AdamNumbers& k,
                        const float* norm, const float* lr_step) {
    if (n <= 32) return launch_kind<BITS, 32>(c, n, tensors, k, norm, lr_step);
    if (n <= 144) return launch_kind<BITS, 144>(c, n, tensors, k, norm, lr_step);
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
