// RMS norm with the residual's addition, forward and backward.
//
//   h = x + residual, rounded;  rstd = 1 / sqrt(sum h^2 / H + eps)
//   y = h rstd gamma;  q = E4M3(y / scale), the scale from the largest |y| of a
//   row, of 128 elements or (a power of two) of 32
//   hhat = h rstd,  g = dy gamma
//   dx = dh + rstd (g - hhat sum(g hhat) / H),  dgamma = sum_t dy hhat
//
// HBM is the bound: every input read once, every output written once.
//
// Forward: up to 8192 columns a row lies in the registers of one block, and there
// is a block for each row, in order: the SMs finish at different speeds (a fixed
// share of the rows for each costs up to a sixth), so rows are handed out as blocks
// end, and several blocks an SM cover one another's reductions.  Columns of a
// thread (times with residual and MX codes): 32 for many BF16 rows of more than 512
// columns (16384 x 7168: 122 us against 158 with 16 and 275 with 8; 8191 x 2048: 21.5,
// 21.6, 25.7, codes by row 15.7, 18.5, 22.6), 16 for more than 256 columns and for
// FP32 (16383 x 512 BF16: 11.2 against 15.0 with 32 and 13.7 with 8; 8191 x 4096 FP32:
// 65, 73, 67), 8 for short rows (16383 x 128: 6.6 against 8.5 with 16).  gamma is read
// from L1 as it is needed: in registers beside the row it spilled (150 us against 131
// at the same step).  Rows off 16-byte blocks in vectors of less than four elements
// pass through shared memory (8191 x 7167 BF16, residual and MX codes: 161 against
// 333 by elements).  Rows of up to 16384 columns in whole vectors lie in one block of
// up to 512 threads (32 columns of BF16) or 1024 (FP32, and few rows).
//
// Backward: persistent blocks, each thread with the sums of dgamma of its columns
// in registers, so that dy and h are read once for both gradients; the blocks'
// sums go through the workspace to a reduction in a fixed order.  Of rows of more
// than 8192 columns dgamma is a pass of its own.
//
// Longer rows are walked two or three times, the re-reads served by the caches.
//
// Measured on GB300 (copy rate 6.8 TB/s): 16384 x 7168 BF16 with residual and MX
// codes 122 us (6.8 TB/s), with y instead 135 (7.0), y of x alone 79 (5.9), codes
// by row alone 102 (3.4: two looks at gamma and the row's maximum bound it); FP32
// 216, 267, 133, 138.  Backward with dh, 8191 x 7168: BF16 80 us (5.9), FP32 141
// (6.7); from 512 to 4096 columns 38 to 68 % of the copy rate (8191 x 1024 19 us,
// 2000 x 4096 22, from HBM: a block has six or seven rows, and the blocks' sums are
// written and read again).  8191 x 7167 BF16: 141 with residual and y (3.3), backward
// with dh 191 (2.5).  2000 x 16384 BF16: 42 with residual and y (6.3), 41 with MX codes,
// backward with dh 83 (3.2).  1000 x 65536 BF16: 117, 139, 235.  One row of 7168: 3.5.
#include <math.h>

#include "f32x2.cuh"
#include "row_vec.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr float kE4M3Max = 448.0f;

// A row's scale from the largest |y|, and what y is multiplied by.  At least
// 2^-126: the reciprocal stays finite.
__device__ __forceinline__ float linear_scale(float amax) {
    return amax == 0.0f ? 1.0f : fmaxf(amax * (1.0f / kE4M3Max), 1.17549435e-38f);
}
// 1 / scale: the reciprocal within a unit and Newton's correction.
__device__ __forceinline__ float inverse(float scale) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
    return fmaf(fmaf(-scale, r, 1.0f), r, r);
}

// A vector's values in pairs (a single one with 0).
template <typename T_, int VEC>
__device__ __forceinline__ void unpack_pairs(const typename RowVec<T_, VEC>::Raw& r, float2 (&v)[(VEC + 1) / 2]) {
    float u[VEC];
    RowVec<T_, VEC>::unpack(r, u);
#pragma unroll
    for (int k = 0; k < (VEC + 1) / 2; ++k) v[k] = make_float2(u[2 * k], VEC > 1 ? u[(2 * k + 1) % VEC] : 0.0f);
}

template <typename T_, int VEC>
__device__ __forceinline__ typename RowVec<T_, VEC>::Raw pack_pairs(const float2 (&v)[(VEC + 1) / 2]) {
    float u[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) u[k] = k & 1 ? v[k >> 1].y : v[k >> 1].x;
    return RowVec<T_, VEC>::pack(u);
}

// 1 / sqrt(S / H + eps) as the sum of two FP32 numbers, from S in two.  What is
// quantized after it sits on borders (of E4M3's steps, of powers of two) that an
// error of a unit crosses one time in a million; with rstd and h rstd in two
// numbers y is rounded once.
struct Rstd {
    float hi, lo;
};
__device__ __forceinline__ float2 two_sum(float a, float b) {       // a + b = x + y
    const float s = a + b, t = s - a;
    return make_float2(s, (a - (s - t)) + (b - t));
}
__device__ __forceinline__ Rstd rstd_of(float2 sum, float2 inv_h, float eps) {
    const float v = sum.x * inv_h.x;
    const float v_lo = fmaf(sum.x, inv_h.x, -v) + fmaf(sum.x, inv_h.y, sum.y * inv_h.x);
    const float2 t = two_sum(v, eps);
    const float r = rsqrtf(t.x), w = t.x * r;       // Newton's correction: r (1 - t r^2) / 2
    const float lo = 0.5f * r * (fmaf(-w, r, 1.0f) - fmaf(t.x, r, -w) * r - (t.y + v_lo) * r * r);
    return Rstd{r, fabsf(lo) < INFINITY ? lo : 0.0f};
}
// h rstd gamma of two elements, rounded once (but for a unit in some hundreds).  The
// product with rstd comes first: it is sqrt(H) at most, and zero where rstd is, while
// h gamma may pass FP32 (h gamma first: 120.5 us against 121.9 for 16384 x 7168 with
// MX codes, 80.5 against 79.5 for y alone).
__device__ __forceinline__ float2 scaled(float2 h, float2 gamma, Rstd r) {
    const float2 p = mul2(h, both(r.hi)), p_lo = make_float2(fmaf(h.x, r.hi, -p.x), fmaf(h.y, r.hi, -p.y));
    return fma2(p, gamma, mul2(fma2(h, both(r.lo), p_lo), gamma));
}

// Sum over the W warps of a row in two FP32 numbers, and with `most` the row's
// largest m; every thread gets them.
struct RowJoin {
    float2 sum;
    float most;
};
__device__ __forceinline__ RowJoin join_row(float sum, float m, bool most, int W, float2* s) {
    sum = warp_sum(sum);
    if (most) m = warp_largest(m);
    float2 v = make_float2(sum, 0.0f);
    if (W > 1) {
        const int lane = threadIdx.x & 31;
        s += threadIdx.y * W;
        if (lane == 0) s[threadIdx.x >> 5] = make_float2(sum, m);
        __syncthreads();
        const float2 u = lane < W ? s[lane] : make_float2(0.0f, 0.0f);
        v.x = u.x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            if (o < W) {
                const float2 t = two_sum(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
                v = make_float2(t.x, v.y + __shfl_xor_sync(0xffffffffu, v.y, o) + t.y);
            }
        // (lanes past the next power of two have not met the row's)
        v.x = __shfl_sync(0xffffffffu, v.x, 0);
        v.y = __shfl_sync(0xffffffffu, v.y, 0);
        if (most) m = warp_largest(u.y);
    }
    return RowJoin{v, m};
}

// A scale of `amax` by the mode's rule, stored at `to[i]`, and what y is multiplied by.
__device__ __forceinline__ float put_scale(int mode, void* to, int i, float amax, bool writes) {
    if (mode == MOE_SCALE_MX) {
        // mx_block_exp in the fields of FP32: the code is the exponent's less 8, 0 below that (and of infinity)
        const int field = (int)(__float_as_uint(amax) >> 23), code = field < 255 ? max(field - 8, 0) : 0;
        if (writes) static_cast<uint8_t*>(to)[i] = (uint8_t)code;
        return __uint_as_float((uint32_t)(254 - code) << 23);
    }
    const float scale = linear_scale(amax);
    if (writes) static_cast<float*>(to)[i] = scale;
    return inverse(scale);
}

// Four E4M3 codes.
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        " mov.b32 %0, {lo, hi};\n}" : "=r"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* q, float2 (&v)[(VEC + 1) / 2], float inv) {
#pragma unroll
    for (int k = 0; k < (VEC + 1) / 2; ++k) v[k] = mul2(v[k], both(inv));
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q) = make_uint2(e4m3x4(v[0], v[1]), e4m3x4(v[2], v[3]));
    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(q) = e4m3x4(v[0], v[1]);
    else if constexpr (VEC == 2) *reinterpret_cast<uint16_t*>(q) = (uint16_t)f32x2_to_e4m3x2(v[0].x, v[0].y);
    else *q = (uint8_t)f32x2_to_e4m3x2(v[0].x, 0.0f);
}
// The first `count` codes of a vector, at any address.
template <int VEC>
__device__ __forceinline__ void put_codes(uint8_t* q, float2 (&v)[VEC / 2], float inv, int count) {
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) v[k] = mul2(v[k], both(inv));
    uint32_t w[VEC / 4];
#pragma unroll
    for (int k = 0; k < VEC / 4; ++k) w[k] = e4m3x4(v[2 * k], v[2 * k + 1]);
#pragma unroll
    for (int k = 0; k < VEC; ++k)
        if (k < count) q[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
}
// The largest of `m` and the magnitudes of a vector.
template <int VEC>
__device__ __forceinline__ float max_of(float m, const float2 (&v)[(VEC + 1) / 2]) {
#pragma unroll
    for (int k = 0; k < (VEC + 1) / 2; ++k)
        asm("{\n .reg .f32 x, y;\n abs.f32 x, %1;\n abs.f32 y, %2;\n max.f32 %0, %0, x, y;\n}" : "+f"(m) : "f"(v[k].x), "f"(v[k].y));
    return m;
}

// Fetches BYTES (4, 8 or 16) into shared memory behind the thread's back.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    if constexpr (BYTES == 16)      // (past L1)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(BYTES) : "memory");
}

// A row off 16-byte blocks through shared memory: it lies there with its place
// within 16 bytes, so that its whole blocks move in vectors and its ends alone by
// elements, and the threads take and put vectors of the row at that offset.
struct RowSlot {
    static __host__ __device__ size_t bytes(size_t row) { return (row + 63) & ~(size_t)15; }    // with a vector past the end
    static __device__ __forceinline__ uint32_t offset(const void* row) { return (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u; }
    // By `lanes` threads, of which this is the j-th.
    template <typename One>
    static __device__ __forceinline__ void move(uint8_t* slot, uint8_t* row, uint32_t bytes, int j, int lanes, bool out) {
        const uint32_t off = offset(row), lead = min((16u - off) & 15u, bytes), whole = (bytes - lead) & ~15u;
        uint8_t* in_slot = slot + off;
        uint4 *a = reinterpret_cast<uint4*>(in_slot + lead), *b = reinterpret_cast<uint4*>(row + lead);
        for (uint32_t k = j; k < whole / 16; k += lanes) (out ? b : a)[k] = (out ? a : b)[k];
        // up to 15 bytes before and after
        for (uint32_t k = j * sizeof(One); k < 32; k += lanes * sizeof(One)) {
            const uint32_t at = k < 16 ? k : lead + whole + (k - 16);
            if (at < (k < 16 ? lead : bytes)) {
                One *c = reinterpret_cast<One*>(in_slot + at), *d = reinterpret_cast<One*>(row + at);
                *(out ? d : c) = *(out ? c : d);
            }
        }
    }
    // The same into a slot behind the threads' back: `begin`, and after
    // cp.async.wait_all `end`, which puts the thread's element of the ends.
    static __device__ __forceinline__ uint32_t edge(uint32_t off, uint32_t bytes, uint32_t k, bool* there) {
        const uint32_t lead = min((16u - off) & 15u, bytes), whole = (bytes - lead) & ~15u;
        const uint32_t at = k < 16 ? k : lead + whole + (k - 16);
        *there = k < 32 && at < (k < 16 ? lead : bytes);
        return at;
    }
    template <typename One>
    static __device__ __forceinline__ void begin(uint8_t* slot, const uint8_t* row, uint32_t bytes, int j, int lanes, One& end) {
        const uint32_t off = offset(row), lead = min((16u - off) & 15u, bytes), whole = (bytes - lead) & ~15u;
        for (uint32_t k = j * 16; k < whole; k += lanes * 16) copy_async<16>(slot + off + lead + k, row + lead + k);
        bool there;
        const uint32_t at = edge(off, bytes, j * sizeof(One), &there);
        if (there) end = *reinterpret_cast<const One*>(row + at);
    }
    template <typename One>
    static __device__ __forceinline__ void end(uint8_t* slot, const uint8_t* row, uint32_t bytes, int j, One end) {
        bool there;
        const uint32_t at = edge(offset(row), bytes, j * sizeof(One), &there);
        if (there) *reinterpret_cast<One*>(slot + offset(row) + at) = end;
    }
    // Vector c of a row at `off`: two blocks, shifted.  Of the last one `count`
    // elements count, the others become 0.
    template <typename T_>
    static __device__ __forceinline__ uint4 take(const uint8_t* slot, uint32_t off, int c, int count) {
        constexpr int VEC = 16 / sizeof(T_);
        const uint4 lo = reinterpret_cast<const uint4*>(slot)[c], hi = reinterpret_cast<const uint4*>(slot)[c + 1];
        uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = off & 8u ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = off & 4u ? w[i + 1] : w[i];
        if (sizeof(T_) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], off & 2u ? 16 : 0);
        }
        if (count < VEC) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i >= count) w[i * sizeof(T_) / 4] &= sizeof(T_) == 4 ? 0u : i & 1 ? 0xffffu : 0xffff0000u;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    template <typename T_>
    static __device__ __forceinline__ void put(uint8_t* slot, uint32_t off, int c, int count, const uint4& v) {
        constexpr int VEC = 16 / sizeof(T_);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint8_t* to = slot + off + c * 16;
        if (count == VEC && (off & 3u) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(to)[i] = w[i];
        } else if (sizeof(T_) == 2 && count == VEC) {
            *reinterpret_cast<uint16_t*>(to) = (uint16_t)w[0];
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(to + 2 + 4 * i) = __funnelshift_r(w[i], w[i + 1], 16);
            *reinterpret_cast<uint16_t*>(to + 14) = (uint16_t)(w[3] >> 16);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i < count) {
                    if (sizeof(T_) == 2) reinterpret_cast<uint16_t*>(to)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                    else reinterpret_cast<uint32_t*>(to)[i] = w[i & 3];
                }
        }
    }
};

// A thread's columns of gamma, of vector c (0 past the row's end).  RAGGED: the last
// vector may be cut.
template <int VEC, bool RAGGED>
__device__ __forceinline__ void gamma_vector(const float* gamma, int H, int c, bool wide, float2 (&ga)[(VEC + 1) / 2]) {
#pragma unroll
    for (int k = 0; k < (VEC + 1) / 2; ++k) ga[k] = both(0.0f);
    if ((c + 1) * VEC <= H) {
        load_vector<VEC>(gamma, c, wide, ga);
    } else if (RAGGED) {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (c * VEC + k < H) (k & 1 ? ga[k >> 1].y : ga[k >> 1].x) = gamma[c * VEC + k];
    }
}

constexpr int kRowColumns = 8192;   // rows up to here lie in registers,
constexpr int kWideColumns = 16384; // and up to here those in vectors of 16 bytes

// Rows of up to kRowColumns (kWideColumns) columns in registers: C columns a thread, V vectors
// that lie `lanes` vectors apart; W warps a row, eight warps a block or one row
// (a block of 32 W by rows).  STAGED: the rows pass through shared memory (RowSlot).
template <typename T_, int VEC, int C, bool RES, bool Q, bool STAGED, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) rms_rows_kernel(const RmsArgs a, int W, float2 inv_h, bool wide_gamma) {
    using RV = RowVec<T_, VEC>;
    using Raw = typename RV::Raw;
    using One = typename RowVec<T_, 1>::Raw;
    constexpr int V = C / VEC, P = (VEC + 1) / 2;
    static_assert(!STAGED || sizeof(Raw) == 16, "staged rows are taken in whole vectors");
    static_assert(!Q || VEC >= 4, "a block of 128 is a warp's");
    __shared__ float2 s_red[32];
    extern __shared__ __align__(16) uint8_t s_mem[];    // STAGED: a group's slots
    pdl_wait();
    const int lanes = blockDim.x, j = threadIdx.x, g = threadIdx.y, G = blockDim.y;
    const int n = (a.H + VEC - 1) / VEC;                // (not STAGED: H is a multiple)
    const int64_t t = (int64_t)blockIdx.x * G + g;
    const bool live = t < a.T;
    const uint32_t row_bytes = (uint32_t)a.H * sizeof(T_);
    const size_t slot = RowSlot::bytes(row_bytes);
    uint8_t *slot0 = s_mem + g * (STAGED ? 2 * slot + RowSlot::bytes(a.H) : 0), *slot1 = slot0 + slot, *slot_q = slot1 + slot;
    const T_* x = static_cast<const T_*>(a.x) + (live ? t : 0) * a.x_stride;
    const T_* res = RES ? static_cast<const T_*>(a.residual) + (live ? t : 0) * a.residual_stride : nullptr;
    T_* out_h = RES && a.h && live ? static_cast<T_*>(a.h) + t * a.h_stride : nullptr;
    T_* y = a.y && live ? static_cast<T_*>(a.y) + t * a.y_stride : nullptr;
    uint8_t* q = Q && a.q && live ? static_cast<uint8_t*>(a.q) + t * a.H : nullptr;
    if constexpr (STAGED) {
        if (live) RowSlot::move<One>(slot0, (uint8_t*)x, row_bytes, j, lanes, false);
        if (RES && live) RowSlot::move<One>(slot1, (uint8_t*)res, row_bytes, j, lanes, false);
        __syncthreads();
    }
    auto count_of = [&](int c) { return min(VEC, a.H - c * VEC); };
    auto load = [&](const T_* row, const uint8_t* at, int c) -> Raw {
        if (!live || c >= n) return Raw{};
        if constexpr (STAGED) return RowSlot::take<T_>(at, RowSlot::offset(row), c, count_of(c));
        else return reinterpret_cast<const Raw*>(row)[c];
    };
    auto store = [&](T_* row, uint8_t* at, int c, const Raw& v) {
        if constexpr (STAGED) RowSlot::put<T_>(at, RowSlot::offset(row), c, count_of(c), v);
        else reinterpret_cast<Raw*>(row)[c] = v;
    };
    Raw h[V];
    {
        Raw r[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            h[i] = load(x, slot0, j + i * lanes);
            if (RES) r[i] = load(res, slot1, j + i * lanes);
        }
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float2 u[P], v[P];
                unpack_pairs<T_, VEC>(h[i], u);
                unpack_pairs<T_, VEC>(r[i], v);
#pragma unroll
                for (int k = 0; k < P; ++k) u[k] = add2(u[k], v[k]);
                h[i] = pack_pairs<T_, VEC>(u);
                if (!STAGED && out_h && j + i * lanes < n) store(out_h, nullptr, j + i * lanes, h[i]);
            }
        }
    }
    // gamma of vector c (from L1)
    // (past the row's end the last vector's: h is zero there)
    auto gamma_of = [&](int c, float2 (&ga)[P]) {
        if constexpr (STAGED) gamma_vector<VEC, true>(a.gamma, a.H, c, wide_gamma, ga);
        else load_vector<VEC>(a.gamma, min(c, n - 1), wide_gamma, ga);
    };
    const bool by_row = Q && a.scale_mode == MOE_SCALE_ROW;
    // the row's scales of blocks
    uint8_t* scales = static_cast<uint8_t*>(a.scales) +
                      (a.scale_mode == MOE_SCALE_MX ? t * ((a.H + 31) / 32) : t * ((a.H + 127) / 128) * 4);
    float2 sq = both(0.0f);
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float2 u[P];
        unpack_pairs<T_, VEC>(h[i], u);
#pragma unroll
        for (int k = 0; k < P; ++k) sq = fma2(u[k], u[k], sq);
        if (by_row) {
            float2 ga[P];
            gamma_of(j + i * lanes, ga);
#pragma unroll
            for (int k = 0; k < P; ++k) u[k] = mul2(u[k], ga[k]);
            most = max_of<VEC>(most, u);
        }
    }
    const RowJoin row = join_row(sq.x + sq.y, most, by_row, W, s_red);
    const Rstd r = rstd_of(row.sum, inv_h, a.eps);
    if (a.rstd && live && j == 0) a.rstd[t] = r.hi + r.lo;
    float inv = 1.0f;
    // (a product that is NaN, of a row with NaN or an infinity: no y but zeros and NaN)
    if (by_row) inv = put_scale(MOE_SCALE_ROW, a.scales, (int)t, fmaxf(row.most * r.hi, 0.0f), live && j == 0);
    if constexpr (STAGED)
        if (W == 1) __syncthreads();        // (else join_row's: every thread has taken its vectors)
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = j + i * lanes;
        const bool there = live && c < n;
        float2 u[P], ga[P];
        if (STAGED && out_h && there) store(out_h, slot0, c, h[i]);
        unpack_pairs<T_, VEC>(h[i], u);
        gamma_of(c, ga);
#pragma unroll
        for (int k = 0; k < P; ++k) u[k] = scaled(u[k], ga[k], r);
        if (y && there) store(y, slot1, c, pack_pairs<T_, VEC>(u));
        if constexpr (Q) {
            if (!by_row) {
                float m = max_of<VEC>(0.0f, u);
#pragma unroll
                for (int o = 1; o < 32 / VEC; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (a.scale_mode == MOE_SCALE_MX) {
                    inv = put_scale(MOE_SCALE_MX, scales, c / (32 / VEC), m, there && c % (32 / VEC) == 0);
                } else {
#pragma unroll
                    for (int o = 32 / VEC; o < 128 / VEC; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    inv = put_scale(MOE_SCALE_BLOCK128, scales, c / (128 / VEC), m, there && c % (128 / VEC) == 0);
                }
            }
            if (q && there) {
                if constexpr (STAGED) put_codes<VEC>(slot_q + RowSlot::offset(q) + c * VEC, u, inv, count_of(c));
                else store_codes<VEC>(q + (int64_t)c * VEC, u, inv);
            }
        }
    }
    if constexpr (STAGED) {
        __syncthreads();
        if (out_h) RowSlot::move<One>(slot0, reinterpret_cast<uint8_t*>(out_h), row_bytes, j, lanes, true);
        if (y) RowSlot::move<One>(slot1, reinterpret_cast<uint8_t*>(y), row_bytes, j, lanes, true);
        if (q) RowSlot::move<uint8_t>(slot_q, q, (uint32_t)a.H, j, lanes, true);
    }
    pdl_launch_dependents();
}

constexpr int kRmsThreads = 512;

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

// A block a row, which is walked once for each of its results.
template <typename T_, int VEC>
__global__ void __launch_bounds__(kRmsThreads)
    rms_norm_kernel(const RmsArgs a, float2 inv_h, bool wide_gamma) {
    using RV = RowVec<T_, VEC>;
    using Raw = typename RV::Raw;
    constexpr int P = (VEC + 1) / 2, U = VEC > 2 ? 1 : 4 / VEC;     // vectors in flight
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
    // a vector of h, and of gamma
    auto pairs = [&](int c, float2 (&v)[P], float2 (&ga)[P]) {
        float u[VEC];
        row(c, true, u);
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = make_float2(u[2 * k], VEC > 1 ? u[(2 * k + 1) % VEC] : 0.0f);
        load_vector<VEC>(a.gamma, c, wide_gamma, ga);
    };
    float sq = 0.0f;
    for (int c = threadIdx.x; c < n; c += kRmsThreads) {
        float v[VEC];
        row(c, false, v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) sq = fmaf(v[k], v[k], sq);
    }
    const Rstd r = rstd_of(make_float2(block_join<false>(sq, s), 0.0f), inv_h, a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[t] = r.hi + r.lo;
    float inv = 1.0f;
    if (a.q && a.scale_mode == MOE_SCALE_ROW) {
        float most = 0.0f;
#pragma unroll U
        for (int c = threadIdx.x; c < n; c += kRmsThreads) {
            float2 v[P], ga[P];
            pairs(c, v, ga);
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] = mul2(v[k], ga[k]);
            most = max_of<VEC>(most, v);
        }
        most = block_join<true>(most, s);
        inv = put_scale(MOE_SCALE_ROW, a.scales, (int)t, fmaxf(most * r.hi, 0.0f), threadIdx.x == 0);
    } else if (a.q) {
        for (int b = threadIdx.x; b < n32; b += kRmsThreads) s_block[b] = 0.0f;
        __syncthreads();
#pragma unroll U
        for (int c = threadIdx.x; c < n; c += kRmsThreads) {
            float2 v[P], ga[P];
            pairs(c, v, ga);
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] = scaled(v[k], ga[k], r);
            // of non-negative floats the order of the bits is that of the values
            atomicMax(reinterpret_cast<int*>(s_block) + c * VEC / 32, __float_as_int(max_of<VEC>(0.0f, v)));
        }
        __syncthreads();
        if (a.scale_mode == MOE_SCALE_MX) {
            for (int b = threadIdx.x; b < n32; b += kRmsThreads)
                s_block[b] = put_scale(MOE_SCALE_MX, static_cast<uint8_t*>(a.scales) + t * n32, b, s_block[b], true);
        } else {
            const int n128 = (a.H + 127) / 128;
            for (int b = threadIdx.x; b < n128; b += kRmsThreads) {
                float m = 0.0f;
                for (int k = 4 * b; k < 4 * b + 4 && k < n32; ++k) m = fmaxf(m, s_block[k]);
                m = put_scale(MOE_SCALE_BLOCK128, static_cast<float*>(a.scales) + t * n128, b, m, true);
                for (int k = 4 * b; k < 4 * b + 4 && k < n32; ++k) s_block[k] = m;
            }
        }
        __syncthreads();
    }
    Raw* y = a.y ? static_cast<Raw*>(a.y) + t * (a.y_stride / VEC) : nullptr;
    uint8_t* q = a.q ? static_cast<uint8_t*>(a.q) + t * a.H : nullptr;
#pragma unroll U
    for (int c = threadIdx.x; c < n; c += kRmsThreads) {
        float2 v[P], ga[P];
        pairs(c, v, ga);
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = scaled(v[k], ga[k], r);
        if (y) y[c] = pack_pairs<T_, VEC>(v);
        if (q) store_codes<VEC>(q + c * VEC, v, a.scale_mode == MOE_SCALE_ROW ? inv : s_block[c * VEC / 32]);
    }
    pdl_launch_dependents();
}

// ---- backward -----------------------------------------------------------------------

// A block's sums of dgamma, its groups' in order, to the block's row of `part`.
template <int VEC, int V>
__device__ __forceinline__ void put_sums(const RmsGradArgs& a, const float2 (&dg)[V][(VEC + 1) / 2], int j, int lanes, int g,
                                         int G, float* sums) {
    float* out = a.part + (size_t)blockIdx.x * a.H;
    if (G > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int h = (j + i * lanes) * VEC + k;
            const float v = k & 1 ? dg[i][k >> 1].y : dg[i][k >> 1].x;
            if (h < a.H) (G > 1 ? sums + (size_t)g * a.H : out)[h] = v;
        }
    if (G > 1) {
        __syncthreads();
        for (int h = threadIdx.x; h < a.H; h += blockDim.x) {
            float v = 0.0f;
            for (int q = 0; q < G; ++q) v += sums[(size_t)q * a.H + h];
            out[h] = v;
        }
    }
}

// Rows of up to kRowColumns columns: a block walks rows, W warps a row of C columns
// a thread (eight warps a block, or one row), and each thread keeps the sums of
// dgamma for its columns in registers until the end.  The rows wait in a ring of S
// stages in shared memory, where each thread copies and reads its own vectors
// alone.  A turn takes the sum of one row's g hhat and writes the row before it,
// whose sum has met in between: one barrier a turn, and the two rows' reductions
// overlap.  DH: 0 none, 1 in the ring, 2 loaded when it is needed (FP32: three
// stages of all three would not fit).
template <typename T_, int VEC, int C, int DH>
__global__ void __launch_bounds__(512, 1) rms_ring_backward_kernel(const RmsGradArgs a, int W, int S, float inv_h, bool wide_gamma) {
    using RV = RowVec<T_, VEC>;
    using Raw = typename RV::Raw;
    constexpr int V = C / VEC, P = (VEC + 1) / 2, N = DH == 1 ? 3 : 2;
    __shared__ float s_red[2][32];
    extern __shared__ __align__(16) uint8_t s_mem[];    // [S][N][V][threads] vectors; in the end the groups' sums
    pdl_wait();
    const int lanes = W * 32, j = threadIdx.x % lanes, g = threadIdx.x / lanes, G = blockDim.x / lanes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = a.H / VEC;
    const int64_t step = (int64_t)gridDim.x * G, first = (int64_t)blockIdx.x * G + g;
    const Raw* rows[3] = {static_cast<const Raw*>(a.dy) + j, static_cast<const Raw*>(a.h) + j, static_cast<const Raw*>(a.dh) + j};
    const int64_t strides[3] = {a.dy_stride / VEC, a.h_stride / VEC, a.dh_stride / VEC};
    Raw* dx = static_cast<Raw*>(a.dx) + j;
    const int64_t dx_stride = a.dx_stride / VEC;
    Raw* ring = reinterpret_cast<Raw*>(s_mem) + threadIdx.x;
    auto at = [&](int stage, int k, int i) { return ring + ((stage * N + k) * V + i) * (int)blockDim.x; };
    auto fetch = [&](int64_t t, int stage) {
        if (t < a.T)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const Raw* row = rows[k] + t * strides[k];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (j + i * lanes < n)
                        copy_async<sizeof(Raw)>(at(stage, k, i), row + i * lanes);
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int q = 0; q < S; ++q) fetch(first + q * step, q);
    float2 ga[V][P], dg[V][P];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        gamma_vector<VEC, false>(a.gamma, a.H, j + i * lanes, wide_gamma, ga[i]);
#pragma unroll
        for (int k = 0; k < P; ++k) dg[i][k] = both(0.0f);
    }
    int stage = 0, before = 0, turn = 0;
    float sum_before = 0.0f, rstd_before = 0.0f, rstd = first < a.T ? a.rstd[first] : 0.0f;
    // turns: row t's sum and row t - step's result; one more than rows.  Uniform over the block
    for (int64_t t = first; t - g - step < a.T; t += step) {
        const bool live = t < a.T, had = t >= step && t - step < a.T && t != first;
        const float rstd_next = t + step < a.T ? a.rstd[t + step] : 0.0f;
        // row t's copies; S - 2 later ones may be under way (row t - step's stage is filled below)
        if (t == first) {
            if (S == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
            else asm volatile("cp.async.wait_group 3;" ::: "memory");
        } else {
            if (S == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 2;" ::: "memory");
        }
        Raw e[V];
        if (DH == 2) {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = had && j + i * lanes < n ? rows[2][(t - step) * strides[2] + i * lanes] : Raw{};
        }
        float2 sum = both(0.0f);
        if (live) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (j + i * lanes < n) {
                    float2 d[P], h[P];
                    unpack_pairs<T_, VEC>(*at(stage, 0, i), d);
                    unpack_pairs<T_, VEC>(*at(stage, 1, i), h);
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const float2 p = mul2(d[k], mul2(h[k], both(rstd)));
                        dg[i][k] = add2(dg[i][k], p);
                        sum = fma2(p, ga[i][k], sum);
                    }
                }
        }
        float s = warp_sum(sum.x + sum.y);
        if (W > 1) {
            if (lane == 0) s_red[turn][warp] = s;
            if (t != first) sum_before = warp_sum(lane < W ? s_red[turn ^ 1][warp / W * W + lane] : 0.0f);
        }
        if (had) {
            const float mean = sum_before * inv_h * rstd_before;
            Raw* out = dx + (t - step) * dx_stride;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (j + i * lanes < n) {
                    float2 d[P], h[P], u[P];
                    unpack_pairs<T_, VEC>(*at(before, 0, i), d);
                    unpack_pairs<T_, VEC>(*at(before, 1, i), h);
                    if (DH == 1) unpack_pairs<T_, VEC>(*at(before, N - 1, i), u);
                    if (DH == 2) unpack_pairs<T_, VEC>(e[i], u);
                    // rstd (g - hhat mean) + dh
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const float2 w = fma2(h[k], both(-mean), mul2(d[k], ga[i][k]));
                        d[k] = DH ? fma2(w, both(rstd_before), u[k]) : mul2(w, both(rstd_before));
                    }
                    out[i * lanes] = pack_pairs<T_, VEC>(d);
                }
        }
        if (t != first) fetch(t + (S - 1) * step, before);      // the stage of row t - step is free
        if (W > 1) __syncthreads();
        sum_before = s;
        rstd_before = rstd;
        rstd = rstd_next;
        before = stage;
        if (++stage == S) stage = 0;
        turn ^= 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    put_sums<VEC, V>(a, dg, j, lanes, g, G, reinterpret_cast<float*>(s_mem));
    pdl_launch_dependents();
}

// The same for rows off 16-byte blocks, in vectors of two bytes: each row through
// slots (RowSlot), the next one on its way meanwhile.  dy, whose slot takes dx, stays
// in registers; h and dh are taken twice (all three in registers spill: 208 us
// against 191 for 8191 x 7167 with dh; one row after the other 251).
template <typename T_, int C, bool DH, int BLOCKS>
__global__ void __launch_bounds__(512, BLOCKS) rms_slot_backward_kernel(const RmsGradArgs a, int W, float inv_h, bool wide_gamma) {
    constexpr int VEC = 16 / sizeof(T_);
    using Raw = typename RowVec<T_, VEC>::Raw;
    using One = typename RowVec<T_, 1>::Raw;
    constexpr int V = C / VEC, P = VEC / 2, N = DH ? 3 : 2;
    __shared__ float s_red[2][32];
    extern __shared__ __align__(16) uint8_t s_mem[];    // [groups][2][N] slots; in the end the groups' sums
    pdl_wait();
    const int lanes = W * 32, j = threadIdx.x % lanes, g = threadIdx.x / lanes, G = blockDim.x / lanes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (a.H + VEC - 1) / VEC;
    const int64_t step = (int64_t)gridDim.x * G, first = (int64_t)blockIdx.x * G + g;
    const T_* rows[3] = {static_cast<const T_*>(a.dy), static_cast<const T_*>(a.h), static_cast<const T_*>(a.dh)};
    const int64_t strides[3] = {a.dy_stride, a.h_stride, a.dh_stride};
    const uint32_t row_bytes = (uint32_t)a.H * sizeof(T_);
    const size_t slot = RowSlot::bytes(row_bytes);
    uint8_t *slots = s_mem + g * 2 * N * slot, *others = slots + N * slot;
    float2 dg[V][P];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < P; ++k) dg[i][k] = both(0.0f);
    One ends[N] = {};
    auto begin = [&](int64_t t, uint8_t* to) {
        if (t < a.T)
#pragma unroll
            for (int k = 0; k < N; ++k)
                RowSlot::begin<One>(to + k * slot, reinterpret_cast<const uint8_t*>(rows[k] + t * strides[k]), row_bytes, j, lanes, ends[k]);
    };
    begin(first, slots);
    int turn = 0;
    for (int64_t t = first; t - g < a.T; t += step) {        // uniform over the block
        const bool live = t < a.T;
        const float rstd = live ? a.rstd[t] : 0.0f;
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (live)
#pragma unroll
            for (int k = 0; k < N; ++k)
                RowSlot::end<One>(slots + k * slot, reinterpret_cast<const uint8_t*>(rows[k] + t * strides[k]), row_bytes, j, ends[k]);
        __syncthreads();            // and the row before has left the other slots
        begin(t + step, others);
        auto take = [&](int k, int c) {
            return live && c < n ? RowSlot::take<T_>(slots + k * slot, RowSlot::offset(rows[k] + t * strides[k]), c, min(VEC, a.H - c * VEC))
                                 : Raw{};
        };
        Raw r[V];
        float2 sum = both(0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = j + i * lanes;
            r[i] = take(0, c);
            float2 d[P], h[P], ga[P];
            unpack_pairs<T_, VEC>(r[i], d);
            unpack_pairs<T_, VEC>(take(1, c), h);
            gamma_vector<VEC, true>(a.gamma, a.H, c, wide_gamma, ga);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const float2 p = mul2(d[k], mul2(h[k], both(rstd)));
                dg[i][k] = add2(dg[i][k], p);
                sum = fma2(p, ga[k], sum);
            }
        }
        float s = warp_sum(sum.x + sum.y);
        if (lane == 0) s_red[turn][warp] = s;
        __syncthreads();            // and every thread has taken its vectors
        if (W > 1) s = warp_sum(lane < W ? s_red[turn][warp / W * W + lane] : 0.0f);
        turn ^= 1;
        const float mean = s * inv_h * rstd;
        T_* out = static_cast<T_*>(a.dx) + (live ? t : 0) * a.dx_stride;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = j + i * lanes;
            float2 d[P], h[P], ga[P], u[P];
            unpack_pairs<T_, VEC>(r[i], d);
            unpack_pairs<T_, VEC>(take(1, c), h);
            if (DH) unpack_pairs<T_, VEC>(take(N - 1, c), u);
            gamma_vector<VEC, true>(a.gamma, a.H, c, wide_gamma, ga);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const float2 w = fma2(h[k], both(-mean), mul2(d[k], ga[k]));
                d[k] = DH ? fma2(w, both(rstd), u[k]) : mul2(w, both(rstd));
            }
            if (live && c < n) RowSlot::put<T_>(slots, RowSlot::offset(out), c, min(VEC, a.H - c * VEC), pack_pairs<T_, VEC>(d));
        }
        __syncthreads();
        if (live) RowSlot::move<One>(slots, reinterpret_cast<uint8_t*>(out), row_bytes, j, lanes, true);
        uint8_t* const now = slots;
        slots = others;
        others = now;
    }
    __syncthreads();
    put_sums<VEC, V>(a, dg, j, lanes, g, G, reinterpret_cast<float*>(s_mem));
    pdl_launch_dependents();
}

// Partial sums of dgamma for longer rows: 256 columns a block and 256 / VEC threads
// a row, VEC rows at a time; blockIdx.y takes a share of the rows.
template <typename T_, int VEC>
__global__ void __launch_bounds__(256) rms_partial_kernel(const RmsGradArgs a) {
    using RV = RowVec<T_, VEC>;
    using Raw = typename RV::Raw;
    __shared__ float s[VEC][256];
    pdl_wait();
    constexpr int kLanes = 256 / VEC;
    const int j = threadIdx.x % kLanes, g = threadIdx.x / kLanes, first = blockIdx.x * 256, c = first / VEC + j;
    float sum[VEC] = {};
    if (c < a.H / VEC) {
        const Raw* dy = static_cast<const Raw*>(a.dy) + c;
        const Raw* h = static_cast<const Raw*>(a.h) + c;
        const int64_t dy_stride = a.dy_stride / VEC, h_stride = a.h_stride / VEC;
#pragma unroll 4
        for (int64_t t = (int64_t)blockIdx.y * VEC + g; t < a.T; t += gridDim.y * VEC) {
            float d[VEC], v[VEC];
            RV::unpack(dy[t * dy_stride], d);
            RV::unpack(h[t * h_stride], v);
            const float rstd = a.rstd[t];
#pragma unroll
            for (int k = 0; k < VEC; ++k) sum[k] = fmaf(d[k], v[k] * rstd, sum[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[g][j * VEC + k] = sum[k];
    __syncthreads();
    const int column = first + threadIdx.x;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < VEC; ++k) v += s[k][threadIdx.x];
    if (column < a.H) a.part[(size_t)blockIdx.y * a.H + column] = v;
    pdl_launch_dependents();
}
// Shares of the rows: eight blocks an SM, each with 64 rows or more.
int partial_shares(int T, int H) {
    const int strips = (H + 255) / 256, most = (152 * 8 + strips - 1) / strips, need = (T + 63) / 64;
    return need < 1 ? 1 : need < most ? need : most;
}

// dgamma from `parts` partial sums [parts][H]: 32 columns a block, a 32nd of the
// parts a warp, then the warps' sums in order.
__global__ void __launch_bounds__(1024) rms_reduce_kernel(int H, int parts, const float* part, float* dgamma) {
    __shared__ float s[32][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (c < H) {
#pragma unroll 8
        for (int p = warp; p < parts; p += 32) sum += part[(size_t)p * H + c];
    }
    s[warp][lane] = sum;
    __syncthreads();
    sum = warp_sum(s[lane][warp]);
    if (lane == 0 && blockIdx.x * 32 + warp < H) dgamma[blockIdx.x * 32 + warp] = sum;
    pdl_launch_dependents();
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

// The same with a row of dy and h in the registers of a block, C columns a thread: 32
// of BF16 and two blocks an SM (2000 x 16384 with dh 83 us, the sums of dgamma among
// them, against 95 with 16 and one block), 16 of FP32 (136).  Reading both twice took
// 127 and 159, one pass for both results through slots 122 (BF16).
template <typename T_, int VEC, int C>
__global__ void __launch_bounds__(16384 / C, C / 16) rms_dx_rows_kernel(const RmsGradArgs a, float inv_h, bool wide_gamma) {
    using RV = RowVec<T_, VEC>;
    using Raw = typename RV::Raw;
    constexpr int V = C / VEC, P = VEC / 2;
    __shared__ float s[32];
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int n = a.H / VEC, lanes = blockDim.x, j = threadIdx.x;
    const Raw* dy = static_cast<const Raw*>(a.dy) + t * (a.dy_stride / VEC);
    const Raw* h = static_cast<const Raw*>(a.h) + t * (a.h_stride / VEC);
    const Raw* dh = a.dh ? static_cast<const Raw*>(a.dh) + t * (a.dh_stride / VEC) : nullptr;
    Raw* dx = static_cast<Raw*>(a.dx) + t * (a.dx_stride / VEC);
    const float rstd = a.rstd[t];
    Raw rd[V], rh[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = j + i * lanes;
        rd[i] = c < n ? dy[c] : Raw{};
        rh[i] = c < n ? h[c] : Raw{};
    }
    // gamma four by four, and the rows unpacked twice: in 32 bits they would spill
    float2 sum = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = min(j + i * lanes, n - 1);            // (past the end dy is zero)
        float2 d[P], v[P], ga[2];
        unpack_pairs<T_, VEC>(rd[i], d);
        unpack_pairs<T_, VEC>(rh[i], v);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            if (k % 2 == 0) {
                asm volatile("" ::: "memory");
                load_vector<4>(a.gamma, c * (VEC / 4) + k / 2, wide_gamma, ga);
            }
            sum = fma2(mul2(d[k], ga[k % 2]), mul2(v[k], both(rstd)), sum);
        }
    }
    const float mean = block_join<false>(sum.x + sum.y, s) * inv_h * rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        asm volatile("" : "+r"(rd[i].x), "+r"(rd[i].y), "+r"(rd[i].z), "+r"(rd[i].w));
        asm volatile("" : "+r"(rh[i].x), "+r"(rh[i].y), "+r"(rh[i].z), "+r"(rh[i].w));
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = j + i * lanes;
        if (c >= n) break;
        float2 d[P], v[P], u[P], ga[2];
        unpack_pairs<T_, VEC>(rd[i], d);
        unpack_pairs<T_, VEC>(rh[i], v);
        unpack_pairs<T_, VEC>(dh ? dh[c] : Raw{}, u);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            if (k % 2 == 0) {
                asm volatile("" ::: "memory");
                load_vector<4>(a.gamma, c * (VEC / 4) + k / 2, wide_gamma, ga);
            }
            const float2 w = mul2(fma2(v[k], both(-mean), mul2(d[k], ga[k % 2])), both(rstd));
            d[k] = dh ? add2(w, u[k]) : w;
        }
        dx[c] = pack_pairs<T_, VEC>(d);
    }
    pdl_launch_dependents();
}

// 1 / H in two FP32 numbers.
float2 inverse_pair(int H) {
    const double inv = 1.0 / H;
    return make_float2((float)inv, (float)(inv - (double)(float)inv));
}

// C columns a thread.
template <typename T_, int VEC, int C, bool Q, bool STAGED, int THREADS, int BLOCKS>
cudaError_t forward_rows(const LaunchCtx& c, const RmsArgs& a) {
    const int W = (a.H + 32 * C - 1) / (32 * C), G = W >= 8 ? 1 : 8 / W;
    const bool wide_gamma = row_at(a.gamma) % 16 == 0;
    const size_t slots = STAGED ? G * (2 * RowSlot::bytes(a.H * sizeof(T_)) + RowSlot::bytes(a.H)) : 0;
    auto kernel = a.residual ? rms_rows_kernel<T_, VEC, C, true, Q, STAGED, THREADS, BLOCKS>
                             : rms_rows_kernel<T_, VEC, C, false, Q, STAGED, THREADS, BLOCKS>;
    return c.launch(kernel, dim3((unsigned)((a.T + G - 1) / G)), dim3(32 * W, G), slots, a, W, inverse_pair(a.H), wide_gamma);
}

template <typename T_, int VEC, bool Q>
cudaError_t forward_short(const LaunchCtx& c, const RmsArgs& a) {
    constexpr int kWhole = 16 / sizeof(T_);
    if constexpr (VEC < 4 && (sizeof(T_) == 2 || Q)) {
        // through shared memory, where a vector (or its codes) is less than eight bytes
        if constexpr (sizeof(T_) == 2)
            if (a.H > 4096) return forward_rows<T_, kWhole, 32, Q, true, 256, 4>(c, a);
        if (a.H > 256) return forward_rows<T_, kWhole, 16, Q, true, 512, 2>(c, a);
        return forward_rows<T_, kWhole, 8, Q, true, 256, 4>(c, a);
    } else {
        if constexpr (sizeof(T_) == 2)
            if (a.H > 512 && a.T > 2 * 152) return forward_rows<T_, VEC, 32, Q, false, 256, 4>(c, a);
        if constexpr (VEC >= 2)
            if (a.H > 256 && a.T > 152)      // (three without codes: FP32 16384 x 7168 133 us against 155)
                return forward_rows<T_, VEC, 16, Q, false, 512, Q ? 2 : 3>(c, a);
        return forward_rows<T_, VEC, 8, Q, false, 1024, 1>(c, a);
    }
}

template <typename T_, int VEC, bool Q>
cudaError_t forward_wide(const LaunchCtx& c, const RmsArgs& a) {
    if constexpr (sizeof(T_) == 2)
        if (a.T > 152) return forward_rows<T_, VEC, 32, Q, false, 512, 2>(c, a);
    return forward_rows<T_, VEC, 16, Q, false, 1024, 1>(c, a);
}

template <typename T_, int VEC>
cudaError_t forward_any(const LaunchCtx& c, const RmsArgs& a) {
    if (a.H <= kRowColumns) return a.q ? forward_short<T_, VEC, true>(c, a) : forward_short<T_, VEC, false>(c, a);
    if constexpr (VEC * sizeof(T_) == 16)
        if (a.H <= kWideColumns) return a.q ? forward_wide<T_, VEC, true>(c, a) : forward_wide<T_, VEC, false>(c, a);
    const size_t smem = a.q && a.scale_mode != MOE_SCALE_ROW ? (size_t)(a.H + 31) / 32 * 4 : 0;
    return c.launch(rms_norm_kernel<T_, VEC>, dim3((unsigned)a.T), dim3(kRmsThreads), smem, a, inverse_pair(a.H),
                    row_at(a.gamma) % 16 == 0);
}
// The shape of the backward kernels of short rows: warps a row, rows a block, and
// blocks on an SM (512 threads, or twice as many for the slots of BF16 rows).
struct BackwardShape {
    int C, W, G, threads, per_sm;
};
BackwardShape backward_shape(int H, bool many) {
    BackwardShape s;
    s.C = H > 256 ? 16 : 8;
    s.W = (H + 32 * s.C - 1) / (32 * s.C);
    s.G = s.W >= 8 ? 1 : 8 / s.W;
    s.threads = s.W * s.G * 32;
    s.per_sm = (many ? 1024 : 512) / s.threads;
    return s;
}
int backward_blocks(int T, const BackwardShape& s) {
    const int need = (T + s.G - 1) / s.G, most = 152 * s.per_sm;
    return need < 1 ? 1 : need < most ? need : most;
}

constexpr int kBackwardSmem = 216 * 1024;
template <typename T_, int VEC, int C>
cudaError_t ring_backward(const LaunchCtx& c, const RmsGradArgs& a, const BackwardShape& s) {
    constexpr int kDh = sizeof(T_) == 2 ? 1 : 2;
    auto kernel = a.dh ? rms_ring_backward_kernel<T_, VEC, C, kDh> : rms_ring_backward_kernel<T_, VEC, C, 0>;
    const int stage = (a.dh && kDh == 1 ? 3 : 2) * s.threads * C * (int)sizeof(T_);
    const int S = 4 * stage <= kBackwardSmem / s.per_sm ? 4 : 3;     // (three of the longest rows' are 144 KB of BF16, 192 of FP32)
    const int sums = s.G > 1 ? s.G * a.H * 4 : 0;
    return c.launch(kernel, dim3(backward_blocks(a.T, s)), dim3(s.threads), S * stage > sums ? S * stage : sums, a, s.W, S,
                    1.0f / (float)a.H, row_at(a.gamma) % 16 == 0);
}
template <typename T_, int C>
cudaError_t slot_backward(const LaunchCtx& c, const RmsGradArgs& a, const BackwardShape& s) {
    constexpr int kBlocks = sizeof(T_) == 2 ? 2 : 1;
    auto kernel = a.dh ? rms_slot_backward_kernel<T_, C, true, kBlocks> : rms_slot_backward_kernel<T_, C, false, kBlocks>;
    const size_t slots = 2 * s.G * (a.dh ? 3 : 2) * RowSlot::bytes(a.H * sizeof(T_)), sums = s.G > 1 ? (size_t)s.G * a.H * 4 : 0;
    return c.launch(kernel, dim3(backward_blocks(a.T, s)), dim3(s.threads), slots > sums ? slots : sums, a, s.W,
                    1.0f / (float)a.H, row_at(a.gamma) % 16 == 0);
}
// Are rows of these vectors taken through slots?  (Asynchronous copies have four bytes at least.)
bool in_slots(int elem, int bytes) { return elem == 2 && bytes == 2; }
template <typename T_, int VEC>
cudaError_t backward_any(const LaunchCtx& c, const RmsGradArgs& a, const BackwardShape& s) {
    if constexpr (VEC * sizeof(T_) < 4) return s.C == 16 ? slot_backward<T_, 16>(c, a, s) : slot_backward<T_, 8>(c, a, s);
    else return s.C == 16 ? ring_backward<T_, VEC, 16>(c, a, s) : ring_backward<T_, VEC, 8>(c, a, s);
}
cudaError_t launch_backward_rows(const LaunchCtx& c, int elem, int bytes, const RmsGradArgs& a, const BackwardShape& s) {
    MOE_ROW_VEC(elem, bytes, backward_any, c, a, s);
}

template <typename T_, int VEC>
cudaError_t partial_any(const LaunchCtx& c, const RmsGradArgs& a, dim3 grid) {
    return c.launch(rms_partial_kernel<T_, VEC>, grid, dim3(256), 0, a);
}
cudaError_t launch_partial(const LaunchCtx& c, int elem, int bytes, const RmsGradArgs& a, dim3 grid) {
    MOE_ROW_VEC(elem, bytes, partial_any, c, a, grid);
}

template <typename T_, int VEC>
cudaError_t dx_any(const LaunchCtx& c, const RmsGradArgs& a) {
    if constexpr (VEC * sizeof(T_) == 16)
        if (a.H <= kWideColumns) {
            constexpr int C = 64 / sizeof(T_);
            return c.launch(rms_dx_rows_kernel<T_, VEC, C>, dim3((unsigned)a.T), dim3((a.H + 32 * C - 1) / (32 * C) * 32), 0, a,
                            1.0f / (float)a.H, row_at(a.gamma) % 16 == 0);
        }
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

namespace {
template <typename K>
void allow(cudaError_t& e, K kernel) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBackwardSmem);
}
template <typename T_, int C, int THREADS, int BLOCKS>
void allow_staged(cudaError_t& e) {
    constexpr int VEC = 16 / sizeof(T_);
    allow(e, rms_rows_kernel<T_, VEC, C, false, true, true, THREADS, BLOCKS>);
    allow(e, rms_rows_kernel<T_, VEC, C, true, true, true, THREADS, BLOCKS>);
    if constexpr (sizeof(T_) == 2) {
        allow(e, rms_rows_kernel<T_, VEC, C, false, false, true, THREADS, BLOCKS>);
        allow(e, rms_rows_kernel<T_, VEC, C, true, false, true, THREADS, BLOCKS>);
    }
}
template <typename T_, int VEC>
void allow_ring(cudaError_t& e) {
    constexpr int kDh = sizeof(T_) == 2 ? 1 : 2;
    allow(e, rms_ring_backward_kernel<T_, VEC, 8, 0>);
    allow(e, rms_ring_backward_kernel<T_, VEC, 8, kDh>);
    allow(e, rms_ring_backward_kernel<T_, VEC, 16, 0>);
    allow(e, rms_ring_backward_kernel<T_, VEC, 16, kDh>);
}
}  // namespace

cudaError_t setup_rms_norm_kernels() {
    cudaError_t e = cudaSuccess;
    allow_staged<__nv_bfloat16, 8, 256, 4>(e);
    allow_staged<__nv_bfloat16, 16, 512, 2>(e);
    allow_staged<__nv_bfloat16, 32, 256, 4>(e);
    allow_staged<float, 8, 256, 4>(e);
    allow_staged<float, 16, 512, 2>(e);
    allow_ring<__nv_bfloat16, 8>(e);
    allow_ring<__nv_bfloat16, 4>(e);
    allow_ring<__nv_bfloat16, 2>(e);
    allow_ring<float, 4>(e);
    allow_ring<float, 2>(e);
    allow_ring<float, 1>(e);
    allow(e, rms_slot_backward_kernel<__nv_bfloat16, 8, false, 2>);
    allow(e, rms_slot_backward_kernel<__nv_bfloat16, 8, true, 2>);
    allow(e, rms_slot_backward_kernel<__nv_bfloat16, 16, false, 2>);
    allow(e, rms_slot_backward_kernel<__nv_bfloat16, 16, true, 2>);
    return e;
}

// Partial sums of dgamma, a row of H for each block of the backward kernels.
size_t rms_norm_workspace_bytes(int T, int H) {
    const int parts = H > kRowColumns ? partial_shares(T, H) : backward_blocks(T, backward_shape(H, true));
    return align_up((uint64_t)parts * H * 4, 256);
}

cudaError_t launch_rms_norm_backward(const LaunchCtx& c, int elem, const RmsGradArgs& args) {
    RmsGradArgs a = args;
    const int bytes = row_vec_bytes(a.H, elem,
                                    row_at(a.dy, a.dy_stride, elem) | row_at(a.dh, a.dh ? a.dh_stride : 0, elem) |
                                        row_at(a.h, a.h_stride, elem) | row_at(a.dx, a.dx_stride, elem));
    const bool rows = a.H <= kRowColumns;
    const BackwardShape s = backward_shape(a.H, in_slots(elem, bytes));
    const int parts = rows ? backward_blocks(a.T, s) : partial_shares(a.T, a.H);
    if (parts == 1) a.part = a.dgamma;          // one block's sums are the result
    cudaError_t e;
    if (rows) {
        e = launch_backward_rows(c, elem, bytes, a, s);
    } else {
        // the column sums first: dx may overwrite dy or h
        e = launch_partial(c, elem, bytes, a, dim3((unsigned)((a.H + 255) / 256), (unsigned)parts));
    }
    if (e == cudaSuccess && parts > 1)
        e = c.launch(rms_reduce_kernel, dim3((unsigned)((a.H + 31) / 32)), dim3(1024), 0, a.H, parts, (const float*)a.part,
                     a.dgamma);
    if (e != cudaSuccess || rows || a.T == 0) return e;
    return launch_dx(c, elem, bytes, a);
}

}  // namespace moe
