// Rows of BF16 or FP32 elements as vectors of VEC elements: the widest of 16,
// 8, 4 and 2 bytes that divides a row and that every row starts on.
#pragma once
#include "common.cuh"

namespace moe {

template <typename T, int VEC>
struct RowVec;

// Two FP32 values rounded to BF16, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <>
struct RowVec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[8]) {
        return pack_bf16x8(v);
    }
};
template <>
struct RowVec<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[4]) {
        v[0] = bf16_lo(r.x);
        v[1] = bf16_hi(r.x);
        v[2] = bf16_lo(r.y);
        v[3] = bf16_hi(r.y);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[4]) {
        return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
};
template <>
struct RowVec<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[2]) {
        v[0] = bf16_lo(r);
        v[1] = bf16_hi(r);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[2]) {
        return pack_bf16x2(v[0], v[1]);
    }
};
template <>
struct RowVec<__nv_bfloat16, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[1]) {
        v[0] = bf16_lo(r);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[1]) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
};
template <>
struct RowVec<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z);
        v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct RowVec<float, 2> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[2]) {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[2]) {
        return make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
    }
};
template <>
struct RowVec<float, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[1]) {
        v[0] = __uint_as_float(r);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[1]) {
        return __float_as_uint(v[0]);
    }
};

// Bytes of the widest vector for rows of H elements in buffers whose first
// elements and row strides (in bytes) are all or'ed into `where`.
inline int row_vec_bytes(int64_t H, int elem, uint64_t where) {
    const uint64_t all = (uint64_t)H * elem | where;
    return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}
inline uint64_t row_at(const void* p, int64_t stride = 0, int elem = 0) {
    return (uint64_t)reinterpret_cast<uintptr_t>(p) | (uint64_t)stride * elem;
}

// Calls f<T_, VEC>() for the element size and the vector's bytes.
#define MOE_ROW_VEC(elem, bytes, f, ...)                                                     \
    do {                                                                                     \
        if ((elem) == 2) {                                                                   \
            switch (bytes) {                                                                 \
                case 16: return f<__nv_bfloat16, 8>(__VA_ARGS__);                            \
                case 8: return f<__nv_bfloat16, 4>(__VA_ARGS__);                             \
                case 4: return f<__nv_bfloat16, 2>(__VA_ARGS__);                             \
                default: return f<__nv_bfloat16, 1>(__VA_ARGS__);                            \
            }                                                                                \
        }                                                                                    \
        switch (bytes) {                                                                     \
            case 16: return f<float, 4>(__VA_ARGS__);                                        \
            case 8: return f<float, 2>(__VA_ARGS__);                                         \
            default: return f<float, 1>(__VA_ARGS__);                                        \
        }                                                                                    \
    } while (0)

}  // namespace moe
