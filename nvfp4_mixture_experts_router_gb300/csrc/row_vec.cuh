// Rows of BF16 or FP32 elements as vectors of VEC elements: 16 bytes where
// every row starts on a 16-byte boundary, else single elements.
#pragma once
#include "common.cuh"

namespace moe {

template <typename T, int VEC>
struct RowVec;

template <>
struct RowVec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[8]) { return pack_bf16x8(v); }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct RowVec<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct RowVec<__nv_bfloat16, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[1]) {
        v[0] = __uint_as_float((uint32_t)r << 16);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[1]) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
    static __device__ __forceinline__ Raw zero() { return 0; }
};
template <>
struct RowVec<float, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[1]) { v[0] = __uint_as_float(r); }
    static __device__ __forceinline__ Raw pack(const float (&v)[1]) { return __float_as_uint(v[0]); }
    static __device__ __forceinline__ Raw zero() { return 0u; }
};

}  // namespace moe
