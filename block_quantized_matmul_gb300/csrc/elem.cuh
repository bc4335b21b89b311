// elem.cuh -- floating-point element types of the MX4 and cache operators: loads of 8 consecutive
// elements as fp32 and stores of 8 fp32 values rounded to the element type (to nearest even).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace qmm {

__device__ __forceinline__ float elem_to_float(float v) { return v; }
__device__ __forceinline__ float elem_to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float elem_to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void float_to_elem(float v, float &o) { o = v; }
__device__ __forceinline__ void float_to_elem(float v, __half &o) { o = __float2half_rn(v); }
__device__ __forceinline__ void float_to_elem(float v, __nv_bfloat16 &o) { o = __float2bfloat16_rn(v); }

// Two fp32 values as one packed word of a 16-bit type (first in the low half).
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

// 8 consecutive elements at p as fp32; VEC: p is 16-byte aligned.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = elem_to_float(p[i]);
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(u[i], T{});
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// 8 fp32 values rounded to T at p; VEC: p is 16-byte aligned.
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) float_to_elem(v[i], p[i]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack2(v[0], v[1], T{}), pack2(v[2], v[3], T{}), pack2(v[4], v[5], T{}), pack2(v[6], v[7], T{}));
    }
}

inline size_t dtype_bytes(qmm_dtype t) { return t == QMM_F32 ? 4 : 2; }

// n / d for n < 2^31 by a multiplication and a shift (the round-up method: with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (high word of m n + n) >> s).
struct FastDiv {
    uint32_t d, mul, shift;
    explicit FastDiv(uint32_t div) : d(div), mul(0), shift(0) {
        while (((uint64_t)1 << shift) < d) ++shift;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(mul, n) + n) >> shift; }
};

// Calls f with a value of the element type (its value does not matter).
template <typename F>
inline cudaError_t with_dtype(qmm_dtype t, F f) {
    switch (t) {
        case QMM_F32: return f(float{});
        case QMM_F16: return f(__half{});
        default: return f(__nv_bfloat16{});
    }
}

}  // namespace qmm
