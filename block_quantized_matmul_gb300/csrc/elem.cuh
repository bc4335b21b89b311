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

// 8 consecutive elements as they lie in memory.
template <typename T>
struct Raw8 {
    uint32_t w[2 * sizeof(T)];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); ++i) w[i] = 0u;
    }
    // VEC: p is 16-byte aligned.
    template <bool VEC>
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        } else {
            const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (uint32_t)q[2 * i] | ((uint32_t)q[2 * i + 1] << 16);
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2(w[i], T{});
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
    // The largest magnitude as the bits of an fp32; infinities and NaN come out on top.
    __device__ __forceinline__ uint32_t top_bits() const {
        if constexpr (sizeof(T) == 4) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
            return m;
        } else {
            uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
            for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
            m = max(m & 0xFFFFu, m >> 16);
            return __float_as_uint(unpack2(m, T{}).x);
        }
    }
};

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
