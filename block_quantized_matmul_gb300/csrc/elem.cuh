// elem.cuh -- floating-point element types of the MX4 and cache operators: loads of consecutive elements,
// their largest magnitude, and stores of fp32 values rounded to the element type (to nearest even).
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

// 32 bytes at a 32-byte aligned address in one access.
__device__ __forceinline__ void ld32(const void *p, uint32_t *w) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void st32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// N (8 or 16) consecutive elements as they lie in memory.
template <typename T, int N>
struct Raw {
    static constexpr int kWords = N * (int)sizeof(T) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // VEC: p is aligned to 32 bytes (16 for 16 bytes of elements).
    template <bool VEC>
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC && kWords == 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kWords / 8; ++i) ld32(reinterpret_cast<const uint32_t *>(p) + 8 * i, w + 8 * i);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        } else {
            const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = (uint32_t)q[2 * i] | ((uint32_t)q[2 * i + 1] << 16);
        }
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return (i & 1) ? unpack2(w[i >> 1], T{}).y : unpack2(w[i >> 1], T{}).x;
    }
    // The largest magnitude as the bits of an fp32; infinities and NaN come out on top.
    __device__ __forceinline__ uint32_t top_bits() const {
        if constexpr (sizeof(T) == 4) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
            return m;
        } else {
            uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
            for (int i = 1; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
            m = max(m & 0xFFFFu, m >> 16);
            return __float_as_uint(unpack2(m, T{}).x);
        }
    }
    // The largest magnitude of the elements without and with a sign bit, as bits of T (-1: there is none).
    __device__ __forceinline__ void top_signed(int &pos, int &neg) const {
        constexpr uint32_t kAbs = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFFu;
        uint32_t u;
        if constexpr (sizeof(T) == 4) {
            int m = (int)w[0];
            u = w[0];
#pragma unroll
            for (int i = 1; i < kWords; ++i) {
                m = max(m, (int)w[i]);
                u = max(u, w[i]);
            }
            pos = m < 0 ? -1 : m;
        } else {
            uint32_t m = w[0];
            u = w[0];
#pragma unroll
            for (int i = 1; i < kWords; ++i) {
                m = __vmaxs2(m, w[i]);
                u = __vmaxu2(u, w[i]);
            }
            pos = max((int)(int16_t)(m & 0xFFFFu), (int)(int16_t)(m >> 16));
            pos = pos < 0 ? -1 : pos;
            u = max(u & 0xFFFFu, u >> 16);
        }
        neg = u > kAbs ? (int)(u & kAbs) : -1;
    }
    __device__ __forceinline__ uint32_t bits(int i) const {        // element i as bits of T
        if constexpr (sizeof(T) == 4) return w[i];
        else return (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    }
};
template <typename T>
__device__ __forceinline__ float bits_to_float(uint32_t b) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(b);
    else return unpack2(b, T{}).x;
}

// N (8 or 16) fp32 values rounded to T at p; VEC: p is aligned as for Raw::load.
template <bool VEC, int N, typename T>
__device__ __forceinline__ void store_values(T *p, const float (&v)[N]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < N; ++i) float_to_elem(v[i], p[i]);
    } else {
        constexpr int kWords = N * (int)sizeof(T) / 4;
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
            else w[i] = pack2(v[2 * i], v[2 * i + 1], T{});
        }
        if constexpr (kWords == 4) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 8; ++i) st32(reinterpret_cast<uint32_t *>(p) + 8 * i, w + 8 * i);
        }
    }
}

inline bool rows_aligned(const void *p, int64_t ld, size_t es) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && (ld * es) % 32 == 0; }

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
