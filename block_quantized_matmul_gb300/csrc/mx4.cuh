// mx4.cuh -- the microscaled 4-bit floating-point (MX4) operand: E2M1 codes with one E8M0 scale per 32
// consecutive elements of a row (the OCP MXFP4 format), in the layout that the block-scaled tensor
// core instruction reads.
//
// Codes: uint8 [R][K/2], element 2i of a row in the low nibble of byte i, element 2i + 1 in the high.
// Scales: 512-byte blocks, each for 128 rows x 4 blocks of 32 (K 128), block (r / 128) * ceil(K / 128)
// + k / 128; inside it row r, block b is byte 16 * (r % 32) + 4 * ((r % 128) / 32) + (b % 4).  That is 32
// lanes of 16 bytes, which tcgen05.cp copies to tensor memory as they are.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace qmm {

constexpr int kMx4ScaleBlock = 512;        // bytes of the scales of 128 rows x 128 k

inline size_t mx4_codes_bytes(int64_t R, int64_t K) { return (size_t)R * (size_t)(K / 2); }
inline size_t mx4_scales_bytes(int64_t R, int64_t K) {
    return (size_t)((R + 127) / 128) * (size_t)((K + 127) / 128) * kMx4ScaleBlock;
}

// Byte offset of the scales of row r, blocks 4 * k128 .. 4 * k128 + 3 (4 bytes, 4-byte aligned).
__host__ __device__ __forceinline__ int64_t mx4_scale_word(int64_t r, int64_t k128, int64_t n128) {
    return ((r >> 7) * n128 + k128) * kMx4ScaleBlock + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

// 2^(e - 127) for an E8M0 scale: 2^-127 is an fp32 subnormal, 255 is NaN.
__device__ __forceinline__ float mx4_scale(uint32_t e) {
    const uint32_t bits = e == 0 ? 0x00400000u : (e == 255 ? 0x7FC00000u : e << 23);
    return __uint_as_float(bits);
}

// Scale of a block from the bits of its largest magnitude: floor(log2 max) - 2, so that the largest
// element lands in [4, 8) (codes end at 6); 255 when the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t mx4_block_scale(uint32_t abs_bits) {
    if (abs_bits >= 0x7F800000u) return 255u;
    const int e = (int)(abs_bits >> 23) - 2;
    return (uint32_t)(e < 0 ? 0 : e);
}

// Codes of 8 elements under scale e (element i in nibble i): E2M1 of x * 2^(127 - e), to nearest even,
// saturating at 6.  The product is exact but for subnormal results, which round to zero anyway.
__device__ __forceinline__ uint32_t mx4_codes8(const float *x, uint32_t e) {
    const float inv = __uint_as_float((254u - e) << 23);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i] * inv;
    uint32_t w;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return e == 255u ? 0u : w;
}

// Values of the 8 codes of a word, without the scale.
__device__ __forceinline__ void mx4_values8(uint32_t w, float *v) {
    uint32_t h[4];
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

}  // namespace qmm
