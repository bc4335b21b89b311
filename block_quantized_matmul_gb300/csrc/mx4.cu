// mx4.cu -- rows of floating-point values to microscaled 4-bit operands (mx4.cuh) and back.
//
// Both directions move each element once and do a few operations on it, so they are bound by memory.
// A warp takes 256 consecutive elements of a row, 8 to a lane: 16- or 32-byte loads, 4-byte code
// words; the four lanes of a block find its largest magnitude with two shuffles, and the scale bytes
// of four blocks leave as one word.
#include "qmm_internal.cuh"

#include "elem.cuh"
#include "mx4.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;

template <bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(const T *__restrict__ x, int64_t R, int64_t K, int64_t ldx,
                                                                uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t nseg = (K + 255) / 256, n128 = (K + 127) / 128;
    const int lane = threadIdx.x & 31;
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < R * nseg;
         i += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t r = i / nseg, seg = i - r * nseg, k = seg * 256 + lane * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (k < K && QMM_DCHECK(r < R && k + 8 <= K)) load8<VEC>(x + r * ldx + k, v);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t e = mx4_block_scale(top);
        if (k < K) *reinterpret_cast<uint32_t *>(codes + (r * K + k) / 2) = mx4_codes8(v, e);
        // the scales of four blocks (16 lanes) as one word; blocks past K hold 0
        uint32_t word = e << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        const int64_t k128 = seg * 2 + (lane >> 4);
        if ((lane & 15) == 0 && k128 < n128) *reinterpret_cast<uint32_t *>(scales + mx4_scale_word(r, k128, n128)) = word;
    }
}

template <bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales, int64_t R, int64_t K,
                                                                  T *__restrict__ y, int64_t ldy) {
    const int64_t nseg = (K + 255) / 256, n128 = (K + 127) / 128;
    const int lane = threadIdx.x & 31;
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < R * nseg;
         i += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t r = i / nseg, seg = i - r * nseg, k = seg * 256 + lane * 8;
        if (k >= K || !QMM_DCHECK(r < R && k + 8 <= K)) continue;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + (r * K + k) / 2);
        const float s = mx4_scale(scales[mx4_scale_word(r, k >> 7, n128) + ((k >> 5) & 3)]);
        float v[8];
        mx4_values8(w, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= s;
        store8<VEC>(y + r * ldy + k, v);
    }
}

unsigned grid_rows(int64_t R, int64_t K) {
    const int64_t warps = R * ((K + 255) / 256), g = (warps + kThreads / 32 - 1) / (kThreads / 32);
    return (unsigned)(g > 152 * 8 ? 152 * 8 : g);
}

}  // namespace

cudaError_t launch_mx4_quantize(qmm_dtype t, const void *x, int64_t R, int64_t K, int64_t ldx, uint8_t *codes, uint8_t *scales,
                                cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using T = decltype(z);
        const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (ldx * sizeof(T)) % 16 == 0;
        auto kern = vec ? mx4_quantize_kernel<true, T> : mx4_quantize_kernel<false, T>;
        return launch_pdl(kern, dim3(grid_rows(R, K)), kThreads, 0, s, static_cast<const T *>(x), R, K, ldx, codes, scales);
    });
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K, qmm_dtype t, void *y,
                                  int64_t ldy, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using T = decltype(z);
        const bool vec = (reinterpret_cast<uintptr_t>(y) & 15u) == 0 && (ldy * sizeof(T)) % 16 == 0;
        auto kern = vec ? mx4_dequantize_kernel<true, T> : mx4_dequantize_kernel<false, T>;
        kern<<<grid_rows(R, K), kThreads, 0, s>>>(codes, scales, R, K, static_cast<T *>(y), ldy);
        return cudaGetLastError();
    });
}

QMM_DCHECK_READER(read_dcheck_mx4)

}  // namespace qmm
