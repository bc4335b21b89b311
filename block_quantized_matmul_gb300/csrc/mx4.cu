// mx4.cu -- rows of floating-point values to microscaled 4-bit operands (mx4.cuh) and back.
//
// Both directions move each element once and do a few operations on it.  A warp takes segments of 256
// consecutive elements of a row, 8 to a lane: 16- or 32-byte loads and 4-byte code words; the four
// lanes of a block find its largest magnitude with two shuffles, and the scale bytes of four blocks
// leave as one word.  A warp loads kBatch segments before it works on the first, so that enough
// bytes are on their way to hide memory's latency.
#include "qmm_internal.cuh"

#include "elem.cuh"
#include "mx4.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;

// `trigger`: the next kernel on the stream may start early (it waits for this one before it reads the
// operand; see launch_mx4_quantize).
template <bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(const T *__restrict__ x, uint32_t items, const FastDiv nseg, int64_t K,
                                                                int64_t ldx, uint8_t *__restrict__ codes,
                                                                uint8_t *__restrict__ scales, int64_t r0, int trigger) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t n128 = (K + 127) / 128;
    const int lane = threadIdx.x & 31;
    const uint32_t warps = gridDim.x * kWarps;
    for (uint32_t base = blockIdx.x * kWarps + (threadIdx.x >> 5); base < items; base += warps * kBatch) {
        Raw8<T> raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * warps, row = nseg(i);
            const int64_t k = (int64_t)(i - row * nseg.d) * 256 + lane * 8;
            raw[u].zero();
            if (i < items && k < K && QMM_DCHECK(k + 8 <= K)) raw[u].template load<VEC>(x + (r0 + row) * ldx + k);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * warps, row = nseg(i);
            if (i >= items) break;
            const int64_t r = r0 + row, seg = i - row * nseg.d, k = seg * 256 + lane * 8;
            uint32_t top = raw[u].top_bits();
            float v[8];
            raw[u].values(v);
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
}

template <bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales, uint32_t items,
                                                                  const FastDiv nseg, int64_t K, T *__restrict__ y, int64_t ldy,
                                                                  int64_t r0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t n128 = (K + 127) / 128;
    const int lane = threadIdx.x & 31;
    const uint32_t warps = gridDim.x * kWarps;
    for (uint32_t base = blockIdx.x * kWarps + (threadIdx.x >> 5); base < items; base += warps * kBatch) {
        uint32_t w[kBatch], e[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * warps, row = nseg(i);
            const int64_t r = r0 + row, k = (int64_t)(i - row * nseg.d) * 256 + lane * 8;
            w[u] = e[u] = 0;
            if (i < items && k < K && QMM_DCHECK(k + 8 <= K)) {
                w[u] = *reinterpret_cast<const uint32_t *>(codes + (r * K + k) / 2);
                e[u] = scales[mx4_scale_word(r, k >> 7, n128) + ((k >> 5) & 3)];
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * warps, row = nseg(i);
            const int64_t k = (int64_t)(i - row * nseg.d) * 256 + lane * 8;
            if (i >= items || k >= K) continue;
            const float s = mx4_scale(e[u]);
            float v[8];
            mx4_values8(w[u], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= s;
            store8<VEC>(y + (r0 + row) * ldy + k, v);
        }
    }
}

// Calls f(first row, rows, segments, grid) for pieces of fewer than 2^31 segments (one piece, but for
// operands beyond 2^39 elements).
template <typename F>
cudaError_t for_rows(int64_t R, int64_t K, F f) {
    const int64_t nseg = (K + 255) / 256, most = 0x3fffffff / nseg;
    for (int64_t r = 0; r < R; r += most) {
        const int64_t rows = R - r < most ? R - r : most, items = rows * nseg;
        const int64_t g = (items + kWarps - 1) / kWarps;
        const cudaError_t e = f(r, (uint32_t)items, FastDiv((uint32_t)nseg), dim3((unsigned)(g > 152 * 6 ? 152 * 6 : g)));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_mx4_quantize(qmm_dtype t, const void *x, int64_t R, int64_t K, int64_t ldx, uint8_t *codes, uint8_t *scales,
                                int trigger, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using T = decltype(z);
        const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (ldx * sizeof(T)) % 16 == 0;
        auto kern = vec ? mx4_quantize_kernel<true, T> : mx4_quantize_kernel<false, T>;
        return for_rows(R, K, [&](int64_t r, uint32_t items, FastDiv nseg, dim3 grid) {
            return launch_pdl(kern, grid, kThreads, 0, s, static_cast<const T *>(x), items, nseg, K, ldx, codes, scales, r, trigger);
        });
    });
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K, qmm_dtype t, void *y,
                                  int64_t ldy, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using T = decltype(z);
        const bool vec = (reinterpret_cast<uintptr_t>(y) & 15u) == 0 && (ldy * sizeof(T)) % 16 == 0;
        auto kern = vec ? mx4_dequantize_kernel<true, T> : mx4_dequantize_kernel<false, T>;
        return for_rows(R, K, [&](int64_t r, uint32_t items, FastDiv nseg, dim3 grid) {
            return launch_pdl(kern, grid, kThreads, 0, s, codes, scales, items, nseg, K, static_cast<T *>(y), ldy, r);
        });
    });
}

QMM_DCHECK_READER(read_dcheck_mx4)

}  // namespace qmm
