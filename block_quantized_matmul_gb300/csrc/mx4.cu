// mx4.cu -- rows of floating-point values to microscaled 4-bit operands (mx4.cuh) and back.
//
// Both directions move each element once and do a few operations on it; what costs beside the bytes is
// instructions.  A lane takes 16 consecutive elements, half a block (a warp: 512 of a row): with 8, the
// addresses, shuffles and scale bytes of a lane's piece weigh twice as much (8192 x 14336 bf16: 77 us, with 16 about
// 50).  Bound by memory: 14336 x 4096 fp32 to MX4 and back, 532 MB, 90 us, 5.9 TB/s.
// Loads and stores are 32 bytes; two lanes of a block agree on its largest magnitude, and the scale
// bytes of four blocks leave as one word.  A warp loads kBatch pieces before it works on the first,
// so that enough bytes are on their way to hide memory's latency.
#include "qmm_internal.cuh"

#include "elem.cuh"
#include "mx4.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 2;
constexpr int kSeg = 512;                   // elements of a warp's piece

// TRIGGER: the next kernel on the stream may start early (it waits for this one before it reads the
// operand; see launch_mx4_quantize).  Six CTAs an SM (as launched) for 16-bit elements: five cost 6 us of 51
// for 8192 x 14336 bf16.
template <bool VEC, bool TRIGGER, typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 6 : 4) mx4_quantize_kernel(const T *__restrict__ x, uint32_t items, const FastDiv nseg, int64_t K,
                                                                int64_t ldx, uint8_t *__restrict__ codes,
                                                                uint8_t *__restrict__ scales, int64_t r0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (TRIGGER) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t n128 = (K + 127) / 128;
    const int lane = threadIdx.x & 31;
    const uint32_t warps = gridDim.x * kWarps;
    for (uint32_t base = blockIdx.x * kWarps + (threadIdx.x >> 5); base < items; base += warps * kBatch) {
        Raw<T, 16> raw[kBatch];
        int64_t row[kBatch], col[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * warps, r = nseg(i);
            row[u] = r0 + r;
            col[u] = i < items ? (int64_t)(i - r * nseg.d) * kSeg + lane * 16 : K;
            raw[u].zero();
            if (col[u] < K && QMM_DCHECK(col[u] + 16 <= K)) raw[u].template load<VEC>(x + row[u] * ldx + col[u]);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            uint32_t top = raw[u].top_bits();
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            const uint32_t e = mx4_block_scale(top);
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = raw[u].value(j);
            if (col[u] < K) *reinterpret_cast<uint2 *>(codes + (row[u] * K + col[u]) / 2) = make_uint2(mx4_codes8(v, e), mx4_codes8(v + 8, e));
            // the scales of four blocks (8 lanes) as one word; blocks past K hold 0
            uint32_t word = e << (4 * (lane & 6));
            word |= __shfl_xor_sync(0xffffffffu, word, 2);
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            if ((lane & 7) == 0 && col[u] < K) *reinterpret_cast<uint32_t *>(scales + mx4_scale_word(row[u], col[u] >> 7, n128)) = word;
        }
    }
    if constexpr (!TRIGGER) {
        // The product for few tokens streams its weight before it waits for the kernel before it, so an operand must be
        // visible device-wide, to bulk copies too, by the time this grid's blocks have exited.
        __threadfence();
        asm volatile("fence.proxy.async.global;" ::: "memory");
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
        uint2 w[kBatch];
        uint32_t e[kBatch];
        int64_t row[kBatch], col[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * warps, r = nseg(i);
            row[u] = r0 + r;
            col[u] = i < items ? (int64_t)(i - r * nseg.d) * kSeg + lane * 16 : K;
            w[u] = make_uint2(0u, 0u);
            e[u] = 0;
            if (col[u] < K && QMM_DCHECK(col[u] + 16 <= K)) {
                w[u] = *reinterpret_cast<const uint2 *>(codes + (row[u] * K + col[u]) / 2);
                e[u] = scales[mx4_scale_word(row[u], col[u] >> 7, n128) + ((lane >> 1) & 3)];
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (col[u] >= K) continue;
            const float s = mx4_scale(e[u]);
            float v[16];
            mx4_values8(w[u].x, v);
            mx4_values8(w[u].y, v + 8);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] *= s;
            store_values<VEC, 16>(y + row[u] * ldy + col[u], v);
        }
    }
}

// Calls f(first row, rows, segments, grid) for pieces of fewer than 2^31 segments (one piece, but for
// operands beyond 2^39 elements).
template <typename F>
cudaError_t for_rows(int64_t R, int64_t K, F f) {
    const int64_t nseg = (K + kSeg - 1) / kSeg, most = 0x3fffffff / nseg;
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
        const bool vec = rows_aligned(x, ldx, sizeof(T));
        auto kern = trigger ? (vec ? mx4_quantize_kernel<true, true, T> : mx4_quantize_kernel<false, true, T>)
                            : (vec ? mx4_quantize_kernel<true, false, T> : mx4_quantize_kernel<false, false, T>);
        return for_rows(R, K, [&](int64_t r, uint32_t items, FastDiv nseg, dim3 grid) {
            return launch_pdl(kern, grid, kThreads, 0, s, static_cast<const T *>(x), items, nseg, K, ldx, codes, scales, r);
        });
    });
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K, qmm_dtype t, void *y,
                                  int64_t ldy, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using T = decltype(z);
        const bool vec = rows_aligned(y, ldy, sizeof(T));
        auto kern = vec ? mx4_dequantize_kernel<true, T> : mx4_dequantize_kernel<false, T>;
        return for_rows(R, K, [&](int64_t r, uint32_t items, FastDiv nseg, dim3 grid) {
            return launch_pdl(kern, grid, kThreads, 0, s, codes, scales, items, nseg, K, static_cast<T *>(y), ldy, r);
        });
    });
}

QMM_DCHECK_READER(read_dcheck_mx4)

}  // namespace qmm
