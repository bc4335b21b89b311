// mx4_gemm.cu -- the product of two microscaled 4-bit operands (mx4.cuh).
//
//   Y[m, n] = sum_b 2^(ea[m, b] + ew[n, b] - 254) * sum_{j < 32} a[m, 32b + j] * w[n, 32b + j]
//
// One thread an output; the lanes of a warp take consecutive n.
#include "qmm_internal.cuh"

#include "elem.cuh"
#include "mx4.cuh"

namespace qmm {
namespace {

template <typename T>
__global__ void __launch_bounds__(256) mx4_matmul_kernel(const uint8_t *__restrict__ wc, const uint8_t *__restrict__ ws, int64_t K,
                                                         int64_t N, const uint8_t *__restrict__ ac,
                                                         const uint8_t *__restrict__ as, int64_t M, T *__restrict__ y,
                                                         int64_t ldy) {
    const int64_t n128 = (K + 127) / 128;
    const int64_t n = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    for (int64_t m = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); m < M; m += (int64_t)gridDim.y * 8) {
        if (n >= N) break;
        float acc = 0.0f;
        for (int64_t b = 0; b < K / 32; ++b) {
            const uint4 a4 = *reinterpret_cast<const uint4 *>(ac + m * (K / 2) + b * 16);
            const uint4 w4 = *reinterpret_cast<const uint4 *>(wc + n * (K / 2) + b * 16);
            const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w}, ww[4] = {w4.x, w4.y, w4.z, w4.w};
            float sum = 0.0f;                                  // exact: multiples of 1/4 below 32 * 36
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float av[8], wv[8];
                mx4_values8(aw[c], av);
                mx4_values8(ww[c], wv);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += av[j] * wv[j];
            }
            const int ea = as[mx4_scale_word(m, b >> 2, n128) + (b & 3)], ew = ws[mx4_scale_word(n, b >> 2, n128) + (b & 3)];
            acc += ea == 255 || ew == 255 ? NAN : ldexpf(sum, ea + ew - 254);   // one exponent: neither factor overflows alone
        }
        float_to_elem(acc, y[m * ldy + n]);
    }
}

}  // namespace

cudaError_t launch_mx4_matmul(const uint8_t *wc, const uint8_t *ws, int64_t K, int64_t N, const uint8_t *ac, const uint8_t *as,
                              int64_t M, qmm_dtype t, void *y, int64_t ldy, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using T = decltype(z);
        const int64_t gm = (M + 7) / 8;
        const dim3 grid((unsigned)((N + 31) / 32), (unsigned)(gm > 65535 ? 65535 : gm));
        mx4_matmul_kernel<T><<<grid, 256, 0, s>>>(wc, ws, K, N, ac, as, M, static_cast<T *>(y), ldy);
        return cudaGetLastError();
    });
}

QMM_DCHECK_READER(read_dcheck_mx4_gemm)

}  // namespace qmm
