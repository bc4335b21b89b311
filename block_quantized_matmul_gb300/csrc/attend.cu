// attend.cu -- attention of a few new tokens of each sequence over the block-quantized cache (cache.cuh).
//
// For new token i of a sequence with n cached tokens, nq of them new, and query head hq (key/value head
// h = hq / (Hq / H)):
//   s_j = scale * sum_d q[i, hq, d] * k[j, h, d]  over the visible j,
//   out[i, hq] = sum_j exp(s_j - max s) v[j, h] / sum_j exp(s_j - max s),   lse = max s + ln(sum);
// j is visible when j < n - nq, or when bit j - (n - nq) of the token's tree word is set (without tree
// words: when j - (n - nq) <= i).  A row that sees nothing is 0 with lse -inf.
//
// One warp a (token, query head): lanes share the head's elements, one pass over the keys with the
// running maximum and sum.
#include "cache.cuh"
#include "elem.cuh"

namespace qmm {
namespace {

constexpr int kWarps = 4;

struct AttendParams {
    const uint8_t *k_cache, *v_cache;
    int64_t n_pages;
    int P, H, D, group;
    const int32_t *pages;
    int64_t ld_pages;
    const int32_t *q_starts, *kv_lens;
    int64_t n_seq, T, ldq, ldo;
    const void *q;
    const uint64_t *tree;
    float scale;
    void *out;
    float *lse;
};

template <int TYPE>
__device__ __forceinline__ float cache_value(const uint8_t *chunk, int P, int D, int off, int e) {
    const int cb = cache_code_bytes(TYPE, D);
    const float d = __half2float(
        __ushort_as_half(*reinterpret_cast<const uint16_t *>(chunk + (int64_t)P * cb + ((int64_t)off * (D / 32) + e / 32) * 2)));
    if constexpr (TYPE == QMM_Q8_0) return d * (float)(int8_t)chunk[(int64_t)off * cb + e];
    const uint32_t b = chunk[(int64_t)off * cb + e / 32 * 16 + e % 16];
    return d * (float)((int)((e % 32 < 16 ? b : b >> 4) & 15u) - 8);
}

template <int TYPE, typename T>
__global__ void __launch_bounds__(kWarps * 32) attend_simple_kernel(const AttendParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t tok = blockIdx.x;
    const int Hq = p.H * p.group, nb = p.D / 32;
    int64_t s = 0;
    while (s + 1 < p.n_seq && p.q_starts[s + 1] <= tok) ++s;
    const int64_t i = tok - p.q_starts[s], nq = p.q_starts[s + 1] - p.q_starts[s];
    if (i < 0 || i >= nq) return;
    int64_t n = p.kv_lens[s];
    const int64_t first = n - nq;
    if (n > p.ld_pages * p.P) n = p.ld_pages * p.P;
    for (int hq = blockIdx.y * kWarps + (threadIdx.x >> 5); hq < Hq; hq += gridDim.y * kWarps) {
        const int h = hq / p.group;
        const T *qp = static_cast<const T *>(p.q) + tok * p.ldq + (int64_t)hq * p.D;
        float q[8], o[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            q[b] = b < nb ? elem_to_float(qp[32 * b + lane]) : 0.0f;
            o[b] = 0.0f;
        }
        float top = -INFINITY, sum = 0.0f;
        for (int64_t j = 0; j < n; ++j) {
            if (j >= first) {
                const int64_t b = j - first;
                if (p.tree ? (b >= 64 || !((p.tree[tok] >> b) & 1)) : b > i) continue;
            }
            const int64_t page = p.pages[s * p.ld_pages + j / p.P];
            if (page < 0 || page >= p.n_pages) continue;
            const int64_t at = cache_chunk(TYPE, p.H, p.D, p.P, page, h);
            const int off = (int)(j % p.P);
            float x = 0.0f;
#pragma unroll
            for (int b = 0; b < 8; ++b)
                if (b < nb) x += q[b] * cache_value<TYPE>(p.k_cache + at, p.P, p.D, off, 32 * b + lane);
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
            x *= p.scale;
            const float m = fmaxf(top, x);
            const float base = m == -INFINITY ? 0.0f : m;
            const float down = __expf(top - base), e = __expf(x - base);
            top = m;
            sum = sum * down + e;
#pragma unroll
            for (int b = 0; b < 8; ++b)
                if (b < nb) o[b] = o[b] * down + e * cache_value<TYPE>(p.v_cache + at, p.P, p.D, off, 32 * b + lane);
        }
        T *op = static_cast<T *>(p.out) + tok * p.ldo + (int64_t)hq * p.D;
#pragma unroll
        for (int b = 0; b < 8; ++b)
            if (b < nb) float_to_elem(sum == 0.0f ? 0.0f : o[b] / sum, op[32 * b + lane]);
        if (p.lse && lane == 0) p.lse[tok * Hq + hq] = sum == 0.0f ? -INFINITY : top + __logf(sum);
    }
}

}  // namespace

size_t attend_workspace_bytes(int64_t, int64_t, int, int, int, int64_t) { return 0; }

cudaError_t launch_cache_attend(qmm_type type, const uint8_t *k_cache, const uint8_t *v_cache, int64_t n_pages, int P, int H, int D,
                                const int32_t *pages, int64_t ld_pages, const int32_t *q_starts, const int32_t *kv_lens,
                                int64_t n_seq, qmm_dtype t, const void *q, int64_t ldq, int64_t T, int Hq, const uint64_t *tree,
                                float scale, int64_t max_new, int64_t max_len, void *out, int64_t ldo, float *lse, void *ws,
                                size_t ws_bytes, cudaStream_t s) {
    const AttendParams p{k_cache, v_cache, n_pages, P, H, D, Hq / H, pages, ld_pages, q_starts, kv_lens, n_seq, T, ldq, ldo, q, tree,
                         scale, out, lse};
    const dim3 grid((unsigned)T, (unsigned)((Hq + kWarps - 1) / kWarps));
    if (type == QMM_Q8_0) {
        if (t == QMM_F16) attend_simple_kernel<QMM_Q8_0, __half><<<grid, kWarps * 32, 0, s>>>(p);
        else attend_simple_kernel<QMM_Q8_0, __nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(p);
    } else {
        if (t == QMM_F16) attend_simple_kernel<QMM_Q4_0, __half><<<grid, kWarps * 32, 0, s>>>(p);
        else attend_simple_kernel<QMM_Q4_0, __nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(p);
    }
    return cudaGetLastError();
}

QMM_DCHECK_READER(read_dcheck_attend)

}  // namespace qmm
