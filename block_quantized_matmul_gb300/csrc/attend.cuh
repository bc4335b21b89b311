// attend.cuh -- what the kernels of the attention over the block-quantized cache share: their parameters, which
// rows and keys a CTA works on, where its results go, and the plain loop for caches that hold infinities
// or NaN.
#pragma once

#include "cache.cuh"
#include "elem.cuh"
#include "pipeline.cuh"
#include "tc_common.cuh"

namespace qmm {

constexpr float kBias = 14.0f;             // p is kept times 2^14

struct AttendParams {
    const uint8_t *k_cache, *v_cache;
    int64_t n_pages;
    int P, log_p, H, group, tile_rows, row_tiles, splits;
    int64_t chunk;                         // keys of a split
    const int32_t *pages;
    int64_t ld_pages;
    const int32_t *q_starts, *kv_lens;
    int64_t n_seq, T, ldq, ldo;
    const void *q;
    const uint64_t *tree;
    float scale;
    int bf16;
    void *out;
    float *lse;
    float *part_o, *part_ml;               // [splits][T * Hq][D], [splits][T * Hq][2]
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) { return tc::h2_bits(__hmul2(tc::bits_h2(a), tc::bits_h2(b))); }
// Ones in the halves of d that are finite.
__device__ __forceinline__ uint32_t finite2(uint32_t d) { return __hlt2_mask(__habs2(tc::bits_h2(d)), tc::bits_h2(0x7C007C00u)); }
constexpr int kSorted = 128;               // sequences up to which a CTA sorts them itself

struct Rows {                              // what a CTA works on
    int64_t s, q0, nq, n, first, k0, k1;
    int h, r0, rows, sp, used;
};

// The CTA's rows and keys, from its index: splits fastest, then row tiles, heads, sequences.  False: it has
// none.  `scratch`: kSorted + 1 ints of shared memory, free again on return.
template <int ROWS>
__device__ __forceinline__ bool find_rows(const AttendParams &p, int *scratch, int threads, Rows &w) {
    uint32_t at = blockIdx.x;
    w.sp = (int)(at % (uint32_t)p.splits);
    at /= (uint32_t)p.splits;
    const int rt = (int)(at % (uint32_t)p.row_tiles);
    at /= (uint32_t)p.row_tiles;
    w.h = (int)(at % (uint32_t)p.H);
    w.s = at / (uint32_t)p.H;
    if (p.n_seq > 1 && p.n_seq <= kSorted) {
        // the longest sequences first: what is started last is then short, and the SMs end together
        int *found = scratch + kSorted;
        for (int i = threadIdx.x; i < (int)p.n_seq; i += threads) scratch[i] = p.kv_lens[i];
        __syncthreads();
        for (int i = threadIdx.x; i < (int)p.n_seq; i += threads) {
            const int n = scratch[i];
            int before = 0;
            for (int j = 0; j < (int)p.n_seq; ++j) before += scratch[j] > n || (scratch[j] == n && j < i);
            if (before == (int)w.s) *found = i;
        }
        __syncthreads();
        w.s = *found;
        __syncthreads();
    }
    w.q0 = p.q_starts[w.s];
    w.nq = p.q_starts[w.s + 1] - w.q0;
    w.n = p.kv_lens[w.s];
    w.r0 = rt * ROWS;
    w.rows = (int)min((int64_t)ROWS, w.nq * p.group - w.r0);
    if (w.rows <= 0) return false;
    w.first = w.n - w.nq;
    w.n = max((int64_t)0, min(w.n, p.ld_pages << p.log_p));
    w.used = (int)min((int64_t)p.splits, max((int64_t)1, (w.n + p.chunk - 1) / p.chunk));
    if (w.sp >= w.used) return false;
    w.k0 = w.sp * p.chunk;
    w.k1 = w.sp == p.splits - 1 ? w.n : min(w.n, w.k0 + p.chunk);
    return true;
}

__device__ __forceinline__ float load_q(const AttendParams &p, int64_t at) {
    return p.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[at]) : __half2float(static_cast<const __half *>(p.q)[at]);
}
__device__ __forceinline__ void store_out(const AttendParams &p, int64_t at, float v) {
    if (p.bf16) float_to_elem(v, static_cast<__nv_bfloat16 *>(p.out)[at]);
    else float_to_elem(v, static_cast<__half *>(p.out)[at]);
}

// Token i of the sequence sees the new token b.
__device__ __forceinline__ bool sees(const uint64_t *tree, int64_t tok, int i, int64_t b) {
    return tree ? b < 64 && ((tree[tok] >> b) & 1) : b <= i;
}

// Where N consecutive elements of a row's result go: the output when its sequence is not split, else this
// split's partial.
template <int N>
__device__ __forceinline__ void write_row(const AttendParams &p, const Rows &w, int D, int row, int d, const float (&o)[N], float top,
                                          float sum) {
    const int r = w.r0 + row, i = r / p.group, hq = w.h * p.group + (r - i * p.group), Hq = p.H * p.group;
    const int64_t at = (w.q0 + i) * Hq + hq;
    if (w.used == 1) {
        const int64_t to = (w.q0 + i) * p.ldo + (int64_t)hq * D + d;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if constexpr (N == 4) {
            const float a = o[0] * inv, b = o[1] * inv, c = o[2] * inv, e = o[3] * inv;
            uint16_t *q = static_cast<uint16_t *>(p.out) + to;   // 8-byte aligned
            *reinterpret_cast<uint2 *>(q) = p.bf16 ? make_uint2(pack2(a, b, __nv_bfloat16{}), pack2(c, e, __nv_bfloat16{}))
                                                   : make_uint2(pack2(a, b, __half{}), pack2(c, e, __half{}));
        } else {
            store_out(p, to, o[0] * inv);
        }
        if (d == 0 && p.lse) p.lse[at] = sum == 0.0f ? -INFINITY : (top + __log2f(sum) - kBias) * 0.6931471805599453f;
    } else {
        const int64_t part = (int64_t)w.sp * p.T * Hq + at;
        if constexpr (N == 4) *reinterpret_cast<float4 *>(p.part_o + part * D + d) = make_float4(o[0], o[1], o[2], o[3]);
        else p.part_o[part * D + d] = o[0];
        if (d == 0) {
            p.part_ml[2 * part] = top;
            p.part_ml[2 * part + 1] = sum;
        }
    }
}

template <int TYPE>
__device__ __forceinline__ float cache_value(const uint8_t *chunk, int P, int D, int off, int e) {
    const int cb = cache_code_bytes(TYPE, D);
    const float d = __half2float(
        __ushort_as_half(*reinterpret_cast<const uint16_t *>(chunk + (int64_t)P * cb + ((int64_t)off * (D / 32) + e / 32) * 2)));
    if constexpr (TYPE == QMM_Q8_0) return d * (float)(int8_t)chunk[(int64_t)off * cb + e];
    const uint32_t b = chunk[(int64_t)off * cb + e / 32 * 16 + e % 16];
    return d * (float)((int)((e % 32 < 16 ? b : b >> 4) & 15u) - 8);
}

// The CTA's rows and keys once more, a warp a row, skipping what the row does not see; rows whose result
// is finite, and was, keep the one they have.
template <int TYPE, int DB, int WARPS>
__device__ __noinline__ void rows_one_by_one(const AttendParams &p, const Rows &w, const int *row_bad) {
    const int lane = threadIdx.x & 31;
    constexpr int D = DB * 32;
    for (int row = threadIdx.x >> 5; row < w.rows; row += WARPS) {
        const int r = w.r0 + row, i = r / p.group, hq = w.h * p.group + r % p.group;
        float q[DB], o[DB];
#pragma unroll
        for (int b = 0; b < DB; ++b) {
            q[b] = load_q(p, (w.q0 + i) * p.ldq + (int64_t)hq * D + 32 * b + lane);
            o[b] = 0.0f;
        }
        float top = -INFINITY, sum = 0.0f;                      // in powers of two
        for (int64_t j = w.k0; j < w.k1; ++j) {
            if (j >= w.first && !sees(p.tree, w.q0 + i, i, j - w.first)) continue;
            const int64_t page = p.pages[w.s * p.ld_pages + (j >> p.log_p)];
            if (page < 0 || page >= p.n_pages) continue;
            const int64_t at = cache_chunk(TYPE, p.H, D, p.P, page, w.h);
            const int off = (int)(j & (p.P - 1));
            float x = 0.0f;
#pragma unroll
            for (int b = 0; b < DB; ++b) x += q[b] * cache_value<TYPE>(p.k_cache + at, p.P, D, off, 32 * b + lane);
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
            x *= p.scale * 1.4426950408889634f;
            const float m = fmaxf(top, x), base = m == -INFINITY ? 0.0f : m;
            const float down = exp2f(top - base), e = exp2f(x - base + kBias);
            top = m;
            sum = sum * down + e;
#pragma unroll
            for (int b = 0; b < DB; ++b) o[b] = o[b] * down + e * cache_value<TYPE>(p.v_cache + at, p.P, D, off, 32 * b + lane);
        }
        bool fine = sum < INFINITY && !row_bad[row];
#pragma unroll
        for (int b = 0; b < DB; ++b) fine = fine && fabsf(o[b]) < INFINITY;
        if (__all_sync(0xffffffffu, fine)) continue;
#pragma unroll
        for (int b = 0; b < DB; ++b) {
            const float v[1] = {o[b]};
            write_row(p, w, D, row, 32 * b + lane, v, top, sum);
        }
    }
}

// More than kMaxMmaRows rows of up to 128 elements (attend_tc.cu): 128 rows to a CTA, one CTA an SM.
constexpr int kTcRows = 128;
cudaError_t launch_attend_tc(qmm_type type, const AttendParams &p, int DB, int64_t ctas, cudaStream_t s);
cudaError_t read_and_clear_attend_status(unsigned *out, cudaStream_t s);
cudaError_t read_dcheck_attend_tc(unsigned *out, cudaStream_t s);

}  // namespace qmm
