// norm.cu -- the norm behind a block, its gate and residual, and the norm before the next block, in one pass:
//   b = w_post ? x / sqrt(mean(x^2) + eps) * w_post : x,   h' = round(h + scale * gate * b),
//   y = h' / sqrt(mean(h'^2) + eps) * w_pre,
// with y as rows, as Q8_0 blocks or as MX4 blocks.
//
// x, h and gate are read once and h' and y written once: a row stays on the SM from its load to its last store.  Each thread
// holds C pieces of 8 consecutive elements, so that four neighbouring threads hold a block of 32.  Rows of up to 1024 elements take
// a warp each, longer ones a CTA; what a thread does once a row (sums, roots, addresses) is about 150 instructions, so it
// takes 16 elements where rows are many.
#include "qmm_internal.cuh"

#include "elem.cuh"
#include "mx4.cuh"

namespace qmm {
namespace {

// Eight elements of a row as they lie in memory (16 bits: the first four words), converted once they are needed.
struct Raw8 {
    uint32_t w[8];
};

// Elements at .. at + 7 of a row of n (those past its end as 0); VEC: 32-byte aligned rows, and all there.
template <bool VEC>
__device__ __forceinline__ void load8(Raw8 &r, const void *row, int type, int at, int n) {
    if constexpr (VEC) {
        if (type == QMM_F32) {
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(row) + at);
            const uint4 a = q[0], b = q[1];
            r = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + at);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        }
    } else if (type == QMM_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = at + i < n ? static_cast<const uint32_t *>(row)[at + i] : 0u;
    } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = at + i < n ? static_cast<const uint16_t *>(row)[at + i] : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = e[2 * i] | e[2 * i + 1] << 16;
    }
}

// The branches on the type are taken for eight elements at a time: selects in their place, element by element, cost three
// times the instructions of everything else.
__device__ __forceinline__ void values8(float (&v)[8], const Raw8 &r, int type) {
    if (type == QMM_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
        }
    } else if (type == QMM_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(r.w[i], __half{});
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// v rounded to the type, as it will lie in memory.
__device__ __forceinline__ void round8(Raw8 &r, const float (&v)[8], int type) {
    if (type == QMM_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = pack2(v[2 * i], v[2 * i + 1], __nv_bfloat16{});
    } else if (type == QMM_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = pack2(v[2 * i], v[2 * i + 1], __half{});
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(const Raw8 &r, void *row, int type, int at, int n) {
    if constexpr (VEC) {
        if (type == QMM_F32) {
            uint4 *q = reinterpret_cast<uint4 *>(static_cast<float *>(row) + at);
            q[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
            q[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + at) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        }
    } else if (type == QMM_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i < n) static_cast<uint32_t *>(row)[at + i] = r.w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i < n) static_cast<uint16_t *>(row)[at + i] = (uint16_t)(r.w[i >> 1] >> (16 * (i & 1)));
    }
}

__device__ __forceinline__ const void *row_of(const void *p, int type, int64_t at) {
    return static_cast<const uint8_t *>(p) + at * (type == QMM_F32 ? 4 : 2);
}

// 1 / sqrt(v): the hardware's approximation and one step of Newton's iteration, within two roundings, where every thread would
// take forty instructions for a root and a division.  (v = 0 gives infinity, an infinite v 0.)
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v), e = fmaf(-v * r, r, 1.0f);
    return v > 0.0f && v < INFINITY ? fmaf(0.5f * r, e, r) : r;
}

// The sum over the threads of a row.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *part) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        const int lane = threadIdx.x & 31;
        if (lane == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < kWarps ? part[lane] : 0.0f;
#pragma unroll
        for (int m = kWarps / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        v = __shfl_sync(0xffffffffu, v, 0);
    }
    return v;
}

// TPR threads take a row, C pieces of 8 elements each.  TYPES: of x, h and y, where the compiler knows them (9 x + 3 h + y), or -1.
// 8192 rows of 4096, both norms and a gate, us (bytes at the copy rate): bf16 45 (40), with an fp32 stream 62 (60), to a Q8_0 operand 55 (36), to
// an MX4 operand 47 (33).  With the types as parameters of the launch bf16 takes 65, for branches and unused registers; fp16 rows, which have no
// instance of their own, 66 (40), their operands 74 (36) and 66 (33), fp32 rows 94 (80).  A ring of asynchronous copies under
// CTAs that go on from row to row: 52.
template <int TPR, int C, bool VEC, int TYPES>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_kernel(const NormParams p) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    static_assert(TPR == 32 || kRows == 1, "a row is a warp's or a CTA's");
    __shared__ float part[2][TPR > 32 ? TPR / 32 : 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int xdt = TYPES < 0 ? p.xdt : TYPES / 9, hdt = TYPES < 0 ? p.hdt : TYPES / 3 % 3, ydt = TYPES < 0 ? p.ydt : TYPES % 3;
    const int t = threadIdx.x % TPR, n = p.N;
    const float inv_n = 1.0f / (float)n;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (row >= p.R) return;                                            // (a whole warp)
    const void *hr = row_of(p.h, hdt, row * p.ldh), *xr = p.x ? row_of(p.x, xdt, row * p.ldx) : nullptr;
    const void *gr = p.gate ? row_of(p.gate, xdt, row * p.ldg) : nullptr;
    // of x the pieces are kept as they lie in memory; a thread of 1024 has no registers for four of them, and loads them again
    // (and with the types unknown still keeps 7 to 24 words of them in local memory: rows of more than 16384)
    constexpr bool kKeep = C < 4 || TPR == 32;
    Raw8 rx[kKeep ? C : 1];
    float h[C][8];
    if (kKeep && xr) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if ((c * TPR + t) * 8 < n) load8<VEC>(rx[c], xr, xdt, (c * TPR + t) * 8, n);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * TPR + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = 0.0f;
        if (at >= n) continue;
        Raw8 r;
        load8<VEC>(r, hr, hdt, at, n);
        values8(h[c], r, hdt);
    }
    if (xr) {
        float r = 1.0f;
        if (p.w_post) {
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int at = (c * TPR + t) * 8;
                if (at >= n) continue;
                float x[8];
                if constexpr (!kKeep) load8<VEC>(rx[0], xr, xdt, at, n);
                values8(x, rx[kKeep ? c : 0], xdt);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
            }
            r = inverse_root(row_sum<TPR>(sum, part[0]) * inv_n + p.eps);
        }
        r *= p.scale;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * 8;
            if (at >= n) continue;
            float x[8], w[8];
            Raw8 raw;
            if constexpr (!kKeep) load8<VEC>(rx[0], xr, xdt, at, n);
            values8(x, rx[kKeep ? c : 0], xdt);
            if (p.w_post) {
                load8<VEC>(raw, p.w_post, QMM_F32, at, n);
                values8(w, raw, QMM_F32);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= w[i];
            }
            if (gr) {
                load8<VEC>(raw, gr, xdt, at, n);
                values8(w, raw, xdt);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] += x[i] * r;
        }
    }
    // ---- h' rounded and stored; its sum of squares ----
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * TPR + t) * 8;
        if (at >= n) continue;
        if (p.h_out) {
            Raw8 r;
            round8(r, h[c], hdt);
            if (QMM_DCHECK(!VEC || at + 8 <= n)) store8<VEC>(r, const_cast<void *>(row_of(p.h_out, hdt, row * p.ldho)), hdt, at, n);
            if (hdt != QMM_F32) values8(h[c], r, hdt);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += VEC || at + i < n ? h[c][i] * h[c][i] : 0.0f;
    }
    const float r = inverse_root(row_sum<TPR>(sum, part[1]) * inv_n + p.eps);
    // ---- y ----
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * TPR + t) * 8;
        const bool in = at < n;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        if (in) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(h[c][i], r);
            if (p.w_pre) {
                Raw8 raw;
                load8<VEC>(raw, p.w_pre, QMM_F32, at, n);
                values8(w, raw, QMM_F32);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(y[i], w[i]);
            }
        }
        if (p.form == kNormRows) {
            Raw8 o;
            round8(o, y, ydt);
            if (in) store8<VEC>(o, const_cast<void *>(row_of(p.y, ydt, row * p.ldy)), ydt, at, n);
            continue;
        }
        // the largest magnitude of the block of 32 that four threads hold, by the rule of the operand: Q8_0 passes over NaN in
        // a block that holds anything else, in MX4 it comes out on top
        if (p.form == kNormQ8) {
            float top = fabsf(y[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float d = q8_scale(top), id = inv_or_zero(d);
            uint32_t b[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i >> 2] |= ((uint32_t)q8_code(y[i], id) & 255u) << (8 * (i & 3));
            if (in) {
                *reinterpret_cast<uint2 *>(static_cast<int8_t *>(p.y) + row * n + at) = make_uint2(b[0], b[1]);
                if ((t & 3) == 0) reinterpret_cast<__half *>(p.scales)[row * (n / 32) + at / 32] = __float2half_rn(d);
            }
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t e = mx4_block_scale(top);
            // the scales of four blocks (16 threads) as one word; blocks past n hold 0
            uint32_t word = in ? e << (2 * (t & 12)) : 0u;
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            word |= __shfl_xor_sync(0xffffffffu, word, 8);
            if (in) {
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.y) + (row * n + at) / 2) = mx4_codes8(y, e);
                if ((t & 15) == 0) *reinterpret_cast<uint32_t *>(p.scales + mx4_scale_word(row, at >> 7, (n + 127) / 128)) = word;
            }
        }
    }
}

template <int TPR, int C, int TYPES>
cudaError_t launch_typed(const NormParams &p, bool vec, cudaStream_t s) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1, kThreads = TPR < 256 ? 256 : TPR;
    const int64_t grid = (p.R + kRows - 1) / kRows;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl(vec ? norm_kernel<TPR, C, true, TYPES> : norm_kernel<TPR, C, false, -1>, dim3((unsigned)grid), kThreads, 0, s, p);
}
template <int TPR, int C>
cudaError_t launch_rows(const NormParams &p, bool vec, cudaStream_t s) {
    // many rows of bf16, with a residual stream of either kind; few rows are bound by latency
    constexpr int kBf16 = QMM_BF16 * 13, kBf16Stream32 = QMM_BF16 * 9 + QMM_F32 * 3 + QMM_BF16;
    if (vec && p.R > 152) {
        const bool y16 = p.form != kNormRows || p.ydt == QMM_BF16, x16 = !p.x || p.xdt == QMM_BF16;
        if (x16 && y16 && p.hdt == QMM_BF16) return launch_typed<TPR, C, kBf16>(p, vec, s);
        if (x16 && y16 && p.hdt == QMM_F32) return launch_typed<TPR, C, kBf16Stream32>(p, vec, s);
    }
    return launch_typed<TPR, C, -1>(p, vec, s);
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, cudaStream_t s) {
    auto fits = [&](const void *q, int type, int64_t ld) { return !q || rows_aligned(q, ld, type == QMM_F32 ? 4 : 2); };
    const bool vec = p.N % 8 == 0 && fits(p.x, p.xdt, p.ldx) && fits(p.h, p.hdt, p.ldh) && fits(p.gate, p.xdt, p.ldg) &&
                     fits(p.h_out, p.hdt, p.ldho) && fits(p.w_post, QMM_F32, 0) && fits(p.w_pre, QMM_F32, 0) &&
                     (p.form != kNormRows || fits(p.y, p.ydt, p.ldy));
    if (p.N <= 256) return launch_rows<32, 1>(p, vec, s);
    if (p.N <= 512) return launch_rows<32, 2>(p, vec, s);
    if (p.N <= 1024) return launch_rows<32, 4>(p, vec, s);
    if (p.N <= 2048) return launch_rows<256, 1>(p, vec, s);
    if (p.N <= 4096) return p.R <= 152 ? launch_rows<512, 1>(p, vec, s) : launch_rows<256, 2>(p, vec, s);
    if (p.N <= 8192) return p.R <= 152 ? launch_rows<1024, 1>(p, vec, s) : launch_rows<512, 2>(p, vec, s);
    if (p.N <= 16384) return launch_rows<1024, 2>(p, vec, s);
    return launch_rows<1024, 4>(p, vec, s);
}

QMM_DCHECK_READER(read_dcheck_norm)

}  // namespace qmm
