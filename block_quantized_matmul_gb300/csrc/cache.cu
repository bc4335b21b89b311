// cache.cu -- keys and values quantized as they are written into the paged cache (cache.cuh), and read
// back from it.
//
// The rules are those of the library's Q8_0 activations and Q4_0 weights, but that the Q8_0 scale is
// max|x| times the fp32 nearest to 1/127; a block is 32 elements of one head of one token.  A block whose scale is not a finite fp16 (an infinity or a NaN among its
// elements, or values beyond the format) is stored with a NaN scale and reads back as NaN, so that
// nothing turns into a finite value on the way.  Both kernels move each byte once and are bound by
// memory: four lanes to a block, 8 elements to a lane.
#include "cache.cuh"
#include "elem.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr float kInv127 = 1.0f / 127.0f;    // rounded once: the Q8_0 scale is a product, not a quotient

// Codes of a lane's 8 elements and the block's scale; the four lanes of a block call it together.
// Q8_0: 8 int8 codes in w[0..1].  Q4_0: nibbles, element i in nibble i of w[0].
template <int TYPE>
__device__ __forceinline__ uint16_t quantize8(const float (&v)[8], uint32_t (&w)[2]) {
    float top = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        top = fmaxf(top, fabsf(v[i]));
        nan |= isnan(v[i]);
    }
    if (nan) top = INFINITY;
    float d, id;
    if constexpr (TYPE == QMM_Q8_0) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        d = __fmul_rn(top, kInv127);
    } else {
        // the signed element of largest magnitude, the first one on ties
        float m = top;
        bool found = false;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!found && fabsf(v[i]) == top) {
                m = v[i];
                found = true;
            }
        const unsigned lane = threadIdx.x & 31u;
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            const float other_top = __shfl_xor_sync(0xffffffffu, top, o), other_m = __shfl_xor_sync(0xffffffffu, m, o);
            if (other_top > top || (other_top == top && (lane & o))) {
                top = other_top;
                m = other_m;
            }
        }
        d = __fdiv_rn(m, -8.0f);
    }
    uint16_t half = __half_as_ushort(__float2half_rn(d));
    const bool fine = (half & 0x7C00u) != 0x7C00u && top < INFINITY;
    id = inv_or_zero(d);
    w[0] = w[1] = 0;
    if (!fine) return 0x7E00u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (TYPE == QMM_Q8_0) {
            w[i >> 2] |= (uint32_t)(q8_code(v[i], id) & 0xFF) << (8 * (i & 3));
        } else {
            const float q = __fadd_rn(__fmul_rn(v[i], id), 8.5f);
            const int c = !(q >= 0.0f) ? 0 : (q >= 15.0f ? 15 : __float2int_rz(q));
            w[0] |= (uint32_t)c << (4 * i);
        }
    }
    return half;
}

// The 4 bytes of nibble pairs of elements 4 at a time: low nibbles of `lo` (elements j..j+3 from its
// 16 bits at shift) under the nibbles of `hi`.
__device__ __forceinline__ uint32_t interleave4(uint32_t lo, uint32_t hi) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= (((lo >> (4 * i)) & 15u) | (((hi >> (4 * i)) & 15u) << 4)) << (8 * i);
    return r;
}

struct WriteParams {
    const void *src[2];
    uint8_t *cache[2];
    int64_t ld[2];
    const int64_t *slots;
    int64_t T, n_slots;
    int H, D, P;
};

// One thread per 8 elements; blockIdx.y: 0 keys, 1 values.
template <int TYPE, bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int which = blockIdx.y;
    const T *src = static_cast<const T *>(p.src[which]);
    uint8_t *cache = p.cache[which];
    const int per_head = p.D / 8, per_tok = p.H * per_head;
    const int64_t total = p.T * per_tok;
    const int cb = cache_code_bytes(TYPE, p.D);
    // total is a multiple of 4 and so is every warp's first index: the four lanes of a block are all
    // in range or all out of it, and all 32 lanes stay in the loop for the shuffles
    for (int64_t base = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31u); base < total; base += (int64_t)gridDim.x * kThreads) {
        const int64_t i = base + (threadIdx.x & 31u);
        const bool in = i < total;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        int64_t slot = -1;
        int h = 0, c = 0;
        if (in) {
            const int64_t tok = i / per_tok;
            const int rest = (int)(i - tok * per_tok);
            h = rest / per_head;
            c = rest - h * per_head;                       // elements 8c .. 8c + 7 of the head
            slot = p.slots[tok];
            if (slot >= p.n_slots) slot = -1;
            if (slot >= 0) load8<VEC>(src + tok * p.ld[which] + (int64_t)h * p.D + 8 * c, v);
        }
        uint32_t w[2];
        const uint16_t d = quantize8<TYPE>(v, w);
        uint32_t other = 0;
        if constexpr (TYPE == QMM_Q4_0) other = __shfl_xor_sync(0xffffffffu, w[0], 2);
        if (slot < 0 || !QMM_DCHECK(h < p.H && 8 * c + 8 <= p.D)) continue;
        const int64_t page = slot / p.P;
        const int off = (int)(slot - page * p.P);
        uint8_t *chunk = cache + cache_chunk(TYPE, p.H, p.D, p.P, page, h);
        if constexpr (TYPE == QMM_Q8_0) {
            *reinterpret_cast<uint2 *>(chunk + (int64_t)off * cb + 8 * c) = make_uint2(w[0], w[1]);
        } else {
            // lanes 0, 1 hold elements 0..15 of the block, lanes 2, 3 elements 16..31; bytes 8 (lane & 1)
            // .. + 7 pair them: the lower lane writes the first four, the upper lane the others
            const bool upper = (c & 2) != 0;
            const uint32_t lo = upper ? other : w[0], hi = upper ? w[0] : other;
            const uint32_t word = upper ? interleave4(lo >> 16, hi >> 16) : interleave4(lo, hi);
            *reinterpret_cast<uint32_t *>(chunk + (int64_t)off * cb + (c >> 2) * 16 + (c & 1) * 8 + (upper ? 4 : 0)) = word;
        }
        if ((c & 3) == 0)
            *reinterpret_cast<uint16_t *>(chunk + (int64_t)p.P * cb + ((int64_t)off * (p.D / 32) + (c >> 2)) * 2) = d;
    }
}

struct ReadParams {
    const uint8_t *cache[2];
    void *dst[2];
    int64_t ld[2];
    const int32_t *pages;
    int64_t ld_pages, n_pages;
    const int32_t *starts;
    int64_t n_seq, T;
    int H, D, P;
};

// The sequence that token t of the concatenated ones belongs to: the last s with starts[s] <= t.
__device__ __forceinline__ int64_t find_seq(const int32_t *starts, int64_t n_seq, int64_t t) {
    int64_t lo = 0, hi = n_seq - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One thread per 8 elements; blockIdx.y: 0 keys, 1 values.  A token that no valid page holds reads as 0.
template <int TYPE, bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int which = blockIdx.y;
    const uint8_t *cache = p.cache[which];
    T *dst = static_cast<T *>(p.dst[which]);
    if (!dst) return;
    const int per_head = p.D / 8, per_tok = p.H * per_head;
    const int64_t total = p.T * per_tok;
    const int cb = cache_code_bytes(TYPE, p.D);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t tok = i / per_tok;
        const int rest = (int)(i - tok * per_tok);
        const int h = rest / per_head, c = rest - h * per_head;
        const int64_t s = find_seq(p.starts, p.n_seq, tok);
        const int64_t pos = tok - p.starts[s], pi = pos / p.P;
        const int64_t page = pos >= 0 && pi < p.ld_pages ? p.pages[s * p.ld_pages + pi] : -1;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (page >= 0 && page < p.n_pages) {
            const int off = (int)(pos - pi * p.P);
            const uint8_t *chunk = cache + cache_chunk(TYPE, p.H, p.D, p.P, page, h);
            const float d = __half2float(__ushort_as_half(
                *reinterpret_cast<const uint16_t *>(chunk + (int64_t)p.P * cb + ((int64_t)off * (p.D / 32) + (c >> 2)) * 2)));
            if constexpr (TYPE == QMM_Q8_0) {
                const uint2 w = *reinterpret_cast<const uint2 *>(chunk + (int64_t)off * cb + 8 * c);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = d * (float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(chunk + (int64_t)off * cb + (c >> 2) * 16 + (c & 1) * 8);
                const int sh = (c & 2) ? 4 : 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = d * (float)((int)(((j < 4 ? w.x : w.y) >> (8 * (j & 3) + sh)) & 15u) - 8);
            }
        }
        store8<VEC>(dst + tok * p.ld[which] + (int64_t)h * p.D + 8 * c, v);
    }
}

unsigned grid_for(int64_t work) {
    const int64_t g = (work + kThreads - 1) / kThreads;
    return (unsigned)(g > 152 * 8 ? 152 * 8 : (g < 1 ? 1 : g));
}
bool vec_ok(const void *p, int64_t ld, size_t es) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0; }

}  // namespace

cudaError_t launch_cache_write(qmm_type type, qmm_dtype t, const void *k, const void *v, int64_t ldk, int64_t ldv, int64_t T,
                               int H, int D, const int64_t *slots, uint8_t *k_cache, uint8_t *v_cache, int64_t n_pages, int P,
                               cudaStream_t s) {
    const WriteParams p{{k, v}, {k_cache, v_cache}, {ldk, ldv}, slots, T, n_pages * P, H, D, P};
    return with_dtype(t, [&](auto z) {
        using E = decltype(z);
        const bool vec = vec_ok(k, ldk, sizeof(E)) && vec_ok(v, ldv, sizeof(E));
        auto kern = type == QMM_Q8_0 ? (vec ? cache_write_kernel<QMM_Q8_0, true, E> : cache_write_kernel<QMM_Q8_0, false, E>)
                                     : (vec ? cache_write_kernel<QMM_Q4_0, true, E> : cache_write_kernel<QMM_Q4_0, false, E>);
        return launch_pdl(kern, dim3(grid_for(T * H * (D / 8)), 2), kThreads, 0, s, p);
    });
}

cudaError_t launch_cache_read(qmm_type type, const uint8_t *k_cache, const uint8_t *v_cache, int64_t n_pages, int P, int H, int D,
                              const int32_t *pages, int64_t ld_pages, const int32_t *starts, int64_t n_seq, int64_t T, qmm_dtype t,
                              void *k, void *v, int64_t ldk, int64_t ldv, cudaStream_t s) {
    const ReadParams p{{k_cache, v_cache}, {k, v}, {ldk, ldv}, pages, ld_pages, n_pages, starts, n_seq, T, H, D, P};
    return with_dtype(t, [&](auto z) {
        using E = decltype(z);
        const bool vec = (!k || vec_ok(k, ldk, sizeof(E))) && (!v || vec_ok(v, ldv, sizeof(E)));
        auto kern = type == QMM_Q8_0 ? (vec ? cache_read_kernel<QMM_Q8_0, true, E> : cache_read_kernel<QMM_Q8_0, false, E>)
                                     : (vec ? cache_read_kernel<QMM_Q4_0, true, E> : cache_read_kernel<QMM_Q4_0, false, E>);
        return launch_pdl(kern, dim3(grid_for(T * H * (D / 8)), 2), kThreads, 0, s, p);
    });
}

QMM_DCHECK_READER(read_dcheck_cache)

}  // namespace qmm
