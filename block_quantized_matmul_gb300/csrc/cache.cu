// cache.cu -- keys and values quantized as they are written into the paged cache (cache.cuh), and read
// back from it.
//
// The rules are those of the library's Q8_0 activations and Q4_0 weights, but that the Q8_0 scale is
// max|x| times the fp32 nearest to 1/127; a block is 32 elements of one head of one token.  A block whose scale is not a finite fp16 (an infinity or a NaN among its
// elements, or values beyond the format) is stored with a NaN scale and reads back as NaN, so that
// nothing turns into a finite value on the way.  Both kernels move each byte once and are bound by
// memory: four lanes to a block, 8 elements to a lane.
#include <type_traits>

#include "cache.cuh"
#include "elem.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;                   // pieces of 8 elements that a thread loads before it works on the first
constexpr float kInv127 = 1.0f / 127.0f;    // rounded once: the Q8_0 scale is a product, not a quotient

// The low bits of 2^23 + v rounded towards zero are trunc(v), 0 <= v < 2^23: an addition where a
// conversion would take a slower pipe.
__device__ __forceinline__ uint32_t trunc_bits(float v) { return __float_as_uint(__fadd_rz(v, 8388608.0f)); }

// Codes of a lane's 8 elements and the block's scale; the four lanes of a block (and so, for the
// shuffles, the warp) call it together.  Q8_0: 8 int8 codes in w[0..1].  Q4_0: element i in nibble i of w[0].
template <int TYPE, typename T>
__device__ __forceinline__ uint16_t quantize8(const Raw8<T> &raw, uint32_t (&w)[2]) {
    float v[8];
    raw.values(v);
    uint32_t bits = raw.top_bits();
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 2));
    float d;
    if constexpr (TYPE == QMM_Q8_0) {
        d = __fmul_rn(__uint_as_float(bits), kInv127);
    } else {
        // its sign: the block's first element of that magnitude.  First the lane's own: bit i of at.
        const unsigned group = 0xfu << (threadIdx.x & 28u);
        uint32_t sign = 0;
        bool have = false;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const uint32_t x = __float_as_uint(v[i]);
            if ((x & 0x7FFFFFFFu) == bits) {
                sign = x & 0x80000000u;
                have = true;
            }
        }
        const unsigned holders = __ballot_sync(0xffffffffu, have) & group;
        const int from = holders ? __ffs((int)holders) - 1 : 0;
        sign = __shfl_sync(0xffffffffu, sign, from);
        d = __fmul_rn(__uint_as_float(bits | sign), -0.125f);
    }
    const uint16_t half = __half_as_ushort(__float2half_rn(d));
    w[0] = w[1] = 0;
    if (bits >= 0x7F800000u || (half & 0x7C00u) == 0x7C00u) return 0x7E00u;
    const float id = d != 0.0f ? __frcp_rn(d) : 0.0f;
    if (!(fabsf(id) < INFINITY)) {
        // 1 / d overflows: element by element, with the products' infinities and NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (TYPE == QMM_Q8_0) {
                w[i >> 2] |= (uint32_t)(q8_code(v[i], id) & 0xFF) << (8 * (i & 3));
            } else {
                const float q = __fadd_rn(__fmul_rn(v[i], id), 8.5f);
                w[0] |= (uint32_t)(!(q >= 0.0f) ? 0 : (q >= 15.0f ? 15 : __float2int_rz(q))) << (4 * i);
            }
        }
        return half;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = __fmul_rn(v[i], id);
        if constexpr (TYPE == QMM_Q8_0) {
            // half away from zero: trunc(|q| + 1/2), the sum rounded towards zero so that it cannot reach the next integer
            const uint32_t m = trunc_bits(__fadd_rz(fminf(fabsf(q), 127.0f), 0.5f)), neg = (uint32_t)((int32_t)__float_as_uint(q) >> 31);
            w[i >> 2] |= (((m ^ neg) - neg) & 0xFFu) << (8 * (i & 3));
        } else {
            w[0] |= (trunc_bits(fminf(fmaxf(__fadd_rn(q, 8.5f), 0.0f), 15.0f)) & 15u) << (4 * i);
        }
    }
    return half;
}

// The low 16 bits' four nibbles spread to the low nibbles of four bytes.
__device__ __forceinline__ uint32_t spread4(uint32_t x) {
    x = (x | (x << 8)) & 0x00FF00FFu;
    return (x | (x << 4)) & 0x0F0F0F0Fu;
}

struct WriteParams {
    const void *src[2];
    uint8_t *cache[2];
    int64_t ld[2];
    const int64_t *slots;
    int64_t n_slots;
    uint32_t items;                         // tokens * H * D / 8
    FastDiv per_tok;                        // H * D / 8
    int H, log_p;
};

// Where the pieces of a token are in a cache of heads of 32 * DB elements.
template <int TYPE, int DB>
struct Place {
    static constexpr int kCodes = DB * (TYPE == QMM_Q8_0 ? 32 : 16), kToken = kCodes + DB * 2;
    int64_t chunk;                          // start of the head's chunk
    int off, P;
    __device__ __forceinline__ Place(int64_t slot_page, int h, int H, int off_, int log_p)
        : chunk(((slot_page * H + h) << log_p) * kToken), off(off_), P(1 << log_p) {}
    __device__ __forceinline__ int64_t codes(int block, int in) const { return chunk + (off * kCodes + block * (kCodes / DB) + in); }
    __device__ __forceinline__ int64_t scale(int block) const { return chunk + (P * kCodes + (off * DB + block) * 2); }
};

// A thread takes pieces of 8 elements; blockIdx.y: 0 keys, 1 values.
template <int TYPE, int DB, bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ WriteParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int which = blockIdx.y;
    const T *src = static_cast<const T *>(p.src[which]);
    uint8_t *cache = p.cache[which];
    const uint32_t step = gridDim.x * kThreads;
    // items is a multiple of 4 and so is every warp's first index: the four lanes of a block are all in
    // range or all out of it, and all 32 lanes stay in the loop for the shuffles
    for (uint32_t base = blockIdx.x * kThreads + (threadIdx.x & ~31u); base < p.items; base += step * kBatch) {
        Raw8<T> raw[kBatch];
        int64_t slot[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * step + (threadIdx.x & 31u), tok = p.per_tok(i);
            slot[u] = -1;
            raw[u].zero();
            if (i < p.items) {
                slot[u] = p.slots[tok];
                raw[u].template load<VEC>(src + tok * p.ld[which] + (int64_t)(i - tok * p.per_tok.d) * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * step >= p.items) break;
            const uint32_t i = base + u * step + (threadIdx.x & 31u), in_tok = i - p.per_tok(i) * p.per_tok.d;
            uint32_t w[2];
            const uint16_t d = quantize8<TYPE>(raw[u], w);
            uint32_t other = 0;
            if constexpr (TYPE == QMM_Q4_0) other = __shfl_xor_sync(0xffffffffu, w[0], 2);
            if (slot[u] < 0 || slot[u] >= p.n_slots) continue;
            const int h = (int)(in_tok / (4 * DB)), c = (int)(in_tok % (4 * DB));      // elements 8c .. 8c + 7 of the head
            if (!QMM_DCHECK(h < p.H)) continue;
            const Place<TYPE, DB> at(slot[u] >> p.log_p, h, p.H, (int)(slot[u] & ((1 << p.log_p) - 1)), p.log_p);
            if constexpr (TYPE == QMM_Q8_0) {
                *reinterpret_cast<uint2 *>(cache + at.codes(c >> 2, 8 * (c & 3))) = make_uint2(w[0], w[1]);
            } else {
                // lanes 0, 1 hold elements 0..15 of the block, lanes 2, 3 elements 16..31; bytes 8 (lane & 1)
                // .. + 7 pair them: the lower lane writes the first four, the upper lane the others
                const bool upper = (c & 2) != 0;
                const uint32_t lo = upper ? other >> 16 : w[0], hi = upper ? w[0] >> 16 : other;
                *reinterpret_cast<uint32_t *>(cache + at.codes(c >> 2, (c & 1) * 8 + (upper ? 4 : 0))) =
                    spread4(lo & 0xFFFFu) | (spread4(hi & 0xFFFFu) << 4);
            }
            if ((c & 3) == 0) *reinterpret_cast<uint16_t *>(cache + at.scale(c >> 2)) = d;
        }
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
    FastDiv per_tok;                        // H * D / 8
    int H, log_p;
};
constexpr int kReadTokens = 32;             // tokens a CTA looks up at a time

// The sequence that token t of the concatenated ones belongs to: the last s with starts[s] <= t.
__device__ __forceinline__ int64_t find_seq(const int32_t *starts, int64_t n_seq, int64_t t) {
    int64_t lo = 0, hi = n_seq - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A CTA takes 32 tokens: one warp finds their pages, then a thread takes pieces of 8 elements;
// blockIdx.y: 0 keys, 1 values.  A token that no valid page holds reads as 0.
template <int TYPE, int DB, bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int64_t s_page[kReadTokens];
    __shared__ int s_off[kReadTokens];
    const int which = blockIdx.y;
    const uint8_t *cache = p.cache[which];
    T *dst = static_cast<T *>(p.dst[which]);
    if (!dst) return;
    for (int64_t t0 = (int64_t)blockIdx.x * kReadTokens; t0 < p.T; t0 += (int64_t)gridDim.x * kReadTokens) {
        __syncthreads();
        if (threadIdx.x < kReadTokens) {
            const int64_t tok = t0 + threadIdx.x;
            int64_t page = -1;
            int off = 0;
            if (tok < p.T) {
                const int64_t s = find_seq(p.starts, p.n_seq, tok), pos = tok - p.starts[s], pi = pos >> p.log_p;
                if (pos >= 0 && pi < p.ld_pages) page = p.pages[s * p.ld_pages + pi];
                if (page >= p.n_pages) page = -1;
                off = (int)(pos & ((1 << p.log_p) - 1));
            }
            s_page[threadIdx.x] = page;
            s_off[threadIdx.x] = off;
        }
        __syncthreads();
        const uint32_t items = (uint32_t)min((int64_t)kReadTokens, p.T - t0) * p.per_tok.d;
        for (uint32_t base = threadIdx.x; base < items; base += kThreads * kBatch) {
            uint2 w[kBatch];
            uint16_t d[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t i = base + u * kThreads, tok = p.per_tok(i), in_tok = i - tok * p.per_tok.d;
                // codes and scale of a zero (Q4_0: 8 is 0)
                w[u] = TYPE == QMM_Q8_0 ? make_uint2(0u, 0u) : make_uint2(0x88888888u, 0x88888888u);
                d[u] = 0;
                if (i < items && s_page[tok] >= 0) {
                    const int h = (int)(in_tok / (4 * DB)), c = (int)(in_tok % (4 * DB));
                    const Place<TYPE, DB> at(s_page[tok], h, p.H, s_off[tok], p.log_p);
                    d[u] = *reinterpret_cast<const uint16_t *>(cache + at.scale(c >> 2));
                    w[u] = *reinterpret_cast<const uint2 *>(cache + at.codes(c >> 2, 8 * (TYPE == QMM_Q8_0 ? c & 3 : c & 1)));
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t i = base + u * kThreads, tok = p.per_tok(i), in_tok = i - tok * p.per_tok.d;
                if (i >= items) break;
                const float s = __half2float(__ushort_as_half(d[u]));
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t x = j < 4 ? w[u].x : w[u].y;
                    // 2^23 + 128 + q (or + q) is exact, and so is the difference
                    if constexpr (TYPE == QMM_Q8_0) {
                        v[j] = s * (__uint_as_float(__byte_perm(x ^ 0x80808080u, 0x4B000000u, 0x7440 | (j & 3))) - 8388736.0f);
                    } else {
                        const uint32_t q = (x >> (8 * (j & 3) + ((in_tok & 2) ? 4 : 0))) & 15u;
                        v[j] = s * (__uint_as_float(q | 0x4B000000u) - 8388616.0f);
                    }
                }
                store8<VEC>(dst + (t0 + tok) * p.ld[which] + (int64_t)in_tok * 8, v);
            }
        }
    }
}

unsigned grid_for(int64_t work, int64_t per_cta) {
    const int64_t g = (work + per_cta - 1) / per_cta;
    return (unsigned)(g > 152 * 8 ? 152 * 8 : (g < 1 ? 1 : g));
}
bool vec_ok(const void *p, int64_t ld, size_t es) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0; }

}  // namespace

namespace {

// Calls f with the head size in blocks of 32 as a constant.
template <typename F>
cudaError_t with_blocks(int DB, F f) {
    switch (DB) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 5: return f(std::integral_constant<int, 5>{});
        case 6: return f(std::integral_constant<int, 6>{});
        case 7: return f(std::integral_constant<int, 7>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}

template <int TYPE>
cudaError_t write_typed(qmm_dtype t, int DB, bool vec, WriteParams p, int64_t T, const void *k, const void *v, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using E = decltype(z);
        return with_blocks(DB, [&](auto b) {
            constexpr int N = decltype(b)::value;
            auto kern = vec ? cache_write_kernel<TYPE, N, true, E> : cache_write_kernel<TYPE, N, false, E>;
            // pieces are counted in 31 bits: more tokens go in several launches
            const int64_t most = 0x3fffffff / p.per_tok.d;
            WriteParams q = p;
            for (int64_t t0 = 0; t0 < T; t0 += most) {
                const int64_t n = T - t0 < most ? T - t0 : most;
                q.src[0] = static_cast<const E *>(k) + t0 * p.ld[0];
                q.src[1] = static_cast<const E *>(v) + t0 * p.ld[1];
                q.slots = p.slots + t0;
                q.items = (uint32_t)n * p.per_tok.d;
                const cudaError_t e = launch_pdl(kern, dim3(grid_for(q.items, kThreads), 2), kThreads, 0, s, q);
                if (e != cudaSuccess) return e;
            }
            return cudaSuccess;
        });
    });
}

template <int TYPE>
cudaError_t read_typed(qmm_dtype t, int DB, bool vec, const ReadParams &p, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using E = decltype(z);
        return with_blocks(DB, [&](auto b) {
            constexpr int N = decltype(b)::value;
            auto kern = vec ? cache_read_kernel<TYPE, N, true, E> : cache_read_kernel<TYPE, N, false, E>;
            return launch_pdl(kern, dim3(grid_for(p.T, kReadTokens), 2), kThreads, 0, s, p);
        });
    });
}

int log2_of(int P) {
    int l = 0;
    while ((1 << l) < P) ++l;
    return l;
}

}  // namespace

cudaError_t launch_cache_write(qmm_type type, qmm_dtype t, const void *k, const void *v, int64_t ldk, int64_t ldv, int64_t T,
                               int H, int D, const int64_t *slots, uint8_t *k_cache, uint8_t *v_cache, int64_t n_pages, int P,
                               cudaStream_t s) {
    const size_t es = dtype_bytes(t);
    const bool vec = vec_ok(k, ldk, es) && vec_ok(v, ldv, es);
    const WriteParams p{{k, v}, {k_cache, v_cache}, {ldk, ldv}, slots, n_pages * P, 0, FastDiv((uint32_t)(H * (D / 8))), H, log2_of(P)};
    return type == QMM_Q8_0 ? write_typed<QMM_Q8_0>(t, D / 32, vec, p, T, k, v, s) : write_typed<QMM_Q4_0>(t, D / 32, vec, p, T, k, v, s);
}

cudaError_t launch_cache_read(qmm_type type, const uint8_t *k_cache, const uint8_t *v_cache, int64_t n_pages, int P, int H, int D,
                              const int32_t *pages, int64_t ld_pages, const int32_t *starts, int64_t n_seq, int64_t T, qmm_dtype t,
                              void *k, void *v, int64_t ldk, int64_t ldv, cudaStream_t s) {
    const size_t es = dtype_bytes(t);
    const bool vec = (!k || vec_ok(k, ldk, es)) && (!v || vec_ok(v, ldv, es));
    const ReadParams p{{k_cache, v_cache}, {k, v}, {ldk, ldv}, pages, ld_pages, n_pages, starts, n_seq, T, FastDiv((uint32_t)(H * (D / 8))), H, log2_of(P)};
    return type == QMM_Q8_0 ? read_typed<QMM_Q8_0>(t, D / 32, vec, p, s) : read_typed<QMM_Q4_0>(t, D / 32, vec, p, s);
}

QMM_DCHECK_READER(read_dcheck_cache)

}  // namespace qmm
