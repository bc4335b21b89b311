// cache.cu -- keys and values quantized as they are written into the paged cache (cache.cuh), and read
// back from it.
//
// The rules are those of the library's Q8_0 activations and Q4_0 weights, but that the Q8_0 scale is
// max|x| times the fp32 nearest to 1/127; a block is 32 elements of one head of one token.  A block whose
// scale is not a finite fp16 (an infinity or a NaN among its elements, or values beyond the format) is
// stored with a NaN scale and reads back as NaN, so that nothing turns into a finite value on the way.
//
// Both kernels move each byte once and are bound by that: 38768 tokens of 8 heads of 128, fp16 to Q4_0 and back, 407
// MB, take 81 us, 5.0 TB/s.  What costs beside the bytes is instructions, so a lane takes 16 elements, half
// a block: with 8, addresses and shuffles weigh twice as much.  A decode step's few tokens cost a launch each.
#include <type_traits>

#include "cache.cuh"
#include "elem.cuh"
#include "tc_common.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 2;                   // pieces of 16 elements that a thread loads before it works on the first
constexpr float kInv127 = 1.0f / 127.0f;    // rounded once: the Q8_0 scale is a product, not a quotient

// The low bits of 2^23 + v rounded towards zero are trunc(v), 0 <= v < 2^23: an addition where a
// conversion would take a slower pipe.
__device__ __forceinline__ uint32_t trunc_bits(float v) { return __float_as_uint(__fadd_rz(v, 8388608.0f)); }

// Four values' low bytes as one word.
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Codes of a lane's 16 elements, a byte each (Q4_0: 0..15), and the block's scale; the two lanes of a block
// (and so, for the shuffles, the warp) call it together.
template <int TYPE, typename T>
__device__ __forceinline__ uint16_t quantize16(const Raw<T, 16> &raw, uint32_t (&w)[4]) {
    float d;
    if constexpr (TYPE == QMM_Q8_0) {
        uint32_t bits = raw.top_bits();
        bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
        d = bits >= 0x7F800000u ? INFINITY : __fmul_rn(__uint_as_float(bits), kInv127);
    } else {
        int pos, neg;
        raw.top_signed(pos, neg);
        pos = max(pos, __shfl_xor_sync(0xffffffffu, pos, 1));
        neg = max(neg, __shfl_xor_sync(0xffffffffu, neg, 1));
        bool minus = neg > pos;
        if (__any_sync(0xffffffffu, neg == pos)) {
            // both signs reach the largest magnitude: the block's first element of it counts
            constexpr uint32_t kSign = sizeof(T) == 4 ? 0x80000000u : 0x8000u;
            uint32_t first = 0;                                  // the lane's: 2 found, 1 its sign
#pragma unroll
            for (int i = 15; i >= 0; --i) {
                const uint32_t b = raw.bits(i);
                if ((int)(b & ~kSign) == pos) first = 2u | (b & kSign ? 1u : 0u);
            }
            const uint32_t other = __shfl_xor_sync(0xffffffffu, first, 1);
            const uint32_t lower = threadIdx.x & 1 ? other : first, upper = threadIdx.x & 1 ? first : other;
            if (neg == pos) minus = ((lower & 2u ? lower : upper) & 1u) != 0;
        }
        const float m = bits_to_float<T>((uint32_t)max(pos, neg));
        // infinities and NaN have no scale
        d = m < INFINITY ? __fmul_rn(minus ? -m : m, -0.125f) : INFINITY;
    }
    const uint16_t half = __half_as_ushort(__float2half_rn(d));
    w[0] = w[1] = w[2] = w[3] = 0;
    if ((half & 0x7C00u) == 0x7C00u) {
        return 0x7E00u;
    }
    const float id = d != 0.0f ? __frcp_rn(d) : 0.0f;
    const bool slow = !(fabsf(id) < INFINITY);                  // 1 / d overflows: products may be infinities and NaN
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = __fmul_rn(raw.value(4 * c + i), id);
            if constexpr (TYPE == QMM_Q8_0) {
                // half away from zero: trunc(|x| + 1/2), the sum rounded towards zero so that it cannot reach the next integer
                const uint32_t m = trunc_bits(__fadd_rz(fminf(fabsf(x), 127.0f), 0.5f)), neg = (uint32_t)((int32_t)__float_as_uint(x) >> 31);
                q[i] = (m ^ neg) - neg;
            } else {
                q[i] = trunc_bits(fminf(fmaxf(__fadd_rn(x, 8.5f), 0.0f), 15.0f));
            }
            if (slow && isnan(x)) q[i] = 0;
        }
        w[c] = bytes4(q[0], q[1], q[2], q[3]);
    }
    return half;
}

struct WriteParams {
    const void *src[2];
    uint8_t *cache[2];
    int64_t ld[2];
    const int64_t *slots;
    int64_t n_slots;
    uint32_t items;                         // tokens * H * D / 16
    FastDiv per_tok;                        // H * D / 16
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
    // A block's codes and scale lie in a cache of so many pages (for checks).
    __device__ __forceinline__ bool inside(int64_t pages, int H, int block) const {
        return off >= 0 && off < P && block >= 0 && block < DB && chunk >= 0 && chunk + (int64_t)P * kToken <= pages * H * P * kToken;
    }
};

// A thread takes pieces of 16 elements; blockIdx.y: 0 keys, 1 values.
template <int TYPE, int DB, bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ WriteParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int which = blockIdx.y;
    const T *src = static_cast<const T *>(p.src[which]);
    uint8_t *cache = p.cache[which];
    const uint32_t step = gridDim.x * kThreads;
    // items is even and so is every warp's first index: the two lanes of a block are both in range or both
    // out of it, and all 32 lanes stay in the loop for the shuffles
    for (uint32_t base = blockIdx.x * kThreads + (threadIdx.x & ~31u); base < p.items; base += step * kBatch) {
        Raw<T, 16> raw[kBatch];
        int64_t slot[kBatch];
        uint32_t in_tok[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * step + (threadIdx.x & 31u), tok = p.per_tok(i);
            in_tok[u] = i - tok * p.per_tok.d;
            slot[u] = -1;
            raw[u].zero();
            if (i < p.items) {
                slot[u] = p.slots[tok];
                raw[u].template load<VEC>(src + tok * p.ld[which] + (int64_t)in_tok[u] * 16);
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            uint32_t w[4];
            const uint16_t d = quantize16<TYPE>(raw[u], w);
            uint32_t o0 = 0, o1 = 0;
            const bool upper = threadIdx.x & 1;                  // elements 16..31 of the block
            if constexpr (TYPE == QMM_Q4_0) {
                // byte j pairs elements j and j + 16: the lower lane writes bytes 0..7, the upper lane 8..15
                o0 = __shfl_xor_sync(0xffffffffu, upper ? w[0] : w[2], 1);
                o1 = __shfl_xor_sync(0xffffffffu, upper ? w[1] : w[3], 1);
            }
            if (slot[u] < 0 || slot[u] >= p.n_slots) continue;
            const int h = (int)(in_tok[u] / (2 * DB)), c = (int)(in_tok[u] % (2 * DB));      // elements 16c .. 16c + 15 of the head
            const Place<TYPE, DB> at(slot[u] >> p.log_p, h, p.H, (int)slot[u] & ((1 << p.log_p) - 1), p.log_p);
            if (!QMM_DCHECK(h < p.H && at.inside(p.n_slots >> p.log_p, p.H, c >> 1))) continue;
            if constexpr (TYPE == QMM_Q8_0) {
                *reinterpret_cast<uint4 *>(cache + at.codes(c >> 1, 16 * (c & 1))) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                *reinterpret_cast<uint2 *>(cache + at.codes(c >> 1, 8 * (c & 1))) =
                    upper ? make_uint2(o0 | (w[2] << 4), o1 | (w[3] << 4)) : make_uint2(w[0] | (o0 << 4), w[1] | (o1 << 4));
            }
            if (!upper) *reinterpret_cast<uint16_t *>(cache + at.scale(c >> 1)) = d;
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
    FastDiv per_tok;                        // H * D / 16
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

// Codes times scale, rounded to T: exact in fp32 (8 by 11 bits), so one rounding either way.  q: two
// half2 words of four codes.
template <typename T>
__device__ __forceinline__ void scale4(uint32_t q01, uint32_t q23, uint32_t d2, uint32_t *w) {
    if constexpr (std::is_same<T, __half>::value) {
        w[0] = tc::h2_bits(__hmul2(tc::bits_h2(q01), tc::bits_h2(d2)));
        w[1] = tc::h2_bits(__hmul2(tc::bits_h2(q23), tc::bits_h2(d2)));
    } else {
        const float d = __low2float(tc::bits_h2(d2));
        const float2 a = __half22float2(tc::bits_h2(q01)), b = __half22float2(tc::bits_h2(q23));
        if constexpr (sizeof(T) == 4) {
            w[0] = __float_as_uint(a.x * d);
            w[1] = __float_as_uint(a.y * d);
            w[2] = __float_as_uint(b.x * d);
            w[3] = __float_as_uint(b.y * d);
        } else {
            w[0] = pack2(a.x * d, a.y * d, T{});
            w[1] = pack2(b.x * d, b.y * d, T{});
        }
    }
}

// Words of N elements of T at p.
template <bool VEC, int N, typename T>
__device__ __forceinline__ void store_words(T *p, const uint32_t *w) {
    constexpr int kWords = N * (int)sizeof(T) / 4;
    if constexpr (VEC && kWords == 4) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kWords / 8; ++i) st32(reinterpret_cast<uint32_t *>(p) + 8 * i, w + 8 * i);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}

// A CTA takes 32 tokens: one warp finds their pages, then a thread takes pieces of 16 elements;
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
                if (pos >= 0 && pi < p.ld_pages && QMM_DCHECK(s < p.n_seq)) page = p.pages[s * p.ld_pages + pi];
                if (page >= p.n_pages) page = -1;
                off = (int)(pos & ((1 << p.log_p) - 1));
            }
            s_page[threadIdx.x] = page;
            s_off[threadIdx.x] = off;
        }
        __syncthreads();
        const uint32_t items = (uint32_t)min((int64_t)kReadTokens, p.T - t0) * p.per_tok.d;
        for (uint32_t base = threadIdx.x; base < items; base += kThreads * kBatch) {
            // Q8_0: 16 codes in a row.  Q4_0: 8 bytes, elements 8v .. 8v + 7 of a block in the low nibbles and
            // 16 + 8v .. in the high ones, v = the piece's place in its block
            uint4 w[kBatch];
            uint16_t d[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t i = base + u * kThreads, tok = p.per_tok(i), in_tok = i - tok * p.per_tok.d;
                w[u] = make_uint4(0u, 0u, 0u, 0u);
                d[u] = 0;                                        // any code times 0
                if (i < items && s_page[tok] >= 0) {
                    const int h = (int)(in_tok / (2 * DB)), c = (int)(in_tok % (2 * DB));
                    const Place<TYPE, DB> at(s_page[tok], h, p.H, s_off[tok], p.log_p);
                    if (!QMM_DCHECK(h < p.H && at.inside(p.n_pages, p.H, c >> 1))) continue;
                    d[u] = *reinterpret_cast<const uint16_t *>(cache + at.scale(c >> 1));
                    if constexpr (TYPE == QMM_Q8_0) {
                        w[u] = *reinterpret_cast<const uint4 *>(cache + at.codes(c >> 1, 16 * (c & 1)));
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(cache + at.codes(c >> 1, 8 * (c & 1)));
                        w[u].x = v.x;
                        w[u].y = v.y;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t i = base + u * kThreads, tok = p.per_tok(i), in_tok = i - tok * p.per_tok.d;
                if (i >= items || !QMM_DCHECK(t0 + tok < p.T)) break;
                const uint32_t d2 = d[u] * 0x00010001u;
                constexpr int kW4 = sizeof(T);                   // words of four elements
                uint32_t v[4 * kW4];
                const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                T *out = dst + (t0 + tok) * p.ld[which] + (int64_t)(in_tok >> 1) * 32;
                if constexpr (TYPE == QMM_Q8_0) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t q01, q23;
                        tc::i8x4_to_h2x2(x[c], q01, q23);
                        scale4<T>(q01, q23, d2, v + c * kW4);
                    }
                    store_words<VEC, 16>(out + 16 * (in_tok & 1), v);
                } else {
                    const __half2 eight = __halves2half2(__float2half_rn(1032.0f), __float2half_rn(1032.0f));
#pragma unroll
                    for (int c = 0; c < 4; ++c) {               // low nibbles of x[0], x[1], then high ones
                        const uint32_t n = (c < 2 ? x[c & 1] : x[c & 1] >> 4) & 0x0F0F0F0Fu;
                        const uint32_t q01 = tc::h2_bits(__hsub2(tc::bits_h2(__byte_perm(n, 0x64646464u, 0x4140u)), eight));
                        const uint32_t q23 = tc::h2_bits(__hsub2(tc::bits_h2(__byte_perm(n, 0x64646464u, 0x4342u)), eight));
                        scale4<T>(q01, q23, d2, v + c * kW4);
                    }
                    store_words<VEC, 8>(out + 8 * (in_tok & 1), v);
                    store_words<VEC, 8>(out + 16 + 8 * (in_tok & 1), v + 2 * kW4);
                }
            }
        }
    }
}

unsigned grid_for(int64_t work, int64_t per_cta) {
    const int64_t g = (work + per_cta - 1) / per_cta;
    return (unsigned)(g > 152 * 8 ? 152 * 8 : (g < 1 ? 1 : g));
}

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
    const bool vec = rows_aligned(k, ldk, es) && rows_aligned(v, ldv, es);
    const WriteParams p{{k, v}, {k_cache, v_cache}, {ldk, ldv}, slots, n_pages * P, 0, FastDiv((uint32_t)(H * (D / 16))), H, log2_of(P)};
    return type == QMM_Q8_0 ? write_typed<QMM_Q8_0>(t, D / 32, vec, p, T, k, v, s) : write_typed<QMM_Q4_0>(t, D / 32, vec, p, T, k, v, s);
}

cudaError_t launch_cache_read(qmm_type type, const uint8_t *k_cache, const uint8_t *v_cache, int64_t n_pages, int P, int H, int D,
                              const int32_t *pages, int64_t ld_pages, const int32_t *starts, int64_t n_seq, int64_t T, qmm_dtype t,
                              void *k, void *v, int64_t ldk, int64_t ldv, cudaStream_t s) {
    const size_t es = dtype_bytes(t);
    const bool vec = (!k || rows_aligned(k, ldk, es)) && (!v || rows_aligned(v, ldv, es));
    const ReadParams p{{k_cache, v_cache}, {k, v}, {ldk, ldv}, pages, ld_pages, n_pages, starts, n_seq, T, FastDiv((uint32_t)(H * (D / 16))), H, log2_of(P)};
    return type == QMM_Q8_0 ? read_typed<QMM_Q8_0>(t, D / 32, vec, p, s) : read_typed<QMM_Q4_0>(t, D / 32, vec, p, s);
}

QMM_DCHECK_READER(read_dcheck_cache)

}  // namespace qmm
