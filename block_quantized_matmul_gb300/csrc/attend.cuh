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
    int P, log_p, H, group, tile_rows, row_tiles;
    int splits, budget, waves;             // of a sequence at most; of all together in a wave, and the waves to choose from
    int fixed;                             // steps of keys that a CTA's start and end are worth
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
    const int32_t *chosen;                 // [T][H][list_len]: the pages chosen for each token and head (attend_chosen.cu)
    int list_len;
    uint32_t chunk;                        // keys of such a list in a split
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

// Splits are multiples of it, and may be as short: 777 tokens of 8 heads take 8.4 us with one step at least, 8.7 with two,
// 10.1 with four (a tile of 32 keys takes a warp longer than the join takes for another part).
constexpr int kStep = 128;

// Tokens that a sequence has in the cache.
__device__ __forceinline__ int64_t cached(const AttendParams &p, int len) { return max((int64_t)0, min((int64_t)len, p.ld_pages << p.log_p)); }

// The length of sequence base + lane (0: there is none).
__device__ __forceinline__ int len_at(const AttendParams &p, int base) {
    const int s = base + (int)(threadIdx.x & 31);
    return s < (int)p.n_seq ? __ldcg(p.kv_lens + s) : 0;
}

__device__ __forceinline__ uint32_t steps_of(const AttendParams &p, int len) { return ((uint32_t)cached(p, len) + kStep - 1) / kStep; }
__device__ __forceinline__ uint32_t steps_at(const AttendParams &p, int base) { return steps_of(p, len_at(p, base)); }

// Steps of keys in a split: the fewest (to within a thousandth) with which no sequence has more splits than
// p.splits, and all together no more than `budget`.  By one warp, which looks at 32 sizes at a time.  `mine`: steps
// of sequence `lane`, sum and most of all.
__device__ __forceinline__ uint32_t fewest_steps(const AttendParams &p, uint32_t mine, uint32_t sum, uint32_t most, uint32_t budget) {
    const int lane = threadIdx.x & 31, n = (int)p.n_seq;
    uint32_t lo = max(1u, max((most + p.splits - 1) / p.splits, (sum + budget - 1) / budget));
    uint32_t hi = max(lo, most);                                 // one split a sequence: not more than the budget
    for (int round = 0; round < 2 && lo < hi; ++round) {
        const uint32_t c = lo + (uint32_t)((uint64_t)(hi - lo) * lane / 31);
        // t / c, rounded up, by a multiplication (at times one too many for t * c >= 2^32; for c = 1, where 2^32 / c does not
        // fit, (t + 1) (2^32 - 1) / 2^32 = t)
        const uint32_t inv = 0xFFFFFFFFu / c + (c > 1), up = max(c - 1, 1u);
        uint32_t used = 0;
        for (int base = 0; base < n; base += 32) {
            const uint32_t t = base == 0 ? mine : steps_at(p, base);
            for (int l = 0; l < min(32, n - base); ++l) used += max(1u, __umulhi(__shfl_sync(0xffffffffu, t, l) + up, inv));
        }
        const int first = __ffs(__ballot_sync(0xffffffffu, used <= budget)) - 1;     // more keys, fewer splits: lane 31's fit
        hi = __shfl_sync(0xffffffffu, c, first);
        if (first == 0) break;
        lo = __shfl_sync(0xffffffffu, c, first - 1) + 1;
    }
    return hi;
}

// Keys of a split, so that the CTAs come out even whatever the lengths are: for one wave of CTAs, or two where those
// end sooner (a CTA's start, end and partial result cost about as much as p.fixed steps).  By one warp; `len`:
// len_at(p, 0).  (25 sequences of 8 heads, 304 places: 8192 tokens each, 85 us with two waves, 104 without; 0 to
// 8192 tokens, 58 us with two, 53 with one.)
__device__ __forceinline__ uint32_t chunk_of(const AttendParams &p, int len) {
    const uint32_t mine = steps_of(p, len);
    if (p.n_seq == 1) return max(1u, max((mine + p.splits - 1) / p.splits, (mine + p.budget - 1) / p.budget)) * kStep;
    uint32_t sum = mine, most = mine;                            // (a sum past 32 bits only makes the first guess low)
    for (int base = 32; base < (int)p.n_seq; base += 32) {
        const uint32_t t = steps_at(p, base);
        sum += t;
        most = max(most, t);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    most = __reduce_max_sync(0xffffffffu, most);
    uint32_t c = fewest_steps(p, mine, sum, most, p.budget);
    if (p.waves == 2) {
        const uint32_t c2 = fewest_steps(p, mine, sum, most, 2 * p.budget);
        if (2 * (c2 + p.fixed) < c + p.fixed) c = c2;
    }
    return c * kStep;
}
__device__ __forceinline__ int splits_of(int64_t n, uint32_t chunk) { return (int)max(1u, ((uint32_t)n + chunk - 1) / chunk); }

struct Rows {                              // what a CTA works on
    int64_t s, q0, nq, n, first, k0, k1;
    int h, r0, rows, sp, used;
    // of a list of chosen pages: the list, and the places that its token sees: all below `upto`, but with tree words of those
    // from `first` on the ones whose bit is set
    const int32_t *list;
    int64_t upto;
    uint64_t word;
    bool tree;
};

// Which of the places at .. at + 15 the token of a list sees, as bits.
__device__ __forceinline__ uint32_t seen16(const Rows &w, int64_t at) {
    if (at < 0 || at >= w.upto) return 0u;
    uint32_t m = w.upto - at >= 16 ? 0xffffu : (1u << (int)(w.upto - at)) - 1u;
    if (w.tree && at + 16 > w.first) {
        // bit k: place at + k is new token b + k of the sequence
        const int64_t b = at - w.first;
        if (b >= 64) m = 0u;
        else if (b >= 0) m &= (uint32_t)(w.word >> b);
        else m &= (uint32_t)(w.word << -b) | ((1u << (int)-b) - 1u);
    }
    return m;
}

// The CTA's rows and keys, from its index: row tiles fastest, then heads, then sequences (longest first) or, where
// they are split, all whole splits and then the rest of each sequence.  False: it has none.  `scratch`: kSorted + 1 ints of shared
// memory, free again on return.
template <int ROWS>
__device__ __forceinline__ bool find_rows(const AttendParams &p, int *scratch, int threads, Rows &w) {
    const int lane = threadIdx.x & 31;
    uint32_t at = blockIdx.x;
    const int rt = (int)(at % (uint32_t)p.row_tiles);
    at /= (uint32_t)p.row_tiles;
    w.h = (int)(at % (uint32_t)p.H);
    w.s = at / (uint32_t)p.H;
    w.sp = 0;
    w.used = 1;
    uint32_t chunk = 0;
    int q0 = 0, q1 = 0, len = 0;
    if (p.splits > 1 && p.n_seq == 1) {
        len = __ldcg(p.kv_lens);
        q0 = __ldcg(p.q_starts);
        q1 = __ldcg(p.q_starts + 1);
        chunk = chunk_of(p, len);
        w.used = splits_of(cached(p, len), chunk);
        w.sp = (int)w.s;
        w.s = 0;
        if (w.sp >= w.used) return false;
    } else if (p.splits > 1) {
        // a lane a sequence: all that is loaded is under way at once
        const bool have = lane < (int)p.n_seq;
        const int lens = len_at(p, 0), from = have ? __ldcg(p.q_starts + lane) : 0, to = have ? __ldcg(p.q_starts + lane + 1) : 0;
        chunk = chunk_of(p, lens);
        int j = (int)w.s, s = -1;                                // place in the line of splits
        for (int base = 0; base < (int)p.n_seq; base += 32) {
            len = base == 0 ? lens : len_at(p, base);
            const int whole = base + lane < (int)p.n_seq ? splits_of(cached(p, len), chunk) - 1 : 0;
            int upto = whole;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, m);
                if (lane >= m) upto += x;
            }
            const unsigned past = __ballot_sync(0xffffffffu, upto > j);
            if (past) {
                const int l = __ffs(past) - 1;
                s = base + l;
                w.sp = j - (__shfl_sync(0xffffffffu, upto, l) - __shfl_sync(0xffffffffu, whole, l));
                break;
            }
            j -= __shfl_sync(0xffffffffu, upto, 31);
        }
        const bool rest = s < 0;
        if (rest) s = j;
        if (s >= (int)p.n_seq) return false;
        // every split has a CTA: the whole ones before this rest, and a rest of each sequence
        if (rest) (void)QMM_DCHECK(((int)w.s - j + (int)p.n_seq) * p.H * p.row_tiles <= (int)gridDim.x);
        if (s < 32) {
            len = __shfl_sync(0xffffffffu, lens, s);
            q0 = __shfl_sync(0xffffffffu, from, s);
            q1 = __shfl_sync(0xffffffffu, to, s);
        } else {
            len = __ldcg(p.kv_lens + s);
            q0 = __ldcg(p.q_starts + s);
            q1 = __ldcg(p.q_starts + s + 1);
        }
        w.s = s;
        w.used = splits_of(cached(p, len), chunk);
        if (rest) w.sp = w.used - 1;
    } else {
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
        q0 = p.q_starts[w.s];
        q1 = p.q_starts[w.s + 1];
        len = p.kv_lens[w.s];
    }
    w.q0 = q0;
    w.nq = (int64_t)q1 - q0;
    if (q0 < 0 || q1 > p.T) return false;                        // not rows of q
    w.r0 = rt * ROWS;
    w.rows = (int)min((int64_t)ROWS, w.nq * p.group - w.r0);
    if (w.rows <= 0) return false;
    w.first = len - w.nq;
    w.n = cached(p, len);
    w.k0 = (int64_t)w.sp * chunk;
    w.k1 = w.sp == w.used - 1 ? w.n : min(w.n, w.k0 + chunk);
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
    if (!QMM_DCHECK(row < w.rows && w.q0 + i < p.T && hq < Hq && d + N <= D && w.sp < w.used && (w.used == 1 || w.used <= p.splits))) return;
    if (w.used == 1) {
        const int64_t to = (w.q0 + i) * p.ldo + (int64_t)hq * D + d;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if constexpr (N == 8) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float a = o[2 * k] * inv, b = o[2 * k + 1] * inv;
                x[k] = p.bf16 ? pack2(a, b, __nv_bfloat16{}) : pack2(a, b, __half{});
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + to) = make_uint4(x[0], x[1], x[2], x[3]);
        } else if constexpr (N == 4) {
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
        if constexpr (N == 8) st32(p.part_o + part * D + d, reinterpret_cast<const uint32_t *>(o));
        else if constexpr (N == 4) *reinterpret_cast<float4 *>(p.part_o + part * D + d) = make_float4(o[0], o[1], o[2], o[3]);
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
template <int TYPE, int DB, int WARPS, bool CHOSEN = false>
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
            int64_t number = j >> p.log_p;
            if constexpr (CHOSEN) {
                if (!QMM_DCHECK(number < p.list_len)) continue;
                number = w.list[number];
                if (!((seen16(w, (number << p.log_p) + (j & (p.P - 16))) >> (j & 15)) & 1)) continue;
            } else {
                if (j >= w.first && !sees(p.tree, w.q0 + i, i, j - w.first)) continue;
            }
            if (!QMM_DCHECK(number < p.ld_pages && w.s < p.n_seq)) continue;
            const int64_t page = p.pages[w.s * p.ld_pages + number];
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

// More than 32 rows of up to 128 elements (attend_tc.cu): 128 rows to a CTA, one CTA an SM.
constexpr int kTcRows = 128;
cudaError_t launch_attend_tc(qmm_type type, const AttendParams &p, int DB, int64_t ctas, cudaStream_t s);
cudaError_t read_and_clear_attend_status(unsigned *out, cudaStream_t s);
cudaError_t read_dcheck_attend_tc(unsigned *out, cudaStream_t s);

}  // namespace qmm
