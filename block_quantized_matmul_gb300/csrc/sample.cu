// sample.cu -- one token of each row of logits z, from a random number u:
//   w_i = exp((z_i - max z) / temperature); kept are, in the order of z (the earlier index first on ties), the top_k first, of
//   those the ones before which the others sum to less than top_p of the whole, of those the ones with w >= min_p; the token
//   is the first index at which the running sum of the kept w exceeds u times their sum.
//
// Every cut is a prefix of one order, that of (z descending, index ascending), so what is kept is all up to a border element.
// The border is found by a histogram of 2048 bins over the distance from the maximum, of counts for top_k and of
// sums of w for top_p; the elements of the border's bin are then gathered in one CTA and sorted.  Where the first
// top_k elements and the rest of their bin fit there, that CTA does all that is left with them alone.  Where a bin holds too
// much (logits of few values, or of a scale far from the temperature's), the border is found digit by digit instead.
//
// Borders of sums have to fall where the formula's do, to within an error far below one token's share: fp32 sums over 10^5 tokens
// would not do, and fp64 is too slow on this GPU for every logit.  So w is a whole number, 2^43 for the largest (`weight`), and
// all sums are sums of integers: exact, and the same in any order, so histograms may be filled by atomics.
//
// A cluster of up to 8 CTAs takes a row, each CTA a slice of it that stays in shared memory from the first pass on.  What the
// CTAs find is exchanged through distributed shared memory: each adds up all histograms for itself.
//
// What bounds it.  Few rows: a chain of passes, barriers of the cluster (about a microsecond each) and sorts: greedy 4.7 us, plain 10.9,
// top_k = 50 16.5, top_p = 0.95 26.2 (128256 logits).  Many rows: 130 us for 256 rows of 128256 fp32 logits, plain, for 19.6 us of
// bytes, at 84 instructions a logit (executed, of 64 such rows): 36 for staging, the table, the passes and the search, 37 for `weight` in 30 bits, and 12 on
// average for its way in 64 bits, which half of the warps take besides (5 % of the logits lie within 2^-14 of the largest).  They fill 52 to 60 %
// of the issue slots; barriers and loads take the rest.  With top_p its atomic additions.
#include <climits>

#include "qmm_internal.cuh"

#include "elem.cuh"

namespace qmm {
namespace {

constexpr int kBins = 2048, kSums = 512, kMaxCluster = 8;     // bins of a slice's histogram, and sums of four of them that the CTAs exchange
constexpr int kCand = 1024;                 // elements that one CTA sorts
constexpr int kMaxWarps = 32;
constexpr int kOne = 43;                    // w of the largest logit is 2^kOne
constexpr int kPowers = 2048;

// 2^(j / kPowers) times 2^kOne, from the square roots of 2: eleven factors at most, each within 2^-52.
struct Powers {
    uint64_t v[kPowers];
};
constexpr Powers make_powers() {
    double root[11] = {};
    double x = 2.0;
    for (int i = 0; i < 11; ++i) {
        double r = 1.0 + (x - 1.0) / 2;     // Newton's iteration for the square root of x, 1 < x <= 2
        for (int k = 0; k < 6; ++k) r = 0.5 * (r + x / r);
        root[i] = x = r;
    }
    Powers p = {};
    for (int j = 0; j < kPowers; ++j) {
        double v = 1.0;
        for (int i = 0; i < 11; ++i)
            if (j & (kPowers / 2 >> i)) v *= root[i];
        p.v[j] = (uint64_t)(v * (double)((uint64_t)1 << kOne) + 0.5);
    }
    return p;
}
__device__ const Powers g_powers = make_powers();

// What the CTAs of a row share about it.
struct Row {
    float top, scale;                       // largest logit; bins of a histogram for a unit of distance from it
    float ch, cl;                           // c = log2(e) / temperature in two terms
    float y0, gh, gl;                       // top * c; what is left of it above y0's multiple n0 of 1 / kPowers, in two terms
    int n0;
    int wide;                               // too far apart for `weight`
    uint64_t least;                         // w that min_p asks for
};

struct alignas(16) Shared {
    uint32_t powers[kPowers];               // g_powers in units of 2^-30,
    uint16_t more[kPowers];                 // and the 13 bits below
    uint32_t lo[kBins], hi[kBins];          // the histogram of this CTA's slice: counts (lo), or sums in two words
    uint64_t cand[kCand];                   // of the row's first CTA: gathered elements, ~ordered(z) << 32 | index
    uint64_t list[kCand];                   // this CTA's part of them
    uint32_t n_cand, n_list, list_at;
    uint64_t sums[kSums];                   // the histogram, four bins to a sum
    uint64_t seg_sum[kMaxWarps];            // sum of the kept w of each warp's segment
    uint64_t part[kMaxWarps];
    float top, bottom;                      // the slice's largest, and smallest finite, logit
    int first;
    Row row;
    // what one thread finds for all
    int bin;
    uint64_t left, upto, border;            // border: a place
    int seg;
    uint64_t target;
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// The address of a variable of this CTA's shared memory in that of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void *p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t remote_u32(const void *p, int rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t remote_u64(const void *p, int rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint4 remote_u128(const void *p, int rank) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(remote(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t remote_add(const void *p, int rank, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(remote(p, rank)), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void remote_store(const void *p, int rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}

__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
// An element's place in the order: the smaller the earlier.  (-0 is 0.)
__device__ __forceinline__ uint64_t place_of(float z, int index) { return (uint64_t)~ordered(z + 0.0f) << 32 | (uint32_t)index; }
__device__ __forceinline__ float logit_of(uint64_t place) { return unordered(~(uint32_t)(place >> 32)); }

// w = base * (1 + p) 2^-down for base of 2^kOne .. 2^(kOne + 1), |p| < 2^-11.
__device__ __forceinline__ uint64_t scaled(uint64_t base, int p_2_42, int down) {
    const uint64_t w = base + (uint64_t)(((int64_t)p_2_42 * (int64_t)(int32_t)(base >> 13)) >> 29);
    return down <= 0 ? w : (w + ((uint64_t)1 << (down - 1))) >> down;
}

// w of a logit in a row whose logits or temperature are so far from 1 that `weight`'s steps would not hold: z - top and its
// product with c as pairs of fp32, within 2^-40.
__device__ __noinline__ uint64_t weight_wide(float z, float top, float ch, float cl) {
    if (z == top) return (uint64_t)1 << kOne;
    const float hi = __fsub_rn(z, top), b = __fsub_rn(hi, z), lo = __fadd_rn(__fsub_rn(z, __fsub_rn(hi, b)), __fsub_rn(-top, b));
    const float yh = __fmul_rn(hi, ch), yl = __fadd_rn(__fmaf_rn(hi, ch, -yh), __fmaf_rn(hi, cl, __fmul_rn(lo, ch)));
    if (!(yh > -(float)(kOne + 1))) return 0;                          // (and for z = -inf)
    const float magic = 12582912.0f, k = __fmaf_rn(yh, (float)kPowers, magic);
    const int n = __float_as_int(k) - __float_as_int(magic);
    const float g = __fmaf_rn(__fsub_rn(k, magic), -1.0f / kPowers, yh);
    const float ln2h = 0.693147182464599609375f, ln2l = -1.9046542943909386e-9f;      // ln 2 and what fp32 leaves of it
    const float th = __fmul_rn(g, ln2h), tl = __fadd_rn(__fmaf_rn(g, ln2h, -th), __fmaf_rn(g, ln2l, __fmul_rn(yl, ln2h)));
    const float t = __fadd_rn(th, tl), small = __fmaf_rn(__fmul_rn(t, t), __fmaf_rn(t, 1.0f / 6.0f, 0.5f), tl);
    const float unit = 4398046511104.0f;                               // 2^42
    return scaled(g_powers.v[n & (kPowers - 1)], __float2int_rn(__fmul_rn(th, unit)) + __float2int_rn(__fmul_rn(small, unit)), -(n >> 11));
}

// w of logit z: 2^kOne * 2^y, y = (z - top) * c, as a whole number within 9/8 and 2^-34 of itself; 0 for NaN.
// y = z c - top c = n / kPowers + f with |f| <= 1 / kPowers, where the multiple of 1 / kPowers and the rest are taken apart
// for z c (a product in two terms) and for top c (once a row); 2^f - 1 = t + t^2/2 + t^3/6, t = f ln 2 (the next term
// is 2^-50).  Down to 2^-13 of the largest it is the nearest to within 2^-34 of itself.  Below, 30 bits hold what of w counts (2^14 logits at
// most lie higher, and mostly a few): the table's word and the product are cut to them, which takes up to one off, and the fraction p
// is a multiple of 2^-32, an eighth.  So w comes out low there, by a quarter on average at 2^-14 and half as much with each power of
// two below; a sum over 2^20 such logits by 2^18, of at least 2^49.
__device__ __forceinline__ uint64_t weight(const Row &r, float z, const Shared &sh) {
    if (r.wide) return weight_wide(z, r.top, r.ch, r.cl);
    const float yh = __fmul_rn(z, r.ch), y = __fsub_rn(yh, r.y0);
    if (!(y > -(float)(kOne + 1) - 0.25f)) return 0;
    const float yl = __fmaf_rn(z, r.cl, __fmaf_rn(z, r.ch, -yh));
    const float magic = 12582912.0f, k = __fmaf_rn(yh, (float)kPowers, magic);
    const float g = __fmaf_rn(__fsub_rn(k, magic), -1.0f / kPowers, yh);
    const float t = __fmul_rn(__fadd_rn(__fsub_rn(g, r.gh), __fsub_rn(yl, r.gl)), 0.693147182464599609375f);
    const float p = __fmaf_rn(__fmul_rn(t, t), __fmaf_rn(t, 1.0f / 6.0f, 0.5f), t);
    const int n = __float_as_int(k) - __float_as_int(magic) - r.n0, down = -(n >> 11), j = n & (kPowers - 1);
    const uint32_t base = sh.powers[j];
    if (down < 14) {
        if (z == r.top) return (uint64_t)1 << kOne;
        return scaled((uint64_t)base << (kOne - 30) | sh.more[j], __float2int_rn(__fmul_rn(p, 4398046511104.0f)), down);
    }
    const int q = __float_as_int(__fmaf_rn(p, 4294967296.0f, magic)) - __float_as_int(magic);
    const uint32_t w = base + (uint32_t)__mulhi((int)base, q);
    uint32_t a;
    asm("shr.u32 %0, %1, %2;" : "=r"(a) : "r"(w), "r"(down - 14));     // (by 32 and more: 0)
    return (a >> 1) + (a & 1);
}
// The same where time does not matter: the code of all phases has to come to the SMs too.
__device__ __noinline__ uint64_t weight_of_few(const Shared &sh, float z) { return weight(sh.row, z, sh); }

// ceil or floor of f * x for 0 <= f <= 1.
__device__ __forceinline__ uint64_t times(float f, uint64_t x, bool up) {
    const uint32_t b = __float_as_uint(f);
    const int e = (int)(b >> 23);
    const uint64_t mant = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
    int shift = 150 - (e ? e : 1);                                     // f = mant 2^-shift, shift >= 23
    const uint64_t hi = __umul64hi(x, mant), lo = x * mant;            // below 2^88
    uint64_t q, rest;
    if (shift < 64) {
        q = hi << (64 - shift) | lo >> shift;
        rest = lo << (64 - shift);
    } else {
        shift -= 64;
        q = shift < 64 ? hi >> shift : 0;
        rest = lo | (shift == 0 ? 0 : (shift < 64 ? hi << (64 - shift) : hi));
    }
    return q + (up && rest ? 1 : 0);
}

// (z - top) / temperature - ln(total / 2^kOne), rounded once but for 2^-30 of itself: the quotient and the logarithm as pairs
// of fp32.  ln(total / 2^kOne) = ln 2 * (e + j / kPowers) + ln(1 + x), x = total / (2^e g_powers[j]) - 1.
__device__ __noinline__ float log_share(const Shared &sh, float z, float top, float temperature, uint64_t total) {
    float y = 0.0f, y1 = 0.0f;
    if (z != top) {
        const float d = __fsub_rn(z, top), b = __fsub_rn(d, z), low = __fadd_rn(__fsub_rn(z, __fsub_rn(d, b)), __fsub_rn(-top, b));
        y = __fdiv_rn(d, temperature);
        if (fabsf(y) < INFINITY && fabsf(d) < INFINITY && fabsf(y) > 1e-30f) y1 = __fdiv_rn(__fadd_rn(__fmaf_rn(-y, temperature, d), low), temperature);
    }
    const int e = 63 - __clzll((long long)total) - kOne;               // total >= 2^kOne
    const uint64_t m = total >> e;
    const int j = min(kPowers - 1, max(0, (int)(__log2f((float)m * (1.0f / 8796093022208.0f)) * kPowers)));
    const uint64_t base = (uint64_t)sh.powers[j] << (kOne - 30) | sh.more[j];
    const float x = __fdiv_rn((float)(int64_t)(m - base), (float)base);
    const float ln2h = 0.693147182464599609375f, ln2l = -1.9046542943909386e-9f;
    const float k = (float)e + (float)j * (1.0f / kPowers), l = __fmul_rn(k, ln2h);
    const float l1 = __fadd_rn(__fmaf_rn(k, ln2l, __fmaf_rn(k, ln2h, -l)), __fmaf_rn(__fmul_rn(x, x), __fmaf_rn(x, 1.0f / 3.0f, -0.5f), x));
    const float s = __fsub_rn(y, l), back = __fsub_rn(s, y);
    return __fadd_rn(s, __fadd_rn(__fadd_rn(__fsub_rn(y, __fsub_rn(s, back)), __fsub_rn(-l, back)), __fsub_rn(y1, l1)));
}

// Sums of v over the threads before this one; `all`: over all of them.
template <int WARPS>
__device__ __noinline__ uint64_t sums_before(uint64_t v, uint64_t *part, uint64_t &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    uint64_t s = lane < WARPS ? part[lane] : 0;
#pragma unroll
    for (int m = 1; m < WARPS; m <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, s, m);
        if (lane >= m) s += y;
    }
    all = __shfl_sync(0xffffffffu, s, WARPS - 1);
    const uint64_t before = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
    __syncthreads();
    return (warp ? before : 0) + x - v;
}

// a[0 .. n) ascending, by the whole CTA (up to 64 elements by its first warp); n <= kCand, room for the next power of two.
// (In registers, with shuffles between the lanes of a warp: 64 elements as fast, 1024 in 512 threads slower.)
__device__ __noinline__ void sort(uint64_t *a, int n) {
    int n2 = 2;
    while (n2 < n) n2 *= 2;
    for (int i = n + (int)threadIdx.x; i < n2; i += (int)blockDim.x) a[i] = ~(uint64_t)0;
    __syncthreads();
    const int t = (int)threadIdx.x;
    if (n2 > 64 || t < 32) {
#pragma unroll 1
        for (int size = 2; size <= n2; size *= 2)
#pragma unroll 1
            for (int half = size / 2; half > 0; half /= 2) {
                const int i = 2 * t - (t & (half - 1)), j = i + half;
                if (j < n2) {
                    const uint64_t x = a[i], y = a[j];
                    if ((x > y) == ((i & size) == 0)) {
                        a[i] = y;
                        a[j] = x;
                    }
                }
                if (n2 > 64) __syncthreads();
                else __syncwarp();
            }
    }
    __syncthreads();
}

// STAGED: the slice lies in shared memory after the first pass, otherwise it is read again each time.
template <typename T, bool STAGED, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) sample_kernel(const SampleParams p, int ctas, int per, int vec) {
    constexpr int kThreads = THREADS, kWarps = THREADS / 32;
    constexpr bool kClean = STAGED && sizeof(T) == 4;                   // fp32: NaN is taken out as the slice is staged
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    T *stage = reinterpret_cast<T *>(smem + sizeof(Shared));
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)(blockIdx.x % (unsigned)ctas);
    const int64_t row = blockIdx.x / (unsigned)ctas;
    for (int i = tid; i < kPowers; i += kThreads) {
        const uint64_t v = g_powers.v[i];
        sh.powers[i] = (uint32_t)(v >> (kOne - 30));
        sh.more[i] = (uint16_t)(v & ((1u << (kOne - 30)) - 1));
    }
    if (tid == 0) {
        sh.n_cand = sh.n_list = 0;
        sh.seg = -1;
        sh.bin = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto barrier = [&] {
        if (ctas > 1) cluster_sync();
        else __syncthreads();
    };
    const int from = min(rank * per, p.V), n = min(per, p.V - from);
    const T *src = static_cast<const T *>(p.logits) + row * p.ld + from;
    // NaN counts as -inf
    auto logit = [&](int i) {
        const float v = elem_to_float(STAGED ? stage[i] : src[i]);
        return kClean || !isnan(v) ? v : -INFINITY;
    };

    // ---- the first pass: the slice to shared memory, its largest and smallest finite logit ----
    float top = -INFINITY, bottom = INFINITY;
    auto look = [&](float v) {                                         // (fmaxf and fminf pass over NaN)
        top = fmaxf(top, v);
        bottom = fminf(bottom, v == -INFINITY ? INFINITY : v);
    };
    constexpr int kVec = 16 / (int)sizeof(T), kAhead = 4;
    int done = 0;
    if (vec) {
        const int pieces = n / kVec;
        for (int i = tid; i < pieces; i += kThreads * kAhead) {
            uint4 v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i + u * kThreads < pieces) v[u] = reinterpret_cast<const uint4 *>(src)[i + u * kThreads];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (i + u * kThreads >= pieces) continue;
                if constexpr (kClean) {
                    float *e = reinterpret_cast<float *>(&v[u]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[k] = isnan(e[k]) ? -INFINITY : e[k];
                }
                if constexpr (STAGED) reinterpret_cast<uint4 *>(stage)[i + u * kThreads] = v[u];
                const T *e = reinterpret_cast<const T *>(&v[u]);
#pragma unroll
                for (int k = 0; k < kVec; ++k) look(elem_to_float(e[k]));
            }
        }
        done = pieces * kVec;
    }
    for (int i = done + tid; i < n; i += kThreads) {
        T v = src[i];
        if constexpr (kClean) v = isnan(v) ? -INFINITY : v;
        if constexpr (STAGED) stage[i] = v;
        look(elem_to_float(v));
    }
    const float own_top = top;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        bottom = fminf(bottom, __shfl_xor_sync(0xffffffffu, bottom, m));
    }
    if (lane == 0) sh.part[warp] = (uint64_t)__float_as_uint(top) << 32 | __float_as_uint(bottom);
    const float temperature = p.temperature ? p.temperature[row] : 1.0f, top_p = p.top_p ? p.top_p[row] : 1.0f, min_p = p.min_p ? p.min_p[row] : 0.0f;
    const int top_k = p.top_k ? p.top_k[row] : 0;
    const float u = p.u[row];
    __syncthreads();
    if (warp == 0) {
        const uint64_t both = sh.part[lane % kWarps];
        top = __uint_as_float((uint32_t)(both >> 32));
        bottom = __uint_as_float((uint32_t)both);
#pragma unroll
        for (int m = kWarps / 2; m > 0; m >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
            bottom = fminf(bottom, __shfl_xor_sync(0xffffffffu, bottom, m));
        }
        if (lane == 0) {
            sh.top = top;
            sh.bottom = bottom;
        }
    }
    barrier();
    if (warp == 0) {
        top = lane < ctas ? __uint_as_float(remote_u32(&sh.top, lane)) : -INFINITY;
        bottom = lane < ctas ? __uint_as_float(remote_u32(&sh.bottom, lane)) : INFINITY;
#pragma unroll
        for (int m = kMaxCluster / 2; m > 0; m >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
            bottom = fminf(bottom, __shfl_xor_sync(0xffffffffu, bottom, m));
        }
        if (lane == 0) {
            Row &r = sh.row;
            // (pairs of fp32: a chain of fp64 operations takes microseconds on this GPU)
            const float log2e_h = 1.44269502162933349609375f, log2e_l = 1.92596299112661746e-8f;      // log2(e) and what fp32 leaves of it
            r.top = top + 0.0f;
            r.scale = (float)(kBins - 1) / fminf(__fsub_rn(top, bottom), 64.0f * fmaxf(1.0f, temperature));   // (bottom = inf: 0 or less)
            r.ch = __fdiv_rn(log2e_h, temperature);
            r.cl = r.ch < INFINITY ? __fdiv_rn(__fadd_rn(__fmaf_rn(-r.ch, temperature, log2e_h), log2e_l), temperature) : 0.0f;
            r.y0 = __fmul_rn(r.top, r.ch);
            r.wide = !(fabsf(r.y0) < 900.0f) || r.ch < 1e-30f;         // (below that the remainder of the division is lost)
            const float n0 = r.wide ? 0.0f : rintf(r.y0 * kPowers), y1 = __fmaf_rn(r.top, r.cl, __fmaf_rn(r.top, r.ch, -r.y0));
            const float g = __fmaf_rn(n0, -1.0f / kPowers, r.y0);
            r.n0 = (int)n0;
            r.gh = __fadd_rn(g, y1);
            const float back = __fsub_rn(r.gh, g);
            r.gl = __fadd_rn(__fsub_rn(g, __fsub_rn(r.gh, back)), __fsub_rn(y1, back));
            r.least = min_p > 0.0f && min_p <= 1.0f ? times(min_p, (uint64_t)1 << kOne, true) : 0;
        }
    }
    __syncthreads();
    const Row r = sh.row;
    auto write = [&](int index, float z, uint64_t total) {
        if (!QMM_DCHECK(index >= 0 && index < p.V)) return;
        p.tokens[row] = index;
        if (!p.logp) return;
        p.logp[row] = log_share(sh, z, r.top, temperature, total);
    };

    if (r.top == -INFINITY || !(temperature > 0.0f) || top_k == 1 || min_p > 1.0f || top_p <= 0.0f) {
        // ---- the first in rank alone, or nothing ----
        int first = INT_MAX;
        for (int i = tid; i < n; i += kThreads)
            if (logit(i) == r.top) first = min(first, from + i);
        first = __reduce_min_sync(0xffffffffu, first);
        if (tid == 0) sh.first = INT_MAX;
        __syncthreads();
        if (lane == 0) atomicMin(&sh.first, first);
        __syncthreads();
        barrier();
        if (rank == 0 && warp == 0) {
            first = lane < ctas ? (int)remote_u32(&sh.first, lane) : INT_MAX;
            first = __reduce_min_sync(0xffffffffu, first);
            if (lane == 0) {
                p.tokens[row] = r.top == -INFINITY ? -1 : first;
                if (p.logp) p.logp[row] = r.top == -INFINITY ? -INFINITY : 0.0f;
            }
        }
        barrier();                                                     // nobody leaves while its memory is read
        return;
    }

    // ---- what is kept: places up to that of index border_i at logit border_z ----
    float border_z = -INFINITY;
    int border_i = INT_MAX;
    auto kept = [&](float z, int i) { return z > border_z || (z == border_z && from + i <= border_i); };
    auto set_border = [&](uint64_t place) {
        border_z = logit_of(place);
        border_i = (int)(uint32_t)place;
    };
    auto clear = [&] {
        for (int i = tid; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0;
        __syncthreads();
    };
    auto add = [&](int bin, uint64_t w) {
        const uint32_t x = (uint32_t)w, old = atomicAdd(&sh.lo[bin], x), up = (uint32_t)(w >> 32) + (old + x < x ? 1u : 0u);
        if (up) atomicAdd(&sh.hi[bin], up);
    };
    // Of the four bins that find_bins has found the one in question, as sh.bin, sh.left and sh.upto.  (The CTAs exchange sums of
    // four bins, for all bins a CTA would read 64 KB of the others' memory: 3 us.)
    auto find_bin_of_four = [&](bool sums) {
        if (warp == 0) {
            uint64_t s[4] = {0, 0, 0, 0};
            if (lane < ctas) {
                const uint4 lo = remote_u128(&sh.lo[sh.bin], lane);
                s[0] = lo.x; s[1] = lo.y; s[2] = lo.z; s[3] = lo.w;
                if (sums) {
                    const uint4 hi = remote_u128(&sh.hi[sh.bin], lane);
                    s[0] += (uint64_t)hi.x << 32; s[1] += (uint64_t)hi.y << 32; s[2] += (uint64_t)hi.z << 32; s[3] += (uint64_t)hi.w << 32;
                }
            }
            uint64_t all = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int m = 1; m < kMaxCluster; m <<= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], m);
                all += s[k];
            }
            if (lane == 0) {
                uint64_t before = 0, left = sh.left, upto = sh.upto - all;
                int bin = 0;
                uint64_t in = s[0];
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    if (bin == k - 1 && before + in < left) {
                        before += in;
                        in = s[k];
                        bin = k;
                    }
                }
                sh.bin += bin;
                sh.left = left - before;
                sh.upto = upto + before + in;
            }
        }
        __syncthreads();
    };
    // Adds up the CTAs' histograms and finds the four bins in which the sum from bin 0 on reaches want(sum of all): sh.bin (the
    // first of them), what is wanted of them sh.left, and the sum up to their end sh.upto.
    auto find_bins = [&](bool sums, auto want) {
        __syncthreads();
        if (tid < kSums) {
            uint64_t s = 0;
            const uint4 lo = *reinterpret_cast<const uint4 *>(&sh.lo[4 * tid]);
            s = (uint64_t)lo.x + lo.y + lo.z + lo.w;
            if (sums) {
                const uint4 hi = *reinterpret_cast<const uint4 *>(&sh.hi[4 * tid]);
                s += ((uint64_t)hi.x + hi.y + hi.z + hi.w) << 32;
            }
            sh.sums[tid] = s;
        }
        __syncthreads();
        barrier();
        uint64_t s = 0;
        if (tid < kSums) {
            uint64_t of[kMaxCluster];                                  // all under way before the first is added
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) of[c] = c < ctas ? remote_u64(&sh.sums[tid], c) : 0;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) s += of[c];
        }
        uint64_t all;
        const uint64_t before = sums_before<kWarps>(s, sh.part, all), w = want(all);
        if (before < w && before + s >= w) {
            sh.bin = 4 * tid;
            sh.left = w - before;
            sh.upto = before + s;
        }
        __syncthreads();
    };
    // The bin of a logit by its distance from the largest: subtraction and product are monotonic, so bins follow the order.
    auto bin_of = [&](float z) { return min(kBins - 1, __float2int_rz(__fmul_rn(__fsub_rn(r.top, z), r.scale))); };   // (NaN gives bin 0: inf - inf)
    // The kept elements of bins first .. last to the first CTA (at most kCand of them; all are counted).
    auto gather = [&](int first, int last) {
#pragma unroll 4
        for (int i = tid; i < n; i += kThreads) {
            const float z = logit(i);
            const int b = bin_of(z);
            if (b < first || b > last || !kept(z, i)) continue;        // (they are few)
            const uint32_t at = atomicAdd(&sh.n_list, 1u);
            if (at < kCand) sh.list[at] = place_of(z, from + i);
        }
        __syncthreads();
        const uint32_t count = sh.n_list;
        if (tid == 0 && count) sh.list_at = remote_add(&sh.n_cand, 0, count);
        __syncthreads();
        for (uint32_t k = tid; k < min(count, (uint32_t)kCand); k += kThreads)
            if (sh.list_at + k < kCand) remote_store(&sh.cand[sh.list_at + k], 0, sh.list[k]);
        if (tid == 0) sh.n_list = 0;
        __syncthreads();
        barrier();
    };
    // The border among the gathered: the left-th of them, or the one at which the sum of w reaches `left`.
    auto border_of_gathered = [&](bool sums, uint64_t left) {
        if (rank == 0) {
            const int m = (int)sh.n_cand;
            sort(sh.cand, m);
            if (sums) {
                uint64_t w[2], all;
#pragma unroll
                for (int k = 0; k < 2; ++k) w[k] = 2 * tid + k < m ? weight_of_few(sh, logit_of(sh.cand[2 * tid + k])) : 0;
                uint64_t before = sums_before<kWarps>(w[0] + w[1], sh.part, all);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (before < left && before + w[k] >= left) sh.border = sh.cand[2 * tid + k];
                    before += w[k];
                }
            } else if (tid == 0) {
                sh.border = sh.cand[min((int)left, m) - 1];
            }
            if (tid == 0) sh.n_cand = 0;
            __syncthreads();
        }
        barrier();
        set_border(remote_u64(&sh.border, 0));
    };
    // The border by the digits of the places, 9 bits at a time, 32 of the logit and 20 of the index: whatever the logits.
    auto border_by_digits = [&](bool sums, uint64_t left) {
        uint64_t prefix = 0;
#pragma unroll 1
        for (int digit = 0; digit < 7; ++digit) {
            const int shift = digit < 4 ? 32 + (digit < 3 ? 23 - 9 * digit : 0) : (digit == 4 ? 11 : (digit == 5 ? 2 : 0));
            const int bits = digit == 3 ? 5 : (digit == 6 ? 2 : 9);
            clear();
            for (int i = tid; i < n; i += kThreads) {
                const float z = logit(i);
                const uint64_t place = place_of(z, from + i);
                if (place >> shift >> bits != prefix || !kept(z, i)) continue;
                const int bin = 4 * (int)((place >> shift) & ((1u << bits) - 1));
                if (!sums) {
                    atomicAdd(&sh.lo[bin], 1u);
                } else {
                    const uint64_t w = weight_of_few(sh, z);
                    if (w) add(bin, w);
                }
            }
            find_bins(sums, [&](uint64_t) { return left; });
            prefix = prefix << bits | (uint32_t)(sh.bin / 4);
            left = sh.left;
            if (digit == 3) {
                prefix <<= 12;                                         // (an index has 20 bits)
                if (sums) {
                    // the logit is found: of its equals so many are kept
                    const uint64_t w = weight_of_few(sh, unordered(~(uint32_t)(prefix >> 12)));
                    left = w ? (left + w - 1) / w : 1;
                    sums = false;
                }
            }
            barrier();                                                 // before the histograms are cleared
        }
        set_border(prefix);
    };

    // ---- the cuts, of counts and of sums ----
#pragma unroll 1
    for (int cut = 0; cut < 2; ++cut) {
        const bool sums = cut == 1;
        if (sums ? !(top_p < 1.0f) : !(top_k > 0 && top_k < p.V)) continue;
        // The k largest logits lie no lower than the k-th largest of the threads' maxima: where k is small a histogram of those alone,
        // one logit a thread, leaves few candidates.  (Shared memory takes about two atomic additions a cycle.)
        bool alone, quick = !sums && 8 * top_k <= kThreads * ctas;
        int bin;
        uint64_t left, upto, want;
#pragma unroll 1
        while (true) {
            clear();
            if (quick) {
                atomicAdd(&sh.lo[bin_of(own_top)], 1u);
            } else if (!sums) {
#pragma unroll 4
                for (int i = tid; i < n; i += kThreads) atomicAdd(&sh.lo[bin_of(logit(i))], 1u);
            } else {
#pragma unroll 2
                for (int i = tid; i < n; i += kThreads) {
                    const float z = logit(i);
                    const uint64_t w = kept(z, i) ? weight(r, z, sh) : 0;
                    if (w) add(bin_of(z), w);
                }
            }
            find_bins(sums, [&](uint64_t all) { return want = sums ? max((uint64_t)1, times(top_p, all, true)) : (uint64_t)top_k; });
            find_bin_of_four(sums);
            bin = sh.bin;
            left = sh.left;
            alone = quick || (!sums && sh.upto <= kCand);
            gather(alone ? 0 : bin, bin);
            upto = remote_u32(&sh.n_cand, 0);
            barrier();                                                 // the count is read before it is cleared
            if (!quick || upto <= kCand) break;
            if (rank == 0 && tid == 0) sh.n_cand = 0;
            quick = false;
        }
        if (alone) {
            // ---- the first CTA alone: cuts in the order of the logits, then the token in the order of the indexes ----
            if (rank != 0) return;
            uint64_t *ws = reinterpret_cast<uint64_t *>(sh.lo), *order = reinterpret_cast<uint64_t *>(sh.hi);
            if (tid == 0) sh.first = (int)upto;
            sort(sh.cand, (int)upto);
            uint64_t w[2], all, total;
#pragma unroll
            for (int k = 0; k < 2; ++k) w[k] = 2 * tid + k < top_k && 2 * tid + k < (int)upto ? weight_of_few(sh, logit_of(sh.cand[2 * tid + k])) : 0;
            uint64_t before = sums_before<kWarps>(w[0] + w[1], sh.part, all);
            const uint64_t want = top_p < 1.0f ? max((uint64_t)1, times(top_p, all, true)) : ~(uint64_t)0;
            // kept are the elements before the first one that a cut takes: weights of neighbouring logits can lie a unit the wrong way
            // round, so one behind it may be large enough again
            int first = INT_MAX;
#pragma unroll
            for (int k = 1; k >= 0; --k) {
                const int i = 2 * tid + k;
                if (i >= top_k || i >= (int)upto || (k ? before + w[0] : before) >= want || (i > 0 && w[k] < r.least)) first = i;
            }
            first = __reduce_min_sync(0xffffffffu, first);
            if (lane == 0 && first < INT_MAX) atomicMin(&sh.first, first);
            __syncthreads();
            const int m = sh.first;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = 2 * tid + k;
                if (i >= m) continue;
                ws[i] = w[k];
                order[i] = (uint64_t)(uint32_t)sh.cand[i] << 32 | (uint32_t)i;
            }
            sort(order, m);
#pragma unroll
            for (int k = 0; k < 2; ++k) w[k] = 2 * tid + k < m ? ws[(uint32_t)order[2 * tid + k]] : 0;
            before = sums_before<kWarps>(w[0] + w[1], sh.part, total);
            const uint64_t target = u >= 1.0f ? total - 1 : (u > 0.0f ? times(u, total, false) : 0);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (before <= target && target < before + w[k]) {
                    const uint64_t place = sh.cand[(uint32_t)order[2 * tid + k]];
                    write((int)(uint32_t)place, logit_of(place), total);
                }
                before += w[k];
            }
            return;
        }
        if (upto <= kCand) {
            border_of_gathered(sums, left);
        } else {
            if (rank == 0 && tid == 0) sh.n_cand = 0;
            border_by_digits(sums, want);
        }
    }

    // ---- sums of the warps' segments, in the order of the indexes ----
    const int seg_len = (per + kWarps * 32 - 1) / (kWarps * 32) * 32;
    auto weight_of = [&](int i) -> uint64_t {
        const float z = logit(i);
        if (!kept(z, i)) return 0;
        const uint64_t w = weight_of_few(sh, z);
        return w >= r.least ? w : 0;
    };
    {
        uint64_t sum = 0;
        const int end = min(n, (warp + 1) * seg_len);
        if (border_i == INT_MAX && r.least == 0) {                     // all are kept
#pragma unroll 4
            for (int i = warp * seg_len + lane; i < end; i += 32) sum += weight(r, logit(i), sh);
        } else if (border_i == INT_MAX) {
#pragma unroll 2
            for (int i = warp * seg_len + lane; i < end; i += 32) {
                const uint64_t w = weight(r, logit(i), sh);
                sum += w >= r.least ? w : 0;
            }
        } else {
            // those kept are lined up first: their weights, in any order, are then a whole warp's work (64 rows, top_p = 0.95: 89 us,
            // with each weight where it lies 99)
            float *line = reinterpret_cast<float *>(sh.list) + 64 * warp;
            int waiting = 0;
            auto take = [&](bool have) {
                const uint64_t w = have ? weight(r, line[lane], sh) : 0;
                sum += w >= r.least ? w : 0;
            };
            for (int i = warp * seg_len + lane; i - lane < end; i += 32) {
                const float z = i < end ? logit(i) : 0.0f;
                const bool in = i < end && kept(z, i);
                const unsigned mask = __ballot_sync(0xffffffffu, in);
                if (in) line[waiting + __popc(mask & ((1u << lane) - 1))] = z;
                waiting += __popc(mask);
                if (waiting < 32) continue;
                __syncwarp();
                take(true);
                const float next = line[32 + lane];
                __syncwarp();
                waiting -= 32;
                if (lane < waiting) line[lane] = next;                 // (the places behind are other lanes' to write)
            }
            __syncwarp();
            take(lane < waiting);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) sh.seg_sum[warp] = sum;
    }
    __syncthreads();
    barrier();
    uint64_t total;
    {
        // thread j has segment j % kWarps of CTA j / kWarps
        const uint64_t sum = tid < ctas * kWarps ? remote_u64(&sh.seg_sum[tid % kWarps], tid / kWarps) : 0;
        const uint64_t before = sums_before<kWarps>(sum, sh.part, total);
        // u beyond [0, 1) counts as its nearest end, NaN as 0
        const uint64_t target = u >= 1.0f ? total - 1 : (u > 0.0f ? times(u, total, false) : 0);
        if (before <= target && target < before + sum) {
            sh.seg = tid;
            sh.target = target - before;
        }
    }
    barrier();                                                         // nobody reads another CTA's memory from here on
    const int seg = sh.seg;
    if (seg < 0 || seg / kWarps != rank) return;

    // ---- the token: this CTA's threads share the segment ----
    const int begin = (seg % kWarps) * seg_len, end = min(n, begin + seg_len), each = (seg_len + kThreads - 1) / kThreads;
    const int i0 = min(end, begin + tid * each), i1 = min(end, i0 + each);
    uint64_t all, sum = 0;
    for (int i = i0; i < i1; ++i) sum += weight_of(i);
    uint64_t before = sums_before<kWarps>(sum, sh.part, all);
    if (before <= sh.target && sh.target < before + sum) {
        for (int i = i0; i < i1; ++i) {
            before += weight_of(i);
            if (sh.target < before) {
                write(from + i, logit(i), total);
                break;
            }
        }
    }
}

template <typename T, bool STAGED, int THREADS>
cudaError_t launch(const SampleParams &p, int ctas, int per, int vec, cudaStream_t s) {
    const size_t smem = sizeof(Shared) + (STAGED ? ((size_t)per * sizeof(T) + 15) / 16 * 16 : 0);
    static int done[4] = {0, 0, 0, 0};
    const cudaError_t e = ensure_smem_limit(sample_kernel<T, STAGED, THREADS>, 227 * 1024, done);
    if (e != cudaSuccess) return e;
    if (p.R * ctas > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl_cluster(sample_kernel<T, STAGED, THREADS>, dim3((unsigned)(p.R * ctas)), (unsigned)ctas, THREADS, smem, s, p, ctas, per, vec);
}

}  // namespace

cudaError_t launch_sample(qmm_dtype t, const SampleParams &p, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using T = decltype(z);
        // Slices of 60 KB, two CTAs an SM; smaller ones where rows are few, and there one CTA of twice the threads; the largest ones of which
        // an SM holds two where rows are so many that their CTAs are more than two waves.  (128256 bf16 logits, clusters of 8 and of 4, us:
        // 128 rows of mixed requests 87 and 86, of top_k = 50 63 and 43, of top_p = 0.95 168 and 141; 64 rows 53 and 63, 38 and
        // 22, 91 and 79: in one wave the slowest request's own time counts.)
        constexpr int kSlice = 60 * 1024 / (int)sizeof(T), kLargest = (228 * 512 - 1024 - (int)sizeof(Shared)) / 128 * 128 / (int)sizeof(T);
        auto clusters = [&](int slice) {
            int ctas = 1;
            while (ctas < kMaxCluster && (int64_t)ctas * slice < p.V) ctas *= 2;
            return ctas;
        };
        int ctas = clusters(kSlice);
        if (p.R * ctas > 2 * 304) ctas = clusters(kLargest);
        while (ctas < kMaxCluster && p.R * ctas * 2 <= 152 && p.V / (ctas * 2) >= 2048) ctas *= 2;
        const int per = ((p.V + ctas - 1) / ctas + 15) / 16 * 16;
        const bool vec = (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && (p.ld * (int64_t)sizeof(T)) % 16 == 0;
        if (sizeof(Shared) + (size_t)per * sizeof(T) > 227 * 1024) return launch<T, false, 512>(p, ctas, per, vec, s);
        return p.R * ctas <= 152 ? launch<T, true, 1024>(p, ctas, per, vec, s) : launch<T, true, 512>(p, ctas, per, vec, s);
    });
}

QMM_DCHECK_READER(read_dcheck_sample)

}  // namespace qmm
