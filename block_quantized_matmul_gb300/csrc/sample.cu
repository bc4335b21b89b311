// sample.cu -- one token of each row of logits z, from a random number u:
//   w_i = exp((z_i - max z) / temperature); kept are, in the order of z (the earlier index first on ties), the top_k first, of
//   those the ones before which the others sum to less than top_p of the whole, of those the ones with w >= min_p; the token
//   is the first index at which the running sum of the kept w exceeds u times their sum.
//
// Every cut is a prefix of the order of z, so what is kept is "z above a border, and the t first of those at it".  The
// border is found digit by digit of z as an ordered 32-bit number (11, 11 and 10 bits): a histogram of counts for top_k, of
// sums of w for top_p.
//
// Borders of sums have to fall where the formula's do, to within an error far below one token's share: fp32 sums over 10^5 tokens
// would not do, and fp64 is too slow on this GPU for every logit.  So w is a whole number, 2^43 for the largest, computed in
// pairs of fp32 and 64-bit integers (`weight`, within 2^-42), and all sums are sums of integers: exact, and
// the same in any order, so histograms may be filled by atomics.
//
// A cluster of up to 8 CTAs takes a row, each CTA a slice of it that stays in shared memory from the first pass on.  What the
// CTAs find is exchanged through distributed shared memory: each adds up all histograms for itself, so a digit costs one cluster
// barrier.
#include "qmm_internal.cuh"

#include "elem.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 2048, kMaxCluster = 8;
constexpr int kOne = 43;                    // w of the largest logit is 2^kOne

// 2^(j / 1024) times 2^kOne, from the square roots of 2: ten factors at most, each within 2^-52.
struct Powers {
    uint64_t v[1024];
};
constexpr Powers make_powers() {
    double root[10] = {};
    double x = 2.0;
    for (int i = 0; i < 10; ++i) {
        double r = 1.0 + (x - 1.0) / 2;     // Newton's iteration for the square root of x, 1 < x <= 2
        for (int k = 0; k < 6; ++k) r = 0.5 * (r + x / r);
        root[i] = x = r;
    }
    Powers p = {};
    for (int j = 0; j < 1024; ++j) {
        double v = 1.0;
        for (int i = 0; i < 10; ++i)
            if (j & (512 >> i)) v *= root[i];
        p.v[j] = (uint64_t)(v * (double)((uint64_t)1 << kOne) + 0.5);
    }
    return p;
}
__device__ const Powers g_powers = make_powers();

struct alignas(16) Shared {
    uint64_t powers[1024];
    uint32_t lo[2][kBins], hi[2][kBins];    // a histogram of counts (lo), or of sums in two words, of this CTA's slice
    uint64_t seg_sum[kWarps];               // of each warp's segment: sum of w above the border, and how many are at it
    uint32_t seg_ties[kWarps];
    uint64_t part[kWarps];
    float top, ch, cl;                      // the slice's maximum; log2(e) / temperature in two terms
    uint64_t least;                         // w that min_p asks for
    // what one thread finds for all
    uint32_t prefix;
    uint64_t left, all;
    int seg;
    uint64_t target;
    uint64_t quota;
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

__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// w of logit z under the maximum m: 2^kOne * 2^y, y = (z - m) * (ch + cl), to the nearest whole number but for 2^-42 of itself.
// z - m and the product are pairs of fp32 (46 bits or more); y = n / 1024 + g, |g| <= 1/2048, and 2^g - 1 = t + t^2/2 + t^3/6
// with t = g ln 2 in two terms (the next term is below 2^-50), as a whole number of 2^-42.
__device__ __forceinline__ uint64_t weight(float z, float m, float ch, float cl, const uint64_t *powers) {
    if (z == m) return (uint64_t)1 << kOne;
    const float hi = __fsub_rn(z, m), b = __fsub_rn(hi, z), lo = __fadd_rn(__fsub_rn(z, __fsub_rn(hi, b)), __fsub_rn(-m, b));
    const float yh = __fmul_rn(hi, ch), yl = __fadd_rn(__fmaf_rn(hi, ch, -yh), __fmaf_rn(hi, cl, __fmul_rn(lo, ch)));
    if (!(yh > -(float)(kOne + 1))) return 0;                          // (and for z = -inf)
    const float magic = 12582912.0f, r = __fmaf_rn(yh, 1024.0f, magic);
    const int n = __float_as_int(r) - __float_as_int(magic);
    const float g = __fmaf_rn(__fsub_rn(r, magic), -1.0f / 1024.0f, yh);
    const float ln2h = 0.693147182464599609375f, ln2l = -1.9046542943909386e-9f;      // ln 2 and what fp32 leaves of it
    const float th = __fmul_rn(g, ln2h), tl = __fadd_rn(__fmaf_rn(g, ln2h, -th), __fmaf_rn(g, ln2l, __fmul_rn(yl, ln2h)));
    const float t = __fadd_rn(th, tl), small = __fmaf_rn(__fmul_rn(t, t), __fmaf_rn(t, 1.0f / 6.0f, 0.5f), tl);
    const float unit = 4398046511104.0f;                               // 2^42
    const int p = __float2int_rn(__fmul_rn(th, unit)) + __float2int_rn(__fmul_rn(small, unit));
    const uint64_t base = powers[n & 1023];
    const uint64_t w = base + (uint64_t)(((int64_t)p * (int64_t)(int32_t)(base >> 13)) >> 29);
    const int down = -(n >> 10);                                       // 0 .. kOne + 1
    return down <= 0 ? w : (w + ((uint64_t)1 << (down - 1))) >> down;
}

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

// Sums of v over the threads before this one; `all`: over all of them.
__device__ __forceinline__ uint64_t sums_before(uint64_t v, uint64_t *part, uint64_t &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    uint64_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint64_t y = part[w];
        if (w < warp) before += y;
        all += y;
    }
    __syncthreads();
    return before + x - v;
}

// STAGED: the slice lies in shared memory after the first pass, otherwise it is read again each time.
template <typename T, bool STAGED>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p, int ctas, int per, int vec) {
    constexpr int kLevels = sizeof(T) == 4 ? 3 : 2;                    // 16-bit logits as fp32 end within 22 bits
    constexpr uint32_t kKey = sizeof(T) == 4 ? 0xFFFFFFFFu : 0xFFFFFC00u;
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    T *stage = reinterpret_cast<T *>(smem + sizeof(Shared));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = (int)(blockIdx.x % (unsigned)ctas);
    const int64_t row = blockIdx.x / (unsigned)ctas;
    for (int i = threadIdx.x; i < 1024; i += kThreads) sh.powers[i] = g_powers.v[i];
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.lo[0][i] = sh.lo[1][i] = sh.hi[0][i] = sh.hi[1][i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int from = min(rank * per, p.V), n = min(per, p.V - from);
    const T *src = static_cast<const T *>(p.logits) + row * p.ld + from;
    // NaN counts as -inf, -0 as 0
    auto clean = [](float v) { return isnan(v) ? -INFINITY : v + 0.0f; };
    auto logit = [&](int i) { return clean(elem_to_float(STAGED ? stage[i] : src[i])); };

    // ---- the first pass: the slice to shared memory, its maximum ----
    float top = -INFINITY;
    constexpr int kVec = 16 / (int)sizeof(T), kAhead = 4;
    int done = 0;
    if (vec) {
        const int pieces = n / kVec;
        for (int i = threadIdx.x; i < pieces; i += kThreads * kAhead) {
            uint4 v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i + u * kThreads < pieces) v[u] = reinterpret_cast<const uint4 *>(src)[i + u * kThreads];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (i + u * kThreads >= pieces) continue;
                if constexpr (STAGED) reinterpret_cast<uint4 *>(stage)[i + u * kThreads] = v[u];
                const T *e = reinterpret_cast<const T *>(&v[u]);
#pragma unroll
                for (int k = 0; k < kVec; ++k) top = fmaxf(top, elem_to_float(e[k]));      // (fmaxf passes over NaN)
            }
        }
        done = pieces * kVec;
    }
    for (int i = done + threadIdx.x; i < n; i += kThreads) {
        const T v = src[i];
        if constexpr (STAGED) stage[i] = v;
        top = fmaxf(top, elem_to_float(v));
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    if (lane == 0) sh.part[warp] = __float_as_uint(top);
    const float temperature = p.temperature ? p.temperature[row] : 1.0f, top_p = p.top_p ? p.top_p[row] : 1.0f, min_p = p.min_p ? p.min_p[row] : 0.0f;
    const int top_k = p.top_k ? p.top_k[row] : 0;
    if (threadIdx.x == 0) {
        const double c = 1.4426950408889634074 / (double)temperature;
        sh.ch = (float)c;
        sh.cl = fabsf(sh.ch) < INFINITY ? (float)(c - (double)sh.ch) : 0.0f;
        sh.least = min_p > 0.0f && min_p <= 1.0f ? (uint64_t)ceil((double)min_p * (double)((uint64_t)1 << kOne)) : 0;
    }
    __syncthreads();
    if (warp == 0) {
        top = lane < kWarps ? __uint_as_float((uint32_t)sh.part[lane]) : -INFINITY;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        if (lane == 0) sh.top = top;
    }
    __syncthreads();
    if (ctas > 1) cluster_sync();
    top = -INFINITY;
    for (int c = 0; c < ctas; ++c) top = fmaxf(top, __uint_as_float(remote_u32(&sh.top, c)));
    const float m = top + 0.0f, ch = sh.ch, cl = sh.cl;
    const bool nothing = m == -INFINITY;
    const uint64_t least = nothing ? ~(uint64_t)0 : sh.least;            // (nothing is kept of nothing)

    // ---- what is kept: keys above `border`, and the first `quota` of those at it ----
    uint32_t border = 0;                                               // no logit's key but -inf's, whose w is 0, is as low
    uint64_t quota = 0;
    const bool first_only = !(temperature > 0.0f) || top_k == 1 || min_p > 1.0f || top_p <= 0.0f;
    int round = 0;                                                     // histograms so far: they use two buffers in turn
    // Adds up the CTAs' histograms and finds the bin in which the sum from above reaches `want`; sh.prefix: the
    // bin, sh.left: what is wanted of it.  want(all) gives the sum that is wanted.
    auto find_bin = [&](bool sums, auto want) {
        const int buf = round & 1;
        ++round;
        __syncthreads();
        if (ctas > 1) cluster_sync();
        uint64_t bin[4] = {0, 0, 0, 0};                                // 4 i .. 4 i + 3 from the top
        const int at = kBins - 4 - 4 * (int)threadIdx.x;
        for (int c = 0; c < ctas; ++c) {
            const uint4 lo = remote_u128(&sh.lo[buf][at], c);
            bin[3] += lo.x; bin[2] += lo.y; bin[1] += lo.z; bin[0] += lo.w;
            if (sums) {
                const uint4 hi = remote_u128(&sh.hi[buf][at], c);
                bin[3] += (uint64_t)hi.x << 32; bin[2] += (uint64_t)hi.y << 32; bin[1] += (uint64_t)hi.z << 32; bin[0] += (uint64_t)hi.w << 32;
            }
        }
        // the buffer of the round before is read by nobody any more: zeros for the next round
        for (int i = threadIdx.x; i < kBins; i += kThreads) sh.lo[buf ^ 1][i] = sh.hi[buf ^ 1][i] = 0;
        uint64_t all;
        uint64_t before = sums_before(bin[0] + bin[1] + bin[2] + bin[3], sh.part, all);
        const uint64_t w = want(all);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (before < w && before + bin[k] >= w) {
                sh.prefix = (uint32_t)(kBins - 1 - 4 * (int)threadIdx.x - k);
                sh.left = w - before;
            }
            before += bin[k];
        }
        __syncthreads();
    };
    constexpr int kShift[3] = {21, 10, 0};
    if (first_only) {
        border = ordered(m) & kKey;
        quota = 1;
    } else if (!nothing) {
        if (top_k > 0 && top_k < p.V) {
            uint64_t left = (uint64_t)top_k;
            uint32_t prefix = 0, mask = 0;
#pragma unroll
            for (int level = 0; level < kLevels; ++level) {
                uint32_t *hist = sh.lo[round & 1];
                const int shift = kShift[level], bits = level == 2 ? 10 : 11;
                for (int i = threadIdx.x; i < n; i += kThreads) {
                    const uint32_t key = ordered(logit(i));
                    if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1u);
                }
                find_bin(false, [&](uint64_t) { return left; });
                prefix |= sh.prefix << shift;
                mask |= ((1u << bits) - 1) << shift;
                left = sh.left;
            }
            border = prefix;
            quota = left;
        }
        if (top_p < 1.0f) {
            // the ones at the border of top_k count as one element of their common w
            const uint32_t kth = border;
            const uint64_t kth_quota = quota;
            const float kth_z = unordered(kKey != 0xFFFFFFFFu && !(kth & 0x80000000u) ? kth | ~kKey : kth);
            uint64_t left = 0;
            uint32_t prefix = 0, mask = 0;
#pragma unroll
            for (int level = 0; level < kLevels; ++level) {
                uint32_t *lo = sh.lo[round & 1], *hi = sh.hi[round & 1];
                const int shift = kShift[level], bits = level == 2 ? 10 : 11;
                auto add = [&](uint32_t key, uint64_t w) {
                    const uint32_t bin = (key >> shift) & ((1u << bits) - 1), x = (uint32_t)w, old = atomicAdd(&lo[bin], x);
                    const uint32_t up = (uint32_t)(w >> 32) + (old + x < x ? 1u : 0u);
                    if (up) atomicAdd(&hi[bin], up);
                };
                for (int i = threadIdx.x; i < n; i += kThreads) {
                    const float z = logit(i);
                    const uint32_t key = ordered(z);
                    if ((key & mask) != prefix || (key & kKey) <= kth) continue;
                    const uint64_t w = weight(z, m, ch, cl, sh.powers);
                    if (w) add(key, w);
                }
                if (rank == 0 && threadIdx.x == 0 && kth_quota && (kth & mask) == prefix) {
                    const uint64_t w = kth_quota * weight(kth_z, m, ch, cl, sh.powers);
                    if (w) add(kth, w);
                }
                if (level == 0) {
                    find_bin(true, [&](uint64_t all) {
                        const uint64_t w = times(top_p, all, true);
                        return w ? w : (uint64_t)1;
                    });
                } else {
                    find_bin(true, [&](uint64_t) { return left; });
                }
                prefix |= sh.prefix << shift;
                mask |= ((1u << bits) - 1) << shift;
                left = sh.left;
            }
            border = prefix;
            const float z = unordered(kKey != 0xFFFFFFFFu && !(prefix & 0x80000000u) ? prefix | ~kKey : prefix);
            const uint64_t w = weight(z, m, ch, cl, sh.powers);
            quota = w ? (left + w - 1) / w : 1;
        }
    }

    // ---- sums of the warps' segments, in the order of the indexes ----
    const float border_z = border == 0 ? -INFINITY : unordered(kKey != 0xFFFFFFFFu && !(border & 0x80000000u) ? border | ~kKey : border);
    uint64_t at_border = border == 0 ? 0 : weight(border_z, m, ch, cl, sh.powers);
    if (at_border < least) at_border = 0;
    const int seg_len = (per + kWarps * 32 - 1) / (kWarps * 32) * 32;
    {
        uint64_t sum = 0;
        uint32_t ties = 0;
        const int end = min(n, (warp + 1) * seg_len);
        for (int i = warp * seg_len + lane; i < end; i += 32) {
            const float z = logit(i);
            const uint32_t key = ordered(z) & kKey;
            if (key > border) {
                const uint64_t w = weight(z, m, ch, cl, sh.powers);
                if (w >= least) sum += w;
            }
            ties += key == border;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        ties = __reduce_add_sync(0xffffffffu, ties);
        if (lane == 0) {
            sh.seg_sum[warp] = sum;
            sh.seg_ties[warp] = ties;
        }
    }
    if (threadIdx.x == 0) sh.seg = -1;
    __syncthreads();
    if (ctas > 1) cluster_sync();
    uint64_t total;
    {
        // thread j has segment j % kWarps of CTA j / kWarps
        const int j = threadIdx.x;
        uint64_t sum = 0, ties = 0, all;
        if (j < ctas * kWarps) {
            sum = remote_u64(&sh.seg_sum[j % kWarps], j / kWarps);
            ties = remote_u32(&sh.seg_ties[j % kWarps], j / kWarps);
        }
        const uint64_t ties_before = sums_before(ties, sh.part, all);
        const uint64_t mine = quota > ties_before ? min(ties, quota - ties_before) : 0;
        sum += mine * at_border;
        const uint64_t before = sums_before(sum, sh.part, total);
        // u beyond [0, 1) counts as its nearest end, NaN as 0
        const float u = p.u[row];
        const uint64_t target = u >= 1.0f ? total - 1 : (u > 0.0f ? times(u, total, false) : 0);
        if (before <= target && target < before + sum) {
            sh.seg = j;
            sh.target = target - before;
            sh.quota = mine;
        }
    }
    if (ctas > 1) cluster_sync();                                      // nobody reads another CTA's memory from here on
    else __syncthreads();
    const int seg = sh.seg;
    if (seg < 0) {
        // nothing to choose from: every logit is -inf or NaN
        if (rank == 0 && threadIdx.x == 0) {
            p.tokens[row] = -1;
            if (p.logp) p.logp[row] = -INFINITY;
        }
        return;
    }
    if (seg / kWarps != rank) return;

    // ---- the token: this CTA's threads share the segment ----
    const int begin = (seg % kWarps) * seg_len, end = min(n, begin + seg_len), each = (seg_len + kThreads - 1) / kThreads;
    const int i0 = min(end, begin + (int)threadIdx.x * each), i1 = min(end, i0 + each);
    uint64_t all, ties = 0, sum = 0;
    for (int i = i0; i < i1; ++i) ties += (ordered(logit(i)) & kKey) == border;
    uint64_t tie = sums_before(ties, sh.part, all);
    const uint64_t mine = sh.quota > tie ? sh.quota - tie : 0;         // of this thread's, so many at the border are kept
    uint64_t kept = 0;
    auto weight_of = [&](int i) -> uint64_t {
        const float z = logit(i);
        const uint32_t key = ordered(z) & kKey;
        if (key > border) {
            const uint64_t w = weight(z, m, ch, cl, sh.powers);
            return w >= least ? w : 0;
        }
        return key == border && kept++ < mine ? at_border : 0;
    };
    for (int i = i0; i < i1; ++i) sum += weight_of(i);
    uint64_t before = sums_before(sum, sh.part, all);
    if (before <= sh.target && sh.target < before + sum) {
        kept = 0;
        for (int i = i0; i < i1; ++i) {
            before += weight_of(i);
            if (sh.target < before) {
                if (!QMM_DCHECK(from + i < p.V)) break;
                p.tokens[row] = from + i;
                if (p.logp) {
                    const float z = logit(i);
                    const double y = z == m || first_only ? 0.0 : ((double)z - (double)m) / (double)temperature;
                    p.logp[row] = (float)(y - log((double)total * (1.0 / (double)((uint64_t)1 << kOne))));
                }
                break;
            }
        }
    }
}

template <typename T, bool STAGED>
cudaError_t launch(const SampleParams &p, int ctas, int per, int vec, cudaStream_t s) {
    const size_t smem = sizeof(Shared) + (STAGED ? ((size_t)per * sizeof(T) + 15) / 16 * 16 : 0);
    static int done[4] = {0, 0, 0, 0};
    const cudaError_t e = ensure_smem_limit(sample_kernel<T, STAGED>, 227 * 1024, done);
    if (e != cudaSuccess) return e;
    if (p.R * ctas > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl_cluster(sample_kernel<T, STAGED>, dim3((unsigned)(p.R * ctas)), (unsigned)ctas, kThreads, smem, s, p, ctas, per, vec);
}

}  // namespace

cudaError_t launch_sample(qmm_dtype t, const SampleParams &p, cudaStream_t s) {
    return with_dtype(t, [&](auto z) {
        using T = decltype(z);
        // slices of 64 KB, two CTAs an SM; smaller ones where rows are few
        constexpr int kSlice = 64 * 1024 / (int)sizeof(T);
        int ctas = 1;
        while (ctas < kMaxCluster && (int64_t)ctas * kSlice < p.V) ctas *= 2;
        while (ctas < kMaxCluster && p.R * ctas * 2 <= 152 && p.V / (ctas * 2) >= 2048) ctas *= 2;
        const int per = ((p.V + ctas - 1) / ctas + 15) / 16 * 16;
        const bool vec = (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && (p.ld * (int64_t)sizeof(T)) % 16 == 0;
        if (sizeof(Shared) + (size_t)per * sizeof(T) <= 227 * 1024) return launch<T, true>(p, ctas, per, vec, s);
        return launch<T, false>(p, ctas, per, vec, s);
    });
}

QMM_DCHECK_READER(read_dcheck_sample)

}  // namespace qmm
