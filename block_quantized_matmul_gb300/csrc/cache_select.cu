// cache_select.cu -- which pages of the block-quantized cache (cache.cuh) a new token attends over.
//
// Bounds.  For a page, a head and an element e: lo = min_j k[j, e], hi = max_j k[j, e] over the page's tokens, in codes of 8
// bits with one scale a block of 32 for both, rounded outwards: d = up16(max(|lo|, |hi|) / 127), floor(lo / d), ceil(hi / d).
// Minima and maxima do not depend on an order, so a page's bounds are a function of its keys alone.
//
// Score.  sum_e q_e k_e <= sum_e (q_e > 0 ? q_e hi_e : q_e lo_e) for every key of the page.  The query row is quantized by the
// activations' rule, so the sum over a block of 32 is a whole number S below 2^20, exact in any order, and
//   score = sum_b (dq_b d_b) S_b  takes three fp32 roundings a block in the order of the blocks: every way of computing it
// gives the same bits, and so the same choice of pages.
//
// What bounds them.  Bounds: latency, the loads of a page's keys in rounds (5.2 us for the pages of 64 new tokens); with many pages also
// instructions, 9.6 an element with the join of the lanes and the codes of the bounds (17 us for the 22 MB of Q4_0 keys of four prompts of 3000 to 16384
// tokens and 8 heads: 58 % of the issue slots; with 94 registers a thread four warps share a scheduler, and a third of the time in which
// a warp does not issue is a wait for loads).  A step's grid is its sequences times the pages of the longest prompt, most of them of no use
// where prompts and single tokens come together: 255 sequences with a token each and a prompt of 2048 take 22 us, 256 such sequences 6.7
// (4096 to 8096 cached tokens, Q8_0, 8 heads, pages of 64).
// Scores: on mma, so that a page's codes are converted once for eight query rows: 128 tokens of 8 x 4 heads of 128 over 1024
// pages take 36 us (cold; 62 with products of bytes on the ALUs, 42 before query rows were loaded four at a time and page numbers a turn
// ahead), with the choice 47 in a graph: half of the issue slots.  Tokens of several sequences in a tile are scored one sequence after the
// other: the choice takes 289 us for those 255 tokens and the prompt, and 50 for the 256 tokens, a tile each.  Choice: latency, a
// histogram or two and a ranking (9 us).
#include "cache.cuh"
#include "elem.cuh"
#include "tc_common.cuh"

namespace qmm {
namespace {

// ---------------------------------------------------------------------------------------------
// Bounds
// ---------------------------------------------------------------------------------------------
struct BoundsParams {
    const uint8_t *k_cache;
    int64_t n_pages, ld_pages, n_seq, T, max_new;
    int H, log_p, per_seq;                  // pages of a sequence that may hold new tokens
    const int32_t *pages, *q_starts, *kv_lens;
    uint8_t *bounds;
};

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}

constexpr int kBoundWarps = 4;

// Bytes of w as fp32, the sign bits flipped (0 .. 255: 128 + the value): the low bits of 2^23 + v, no conversion.
__device__ __forceinline__ float byte_float(uint32_t w, int k) { return __fsub_rn(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | k)), 8388736.0f); }
// Nibble k of w as fp32, minus 8.
__device__ __forceinline__ float nibble_float(uint32_t w, int k) {
    return __fsub_rn(__uint_as_float(((w >> (4 * k)) & 15u) | 0x4B000000u), 8388616.0f);
}

// A warp takes a page of a head.  Lanes: PK pieces of 16 bytes of codes make a token (Q8_0: half a block each,
// Q4_0: a block), TOK = 32 / PK tokens at a time.  In the end the TOK lanes of a piece share its E elements out: half after half
// is exchanged for a partner's, until each has E / TOK of them over all tokens, to quantize and store.  (Where PK is no power of two
// the first PK lanes take all of them.)
template <int TYPE, int DB>
__global__ void __launch_bounds__(kBoundWarps * 32) cache_bounds_kernel(const BoundsParams p) {
    constexpr int CB = DB * (TYPE == QMM_Q8_0 ? 32 : 16), PK = CB / 16, TOK = 32 / PK, E = TYPE == QMM_Q8_0 ? 16 : 32, D = DB * 32;
    constexpr bool kShare = (PK & (PK - 1)) == 0;
    constexpr int N = kShare ? E / TOK : E;                            // elements of a lane in the end
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, P = 1 << p.log_p;
    int64_t unit = (int64_t)blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
    const int h = (int)(unit % p.H);
    unit /= p.H;
    const int64_t s = unit / p.per_seq;
    if (s >= p.n_seq) return;
    const int64_t q0 = p.q_starts[s], q1 = p.q_starts[s + 1], n = max((int64_t)0, min((int64_t)p.kv_lens[s], p.ld_pages << p.log_p));
    if (q0 < 0 || q1 > p.T || q1 <= q0 || n == 0) return;
    const int64_t from = max((int64_t)0, (int64_t)p.kv_lens[s] - min(q1 - q0, p.max_new)) >> p.log_p, number = from + unit % p.per_seq;
    if (number > (n - 1) >> p.log_p || !QMM_DCHECK(number < p.ld_pages)) return;
    const int64_t page = p.pages[s * p.ld_pages + number];
    if (page < 0 || page >= p.n_pages) return;
    const int have = (int)min((int64_t)P, n - (number << p.log_p));
    const uint8_t *chunk = p.k_cache + cache_chunk(TYPE, p.H, D, P, page, h);
    const uint16_t *scales = reinterpret_cast<const uint16_t *>(chunk + (int64_t)P * CB);
    const int piece = lane % PK, turn = min(lane / PK, TOK - 1), block = TYPE == QMM_Q8_0 ? piece / 2 : piece;
    float lo[E], hi[E];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        lo[i] = INFINITY;
        hi[i] = -INFINITY;
    }
    // tokens past the last stand for the last once more; two at a time
    for (int j = turn; j < have; j += 2 * TOK) {
        const int j2 = min(j + TOK, have - 1);
        const uint4 c = *reinterpret_cast<const uint4 *>(chunk + (int64_t)j * CB + piece * 16), c2 = *reinterpret_cast<const uint4 *>(chunk + (int64_t)j2 * CB + piece * 16);
        const float d = __half2float(__ushort_as_half(scales[j * DB + block])), d2 = __half2float(__ushort_as_half(scales[j2 * DB + block]));
        odd |= !(fabsf(d) < INFINITY) || !(fabsf(d2) < INFINITY);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w}, w2[4] = {c2.x, c2.y, c2.z, c2.w};
        auto take = [&](int e, float v, float u) {
            lo[e] = fminf(fminf(lo[e], v), u);
            hi[e] = fmaxf(fmaxf(hi[e], v), u);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == QMM_Q8_0) {
                const uint32_t x = w[i] ^ 0x80808080u, x2 = w2[i] ^ 0x80808080u;
#pragma unroll
                for (int k = 0; k < 4; ++k) take(4 * i + k, d * byte_float(x, k), d2 * byte_float(x2, k));
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) take(4 * i + k / 2 + 16 * (k & 1), d * nibble_float(w[i], k), d2 * nibble_float(w2[i], k));
            }
        }
    }
    // (a lane whose first token is past the last has found nothing; the others of its piece have)
    float top = 0.0f;
    if constexpr (kShare) {
#pragma unroll
        for (int m = TOK / 2, count = E / 2; m > 0; m /= 2, count /= 2) {
            const bool upper = (turn & m) != 0;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                if (i >= count) break;
                const float a = __shfl_xor_sync(0xffffffffu, upper ? lo[i] : lo[i + count], m * PK);
                const float b = __shfl_xor_sync(0xffffffffu, upper ? hi[i] : hi[i + count], m * PK);
                lo[i] = fminf(upper ? lo[i + count] : lo[i], a);
                hi[i] = fmaxf(upper ? hi[i + count] : hi[i], b);
            }
        }
    } else {
        for (int m = 1; m < TOK; ++m) {
            const int src = (lane + m * PK) & 31;
            const bool other = lane < PK;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float a = __shfl_sync(0xffffffffu, lo[i], src), b = __shfl_sync(0xffffffffu, hi[i], src);
                if (other) {
                    lo[i] = fminf(lo[i], a);
                    hi[i] = fmaxf(hi[i], b);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
    // over the lanes of a block: its pieces, and the turns of each
    uint32_t worst = odd ? 0x7FC00000u : __float_as_uint(top);         // a scale that is not finite comes out on top
    if constexpr (kShare) {
#pragma unroll
        for (int m = PK; m < 32; m *= 2) worst = max(worst, __shfl_xor_sync(0xffffffffu, worst, m));
    } else {
        uint32_t all = worst;
        for (int m = 1; m < TOK; ++m) {
            const uint32_t x = __shfl_sync(0xffffffffu, worst, (lane + m * PK) & 31);
            if (x > 0x7F800000u) all = max(all, x);                    // (the others' tops are not joined yet)
        }
        worst = all;
    }
    if constexpr (TYPE == QMM_Q8_0) worst = max(worst, __shfl_xor_sync(0xffffffffu, worst, 1));
    if (!kShare && lane >= PK) return;
    const bool bad = worst >= 0x7F800000u;
    const __half half = bad ? __ushort_as_half(0x7E00u) : __float2half_ru(__fdiv_rn(__uint_as_float(worst), 127.0f));
    const float d = bad ? 0.0f : __half2float(half);
    uint8_t *out = p.bounds + (page * p.H + h) * cache_bound_bytes(D);
    const int e0 = piece * E + (kShare ? turn * N : 0);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        int q[N < 4 ? 4 : N] = {};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float v = d > 0.0f ? __fdiv_rn(x ? hi[i] : lo[i], d) : 0.0f;
            q[i] = (int)fminf(fmaxf(x ? ceilf(v) : floorf(v), -127.0f), 127.0f);
        }
        uint8_t *to = out + x * D + e0;
        if constexpr (N == 1) *to = (uint8_t)q[0];
        else if constexpr (N == 2) *reinterpret_cast<uint16_t *>(to) = (uint16_t)(pack4(q[0], q[1], 0, 0));
        else {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) reinterpret_cast<uint32_t *>(to)[i] = pack4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
        }
    }
    if ((!kShare || turn == 0) && (TYPE == QMM_Q4_0 || (piece & 1) == 0)) reinterpret_cast<__half *>(out + 2 * D)[block] = half;
    if (lane == 0)
        for (int i = D + DB; i < cache_bound_bytes(D) / 2; ++i) reinterpret_cast<uint16_t *>(out)[i] = 0;
}

// ---------------------------------------------------------------------------------------------
// Scores
// ---------------------------------------------------------------------------------------------
struct Sequence {
    int64_t s, q0, q1, len;                 // number, rows of q q0 .. q1 - 1 (none: it is not computed), cached tokens
};
// The sequence of a row of q.  By a whole warp.
__device__ __forceinline__ Sequence find_sequence(const SelectParams &p, int64_t row) {
    Sequence q = {last_start(p.q_starts, p.n_seq, row), 0, 0, 0};
    if (q.s < 0 || q.s >= p.n_seq) return q;
    const int64_t q0 = p.q_starts[q.s], q1 = p.q_starts[q.s + 1];
    q.len = p.kv_lens[q.s];
    if (q0 < 0 || q1 > p.T) return q;
    q.q0 = q0;
    q.q1 = q1;
    return q;
}

struct Token {                              // a new token, and the pages in question for it
    int64_t s, seen;                        // its sequence; number of pages (0: none)
    int64_t old;                            // the first of the last ones that are always chosen
};
// The token of a row of q of its sequence; false: the row is past max_new, or not computed.
__device__ __forceinline__ bool find_token(const SelectParams &p, const Sequence &q, int64_t row, Token &t) {
    const int64_t i = row - q.q0;
    if (row >= q.q1 || i >= p.max_new) return false;
    const int64_t n = min(q.len, p.ld_pages << p.log_p), first = q.len - (q.q1 - q.q0);
    // the last place that the token sees, and the place from which the last pages are counted
    const int64_t end = p.tree ? n - 1 : min(first + i, n - 1), from = p.tree ? first : first + i;
    t.s = q.s;
    // (a row of `scores` has whole pages, so a sequence that ends in the last of them has its place there)
    t.seen = end < 0 || (q.len + ((int64_t)1 << p.log_p) - 1) >> p.log_p > p.most ? 0 : (end >> p.log_p) + 1;
    t.old = (from < 0 ? 0 : from >> p.log_p) - (p.recent - 1);
    return true;
}

constexpr int kScoreWarps = 4, kScoreThreads = kScoreWarps * 32, kTokTile = 8, kScorePages = kScoreWarps * 16;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes of a query row's codes in fp16 for one sign: neighbouring rows 64 bytes apart, modulo the banks' 128.
constexpr int score_pitch(int DB) { return DB * 64 + (DB % 2 == 0 ? 64 : 0); }

// Pages are the 16 rows of an mma (m16n8k16), query rows its 8 columns; codes are exact in fp16, and so are their sums in
// fp32 (below 2^20), so the tensor cores give the whole numbers S.  A warp takes 16 pages, whose codes stay in its registers, for
// up to kTokTile tokens (neighbouring rows of q; rows of another sequence load their own pages).  The columns of a
// product are the query heads of one token, 8 at a time, or of 8 / span tokens with span >= group a power of two, so
// that the maximum over a group is one over neighbouring columns.
template <int DB>
__global__ void __launch_bounds__(kScoreThreads) cache_score_kernel(const SelectParams p) {
    constexpr int D = DB * 32, BB = (2 * D + 2 * DB + 15) / 16 * 16, kPitch = score_pitch(DB);
    extern __shared__ __align__(16) uint8_t smem[];
    // the tile's products: tokens s_from[i] .. s_from[i + 1] - 1 of sequence s_seq[i], which ask about s_most[i] pages at most
    __shared__ int s_seen[kTokTile], s_from[kTokTile + 1], s_seq[kTokTile], s_most[kTokTile], s_n;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int h = (int)(blockIdx.y % (unsigned)p.H), lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int64_t row0 = (int64_t)blockIdx.x * p.tok_tile;
    const int cta0 = (int)(blockIdx.y / (unsigned)p.H) * kScorePages, stride = (int)(gridDim.y / (unsigned)p.H) * kScorePages;
    const int toks = (int)min((int64_t)p.tok_tile, p.T - row0);
    const int log_span = p.group > 4 ? 3 : (p.group > 2 ? 2 : p.group - 1), span = 1 << log_span, per = p.group > 8 ? 1 : 8 >> log_span;
    int all = 0;                                                       // pages that any token of the tile asks about
    {
        Sequence of = find_sequence(p, row0);
        int n = 0, from = 0, seq = -1, most = 0;                       // the product that is being filled
        for (int k = 0; k < toks; ++k) {
            if (k > 0 && row0 + k >= of.q1) of = find_sequence(p, row0 + k);
            Token tok;
            // where all pages are chosen, nobody asks for scores
            int seen = 0;
            if (find_token(p, of, row0 + k, tok) && tok.seen > p.budget) seen = (int)tok.seen;
            if (k > 0 && (k - from == per || (int)of.s != seq)) {
                if (threadIdx.x == 0) {
                    s_from[n] = from;
                    s_seq[n] = seq;
                    s_most[n] = most;
                }
                ++n;
                from = k;
                most = 0;
            }
            seq = (int)of.s;
            most = max(most, seen);
            all = max(all, seen);
            if (threadIdx.x == 0) s_seen[k] = seen;
        }
        if (threadIdx.x == 0) {
            s_from[n] = from;
            s_seq[n] = seq;
            s_most[n] = most;
            s_from[n + 1] = toks;
            s_n = n + 1;
        }
    }
    if (all <= cta0) return;
    // ---- the tile's query rows, a warp a row: [row][negative, positive] codes as fp16, [row][DB] scales ----
    const int rows = toks * p.group;
    float *dq = reinterpret_cast<float *>(smem + p.tok_tile * p.group * 2 * kPitch);
    constexpr int kAhead = 4;                                          // rows under way at a time
    for (int r0 = warp; r0 < rows; r0 += kScoreWarps * kAhead) {
        uint16_t raw[kAhead][DB];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + u * kScoreWarps;
            if (r >= rows) break;
            const uint16_t *src = static_cast<const uint16_t *>(p.q) + (row0 + r / p.group) * p.ldq + (int64_t)(h * p.group + r % p.group) * D + lane;
#pragma unroll
            for (int b = 0; b < DB; ++b) raw[u][b] = src[32 * b];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + u * kScoreWarps;
            if (r >= rows) break;
            __half *codes = reinterpret_cast<__half *>(smem + r * 2 * kPitch);
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                const float x = p.bf16 ? __uint_as_float((uint32_t)raw[u][b] << 16) : __half2float(__ushort_as_half(raw[u][b]));
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7FFFFFFFu);
                const bool fine = top < 0x7F800000u;
                const float d = fine ? q8_scale(__uint_as_float(top)) : 0.0f;
                const int a = fine ? q8_code(x, inv_or_zero(d)) : 0;
                codes[32 * b + lane] = __int2half_rn(min(a, 0));
                codes[kPitch / 2 + 32 * b + lane] = __int2half_rn(max(a, 0));
                if (lane == 0) dq[r * DB + b] = fine ? d : NAN;
            }
        }
    }
    __syncthreads();
    // a lane has pages page0 + g and + 8, and of each block of codes the eight from 8 t on
    int ahead[2] = {-1, -1}, ahead_seq = -1, ahead_at = -1;            // numbers in the pool of the pages from ahead_at on, of one sequence
    for (int page0 = cta0 + warp * 16; page0 < all; page0 += stride) {
        uint32_t a[DB][2][2][4];                                       // [block][lowest, highest][k step][registers]
        float d[DB][2];
        int loaded = -1;
        bool there[2] = {false, false};
        for (int i = 0; i < s_n; ++i) {
            if (s_most[i] <= page0) continue;
            if (s_seq[i] != loaded) {
                loaded = s_seq[i];
                auto page_of = [&](int number) { return number < p.ld_pages && number < p.most ? p.pages[loaded * p.ld_pages + number] : -1; };
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int page = loaded == ahead_seq && page0 == ahead_at ? ahead[e] : page_of(page0 + g + 8 * e);
                    there[e] = page >= 0 && page < p.n_pages;
                    const uint8_t *src = p.bounds + ((int64_t)(there[e] ? page : 0) * p.H + h) * BB;
#pragma unroll
                    for (int b = 0; b < DB; ++b) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint2 c = *reinterpret_cast<const uint2 *>(src + x * D + 32 * b + 8 * t);
                            tc::i8x4_to_h2x2(c.x, a[b][x][0][e], a[b][x][0][2 + e]);
                            tc::i8x4_to_h2x2(c.y, a[b][x][1][e], a[b][x][1][2 + e]);
                        }
                        d[b][e] = __half2float(reinterpret_cast<const __half *>(src + 2 * D)[b]);
                    }
                }
                if (ahead_seq < 0 || loaded == ahead_seq) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) ahead[e] = page_of(page0 + stride + g + 8 * e);
                    ahead_seq = loaded;
                    ahead_at = page0 + stride;
                }
            }
            const int k0 = s_from[i], k1 = s_from[i + 1];
            float best[2][2];                                          // [page g, g + 8][column 2t, 2t + 1]
            best[0][0] = best[0][1] = best[1][0] = best[1][1] = -INFINITY;
            for (int turn = 0; turn < p.group; turn += 8) {
                // the query row of a column; the tile's first in the place of those that have none
                auto row_of = [&](int c) {
                    const int k = k0 + (c >> log_span), q = turn + (c & (span - 1));
                    return k < k1 && q < p.group ? k * p.group + q : -1;
                };
                const int r0 = row_of(2 * t), r1 = row_of(2 * t + 1);
                const uint8_t *codes = smem + max(row_of(g), 0) * 2 * kPitch + 16 * t;
                const float *dq0 = dq + max(r0, 0) * DB, *dq1 = dq + max(r1, 0) * DB;
                float score[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
                for (int b = 0; b < DB; ++b) {
                    const uint4 lo = *reinterpret_cast<const uint4 *>(codes + 64 * b), hi = *reinterpret_cast<const uint4 *>(codes + kPitch + 64 * b);
                    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma16816(acc, a[b][0][0], lo.x, lo.y);
                    mma16816(acc, a[b][0][1], lo.z, lo.w);
                    mma16816(acc, a[b][1][0], hi.x, hi.y);
                    mma16816(acc, a[b][1][1], hi.z, hi.w);
                    const float d0 = dq0[b], d1 = dq1[b];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        score[e][0] = __fadd_rn(score[e][0], __fmul_rn(__fmul_rn(d0, d[b][e]), acc[2 * e]));
                        score[e][1] = __fadd_rn(score[e][1], __fmul_rn(__fmul_rn(d1, d[b][e]), acc[2 * e + 1]));
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (r0 >= 0) best[e][0] = isnan(score[e][0]) ? INFINITY : fmaxf(best[e][0], score[e][0]);
                    if (r1 >= 0) best[e][1] = isnan(score[e][1]) ? INFINITY : fmaxf(best[e][1], score[e][1]);
                }
            }
            // the maximum over a token's columns: in its first one; with one column each, a lane has two tokens
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (log_span >= 1) best[e][0] = fmaxf(best[e][0], best[e][1]);
                if (log_span >= 2) best[e][0] = fmaxf(best[e][0], __shfl_xor_sync(0xffffffffu, best[e][0], 1));
                if (log_span >= 3) best[e][0] = fmaxf(best[e][0], __shfl_xor_sync(0xffffffffu, best[e][0], 2));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = 2 * t + c, k = k0 + (col >> log_span);
                if ((col & (span - 1)) != 0 || k >= k1) continue;
                float *out = p.scores + ((row0 + k) * p.H + h) * p.most;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int number = page0 + g + 8 * e;
                    if (number < s_seen[k] && QMM_DCHECK(number < p.most && number < p.ld_pages)) out[number] = there[e] ? best[e][c] : -INFINITY;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// The choice
// ---------------------------------------------------------------------------------------------
constexpr int kChooseThreads = 256;

// fp32 as an unsigned number of the same order (-0 does not occur: sums that begin at +0 do not end there).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kChooseWarps = kChooseThreads / 32, kHeld = 16, kFew = 64;

// A CTA takes a token and head.  The border, the rank-th largest score, is found in histograms of 256 bins over the range
// of the scores that are still in question, until a bin holds a few, which are ranked against each other; then come the pages above it, and
// as many of those at it as are still wanted, the earliest first, in the order of their numbers.  A warp has a run of neighbouring
// pages: up to kHeld * 32 of them (HELD) stay in registers.
template <bool HELD>
__global__ void __launch_bounds__(kChooseThreads) cache_choose_kernel(const SelectParams p) {
    __shared__ uint32_t hist[256], few[kFew], part[2][kChooseWarps], s_lo, s_rank, s_count, s_border, s_ties;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row = blockIdx.x / (unsigned)p.H;
    const int h = (int)(blockIdx.x % (unsigned)p.H), tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Token t;
    if (!find_token(p, find_sequence(p, row), row, t)) return;
    int32_t *out = p.chosen + (row * p.H + h) * p.budget;
    const int seen = (int)t.seen, budget = (int)p.budget;
    if (seen <= budget) {
        for (int i = tid; i < budget; i += kChooseThreads) out[i] = i < seen ? i : -1;
        return;
    }
    const int front = (int)min(p.sinks, t.seen), back = max(front, (int)max((int64_t)0, min(t.old, t.seen)));   // always chosen: below front, from back on
    uint32_t rank = (uint32_t)max(0, budget - (front + seen - back));  // of the pages front .. back - 1
    const float *scores = p.scores + (row * p.H + h) * p.most;
    const int run = (seen + kChooseThreads - 1) / kChooseThreads * 32, begin = warp * run, end = min(seen, begin + run);
    // keys of the pages in question; 0 is no score's
    uint32_t held[HELD ? kHeld : 1];
    auto load = [&](int i) { return i >= front && i < back && i < end ? ordered(scores[i]) : 0u; };
    auto each = [&](auto f) {
        if constexpr (HELD) {
#pragma unroll
            for (int u = 0; u < kHeld; ++u)
                if (begin + 32 * u < end) f(begin + 32 * u + lane, held[u]);
        } else {
            for (int i = begin + lane; i - lane < end; i += 32) f(i, load(i));
        }
    };
    if constexpr (HELD) {
#pragma unroll
        for (int u = 0; u < kHeld; ++u) held[u] = load(begin + 32 * u + lane);
    }
    uint32_t border = 0xFFFFFFFFu, ties = 0;                           // keys above it are chosen, and so many of those at it
    if (rank > 0) {
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
        each([&](int, uint32_t key) {
            if (key) {
                lo = min(lo, key);
                hi = max(hi, key);
            }
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            part[0][warp] = lo;
            part[1][warp] = hi;
        }
        __syncthreads();
        lo = __reduce_min_sync(0xffffffffu, part[0][lane % kChooseWarps]);
        hi = __reduce_max_sync(0xffffffffu, part[1][lane % kChooseWarps]);
        // (a round takes at least eight bits from the range)
        for (int round = 0; round < 5; ++round) {
            // bins of 2^shift keys, 256 of which hold lo .. hi
            const int shift = max(0, 24 - __clz(hi - lo));
            hist[tid] = 0;
            if (tid == 0) s_count = 0;
            __syncthreads();
            each([&](int, uint32_t key) {
                if (key >= lo && key <= hi) atomicAdd(&hist[(key - lo) >> shift], 1u);
            });
            __syncthreads();
            if (warp == 0) {
                // eight bins to a lane, from the top
                uint32_t bin[8], sum = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += bin[k] = hist[255 - 8 * lane - k];
                uint32_t before = sum;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, before, m);
                    if (lane >= m) before += y;
                }
                before -= sum;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (before < rank && before + bin[k] >= rank) {
                        s_lo = lo + ((uint32_t)(255 - 8 * lane - k) << shift);
                        s_rank = rank - before;
                        s_border = bin[k];
                    }
                    before += bin[k];
                }
            }
            __syncthreads();
            const uint32_t count = s_border;
            lo = s_lo;
            if (hi - lo >= 1u << shift) hi = lo + ((1u << shift) - 1);
            rank = s_rank;
            if (shift == 0) {
                border = lo;
                ties = rank;
                break;
            }
            if (count > kFew) {
                __syncthreads();                                       // before hist is cleared
                continue;
            }
            each([&](int, uint32_t key) {
                if (key < lo || key > hi) return;
                const uint32_t to = atomicAdd(&s_count, 1u);
                if (QMM_DCHECK(to < kFew)) few[to] = key;
            });
            __syncthreads();
            if (tid < (int)count) {
                const uint32_t key = few[tid];
                uint32_t above = 0, equal = 0;
                for (int k = 0; k < (int)count; ++k) {
                    above += few[k] > key;
                    equal += few[k] == key;
                }
                if (above < rank && above + equal >= rank) {
                    s_border = key;
                    s_ties = rank - above;
                }
            }
            __syncthreads();
            border = s_border;
            ties = s_ties;
            break;
        }
    }
    // ---- the chosen pages, ascending ----
    uint32_t n_in = 0, n_ties = 0;
    auto state = [&](int i, uint32_t key, bool &in, bool &tie) {
        tie = key != 0 && key == border;
        in = i < end && (i < front || i >= back || key > border);      // (a key of the pages in question is below 0xFFFFFFFF, but NaN's: +inf's)
    };
    each([&](int i, uint32_t key) {
        bool in, tie;
        state(i, key, in, tie);
        n_in += __popc(__ballot_sync(0xffffffffu, in));
        n_ties += __popc(__ballot_sync(0xffffffffu, tie));
    });
    __syncthreads();                                                   // part is read above
    if (lane == 0) {
        part[0][warp] = n_in;
        part[1][warp] = n_ties;
    }
    __syncthreads();
    uint32_t at = 0, tied = 0;                                         // chosen, and at the border, in the runs before
    for (int w = 0; w < warp; ++w) {
        const uint32_t more = part[1][w];
        at += part[0][w] + min(more, ties - min(ties, tied));
        tied += more;
    }
    each([&](int i, uint32_t key) {
        bool in, tie;
        state(i, key, in, tie);
        const unsigned tie_mask = __ballot_sync(0xffffffffu, tie), below = (1u << lane) - 1;
        if (tie && tied + __popc(tie_mask & below) < ties) in = true;
        tied += __popc(tie_mask);
        const unsigned mask = __ballot_sync(0xffffffffu, in);
        const uint32_t to = at + __popc(mask & below);
        if (in && to < (uint32_t)budget) out[to] = i;
        at += __popc(mask);
    });
    // (as many as the budget are chosen: more pages are seen than that)
}

template <int DB>
cudaError_t launch_score(const SelectParams &p, cudaStream_t s) {
    const size_t smem = (size_t)p.tok_tile * p.group * (2 * score_pitch(DB) + DB * 4);    // up to 64 rows: 76 KB
    static int done[4] = {0, 0, 0, 0};
    const cudaError_t e = ensure_smem_limit(cache_score_kernel<DB>, 64 * (2 * score_pitch(DB) + DB * 4), done);
    if (e != cudaSuccess) return e;
    // each CTA prepares the tile's query rows for itself, so it takes as many pages as leave the GPU about three CTAs an SM
    const int64_t x = (p.T + p.tok_tile - 1) / p.tok_tile, chunks = (p.most + kScorePages - 1) / kScorePages;
    int64_t split = (3 * 152 + x * p.H - 1) / (x * p.H);
    split = split < chunks ? split : chunks;
    const int64_t turns = (chunks + split - 1) / split;
    split = (chunks + turns - 1) / turns;
    if (x > 0x7fffffff || split * p.H > 65535) return cudaErrorInvalidValue;
    return launch_pdl(cache_score_kernel<DB>, dim3((unsigned)x, (unsigned)(split * p.H)), kScoreThreads, smem, s, p);
}

template <int TYPE, int DB>
cudaError_t launch_bounds(const BoundsParams &p, cudaStream_t s) {
    const int64_t units = p.n_seq * p.per_seq * p.H, grid = (units + kBoundWarps - 1) / kBoundWarps;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl(cache_bounds_kernel<TYPE, DB>, dim3((unsigned)grid), kBoundWarps * 32, 0, s, p);
}

template <int TYPE>
cudaError_t launch_bounds_d(const BoundsParams &p, int D, cudaStream_t s) {
    switch (D / 32) {
        case 1: return launch_bounds<TYPE, 1>(p, s);
        case 2: return launch_bounds<TYPE, 2>(p, s);
        case 3: return launch_bounds<TYPE, 3>(p, s);
        case 4: return launch_bounds<TYPE, 4>(p, s);
        case 5: return launch_bounds<TYPE, 5>(p, s);
        case 6: return launch_bounds<TYPE, 6>(p, s);
        case 7: return launch_bounds<TYPE, 7>(p, s);
        default: return launch_bounds<TYPE, 8>(p, s);
    }
}

}  // namespace

cudaError_t launch_cache_bounds(qmm_type type, const uint8_t *k_cache, int64_t n_pages, int P, int H, int D, const int32_t *pages,
                                int64_t ld_pages, const int32_t *q_starts, const int32_t *kv_lens, int64_t n_seq, int64_t T,
                                int64_t max_new, uint8_t *bounds, cudaStream_t s) {
    BoundsParams p = {k_cache, n_pages, ld_pages, n_seq, T, max_new < T ? max_new : T, H, 0, 0, pages, q_starts, kv_lens, bounds};
    while ((1 << p.log_p) < P) ++p.log_p;
    const int64_t per_seq = (p.max_new + P - 2) / P + 1;               // max_new neighbours lie in so many pages at most
    if (per_seq > 0x7fffffff) return cudaErrorInvalidValue;
    p.per_seq = (int)per_seq;
    return type == QMM_Q8_0 ? launch_bounds_d<QMM_Q8_0>(p, D, s) : launch_bounds_d<QMM_Q4_0>(p, D, s);
}

cudaError_t launch_cache_select(const SelectParams &from, int D, cudaStream_t s) {
    SelectParams p = from;
    if (p.T * p.H > 0x7fffffff) return cudaErrorInvalidValue;
    // rows of one sequence share a page's codes; a single token's CTA is done the sooner without company
    p.tok_tile = p.max_new == 1 ? 1 : kTokTile;
    while (p.tok_tile > 1 && p.tok_tile * p.group > 64) p.tok_tile /= 2;
    cudaError_t e = cudaSuccess;
    if (p.most > p.budget) {
        switch (D / 32) {
            case 1: e = launch_score<1>(p, s); break;
            case 2: e = launch_score<2>(p, s); break;
            case 3: e = launch_score<3>(p, s); break;
            case 4: e = launch_score<4>(p, s); break;
            case 5: e = launch_score<5>(p, s); break;
            case 6: e = launch_score<6>(p, s); break;
            case 7: e = launch_score<7>(p, s); break;
            default: e = launch_score<8>(p, s); break;
        }
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(p.most <= kHeld * kChooseThreads ? cache_choose_kernel<true> : cache_choose_kernel<false>, dim3((unsigned)(p.T * p.H)),
                      kChooseThreads, 0, s, p);
}

QMM_DCHECK_READER(read_dcheck_cache_select)

}  // namespace qmm
