// attend.cu -- attention of a few new tokens of each sequence over the block-quantized cache (cache.cuh).
//
// For new token i of a sequence with n cached tokens, nq of them new, and query head hq (key/value head
// h = hq / G, G = Hq / H):
//   s_j = scale * sum_d q[i, hq, d] * k[j, h, d]  over the visible j,
//   out[i, hq] = sum_j exp(s_j - max s) v[j, h] / sum_j exp(s_j - max s),   lse = max s + ln(sum);
// j is visible when j < n - nq, or when bit j - (n - nq) of the token's tree word is set (without tree
// words: when j - (n - nq) <= i).  A row that sees nothing is 0 with lse -inf.
//
// Both products are taken with the cache as the left factor: S^T = K Q^T and O^T = V^T P^T, so that the mma
// instruction's 16 rows (m16n8k16) are keys or elements of the head, and its 8 columns are the nq * G rows
// of a sequence and key/value head, 8 * NT of them to a CTA.  A decode step's few rows then cost half
// the products, sums and registers of the other way round, where 16 rows are the least.  The codes are
// expanded in registers, once for all rows of the CTA, and never written back; movmatrix turns p from the
// first product's result into the second one's operand.  A CTA takes one chunk of the keys; its warps take
// tiles of 32 keys in turn, each through its own ring of asynchronous copies (no barriers), with its own
// running maximum and sum, and the warps' results are joined at the end.  Sequences longer than a chunk
// leave one partial result per chunk in the workspace, which a second kernel joins.
//
// Arithmetic.  Scores: the codes are exact in fp16, the query row is scaled by a power of two into fp16's
// range (an fp16 or bf16 query loses nothing but elements 2^-14 times smaller than the row's largest),
// the tensor cores add the products of one block of 32 in fp32, and the block's scale multiplies that sum
// in fp32.  Values: p in fp16, times 2^14 so that weights down to 2^-28 keep all 11 bits; v = d * q
// rounded to fp16; sums in fp32.  For fp16 outputs p is taken in two terms, hi + lo: the output's own rounding,
// p's and v's are all of 2^-12, and with all three the error against 64 bits is 1.6 times the output's rounding,
// with two 1.4 times.  A bf16 output's rounding hides both.
//
// A position that a row does not see must not reach it, even if it holds infinities or NaN; 0 * NaN in
// the second product would.  So scales past the end, and value scales that are not finite, count as 0
// there.  Where such a scale (or a value beyond fp16) was met, a plain loop then takes the CTA's rows one
// by one, and replaces those whose result is not finite by either way; no other cache pays for it.
#include "attend.cuh"

namespace qmm {
namespace {

constexpr int kMmaRows = 8;                // columns of an mma
constexpr int kKeys = 32;                  // keys of a tile

// The 16- or 32-byte units of a tile are permuted so that the fragment loads of a warp meet no bank
// twice: block b of row r (DB blocks a row) goes to place b ^ swizzle, U units spanning all banks.
template <int DB, int U>
__device__ __forceinline__ int swz(int r, int b) {
    constexpr int Z = (DB % 8 == 0 && U == 8) ? 8 : (DB % 4 == 0 ? 4 : (DB % 2 == 0 ? 2 : 1));
    return b ^ ((r / (U / Z)) & (Z - 1));
}

template <int TYPE, int DB, int NT>
struct Tile {
    static constexpr int kRowsTile = kMmaRows * NT;
    static constexpr int kUnit = TYPE == QMM_Q8_0 ? 32 : 16;           // bytes of a block's codes
    static constexpr int kSpan = TYPE == QMM_Q8_0 ? 4 : 8;             // units of 128 bytes
    static constexpr int kCodes = kKeys * DB * kUnit;
    static constexpr int kScales = kKeys * DB * 2;
    static constexpr int kK = 0, kV = kCodes, kKs = 2 * kCodes, kVs = kKs + kScales;
    static constexpr int kBytes = kVs + kScales;
    // Two CTAs share an SM, so that one's start and end, mostly latency, pass under the other's tiles: half the
    // shared memory each, and up to 6 warps (170 registers a thread) or 4 (255) with a ring of two tiles at least.
    static constexpr int kRoom = 104 * 1024;
    static constexpr int kWarps = NT == 1 && 2 * 6 * kBytes <= kRoom ? 6 : (2 * 4 * kBytes <= kRoom ? 4 : 3);
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kFit = kRoom / (kWarps * kBytes);
    static constexpr int kStages = kFit > 4 ? 4 : kFit;
    static constexpr int kOut = kWarps * kRowsTile * DB * 32 * 4;      // the warps' results, over the ring
    // query rows in fp16: neighbouring rows 64 bytes apart, modulo the banks' 128
    static constexpr int kQPitch = DB * 64 + (DB % 2 == 0 ? 64 : 0);
    static constexpr int kQ = kRowsTile * kQPitch;
    static constexpr int kRing = kStages * kWarps * kBytes > kOut ? kStages * kWarps * kBytes : kOut;
    static constexpr int kSmem = kRing + kQ + kRowsTile * 8 + kWarps * 4 * 4;
    static_assert(kStages >= 2 && kStages <= 4, "ring depth");
    static_assert(kWarps * kRowsTile * 8 <= kQ, "the warps' maxima and sums lie over the query rows");
    static_assert(kSmem <= 113 * 1024, "two CTAs do not fit an SM");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// An 8 x 8 matrix of 16-bit values, two of a row to a lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Nibbles 0 and 4 of w (Q4_0 codes) as half2, minus 8: exact.
__device__ __forceinline__ uint32_t nib_h2(uint32_t w) {
    uint32_t h;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(h) : "r"(w), "r"(0x000F000Fu), "r"(0x64006400u));
    return tc::h2_bits(__hsub2(tc::bits_h2(h), __halves2half2(__float2half_rn(1032.0f), __float2half_rn(1032.0f))));
}

// Place of element e of a block in a query row: the eight elements of lane t's fragments (two k steps of
// two registers of two) lie together, in the order in which the key codes come out of their words.
template <int TYPE>
__device__ __forceinline__ int query_place(int e) {
    if (TYPE == QMM_Q8_0) return e;
    const int k = e & 3;                       // elements 4t, 4t + 2, 4t + 1, 4t + 3, then 16 + those
    return ((e & 12) << 1) | ((e & 16) >> 2) | (k == 1 ? 2 : (k == 2 ? 1 : k));
}

// The scales of two neighbouring keys, DB each, as DB words: half i is block i of the first key, half
// DB + i block i of the second.
template <int DB>
__device__ __forceinline__ void load_scales(const uint8_t *p, uint32_t (&w)[DB]) {
    if constexpr (DB % 4 == 0) {
#pragma unroll
        for (int i = 0; i < DB / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else if constexpr (DB % 2 == 0) {
#pragma unroll
        for (int i = 0; i < DB / 2; ++i) {
            const uint2 v = reinterpret_cast<const uint2 *>(p)[i];
            w[2 * i] = v.x; w[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < DB; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    }
}
// The scales of one key as fp32.
template <int DB>
__device__ __forceinline__ void load_key_scales(const uint8_t *p, float (&d)[DB]) {
    if constexpr (DB % 2 == 0) {
        uint32_t w[DB / 2];
        if constexpr (DB % 4 == 0) {
#pragma unroll
            for (int i = 0; i < DB / 4; ++i) {
                const uint2 v = reinterpret_cast<const uint2 *>(p)[i];
                w[2 * i] = v.x; w[2 * i + 1] = v.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < DB / 2; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        }
#pragma unroll
        for (int i = 0; i < DB / 2; ++i) {
            d[2 * i] = __low2float(tc::bits_h2(w[i]));
            d[2 * i + 1] = __high2float(tc::bits_h2(w[i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < DB; ++i) d[i] = __half2float(reinterpret_cast<const __half *>(p)[i]);
    }
}
// The scales of block b of both keys as a half2.
template <int DB>
__device__ __forceinline__ uint32_t scale_pair(const uint32_t (&w)[DB], int b) {
    return __byte_perm(w[b >> 1], w[(DB + b) >> 1], (b & 1 ? 0x32 : 0x10) | ((DB + b) & 1 ? 0x7600 : 0x5400));
}

// What bounds it: for up to 8 rows of Q8_0 the cache's bytes (38 sequences of 8192 tokens, 8 heads of 128: 106 us, 6.4 TB/s);
// for Q4_0 (97 us, 3.7 TB/s) and for more rows the instructions that expand the codes and take the exponentials (16
// rows 132 us, 32 rows 198); for short sequences the chain of copy, products, softmax and join (777 tokens: 8.4 us).
// TWO: the kernel can take p in two terms, and does for fp16 outputs (32 rows: 256 us).  Without it 32 rows keep
// their registers.
template <int TYPE, int DB, int NT, bool TWO>
__global__ void __launch_bounds__(Tile<TYPE, DB, NT>::kThreads, 2) attend_kernel(const __grid_constant__ AttendParams p) {
    using L = Tile<TYPE, DB, NT>;
    constexpr int D = DB * 32, S = L::kStages, UNIT = L::kUnit, SPAN = L::kSpan, CB = DB * UNIT;
    constexpr int kWarps = L::kWarps, kThreads = L::kThreads, kRowsTile = L::kRowsTile;
    constexpr bool kQRegs = NT == 1;                                           // the query fragments stay in registers
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *q_rows = smem + L::kRing;
    float *w_top = reinterpret_cast<float *>(q_rows), *w_sum = w_top + kWarps * kRowsTile;   // [warp][row], after the last tile
    float *row_mul = reinterpret_cast<float *>(q_rows + L::kQ);               // score -> power of two
    int *row_bad = reinterpret_cast<int *>(row_mul + kRowsTile);              // its result is not finite
    uint32_t *masks = reinterpret_cast<uint32_t *>(row_bad + kRowsTile);      // [warp][stage]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    Rows w;
    if (!find_rows<kRowsTile>(p, reinterpret_cast<int *>(smem), kThreads, w)) return;

    // ---- the ring: tile i of this warp is keys k0 + 32 * (kWarps i + warp) .. ----
    const uint32_t ring = pipe::smem_u32(smem) + (uint32_t)(warp * S * L::kBytes);
    const int64_t head = (int64_t)w.h * p.P * (CB + 2 * DB), page_bytes = (int64_t)p.H * p.P * (CB + 2 * DB);
    const int tiles = (int)((w.k1 - w.k0 + kKeys - 1) / kKeys);
    const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
    const int32_t *table = p.pages + w.s * p.ld_pages;
    // lanes 0-15 know the page of the tile's first 16 keys, lanes 16-31 that of the others
    auto page_of = [&](int i) -> int {
        const int64_t j = w.k0 + (int64_t)(i * kWarps + warp) * kKeys + (lane & 16);
        return i < mine && j < w.k1 && QMM_DCHECK((j >> p.log_p) < p.ld_pages) ? table[j >> p.log_p] : -1;
    };
    auto issue = [&](int i, int page) {
        if (i < mine) {
            const int slot = i % S;
            const uint32_t dst = ring + (uint32_t)(slot * L::kBytes);
            const int64_t j = w.k0 + (int64_t)(i * kWarps + warp) * kKeys;
            const int pg0 = __shfl_sync(0xffffffffu, page, 0), pg1 = __shfl_sync(0xffffffffu, page, 16);
            const bool ok0 = pg0 >= 0 && pg0 < p.n_pages, ok1 = pg1 >= 0 && pg1 < p.n_pages;
            const int off0 = (int)j & (p.P - 1), off1 = (off0 + 16) & (p.P - 1);
            // where the 16 keys' codes and scales start, each contiguous
            const int64_t c0 = (int64_t)pg0 * page_bytes + head, c1 = (int64_t)pg1 * page_bytes + head;
            const int64_t a0 = c0 + off0 * CB + lane * 16, a1 = c1 + off1 * CB + lane * 16 - 16 * CB;
            constexpr int PK = CB / 16, ITS = kKeys * PK / 32;     // pieces of 16 bytes: of a key, for a lane
#pragma unroll
            for (int it = 0; it < ITS; ++it) {
                const int u = it * 32 + lane, key = u / PK, c = u % PK;
                const bool second = PK % 2 == 0 ? it >= ITS / 2 : key >= 16;
                const int64_t src = (second ? a1 : a0) + it * 512;
                if ((second ? ok1 : ok0) && QMM_DCHECK(src >= 0 && src + 16 <= p.n_pages * page_bytes)) {
                    const int blk = c * 16 / UNIT, in = c * 16 % UNIT;
                    const int vrow = (key & 16) | ((key & 1) << 3) | ((key & 15) >> 1);
                    cp_async16(dst + L::kK + (key * DB + swz<DB, SPAN>(key, blk)) * UNIT + in, p.k_cache + src);
                    cp_async16(dst + L::kV + (vrow * DB + swz<DB, SPAN>(vrow, blk)) * UNIT + in, p.v_cache + src);
                }
            }
            // scales: 2 * DB pieces for 16 keys
            if (lane < 4 * DB) {
                const bool second = lane >= 2 * DB;
                const int64_t src = (second ? c1 + off1 * (2 * DB) - 32 * DB : c0 + off0 * (2 * DB)) + p.P * CB + lane * 16;
                if ((second ? ok1 : ok0) && QMM_DCHECK(src >= 0 && src + 16 <= p.n_pages * page_bytes)) {
                    cp_async16(dst + L::kKs + lane * 16, p.k_cache + src);
                    cp_async16(dst + L::kVs + lane * 16, p.v_cache + src);
                }
            }
            if (lane == 0) {
                const int64_t left = w.k1 - j;
                uint32_t m = left >= 32 ? 0xffffffffu : (1u << (int)left) - 1u;
                if (!ok0) m &= 0xffff0000u;
                if (!ok1) m &= 0x0000ffffu;
                masks[warp * 4 + slot] = m;
            }
        }
        cp_commit();
    };
    int page = page_of(0);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        const int next = page_of(i + 1);
        issue(i, page);
        page = next;
    }

    // ---- the query rows: scaled by a power of two so that the largest element lies in [1, 2) ----
    constexpr int kMine = (kRowsTile + kWarps - 1) / kWarps;
    float qv[kMine][DB];
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
        const int row = warp + u * kWarps, r = w.r0 + row;
        const int64_t base = row < w.rows ? (w.q0 + r / p.group) * p.ldq + (int64_t)(w.h * p.group + r % p.group) * D + lane : 0;
#pragma unroll
        for (int b = 0; b < DB; ++b) qv[u][b] = row < w.rows ? load_q(p, base + 32 * b) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
        const int row = warp + u * kWarps;
        if (row >= kRowsTile) break;
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < DB; ++b) top = fmaxf(top, fabsf(qv[u][b]));
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        const int e = top > 0.0f && top < INFINITY ? max((int)(__float_as_uint(top) >> 23) - 127, -120) : 0;
        const float mul = p.scale * 1.4426950408889634f, down = copysignf(exp2f((float)-e), mul);
        if (lane == 0) {
            // a scale of 0 still has to order -inf below 0
            row_mul[row] = fmaxf(fabsf(mul), 1e-30f) * exp2f((float)e);
            row_bad[row] = 0;
        }
        __half *out = reinterpret_cast<__half *>(q_rows + row * L::kQPitch) + query_place<TYPE>(lane);
#pragma unroll
        for (int b = 0; b < DB; ++b) out[32 * b] = __float2half_rn(qv[u][b] * down);
    }
    __syncthreads();
    auto load_frag = [&](uint32_t (&q)[4], int nt, int b) {
        const uint4 v = *reinterpret_cast<const uint4 *>(q_rows + (nt * 8 + g) * L::kQPitch + b * 64 + t * 16);
        q[0] = v.x; q[1] = v.y; q[2] = v.z; q[3] = v.w;
    };
    uint32_t qr[kQRegs ? DB : 1][4];
    if constexpr (kQRegs) {
#pragma unroll
        for (int b = 0; b < DB; ++b) load_frag(qr[b], 0, b);
    }

    // a lane's rows are 8 nt + 2t and + 1; O^T tile (b, x) holds elements e = 2x (lane g) and 2x + 1 (g + 8) of
    // the four that a lane's code word has of block b
    float o[NT][2 * DB][4];
    float top[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        top[nt][0] = top[nt][1] = -INFINITY;
        sum[nt][0] = sum[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * DB; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
    }
    uint32_t odd = 0;                                            // a value scale that is not finite
    const bool two = TWO && !p.bf16;                                    // p in two terms, where the output keeps 11 bits

    for (int i = 0; i < mine; ++i) {
        cp_wait<S - 2>();
        __syncwarp();
        {
            const int next = page_of(i + S);
            issue(i + S - 1, page);
            page = next;
        }
        const uint8_t *st = smem + warp * S * L::kBytes + (i % S) * L::kBytes;
        const uint32_t in = masks[warp * 4 + i % S];
        const int64_t j0 = w.k0 + (int64_t)(i * kWarps + warp) * kKeys;
        const bool masked = in != 0xffffffffu || j0 + kKeys > w.first;

        // ---- scores: sc[nt][mt] holds keys 16 mt + g (0, 1) and 16 mt + g + 8 (2, 3) of rows 2t, 2t + 1 ----
        float sc[NT][2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float d0[DB], d1[DB];
            load_key_scales<DB>(st + L::kKs + (16 * mt + g) * DB * 2, d0);
            load_key_scales<DB>(st + L::kKs + (16 * mt + g + 8) * DB * 2, d1);
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                uint32_t f[4], h[4];                             // codes of keys g and g + 8
                auto codes = [&](int key, uint32_t (&x)[4]) {
                    const uint8_t *kp = st + L::kK + (key * DB + swz<DB, SPAN>(key, b)) * UNIT;
                    if constexpr (TYPE == QMM_Q8_0) {
                        const uint2 c = *reinterpret_cast<const uint2 *>(kp + 8 * t);
                        tc::i8x4_to_h2x2(c.x, x[0], x[1]);
                        tc::i8x4_to_h2x2(c.y, x[2], x[3]);
                    } else {
                        const uint32_t c = *reinterpret_cast<const uint32_t *>(kp + 4 * t);
                        x[0] = nib_h2(c);
                        x[1] = nib_h2(c >> 8);
                        x[2] = nib_h2(c >> 4);
                        x[3] = nib_h2(c >> 12);
                    }
                };
                codes(16 * mt + g, f);
                codes(16 * mt + g + 8, h);
                const uint32_t a0[4] = {f[0], h[0], f[1], h[1]}, a1[4] = {f[2], h[2], f[3], h[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t q[4];
                    if constexpr (kQRegs) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) q[r] = qr[b][r];
                    } else {
                        load_frag(q, nt, b);
                    }
                    float acc[4];
                    mma16816_first(acc, a0, q[0], q[1]);
                    mma16816(acc, a1, q[2], q[3]);
                    float (&x)[4] = sc[nt][mt];
                    x[0] = b == 0 ? d0[b] * acc[0] : fmaf(d0[b], acc[0], x[0]);
                    x[1] = b == 0 ? d0[b] * acc[1] : fmaf(d0[b], acc[1], x[1]);
                    x[2] = b == 0 ? d1[b] * acc[2] : fmaf(d1[b], acc[2], x[2]);
                    x[3] = b == 0 ? d1[b] * acc[3] : fmaf(d1[b], acc[3], x[3]);
                }
            }
        }
        // ---- what is not seen ----
        if (masked) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = nt * 8 + 2 * t + c, tok = (w.r0 + row) / p.group;
                    const uint64_t word = p.tree && row < w.rows ? p.tree[w.q0 + tok] : 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = 8 * x + g;
                        const int64_t nb = j0 + key - w.first;      // place among the new tokens
                        bool seen = (in >> key) & 1;
                        if (nb >= 0) seen = seen && (p.tree ? nb < 64 && ((word >> nb) & 1) : nb <= tok);
                        if (!seen) sc[nt][x >> 1][2 * (x & 1) + c] = -INFINITY;
                    }
                }
        }
        // ---- running maximum and sum; p to fp16 and transposed: pt[nt][x] holds keys 8x + 2t, + 1 of row g ----
        uint32_t pt[NT][4], pl[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float base[2], down[2], mul[2];
            bool moved = false;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                mul[c] = row_mul[nt * 8 + 2 * t + c];
                float m = fmaxf(fmaxf(sc[nt][0][c], sc[nt][0][2 + c]), fmaxf(sc[nt][1][c], sc[nt][1][2 + c]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                m = fmaxf(m * mul[c], top[nt][c]);
                base[c] = m == -INFINITY ? 0.0f : m;
                down[c] = ex2(top[nt][c] - base[c]);
                moved |= m != top[nt][c];
                top[nt][c] = m;
                base[c] = kBias - base[c];
            }
            if (__any_sync(0xffffffffu, moved)) {
                sum[nt][0] *= down[0];
                sum[nt][1] *= down[1];
#pragma unroll
                for (int n = 0; n < 2 * DB; ++n) {
                    o[nt][n][0] *= down[0];
                    o[nt][n][1] *= down[1];
                    o[nt][n][2] *= down[0];
                    o[nt][n][3] *= down[1];
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float p0 = ex2(fmaf(sc[nt][x >> 1][2 * (x & 1)], mul[0], base[0]));
                const float p1 = ex2(fmaf(sc[nt][x >> 1][2 * (x & 1) + 1], mul[1], base[1]));
                sum[nt][0] += p0;
                sum[nt][1] += p1;
                const uint32_t hi = pack2(p0, p1, __half{});
                pt[nt][x] = transpose8x8(hi);
                if (two) {
                    const float2 h = unpack2(hi, __half{});
                    pl[nt][x] = transpose8x8(pack2(p0 - h.x, p1 - h.y, __half{}));
                }
            }
        }
        // ---- values: 16 keys a step; a lane's keys are 2t, 2t + 1, 2t + 8, 2t + 9 ----
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t w01[DB], w89[DB];
            load_scales<DB>(st + L::kVs + (16 * j + 2 * t) * DB * 2, w01);
            load_scales<DB>(st + L::kVs + (16 * j + 2 * t + 8) * DB * 2, w89);
            if (masked) {
                const uint32_t have = in >> (16 * j + 2 * t);
#pragma unroll
                for (int i2 = 0; i2 < DB; ++i2) {
                    // half 2 i2 and 2 i2 + 1: of the first key below DB, of the second from there
                    constexpr uint32_t kLo = 0xFFFFu, kHi = 0xFFFF0000u;
                    const int lo = 2 * i2 >= DB, hi = 2 * i2 + 1 >= DB;
                    w01[i2] &= ((have >> lo) & 1 ? kLo : 0u) | ((have >> hi) & 1 ? kHi : 0u);
                    w89[i2] &= ((have >> (8 + lo)) & 1 ? kLo : 0u) | ((have >> (8 + hi)) & 1 ? kHi : 0u);
                    const uint32_t f01 = finite2(w01[i2]), f89 = finite2(w89[i2]);
                    odd |= ~(f01 & f89);
                    w01[i2] &= f01;
                    w89[i2] &= f89;
                }
            }
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                const uint32_t d01 = scale_pair<DB>(w01, b), d89 = scale_pair<DB>(w89, b);
                const uint8_t *vp = st + L::kV;
                const int r0 = 16 * j + t;                       // rows of keys 2t, 2t + 8, 2t + 1, 2t + 9: t, t + 4, t + 8, t + 12
                auto row = [&](int r) { return vp + (r * DB + swz<DB, SPAN>(r, b)) * UNIT; };
                uint32_t x[4], y[4];                             // element e: keys 2t, 2t + 1 and 2t + 8, 2t + 9
                if constexpr (TYPE == QMM_Q8_0) {
                    const uint32_t k0w = *reinterpret_cast<const uint32_t *>(row(r0) + 4 * g), k8w = *reinterpret_cast<const uint32_t *>(row(r0 + 4) + 4 * g);
                    const uint32_t k1w = *reinterpret_cast<const uint32_t *>(row(r0 + 8) + 4 * g), k9w = *reinterpret_cast<const uint32_t *>(row(r0 + 12) + 4 * g);
                    tc::i8x4_to_h2x2(__byte_perm(k0w, k1w, 0x5140), x[0], x[1]);
                    tc::i8x4_to_h2x2(__byte_perm(k0w, k1w, 0x7362), x[2], x[3]);
                    tc::i8x4_to_h2x2(__byte_perm(k8w, k9w, 0x5140), y[0], y[1]);
                    tc::i8x4_to_h2x2(__byte_perm(k8w, k9w, 0x7362), y[2], y[3]);
                } else {
                    const uint32_t c01 = (uint32_t)*reinterpret_cast<const uint16_t *>(row(r0) + 2 * g) |
                                         ((uint32_t)*reinterpret_cast<const uint16_t *>(row(r0 + 8) + 2 * g) << 16);
                    const uint32_t c89 = (uint32_t)*reinterpret_cast<const uint16_t *>(row(r0 + 4) + 2 * g) |
                                         ((uint32_t)*reinterpret_cast<const uint16_t *>(row(r0 + 12) + 2 * g) << 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = nib_h2(c01 >> (4 * e));
                        y[e] = nib_h2(c89 >> (4 * e));
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = hmul2(x[e], d01);
                    y[e] = hmul2(y[e], d89);
                }
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const uint32_t a[4] = {x[2 * z], x[2 * z + 1], y[2 * z], y[2 * z + 1]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(o[nt][2 * b + z], a, pt[nt][2 * j], pt[nt][2 * j + 1]);
                        if (two) mma16816(o[nt][2 * b + z], a, pl[nt][2 * j], pl[nt][2 * j + 1]);
                    }
                }
            }
        }
        __syncwarp();
    }
    cp_wait<0>();

    // ---- the warps' results, joined ----
    __syncthreads();                                             // the ring is free
    float *res = reinterpret_cast<float *>(smem) + warp * kRowsTile * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            sum[nt][c] += __shfl_xor_sync(0xffffffffu, sum[nt][c], 4);
            sum[nt][c] += __shfl_xor_sync(0xffffffffu, sum[nt][c], 8);
            sum[nt][c] += __shfl_xor_sync(0xffffffffu, sum[nt][c], 16);
            if (g == 0) {
                w_top[warp * kRowsTile + nt * 8 + 2 * t + c] = top[nt][c];
                w_sum[warp * kRowsTile + nt * 8 + 2 * t + c] = sum[nt][c];
            }
        }
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int row = nt * 8 + 2 * t + (c & 1), e = 2 * z + (c >> 1);
                    // the element whose codes were fed to slot e of lane g
                    const int d = TYPE == QMM_Q8_0 ? 4 * g + e : 2 * g + (e >> 1) + 16 * (e & 1);
                    if (row < w.rows) res[row * D + 32 * b + d] = o[nt][2 * b + z][c];
                }
    }
    __syncthreads();
    // per row: the factor of each warp's part (in place of its maximum), the maximum and the sum
    for (int row = threadIdx.x; row < w.rows; row += kThreads) {
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) m = fmaxf(m, w_top[x * kRowsTile + row]);
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float f = ex2(w_top[x * kRowsTile + row] - base);
            l += f * w_sum[x * kRowsTile + row];
            w_top[x * kRowsTile + row] = f;
        }
        row_mul[row] = m;
        w_sum[row] = l;                                          // warp 0's, read above by this thread alone
    }
    __syncthreads();
    bool bad = odd != 0;
    for (int i = threadIdx.x; i < w.rows * (D / 4); i += kThreads) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float f = w_top[x * kRowsTile + row];
            const float4 u = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem) + (x * kRowsTile + row) * D + d);
            v[0] += f * u.x;
            v[1] += f * u.y;
            v[2] += f * u.z;
            v[3] += f * u.w;
        }
        const float l = w_sum[row];
        // 0 times a number that is not finite is NaN, and stays it through the sum
        if (!(v[0] * 0.0f + v[1] * 0.0f + v[2] * 0.0f + v[3] * 0.0f + l * 0.0f == 0.0f)) {
            bad = true;
            row_bad[row] = 1;
        }
        write_row(p, w, D, row, d, v, row_mul[row], l);
    }
    if (__syncthreads_or(bad)) rows_one_by_one<TYPE, DB, kWarps>(p, w, row_bad);
}

// Joins the partial results of the sequences that were split.  WPR warps take a row, each the splits of
// its number modulo WPR: one warp for a few splits, a CTA's eight where there are many.
constexpr int kJoinWarps = 8;
template <int DB, int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendParams p) {
    constexpr int D = DB * 32;
    __shared__ float s_o[WPR > 1 ? WPR : 1][WPR > 1 ? D : 1];
    __shared__ float2 s_l[WPR > 1 ? WPR : 1];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WPR, Hq = p.H * p.group;
    const int64_t stride = p.T * Hq, at = (int64_t)blockIdx.x * (kJoinWarps / WPR) + warp / WPR;
    const int64_t tok = (uint32_t)at / (uint32_t)Hq;
    const int hq = (int)(at - tok * Hq);
    // The lengths are no results of the kernel before this one, which has waited for whoever wrote them.  Nobody
    // leaves before the wait: a kernel that waits for this one has to find the one before it complete too.
    __shared__ uint32_t s_chunk;
    int s = -1, start = 0, end = 0;                              // the row's sequence: the last that starts at or before it
    for (int base = 0; base <= (int)p.n_seq; base += 32) {
        const int from = base + lane <= (int)p.n_seq ? __ldcg(p.q_starts + base + lane) : INT_MAX;
        const unsigned upto = __ballot_sync(0xffffffffu, from <= tok);
        const int n = __popc(upto);
        if (n > 0) {
            s = base + n - 1;
            start = __shfl_sync(0xffffffffu, from, n - 1);
        }
        if (n < 32) {
            end = __shfl_sync(0xffffffffu, from, n);             // where the next one starts
            break;
        }
    }
    const bool mine = s >= 0 && s < (int)p.n_seq;                // s = n_seq: behind the last
    const int len = mine ? __ldcg(p.kv_lens + s) : 0;
    if (warp == 0) {
        const uint32_t chunk = chunk_of(p, len_at(p, 0));
        if (lane == 0) s_chunk = chunk;
    }
    __syncthreads();
    const int used = splits_of(cached(p, len), s_chunk);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // rows of no sequence, and of those that do not lie in q, were not computed, nor were rows past row_tiles
    if (at >= stride || !mine || start < 0 || end > p.T) return;
    if (used <= 1 || (tok - start) * p.group + hq % p.group >= (int64_t)p.row_tiles * p.tile_rows) return;
    if (!QMM_DCHECK(used <= p.splits && tok < p.T)) return;
    // four parts at a time, each under way before the first is used
    float m = -INFINITY, l = 0.0f, o[DB];
#pragma unroll
    for (int b = 0; b < DB; ++b) o[b] = 0.0f;
    for (int s0 = part; s0 < used; s0 += 4 * WPR) {
        float2 ml[4];
        float v[4][DB];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int sp = s0 + u * WPR;
            ml[u] = make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int b = 0; b < DB; ++b) v[u][b] = 0.0f;
            if (sp < used) {
                ml[u] = *reinterpret_cast<const float2 *>(p.part_ml + 2 * (sp * stride + at));
#pragma unroll
                for (int b = 0; b < DB; ++b) v[u][b] = p.part_o[(sp * stride + at) * D + 32 * b + lane];
            }
        }
        const float top = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m), base = top == -INFINITY ? 0.0f : top;
        const float down = exp2f(m - base);
        m = top;
        l *= down;
#pragma unroll
        for (int b = 0; b < DB; ++b) o[b] *= down;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (ml[u].y == 0.0f) continue;                       // nothing was seen there
            const float f = exp2f(ml[u].x - base);
            l += f * ml[u].y;
#pragma unroll
            for (int b = 0; b < DB; ++b) o[b] += f * v[u][b];
        }
    }
    if constexpr (WPR > 1) {
#pragma unroll
        for (int b = 0; b < DB; ++b) s_o[part][32 * b + lane] = o[b];
        if (lane == 0) s_l[part] = make_float2(m, l);
        __syncthreads();
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) m = fmaxf(m, s_l[w].x);
        const float base = m == -INFINITY ? 0.0f : m;
        float f[WPR];
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            f[w] = s_l[w].y == 0.0f ? 0.0f : exp2f(s_l[w].x - base);
            l += f[w] * s_l[w].y;
        }
        for (int d = threadIdx.x; d < D; d += kJoinWarps * 32) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) v += f[w] * s_o[w][d];
            store_out(p, tok * p.ldo + (int64_t)hq * D + d, l == 0.0f ? 0.0f : v / l);
        }
    } else {
#pragma unroll
        for (int b = 0; b < DB; ++b) store_out(p, tok * p.ldo + (int64_t)hq * D + 32 * b + lane, l == 0.0f ? 0.0f : o[b] / l);
    }
    if (lane == 0 && part == 0 && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (m + __log2f(l) - kBias) * 0.6931471805599453f;
}

// Rows of a CTA: 8, 16 or (of up to 128 elements) 32 on mma; where there are more, and a head has at most 128
// elements, 128 on tcgen05.  (38 sequences of 8192 tokens, 8 heads of 128, bf16 / fp16: 32 rows 198 / 256 us on mma, 33 to
// 128 rows 336 / 354 on tcgen05, where two tiles of 32 would take twice 198 / 256.  Heads of 64: 33 to 64 rows 292 / 297
// on tcgen05, 232 / 307 as two tiles on mma; trees of 60 rows over 200 to 4096 tokens of Q4_0, 31 and 37.)
int tile_rows_of(int64_t max_new, int group, int D) {
    const int64_t rows = max_new * group;
    if (rows <= kMmaRows) return kMmaRows;
    if (rows <= 2 * kMmaRows || D > 128) return 2 * kMmaRows;
    return rows <= 4 * kMmaRows ? 4 * kMmaRows : kTcRows;
}
int64_t row_tiles_of(int64_t max_new, int group, int D) {
    const int rows = tile_rows_of(max_new, group, D);
    return (max_new * group + rows - 1) / rows;
}

// How far sequences may be split.  The GPU has 304 places for the CTAs of attend_kernel (two an SM), 152 for those of
// attend_tc_kernel: as many splits as fill them once, or also twice where whole sequences fill more than half, and none
// where whole sequences fill them.  Three times as many CTAs as places measured slower: one token over 500001
// tokens 124 us for 97.  A sequence that is longer than the others takes up to four times the splits of an even
// batch.  `even`: splits of each sequence in an even batch; the others as in AttendParams.
struct Split {
    int splits, budget, waves, fixed, even;
};
Split split_of(int64_t n_seq, int H, int64_t row_tiles, int tile_rows, int64_t max_len) {
    const bool tc = tile_rows == kTcRows;
    const int64_t places = tc ? 152 : 304, per = H * row_tiles, units = n_seq * per;
    Split s = {1, (int)n_seq, 1, tc ? 2 : 6, 1};
    if (units >= places) return s;
    s.budget = (int)(places / per);
    s.waves = 2 * units > places ? 2 : 1;
    const int64_t all = (int64_t)s.budget * s.waves, even = (all + n_seq - 1) / n_seq;
    const int64_t most = (max_len + kStep - 1) / kStep;
    int64_t want = all - n_seq + 1;
    want = want < 4 * even ? want : 4 * even;
    want = want < most ? want : most;
    s.splits = (int)(want < 1 ? 1 : want);
    s.even = (int)(even < most ? even : most);
    return s;
}
size_t split_bytes(int64_t rows, int D) { return round256((size_t)rows * (size_t)(D + 2) * 4); }

template <int TYPE, int DB, int NT, bool TWO = true>
cudaError_t launch_typed(const AttendParams &p, int64_t ctas, cudaStream_t s) {
    using L = Tile<TYPE, DB, NT>;
    auto kern = attend_kernel<TYPE, DB, NT, TWO>;
    static int attr_done[4] = {0, 0, 0, 0};
    cudaError_t e = ensure_smem_limit(kern, L::kSmem, attr_done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)ctas), L::kThreads, L::kSmem, s, p);
}

template <int DB>
cudaError_t launch_join(const AttendParams &p, int even, cudaStream_t s) {
    const int64_t rows = p.T * p.H * p.group;
    if (even > kJoinWarps) return launch_pdl(attend_join_kernel<DB, kJoinWarps>, dim3((unsigned)rows), kJoinWarps * 32, 0, s, p);
    return launch_pdl(attend_join_kernel<DB, 1>, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), kJoinWarps * 32, 0, s, p);
}

template <int TYPE, int DB>
cudaError_t launch_rows(const AttendParams &p, int64_t ctas, cudaStream_t s) {
    if (p.tile_rows == kMmaRows) return launch_typed<TYPE, DB, 1>(p, ctas, s);
    if constexpr (DB <= 4) {
        if (p.tile_rows == 4 * kMmaRows) return p.bf16 ? launch_typed<TYPE, DB, 4, false>(p, ctas, s) : launch_typed<TYPE, DB, 4>(p, ctas, s);
    }
    return launch_typed<TYPE, DB, 2>(p, ctas, s);
}

template <int DB>
cudaError_t launch_blocks(qmm_type type, const AttendParams &p, int64_t ctas, int even, cudaStream_t s) {
    cudaError_t e;
    if (p.tile_rows == kTcRows) e = launch_attend_tc(type, p, DB, ctas, s);
    else e = type == QMM_Q8_0 ? launch_rows<QMM_Q8_0, DB>(p, ctas, s) : launch_rows<QMM_Q4_0, DB>(p, ctas, s);
    return e != cudaSuccess || p.splits == 1 ? e : launch_join<DB>(p, even, s);
}

}  // namespace

size_t attend_workspace_bytes(int64_t n_seq, int64_t max_new, int H, int Hq, int D, int64_t max_len) {
    const int splits = split_of(n_seq, H, row_tiles_of(max_new, Hq / H, D), tile_rows_of(max_new, Hq / H, D), max_len).splits;
    return splits == 1 ? 0 : (size_t)splits * split_bytes(n_seq * max_new * Hq, D);
}

cudaError_t launch_cache_attend(qmm_type type, const uint8_t *k_cache, const uint8_t *v_cache, int64_t n_pages, int P, int H, int D,
                                const int32_t *pages, int64_t ld_pages, const int32_t *q_starts, const int32_t *kv_lens,
                                int64_t n_seq, qmm_dtype t, const void *q, int64_t ldq, int64_t T, int Hq, const uint64_t *tree,
                                float scale, int64_t max_new, int64_t max_len, void *out, int64_t ldo, float *lse, void *ws,
                                size_t ws_bytes, cudaStream_t s) {
    AttendParams p = {};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.n_pages = n_pages;
    p.P = P;
    while ((1 << p.log_p) < P) ++p.log_p;
    p.H = H;
    p.group = Hq / H;
    if (max_new > T) max_new = T;                                    // no sequence has more
    p.tile_rows = tile_rows_of(max_new, p.group, D);
    const int64_t row_tiles = row_tiles_of(max_new, p.group, D);
    const int64_t units = n_seq * H * row_tiles;
    if (units > 0x7fffffff) return cudaErrorInvalidValue;
    p.row_tiles = (int)row_tiles;
    p.pages = pages;
    p.ld_pages = ld_pages;
    p.q_starts = q_starts;
    p.kv_lens = kv_lens;
    p.n_seq = n_seq;
    p.T = T;
    p.ldq = ldq;
    p.ldo = ldo;
    p.q = q;
    p.tree = tree;
    p.scale = scale;
    p.bf16 = t == QMM_BF16;
    p.out = out;
    p.lse = lse;
    const size_t per_split = split_bytes(T * Hq, D);
    const Split split = split_of(n_seq, H, row_tiles, p.tile_rows, max_len);
    p.splits = split.splits;
    p.budget = split.budget;
    p.waves = split.waves;
    p.fixed = split.fixed;
    if ((size_t)p.splits * per_split > ws_bytes) p.splits = (int)(ws_bytes / per_split);
    if (p.splits < 2) {
        p.splits = 1;
    } else {
        p.part_o = static_cast<float *>(ws);
        p.part_ml = p.part_o + (size_t)p.splits * (size_t)T * (size_t)Hq * (size_t)D;
    }
    const int64_t ctas = p.splits > 1 ? (int64_t)p.budget * p.waves * H * row_tiles : units;
    if (p.splits > 1 && T * Hq > 0x7fffffff) return cudaErrorInvalidValue;       // rows of the join
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    switch (D / 32) {
        case 1: return launch_blocks<1>(type, p, ctas, split.even, s);
        case 2: return launch_blocks<2>(type, p, ctas, split.even, s);
        case 3: return launch_blocks<3>(type, p, ctas, split.even, s);
        case 4: return launch_blocks<4>(type, p, ctas, split.even, s);
        case 5: return launch_blocks<5>(type, p, ctas, split.even, s);
        case 6: return launch_blocks<6>(type, p, ctas, split.even, s);
        case 7: return launch_blocks<7>(type, p, ctas, split.even, s);
        default: return launch_blocks<8>(type, p, ctas, split.even, s);
    }
}

QMM_DCHECK_READER(read_dcheck_attend)

}  // namespace qmm
