// attend_tc.cu -- attention over the block-quantized cache for more rows than a decode step has (trees of
// drafted tokens, pieces of a prompt), on tcgen05: 128 rows (new token x query head of one key/value head)
// to a CTA, heads of up to 128 elements.
//
// The formulas, masks and partial results are those of attend.cu.  With 128 rows the cost is no longer the
// cache's bytes but expanding its codes and the exponentials, so the codes are expanded once a CTA, into
// shared memory, and both products run on the tensor cores from there:
//   S [128 rows x 128 keys] = Q K^T   A = Q, B = K, both K-major in shared memory, S in tensor memory;
//   O [128 rows x D]       = P V      A = P from tensor memory, B = V^T (K-major over the keys).
// A row is a lane of tensor memory and a thread, so that a row's maximum and sum need no exchange between
// threads.  Two groups of four warps take the tiles of keys in turn, each with its own maximum, sum and output:
// a tile's path from scores to p is mostly latency, and the groups' overlap.  The outputs stay in tensor memory.
// p is taken relative to a reference that follows the row's maximum only when that has grown by more than
// 2^8, so that the output is seldom rescaled; the groups' results are joined at the end.
//
// Arithmetic.  k = d * q is split exactly into two fp16 terms, k = hi + lo with hi = fp16(k), which both take part
// (hi alone put 1e-5 into a row's log-sum); v = d * q is rounded to fp16 (2^-12); the query row is scaled by a power
// of two into fp16's range; p is kept in fp16 times 2^7 (at most 2^15), for fp16 outputs in two terms (see attend.cu);
// all sums are fp32.
//
// The raw codes of two tiles of keys come through a ring of asynchronous copies; a key's codes are padded to
// an odd number of 16-byte pieces, so that a warp's 32 keys meet no bank twice.  V^T is written two keys to
// a word: slots 2l and 2l + 1 of a chunk of 64 are keys l and l + 32, the lanes of one load, and K's rows
// (and so the columns of S and p) are in that order too.
//
// Warps: 0-3 and 4-7 rows, of even and odd tiles; 8-15 codes, up to two tiles ahead; 16 products.  (Four warps of
// codes took twice as long as the rows: 277 us for 38 sequences of 8192 tokens, 128 rows, against 113 without.)
// Tensor memory (512 columns): S twice 128 (p overwrites the S that it came from), O twice 128.
//
// What bounds it: a tile's chain (scores, two passes over them, p, values) at two tiles under way, and the instructions of
// the exponentials and of the expansion.  38 sequences of 8192 tokens, 4 heads, 128 rows of bf16: 171 us, 478
// TFLOP/s (2.7 us a tile of 128 keys); trees of 32 tokens x 4 over 8 sequences of 200 to 4096 tokens of Q4_0,
// fp16: 42 us, of which 7 pass before the first scores, 4 in the writing of partial results and 6 in the join.
// The passes over the scores are loops: unrolled, the code of the three roles does not stay in the instruction
// cache (51 us for the trees, 437 for 38 sequences, 8 heads, fp16, against 42 and 354).
// Every wait is bounded; on expiry the kernel records QMM_ERR_TIMEOUT, lets its products land, frees
// tensor memory and returns.
#include <cuda.h>

#include "qmm_internal.cuh"

#include "attend.cuh"

namespace qmm {
namespace {

__device__ unsigned g_attend_status = 0;   // bit 0: a bounded wait gave up

using namespace pipe;
using namespace tc;

constexpr int kKeysTc = 128;
constexpr int kCodeWarps = 8, kCodeThreads = kCodeWarps * 32;
constexpr int kThreadsTc = 256 + kCodeThreads + 32;
constexpr int kColS = 0, kColO = 256;
constexpr float kBiasTc = 7.0f, kSlack = 8.0f;             // p is kept times 2^7; the maximum may pass its reference by 2^8

template <int TYPE, int DB>
struct TcPlan {
    static constexpr int D = DB * 32, CB = DB * (TYPE == QMM_Q8_0 ? 32 : 16);
    static constexpr int NC = (DB + 1) / 2;                // chunks of 64 elements: 128-byte rows
    static constexpr int kChunk = 128 * 128;               // 128 rows of one
    static constexpr int kVChunk = D * 128;                // D rows of 64 keys
    static constexpr int PK = CB / 16, kPitch = (PK | 1) * 16;     // 16-byte pieces of a key's codes, and its pitch
    static constexpr int kQ = 0, kK = kQ + NC * kChunk, kV = kK + 2 * NC * kChunk;   // K: hi, then lo
    static constexpr int kRaw = kV + 2 * kVChunk;          // two stages of: K codes, V codes, K scales, V scales
    static constexpr int kRawV = 128 * kPitch, kRawKs = 2 * 128 * kPitch, kRawVs = kRawKs + 128 * DB * 2, kRawBytes = kRawVs + 128 * DB * 2;
    static constexpr int kBad = kRaw + 2 * kRawBytes;      // rows whose result is not finite
    static constexpr int kStats = kBad + kTcRows * 4;      // [group][row]: reference and sum
    static constexpr int kMul = kStats + 2 * kTcRows * 8;  // score -> power of two
    static constexpr int kBars = kMul + kTcRows * 4;
    static constexpr int kNumBars = 16;
    static constexpr size_t kSmem = 1024 + kBars + kNumBars * 8 + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory plan too large");
};

__device__ __forceinline__ bool wait_tc(uint32_t bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, wait_bounded_on(bar, parity, abort, &g_attend_status, kWaitLimitNs));
}

__device__ __forceinline__ void tmem_ld32x(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
        "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    // the wait writes the registers too, so that no use of them can be scheduled before it
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
    asm volatile(""
                 : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Four unsigned bytes (codes of up to 8 bits) as two half2 of 1024 + byte, minus `off` in both halves.
__device__ __forceinline__ void bytes_h2(uint32_t x, uint32_t off, uint32_t &lo, uint32_t &hi) {
    lo = h2_bits(__hsub2(bits_h2(__byte_perm(x, 0x64646464u, 0x4140u)), bits_h2(off)));
    hi = h2_bits(__hsub2(bits_h2(__byte_perm(x, 0x64646464u, 0x4342u)), bits_h2(off)));
}
__device__ __forceinline__ void swap_halves(uint32_t (&h)[8], bool swap) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t a = swap ? h[4 + k] : h[k], b = swap ? h[k] : h[4 + k];
        h[k] = a;
        h[4 + k] = b;
    }
}
constexpr uint32_t kOff8 = 0x64806480u;    // 1152: int8 codes with the sign bit flipped
constexpr uint32_t kOff4 = 0x64086408u;    // 1032: nibbles

template <int TYPE, int DB>
__global__ void __launch_bounds__(kThreadsTc, 1) attend_tc_kernel(const __grid_constant__ AttendParams p) {
    using L = TcPlan<TYPE, DB>;
    constexpr int D = L::D, CB = L::CB, NC = L::NC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    int *row_bad = reinterpret_cast<int *>(smem + L::kBad);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
    uint64_t *q_full = bars, *k_full = bars + 1, *k_empty = bars + 2, *v_full = bars + 3, *v_empty = bars + 4, *s_full = bars + 5,
             *p_full = bars + 7, *o_full = bars + 9, *raw_full = bars + 11, *raw_empty = bars + 13, *done = bars + 15;
    float2 *stats = reinterpret_cast<float2 *>(smem + L::kStats);
    float *muls = reinterpret_cast<float *>(smem + L::kMul);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::kNumBars);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *odd_flag = reinterpret_cast<int *>(tmem_slot + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    Rows w;
    if (!find_rows<kTcRows>(p, reinterpret_cast<int *>(smem), kThreadsTc, w)) return;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(q_full), 2 * kTcRows);
        mbar_init(smem_u32(done), 1);
        mbar_init(smem_u32(k_full), kCodeThreads);
        mbar_init(smem_u32(k_empty), 1);
        mbar_init(smem_u32(v_full), kCodeThreads);
        mbar_init(smem_u32(v_empty), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&s_full[s]), 1);
            mbar_init(smem_u32(&p_full[s]), kTcRows);
            mbar_init(smem_u32(&o_full[s]), 1);
            mbar_init(smem_u32(&raw_full[s]), kCodeThreads);
            mbar_init(smem_u32(&raw_empty[s]), kCodeThreads);
        }
        *abort = 0;
        *odd_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < kTcRows) row_bad[threadIdx.x] = 0;
    __syncwarp();
    if (warp == 8 + kCodeWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Not before the allocation: a kernel that allocates before it waits for this one, as the products do, could else
    // hold columns of this SM's tensor memory while it waits, and the allocation would wait for them.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tiles = (int)((w.k1 - w.k0 + kKeysTc - 1) / kKeysTc);
    const int32_t *table = p.pages + w.s * p.ld_pages;
    // pages of a tile's eight groups of 16 keys, in lanes 0-7 (-1: past the keys)
    auto pages_of = [&](int i) -> int {
        const int64_t j = w.k0 + (int64_t)i * kKeysTc + 16 * (lane & 7);
        const int page = i < tiles && j < w.k1 && QMM_DCHECK((j >> p.log_p) < p.ld_pages) ? table[j >> p.log_p] : -1;
        return page < p.n_pages ? page : -1;
    };

    const bool two = !p.bf16;                                       // p in two terms, where the output keeps 11 bits
    const int row = threadIdx.x & 127, group = threadIdx.x >> 7;   // of the row warps; row = lane of tensor memory
    const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    if (warp < 8) {
        // =============================== rows ===============================
        const int r = w.r0 + row, i_tok = r / p.group;
        {
            // the query rows, scaled by a power of two so that the largest element lies in [1, 2): sixteen lanes a row, two
            // rows of a warp's sixteen at a time
            const int c = lane & 15;                            // eight elements of the row
            uint4 raw[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int x = 16 * warp + 2 * u + (lane >> 4), rx = w.r0 + x, tok = rx / p.group;
                const int64_t at = (w.q0 + tok) * p.ldq + (int64_t)(w.h * p.group + (rx - tok * p.group)) * D + 8 * c;
                raw[u] = x < w.rows && c < 4 * DB ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int x = 16 * warp + 2 * u + (lane >> 4);
                uint32_t top2 = __vmaxu2(__vmaxu2(raw[u].x & 0x7FFF7FFFu, raw[u].y & 0x7FFF7FFFu), __vmaxu2(raw[u].z & 0x7FFF7FFFu, raw[u].w & 0x7FFF7FFFu));
#pragma unroll
                for (int z = 8; z > 0; z >>= 1) top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, z));
                const uint32_t topb = max(top2 & 0xFFFFu, top2 >> 16);
                const float top = p.bf16 ? bits_to_float<__nv_bfloat16>(topb) : bits_to_float<__half>(topb);
                const int e = top > 0.0f && top < INFINITY ? max((int)(__float_as_uint(top) >> 23) - 127, -120) : 0;
                const float m = p.scale * 1.4426950408889634f, down = copysignf(exp2f((float)-e), m);
                if (c == 0) muls[x] = fmaxf(fabsf(m), 1e-30f) * exp2f((float)e);   // a scale of 0 still has to order -inf below 0
                const uint32_t in[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = p.bf16 ? unpack2(in[k], __nv_bfloat16{}) : unpack2(in[k], __half{});
                    h[k] = pack2(f.x * down, f.y * down, __half{});
                }
                if (c < 8 * NC) *reinterpret_cast<uint4 *>(smem + L::kQ + (c >> 3) * L::kChunk + sw128_off(x, c & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(q_full));
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float mul = muls[row];
        const uint64_t word = p.tree && row < w.rows ? p.tree[w.q0 + i_tok] : 0;
        float ref = -INFINITY, sum[4] = {0.f, 0.f, 0.f, 0.f};
        bool ok = true;
        int page = pages_of(group);
        for (int i = group; i < tiles; i += 2) {
            const uint32_t phase = (uint32_t)((i >> 1) & 1);
            const uint32_t t_s = t_lane + kColS + 128 * group;
            const int64_t j0 = w.k0 + (int64_t)i * kKeysTc;
            const uint32_t groups = __ballot_sync(0xffffffffu, lane < 8 && page >= 0);
            page = pages_of(i + 2);
            if (!wait_tc(smem_u32(&s_full[group]), phase, abort)) { ok = false; break; }
            tc_fence_after();
            const bool masked = groups != 0xFFu || j0 + kKeysTc > w.k1 || j0 + kKeysTc > w.first;
            // keys 32c .. 32c + 31 of this tile that the row sees
            auto keys = [&](int c) -> uint32_t {
                uint32_t m = ((groups >> (2 * c)) & 1 ? 0xFFFFu : 0u) | ((groups >> (2 * c + 1)) & 1 ? 0xFFFF0000u : 0u);
                const int64_t left = w.k1 - (j0 + 32 * c);      // keys of the split from here on
                m &= left >= 32 ? 0xFFFFFFFFu : (left <= 0 ? 0u : (1u << (int)left) - 1u);
                const int64_t nb = j0 + 32 * c - w.first;       // place of the first key among the new tokens
                if (nb > -32) {
                    uint32_t v;                                  // the row's view of new tokens nb .. nb + 31
                    if (p.tree) {
                        v = nb >= 64 ? 0u : (nb >= 0 ? (uint32_t)(word >> nb) : (uint32_t)(word << -nb) | ((1u << -nb) - 1u));
                    } else {
                        const int64_t upto = i_tok - nb + 1;     // it sees that many of them
                        v = upto >= 32 ? 0xFFFFFFFFu : (upto <= 0 ? 0u : (1u << (int)upto) - 1u);
                    }
                    m &= v;
                }
                return m;
            };
            // the same for columns 32c .. 32c + 31: column k is key 16 (c & 1) + k / 2 of the chunk, plus 32 if k is odd
            auto seen = [&](int c) -> uint32_t {
                uint32_t e = keys(c & 2) >> (16 * (c & 1)) & 0xFFFFu, o2 = keys((c & 2) + 1) >> (16 * (c & 1)) & 0xFFFFu;
#pragma unroll
                for (int z = 8; z > 0; z >>= 1) {               // spreads the 16 bits to every second place
                    const uint32_t keep = z == 8 ? 0x00FF00FFu : (z == 4 ? 0x0F0F0F0Fu : (z == 2 ? 0x33333333u : 0x55555555u));
                    e = (e | (e << z)) & keep;
                    o2 = (o2 | (o2 << z)) & keep;
                }
                return e | (o2 << 1);
            };
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                tmem_ld32x(t_s + 32 * c, v);
                if (masked) {
                    const uint32_t bits = seen(c);
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = (bits >> k) & 1 ? v[k] : 0xFF800000u;
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(v[k]));
            }
            const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
            if (__any_sync(0xffffffffu, m > ref + kSlack || (ref == -INFINITY && m > -INFINITY))) {
                const float to = fmaxf(m, ref), down = ex2(ref - (to == -INFINITY ? 0.0f : to));
                ref = to;
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] *= down;
                if (i >= 2) {
                    // the group's products so far, all done, are rescaled
                    if (!wait_tc(smem_u32(&o_full[group]), phase ^ 1u, abort)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 2 * DB; ++c) {
                        uint32_t v[16];
                        tmem_ld16(t_lane + kColO + 128 * group + 16 * c, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * down);
                        tmem_st16(t_lane + kColO + 128 * group + 16 * c, v);
                    }
                }
            }
            const float shift = kBiasTc - (ref == -INFINITY ? 0.0f : ref);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t v[32], h[16];
                tmem_ld32x(t_s + 32 * c, v);
                const uint32_t bits = masked ? seen(c) : 0xFFFFFFFFu;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float p0 = ex2(fmaf(__uint_as_float(v[2 * k]), mul, shift)), p1 = ex2(fmaf(__uint_as_float(v[2 * k + 1]), mul, shift));
                    if (masked) {
                        p0 = (bits >> (2 * k)) & 1 ? p0 : 0.0f;
                        p1 = (bits >> (2 * k + 1)) & 1 ? p1 : 0.0f;
                    }
                    sum[k & 3] += p0 + p1;
                    h[k] = pack2(p0, p1, __half{});
                    if (two) {
                        const float2 hi = unpack2(h[k], __half{});
                        v[k] = pack2(p0 - hi.x, p1 - hi.y, __half{});
                    }
                }
                // over the columns that were read: 16 of hi, 16 of lo
                tmem_st16(t_s + 32 * c, h);
                if (two) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) h[k] = v[k];
                    tmem_st16(t_s + 32 * c + 16, h);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(smem_u32(&p_full[group]));
        }
        if (ok && tiles > group) {
            const int last = (tiles - 1 - group) >> 1;          // the group's last tile, counted among its own
            ok = wait_tc(smem_u32(&o_full[group]), (uint32_t)(last & 1), abort);
        }
        stats[group * kTcRows + row] = make_float2(ref, (sum[0] + sum[1]) + (sum[2] + sum[3]));
    } else if (warp < 8 + kCodeWarps) {
        // =============================== codes ===============================
        const int tid = threadIdx.x - 256, wq = warp - 8;
        constexpr int PK = L::PK;                              // pieces of a key
        constexpr int KP = (128 * PK + kCodeThreads - 1) / kCodeThreads, VW = kCodeWarps / 2, VP = (PK + VW - 1) / VW;
        const int64_t head = (int64_t)w.h * p.P * (CB + 2 * DB), page_bytes = (int64_t)p.H * p.P * (CB + 2 * DB);
        bool odd = false;
        // copies the raw codes and scales of tile i; `page`: its pages, in lanes 0-7
        auto issue = [&](int i, int page) {
            if (i < tiles) {
                const uint32_t st = smem_u32(smem + L::kRaw + (i & 1) * L::kRawBytes);
                const int off0 = (int)(w.k0 + (int64_t)i * kKeysTc) & (p.P - 1);      // P may be below 128
#pragma unroll
                for (int it = 0; it < KP; ++it) {
                    const int u = it * kCodeThreads + tid, key = u / PK, c = u % PK;
                    const int pg = __shfl_sync(0xffffffffu, page, (key >> 4) & 7);
                    const int64_t at = (int64_t)pg * page_bytes + head + ((off0 + key) & (p.P - 1)) * CB + 16 * c;
                    if (pg >= 0 && key < 128 && QMM_DCHECK(at + 16 <= p.n_pages * page_bytes)) {
                        cp_async16(st + key * L::kPitch + 16 * c, p.k_cache + at);
                        cp_async16(st + L::kRawV + key * L::kPitch + 16 * c, p.v_cache + at);
                    }
                }
                // scales: 2 * DB pieces for each group of 16 keys
                const int grp = tid / (2 * DB), c = tid % (2 * DB);
                const int pg = __shfl_sync(0xffffffffu, page, grp & 7);
                const int64_t at = (int64_t)pg * page_bytes + head + p.P * CB + ((off0 + 16 * grp) & (p.P - 1)) * (2 * DB) + 16 * c;
                if (grp < 8 && pg >= 0 && QMM_DCHECK(at + 16 <= p.n_pages * page_bytes)) {
                    cp_async16(st + L::kRawKs + tid * 16, p.k_cache + at);
                    cp_async16(st + L::kRawVs + tid * 16, p.v_cache + at);
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&raw_full[i & 1])) : "memory");
        };
        auto valid = [&](int i, int key, uint32_t groups) { return (groups >> (key >> 4) & 1) && w.k0 + (int64_t)i * kKeysTc + key < w.k1; };
        auto convert_k = [&](int i, uint32_t groups) {
            const uint8_t *raw = smem + L::kRaw + (i & 1) * L::kRawBytes;
            const uint16_t *ks = reinterpret_cast<const uint16_t *>(raw + L::kRawKs);
#pragma unroll
            for (int it = 0; it < KP; ++it) {
                const int u = it * kCodeThreads + tid, key = u / PK, c = u % PK;
                if (key >= 128) break;
                const uint32_t d2 = valid(i, key, groups) ? ks[key * DB + (TYPE == QMM_Q8_0 ? c >> 1 : c)] * 0x00010001u : 0u;
                const uint4 v4 = *reinterpret_cast<const uint4 *>(raw + key * L::kPitch + 16 * c);
                const uint32_t x[4] = {v4.x, v4.y, v4.z, v4.w};
                const int slot = (key & 64) | ((key & 31) << 1) | ((key >> 5) & 1);
                auto store = [&](int chunk, const uint32_t *h) {   // 8 elements
                    uint8_t *at = smem + L::kK + (chunk >> 3) * L::kChunk + sw128_off(slot, chunk & 7);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const __half2 v = __hmul2_rn(bits_h2(h[z]), bits_h2(d2));
                        hi[z] = h2_bits(v);
                        lo[z] = h2_bits(__hfma2(bits_h2(h[z]), bits_h2(d2), __hneg2(v)));     // exact
                    }
                    *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(at + NC * L::kChunk) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                };
                if constexpr (TYPE == QMM_Q8_0) {
                    uint32_t h[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) bytes_h2(x[k] ^ 0x80808080u, kOff8, h[2 * k], h[2 * k + 1]);
                    // lanes of the second chunk of 64 elements take their halves the other way round: the first chunk's
                    // lanes are in the same banks
                    swap_halves(h, c >> 2 & 1);
                    store(2 * c + (c >> 2 & 1), h);
                    store(2 * c + 1 - (c >> 2 & 1), h + 4);
                } else {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {               // elements 0-15 in the low nibbles, 16-31 in the high ones
                        uint32_t h[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) bytes_h2((x[k] >> (4 * n)) & 0x0F0F0F0Fu, kOff4, h[2 * k], h[2 * k + 1]);
                        swap_halves(h, c >> 1 & 1);
                        store(4 * c + 2 * n + (c >> 1 & 1), h);
                        store(4 * c + 2 * n + 1 - (c >> 1 & 1), h + 4);
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(k_full));
        };
        auto convert_v = [&](int i, uint32_t groups) {
            const uint8_t *raw = smem + L::kRaw + (i & 1) * L::kRawBytes;
            const uint16_t *vs = reinterpret_cast<const uint16_t *>(raw + L::kRawVs);
            const int ka = 64 * (wq & 1) + lane, kb = ka + 32;     // slots 2 lane and 2 lane + 1
            const uint32_t have = (valid(i, ka, groups) ? 0xFFFFu : 0u) | (valid(i, kb, groups) ? 0xFFFF0000u : 0u);
            uint8_t *vt = smem + L::kV + (wq & 1) * L::kVChunk + (lane & 3) * 4;
#pragma unroll
            for (int it = 0; it < VP; ++it) {
                const int c = VW * it + (wq >> 1), blk = TYPE == QMM_Q8_0 ? c >> 1 : c;
                if (c >= PK) break;
                uint32_t d2 = have & ((uint32_t)vs[ka * DB + blk] | ((uint32_t)vs[kb * DB + blk] << 16));
                const uint32_t fine = finite2(d2);
                odd |= fine != 0xFFFFFFFFu;
                d2 &= fine;
                const uint4 a4 = *reinterpret_cast<const uint4 *>(raw + L::kRawV + ka * L::kPitch + 16 * c);
                const uint4 b4 = *reinterpret_cast<const uint4 *>(raw + L::kRawV + kb * L::kPitch + 16 * c);
                const uint32_t xa[4] = {a4.x, a4.y, a4.z, a4.w}, xb[4] = {b4.x, b4.y, b4.z, b4.w};
                auto store4 = [&](int d0, uint32_t a, uint32_t bq, uint32_t off) {   // elements d0 .. d0 + 3 of both keys
                    uint32_t h[4];
                    bytes_h2(__byte_perm(a, bq, 0x5140), off, h[0], h[1]);
                    bytes_h2(__byte_perm(a, bq, 0x7362), off, h[2], h[3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t *>(vt + sw128_off(d0 + k, lane >> 2)) = hmul2(h[k], d2);
                };
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (TYPE == QMM_Q8_0) {
                        store4(16 * c + 4 * k, xa[k] ^ 0x80808080u, xb[k] ^ 0x80808080u, kOff8);
                    } else {
                        store4(32 * c + 4 * k, xa[k] & 0x0F0F0F0Fu, xb[k] & 0x0F0F0F0Fu, kOff4);
                        store4(32 * c + 16 + 4 * k, (xa[k] >> 4) & 0x0F0F0F0Fu, (xb[k] >> 4) & 0x0F0F0F0Fu, kOff4);
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(v_full));
        };
        int pg0 = pages_of(0), pg1 = pages_of(1), pg2 = pages_of(2);       // of tiles i, i + 1, i + 2
        issue(0, pg0);
        issue(1, pg1);
        if (tiles > 0 && wait_tc(smem_u32(&raw_full[0]), 0u, abort)) {
            convert_k(0, __ballot_sync(0xffffffffu, lane < 8 && pg0 >= 0));
            for (int i = 0; i < tiles; ++i) {
                const uint32_t groups = __ballot_sync(0xffffffffu, lane < 8 && pg0 >= 0);
                // the keys of the next tile once the scores of this one are computed, then this one's values
                if (i + 1 < tiles) {
                    if (!wait_tc(smem_u32(&raw_full[(i + 1) & 1]), (uint32_t)(((i + 1) >> 1) & 1), abort)) break;
                    if (!wait_tc(smem_u32(k_empty), (uint32_t)(i & 1), abort)) break;
                    convert_k(i + 1, __ballot_sync(0xffffffffu, lane < 8 && pg1 >= 0));
                }
                if (i > 0 && !wait_tc(smem_u32(v_empty), (uint32_t)((i - 1) & 1), abort)) break;
                convert_v(i, groups);
                mbar_arrive(smem_u32(&raw_empty[i & 1]));
                if (i + 2 < tiles) {
                    if (!wait_tc(smem_u32(&raw_empty[i & 1]), (uint32_t)((i >> 1) & 1), abort)) break;
                    issue(i + 2, pg2);
                }
                pg0 = pg1;
                pg1 = pg2;
                pg2 = pages_of(i + 3);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (odd) *odd_flag = 1;
    } else {
        // =============================== products ===============================
        uint32_t e;
        asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
        const bool lead = e != 0;
        const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + L::kQ)), k_desc = smem_desc_sw128(smem_u32(smem + L::kK)),
                       v_desc = smem_desc_sw128(smem_u32(smem + L::kV));
        constexpr uint32_t id_s = idesc_f16(128, kKeysTc), id_o = idesc_f16(128, D);
        auto scores = [&](int i) -> bool {
            if (!wait_tc(smem_u32(k_full), (uint32_t)(i & 1), abort)) return false;
            tc_fence_after();
            if (lead) {
#pragma unroll
                for (int k = 0; k < 4 * DB; ++k) {              // 16 elements a step, of hi, then of lo
                    const int term = k / (2 * DB), el = k % (2 * DB);
                    const uint64_t at = (uint64_t)((el >> 2) * (L::kChunk >> 4) + 2 * (el & 3));
                    mma_f16_ss(tmem + kColS + 128 * (i & 1), q_desc + at, k_desc + at + (uint64_t)(term * NC * (L::kChunk >> 4)), id_s,
                               k > 0 ? 1u : 0u);
                }
                mma_commit(smem_u32(k_empty));
                mma_commit(smem_u32(&s_full[i & 1]));
            }
            __syncwarp();
            return true;
        };
        bool ok = tiles == 0 || (wait_tc(smem_u32(q_full), 0u, abort) && scores(0) && (tiles == 1 || scores(1)));
        for (int i = 0; i < tiles && ok; ++i) {
            const int b = i & 1;
            if (!wait_tc(smem_u32(&p_full[b]), (uint32_t)((i >> 1) & 1), abort)) break;
            if (!wait_tc(smem_u32(v_full), (uint32_t)(i & 1), abort)) break;
            tc_fence_after();
            if (lead) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {                   // 16 keys a step
                    const uint64_t at = (uint64_t)((k >> 2) * (L::kVChunk >> 4) + 2 * (k & 3));
                    const uint32_t pa = tmem + kColS + 128 * b + 32 * (k >> 1) + 8 * (k & 1);
                    mma_f16_ts(tmem + kColO + 128 * b, pa, v_desc + at, id_o, i >= 2 || k > 0 ? 1u : 0u);
                    if (two) mma_f16_ts(tmem + kColO + 128 * b, pa + 16, v_desc + at, id_o, 1u);
                }
                mma_commit(smem_u32(v_empty));
                mma_commit(smem_u32(&o_full[b]));
            }
            __syncwarp();
            // the next scores of this group overwrite the p that the products above read
            if (i + 2 < tiles && (!wait_tc(smem_u32(&o_full[b]), (uint32_t)((i >> 1) & 1), abort) || !scores(i + 2))) break;
        }
        if (lead) {
            // every product issued has landed before tensor memory is released
            mma_commit(smem_u32(done));
            wait_drain(smem_u32(done), 0u);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        // ---- the two groups' results, joined; a group writes its half of the elements ----
        const float2 a = stats[row], b = stats[kTcRows + row];
        const float m = fmaxf(a.x, b.x), base = m == -INFINITY ? 0.0f : m;
        const float fa = ex2(a.x - base), fb = ex2(b.x - base), sum = fa * a.y + fb * b.y;
        float all = sum * 0.0f;                                 // 0 unless something is not finite
#pragma unroll
        for (int c = 0; c < DB; ++c) {
            uint32_t u[16], v[16];
            const uint32_t at = t_lane + kColO + group * (D / 2) + 16 * c;
#pragma unroll
            for (int k = 0; k < 16; ++k) u[k] = v[k] = 0u;
            if (tiles > 0) {
                tmem_ld16(at, u);
                tmem_wait_ld(u);
            }
            if (tiles > 1) {
                tmem_ld16(at + 128, v);
                tmem_wait_ld(v);
            }
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
                float o[8];
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    o[z] = fa * __uint_as_float(u[k + z]) + fb * __uint_as_float(v[k + z]);
                    all = fmaf(o[z], 0.0f, all);
                }
                if (row < w.rows) write_row(p, w, D, row, group * (D / 2) + 16 * c + k, o, m + (kBias - kBiasTc), sum);
            }
        }
        if (row < w.rows && !(all == 0.0f)) {
            row_bad[row] = 1;
            *odd_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8 + kCodeWarps) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
    if (*odd_flag) rows_one_by_one<TYPE, DB, kThreadsTc / 32>(p, w, row_bad);
}

template <int TYPE, int DB>
cudaError_t launch_typed(const AttendParams &p, int64_t ctas, cudaStream_t s) {
    auto kern = attend_tc_kernel<TYPE, DB>;
    static int attr_done[4] = {0, 0, 0, 0};
    const cudaError_t e = ensure_smem_limit(kern, TcPlan<TYPE, DB>::kSmem, attr_done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)ctas), kThreadsTc, TcPlan<TYPE, DB>::kSmem, s, p);
}

}  // namespace

cudaError_t launch_attend_tc(qmm_type type, const AttendParams &p, int DB, int64_t ctas, cudaStream_t s) {
    if (type == QMM_Q8_0) {
        switch (DB) {
            case 1: return launch_typed<QMM_Q8_0, 1>(p, ctas, s);
            case 2: return launch_typed<QMM_Q8_0, 2>(p, ctas, s);
            case 3: return launch_typed<QMM_Q8_0, 3>(p, ctas, s);
            default: return launch_typed<QMM_Q8_0, 4>(p, ctas, s);
        }
    }
    switch (DB) {
        case 1: return launch_typed<QMM_Q4_0, 1>(p, ctas, s);
        case 2: return launch_typed<QMM_Q4_0, 2>(p, ctas, s);
        case 3: return launch_typed<QMM_Q4_0, 3>(p, ctas, s);
        default: return launch_typed<QMM_Q4_0, 4>(p, ctas, s);
    }
}

cudaError_t read_and_clear_attend_status(unsigned *out, cudaStream_t s) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_attend_status, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbolAsync(g_attend_status, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, s);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(s);
}

QMM_DCHECK_READER(read_dcheck_attend_tc)

}  // namespace qmm
