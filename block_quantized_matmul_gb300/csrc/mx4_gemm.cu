// mx4_gemm.cu -- the product of two microscaled 4-bit operands (mx4.cuh) on the block-scaled tensor cores
// (tcgen05.mma, kind::mxf4: E2M1 x E2M1 with one E8M0 scale per 32 of either operand, fp32 sums).
//
//   Y[m, n] = sum_b 2^(ea[m, b] + ew[n, b] - 254) * sum_{j < 32} a[m, 32b + j] * w[n, 32b + j]
//
// The weight rows are the instruction's 128 rows (the lanes of tensor memory), the tokens its columns, TN = 16 or 32 of
// them.  So one token costs no more than the weight's bytes (4096 x 14336: 7.3 us with the token's quantization, 31.2
// MB, 4.3 TB/s; a floor of 4.6 us), and a lane's results of one token are consecutive in y.  More than 32
// tokens take the pairs' kernel below, which is as fast from 33 tokens on for 4096 weight rows, and faster for
// more: 64 tokens x 14336 rows 12.1 us for 19.0.
//
// A stage of the pipeline is 256 of K: 128 weight rows x 128 bytes and TN token rows x 128 bytes by
// tensor copies into the 128-byte-swizzled layout, and the scales of both, which are stored as the
// instruction wants them (512 bytes for 128 rows x 128 K), by plain bulk copies.  tcgen05.cp moves the
// scales on into tensor memory; the same thread issues the copies and the products, so they stay in order.
// Rows past an operand's end and K past its end arrive as zero codes; the scales there are 0 (K) or
// belong to rows whose results are not stored.
//
// Few tokens: the weight's row tiles alone do not fill the GPU, so the CTAs of a cluster share a tile and
// take K in turn; each adds up the parts of its share of the tokens, in the order of the ranks, through
// distributed shared memory.
//
// Long K: after each 16384 of K the sums go on in another accumulator (kDrain), and the result warps add them up in fp32.
//
// Warps: 0 copies, 1 products (and tensor memory), 2-5 results.
// Every wait is bounded; on expiry the kernel records QMM_ERR_TIMEOUT, lets what is in flight land,
// frees tensor memory and returns.
#include <cuda.h>

#include <type_traits>

#include "pipeline.cuh"
#include "qmm_internal.cuh"

#include "elem.cuh"
#include "mx4.cuh"
#include "tc_common.cuh"

namespace qmm {
namespace {

__device__ unsigned g_mx4_status = 0;      // bit 0: a bounded wait gave up

using namespace pipe;
using namespace tc;

constexpr int kRows = 128;                 // weight rows per tile
constexpr int kThreads = 192;
constexpr int kEpilogue = 128;
constexpr int kMaxSplit = 8;               // CTAs of a cluster
// Stages (16384 of K) after which sums go on in a fresh accumulator.  The tensor cores round every addition to a sum towards
// zero, so the error grows with the products added to one: with data of one sign 5.7e-6 of the sum at K = 16384, 1.2e-5 at
// 32768 and 4.5e-5 at 131072 in a single accumulator, and the stated bound is 1e-5.  Pairs pay for it with a pause in the
// products: 2048 x 28672 x 8192 156 us for 150.
constexpr int kDrain = 64;

struct Mx4Params {
    const uint8_t *ws, *as;                // scales of the weight and the activations
    void *y;
    int64_t N, M, ldy;
    int n128;                              // K / 128, rounded up: scale blocks of a row of blocks
    int nk;                                // stages: K / 256, rounded up
    int last_steps;                        // K = 64 products of the last stage (1 to 4)
    int split;                             // CTAs of a cluster, which share a tile's K
    int sums, cols;                        // accumulators of a CTA; columns of tensor memory
    int early_weights;                     // the weight may be read before the kernel before this one is done
    int dtype;
    const void *x;                         // rows to be quantized here (fused)
    int64_t ldx, K;
    int x_vec;                             // they are 32-byte aligned
};

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int *abort) {
    return wait_bounded_on(bar, parity, abort, &g_mx4_status, kWaitLimitNs);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort));
}

// Shared-memory descriptor of 32 lanes x 16 bytes of scales, unswizzled: 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// 512 bytes of scales -> four columns of tensor memory, the 32 lanes repeated in each lane quadrant.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: E2M1 A and B, E8M0 scales, 128 x n; `half` picks the two scales of a K = 64
// product out of the four bytes of a column.
__device__ __forceinline__ constexpr uint32_t idesc_mxf4(int n, int half) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(kRows >> 4) << 24) |
           ((uint32_t)(2 * half) << 29) | ((uint32_t)(2 * half) << 4);
}

// One thread of the (converged) warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
    return ok != 0;
}
// A place in the ring and the phase of its barriers, kept without divisions: the threads that issue copies
// and products have some 500 cycles a stage.
template <int S>
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++s == S) {
            s = 0;
            phase ^= 1u;
        }
    }
};

template <int TN>
struct Plan {
    static constexpr int kW = 0;
    static constexpr int kA = kW + kRows * 128;
    static constexpr int kWS = kA + (TN * 128 + 1023) / 1024 * 1024;
    static constexpr int kAS = kWS + 2 * kMx4ScaleBlock;
    static constexpr int kStageBytes = kAS + 2 * kMx4ScaleBlock;
    static constexpr int kStages = TN >= 32 ? 4 : 5;                     // two CTAs an SM
    // tensor memory: an accumulator of 32 columns for each kDrain stages, then per stage the scales of two K = 128 halves
    // (weight 4 columns, tokens 4)
    static constexpr int kSums = 32;
    static constexpr int kHalfCols = 8;
    static constexpr int cols(int sums) {
        const int used = sums * kSums + kStages * 2 * kHalfCols;
        return used <= 128 ? 128 : (used <= 256 ? 256 : 512);
    }
    static constexpr int kMostSums = (int)(kMaxMatmulK / 256 / kDrain);
    // parts of the other CTAs of a cluster: [rank][token of this CTA's share][row]
    static constexpr int kParts = TN * kRows * 4;
    static constexpr int kPartsAt = kStages * kStageBytes;
    static constexpr int kBars = kPartsAt + kParts;
    static constexpr size_t kSmem = 1024 + kBars + (2 * kStages + 2) * 8 + 16;
    static_assert(TN <= kSums && kMostSums * kSums + kStages * 2 * kHalfCols <= 512 && kSmem <= 227 * 1024, "does not fit");
    // the CTAs of a cluster wait for one another and may share an SM, so that two have to fit its tensor memory
    static_assert(cols(kMostSums / 2) <= 256, "does not fit");
};

// Stores results v[0..n) of tokens m0.. for weight row `row`, those that exist.
template <typename T>
__device__ __forceinline__ void store_tokens(T *y, int64_t ldy, int64_t m0, int64_t M, int64_t row, const uint32_t *v, int n) {
#pragma unroll
    for (int c = 0; c < n; ++c)
        if (m0 + c < M && QMM_DCHECK(row < ldy)) float_to_elem(__uint_as_float(v[c]), y[(m0 + c) * ldy + row]);
}

// XT: void for operands that are quantized already, else the element type of rows that the result warps
// quantize into each stage while its weights arrive.
template <int TN, typename XT>
__global__ void __launch_bounds__(kThreads) mx4_gemm_kernel(const __grid_constant__ Mx4Params p, const __grid_constant__ CUtensorMap w_map,
                                                            const __grid_constant__ CUtensorMap a_map) {
    constexpr bool kFused = !std::is_same<XT, void>::value;
    using L = Plan<TN>;
    constexpr int S = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars), *empty = full + S, *done = empty + S, *parts_in = done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(parts_in + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.split > 1 ? (int)(blockIdx.x % (unsigned)p.split) : 0;
    const int64_t tile = blockIdx.x / (unsigned)p.split;
    const int64_t n0 = tile * kRows, m0 = 0;                     // one tile of tokens
    const int k0 = (int)((int64_t)p.nk * rank / p.split), k1 = (int)((int64_t)p.nk * (rank + 1) / p.split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), kFused ? 1 + kEpilogue / 32 : 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(done), 1);
        mbar_init(smem_u32(parts_in), (uint32_t)(kEpilogue * p.split));
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(p.cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    if (p.split > 1) {
        // the peers' barriers are in place before anything arrives on them
        asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            auto blocks = [&](int k) { return min(2, p.n128 - 2 * k); };
            auto weights = [&](int k, int s) {                 // announces the whole stage
                const uint32_t st = smem_u32(smem + s * L::kStageBytes), bar = smem_u32(&full[s]);
                const uint32_t sb = (uint32_t)blocks(k) * kMx4ScaleBlock;
                // (the stage's wait then runs out)
                if (!QMM_DCHECK(s < S && k < p.nk && blocks(k) > 0 && 2 * k + blocks(k) <= p.n128 && n0 < p.N)) return;
                mbar_arrive_expect_tx(bar, kFused ? (uint32_t)(kRows * 128) + sb
                                                  : (uint32_t)(kRows * 128 + TN * 128) + 2 * sb);
                tma_load_2d(st + L::kW, &w_map, k * 128, (int)n0, bar);
                bulk_g2s(st + L::kWS, p.ws + (tile * p.n128 + 2 * k) * (int64_t)kMx4ScaleBlock, sb, bar);
            };
            auto tokens = [&](int k, int s) {
                if (kFused) return;
                const uint32_t st = smem_u32(smem + s * L::kStageBytes), bar = smem_u32(&full[s]);
                const uint32_t sb = (uint32_t)blocks(k) * kMx4ScaleBlock;
                tma_load_2d(st + L::kA, &a_map, k * 128, (int)m0, bar);
                bulk_g2s(st + L::kAS, p.as + 2 * k * (int64_t)kMx4ScaleBlock, sb, bar);
            };
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&w_map)) : "memory");
            if (!kFused) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a_map)) : "memory");
            const int head = min(S, k1 - k0);
            if (!p.early_weights) asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int i = 0; i < head; ++i) weights(k0 + i, i);
            if (p.early_weights) asm volatile("griddepcontrol.wait;" ::: "memory");
            // Only now: the next kernel may read its weight before it waits, which is sound as long as everything before
            // this kernel is complete (and tensor memory has to be allocated before).
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            for (int i = 0; i < head; ++i) tokens(k0 + i, i);
            int issued = head;
            for (int i = head; i < k1 - k0; ++i) {
                const int s = i % S;
                if (!wait_bounded(smem_u32(&empty[s]), (uint32_t)((i / S - 1) & 1), abort)) break;
                weights(k0 + i, s);
                tokens(k0 + i, s);
                issued = i + 1;
            }
            for (int i = issued > S ? issued - S : 0; i < issued; ++i) wait_drain(smem_u32(&full[i % S]), (uint32_t)((i / S) & 1));
        }
        __syncwarp();
    } else if (warp == 1) {
        const bool lead = elect_one();
        const uint32_t st0 = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
        const uint64_t w_desc = smem_desc_sw128(st0 + L::kW), a_desc = smem_desc_sw128(st0 + L::kA);
        const uint64_t ws_desc = smem_desc_scales(st0 + L::kWS), as_desc = smem_desc_scales(st0 + L::kAS);
        constexpr int kHalf = kMx4ScaleBlock >> 4;                 // in units of a descriptor's address
        asm volatile("griddepcontrol.wait;" ::: "memory");     // here too: however long the kernel before takes, no bounded wait sees it
        Ring<S> r;
        for (int k = k0; k < k1; ++k, r.next()) {
            if (!wait_warp(full0 + 8 * r.s, r.phase, abort)) break;
            tc_fence_after();
            const uint64_t off = (uint64_t)(uint32_t)(r.s * (L::kStageBytes >> 4));
            const uint32_t cols = tmem + (uint32_t)(p.sums * L::kSums + r.s * 2 * L::kHalfCols);
            const int in_sum = (k - k0) % kDrain;
            const uint32_t sum = tmem + (uint32_t)((k - k0) / kDrain * L::kSums);
            const int steps = k == p.nk - 1 ? p.last_steps : 4;
            if (lead) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    copy_scales(cols + h * L::kHalfCols, ws_desc + off + h * kHalf);
                    copy_scales(cols + h * L::kHalfCols + 4, as_desc + off + h * kHalf);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t c = cols + (uint32_t)((q >> 1) * L::kHalfCols);
                    if (q < steps)
                        mma_mxf4(sum, w_desc + off + 2 * q, a_desc + off + 2 * q, idesc_mxf4(TN, q & 1), c, c + 4,
                                 q > 0 ? 1u : (in_sum > 0 ? 1u : 0u));
                }
                mma_commit(empty0 + 8 * r.s);
            }
            __syncwarp();
        }
        if (lead) {
            mma_commit(smem_u32(done));
            wait_drain(smem_u32(done), 0u);
        }
        __syncwarp();
    } else {
        const int qd = warp & 3, row = 32 * qd + lane;
        const int64_t n = n0 + row;
        asm volatile("griddepcontrol.wait;" ::: "memory");     // y may still be read by an earlier kernel, x written
        if constexpr (kFused) {
            // row r of a stage goes to warp r % 4, 8 elements a lane; the next stage's rows are loaded before this
            // one's are worked on
            constexpr int kMine = kMx4FusedTokens / 4;
            const XT *x = static_cast<const XT *>(p.x);
            Raw<XT, 8> raw[kMine];
            auto load = [&](int k) {
                const int64_t at = (int64_t)k * 256 + lane * 8;
#pragma unroll
                for (int u = 0; u < kMine; ++u) {
                    const int64_t r = qd + 4 * u;
                    raw[u].zero();
                    if (r < p.M && at < p.K) {
                        if (p.x_vec) raw[u].template load<true>(x + r * p.ldx + at);
                        else raw[u].template load<false>(x + r * p.ldx + at);
                    }
                }
            };
            load(k0);
            for (int i = 0; i < k1 - k0; ++i) {
                const int s = i % S;
                if (i >= S && !wait_warp(smem_u32(&empty[s]), (uint32_t)((i / S - 1) & 1), abort)) break;
                uint8_t *st = smem + s * L::kStageBytes;
#pragma unroll
                for (int u = 0; u < kMine; ++u) {
                    const int r = qd + 4 * u;
                    if (r >= p.M) break;
                    uint32_t top = raw[u].top_bits();
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = raw[u].value(j);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const uint32_t e = mx4_block_scale(top);
                    *reinterpret_cast<uint32_t *>(st + L::kA + sw128_off(r, lane >> 2) + (lane & 3) * 4) = mx4_codes8(v, e);
                    uint32_t word = e << (8 * ((lane >> 2) & 3));
                    word |= __shfl_xor_sync(0xffffffffu, word, 4);
                    word |= __shfl_xor_sync(0xffffffffu, word, 8);
                    if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(st + L::kAS + (lane >> 4) * kMx4ScaleBlock + 16 * r) = word;
                }
                if (i + 1 < k1 - k0) load(k0 + i + 1);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&full[s]));
            }
        }
        bool ok = wait_warp(smem_u32(done), 0u, abort) && !*abort;
        tc_fence_after();
        const uint32_t t_lane = tmem + ((uint32_t)(32 * qd) << 16);
        constexpr int kChunk = 16;
        const int sums = (k1 - k0 + kDrain - 1) / kDrain;
        // results of tokens c0 .. c0 + 15: the accumulators added up
        auto load_sums = [&](int c0, uint32_t (&v)[16]) {
            tmem_ld16(t_lane + c0, v);
            tmem_wait_ld(v);
            for (int r = 1; r < sums; ++r) {
                uint32_t u[16];
                tmem_ld16(t_lane + r * L::kSums + c0, u);
                tmem_wait_ld(u);
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) + __uint_as_float(u[c]));
            }
        };
        if (p.split == 1) {
#pragma unroll 1
            for (int c0 = 0; c0 < TN && ok; c0 += kChunk) {
                if (m0 + c0 >= p.M) break;
                uint32_t v[16];
                load_sums(c0, v);
                if (n < p.N) {
                    if (p.dtype == QMM_F32) store_tokens(static_cast<float *>(p.y), p.ldy, m0 + c0, p.M, n, v, kChunk);
                    else if (p.dtype == QMM_F16) store_tokens(static_cast<__half *>(p.y), p.ldy, m0 + c0, p.M, n, v, kChunk);
                    else store_tokens(static_cast<__nv_bfloat16 *>(p.y), p.ldy, m0 + c0, p.M, n, v, kChunk);
                }
            }
        } else {
            // token c goes to the CTA of rank c / share, into its slot [this rank][c % share][row]
            const int share = TN / p.split;
            float *parts = reinterpret_cast<float *>(smem + L::kPartsAt);
#pragma unroll 1
            for (int c0 = 0; c0 < TN && ok; c0 += kChunk) {
                uint32_t v[16];
                load_sums(c0, v);
#pragma unroll
                for (int c = 0; c < kChunk; ++c) {
                    if (m0 + c0 + c >= p.M) break;
                    const int to = (c0 + c) / share, at = (rank * share + (c0 + c) % share) * kRows + row;
                    if (!QMM_DCHECK(to < p.split && at < TN * kRows)) break;
                    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(peer_addr(smem_u32(parts + at), (uint32_t)to)), "r"(v[c])
                                 : "memory");
                }
            }
            for (int to = 0; to < p.split; ++to) mbar_arrive_peer(peer_addr(smem_u32(parts_in), (uint32_t)to));
            // nobody leaves before its peers have written here
            const bool in = wait_cluster_bounded(smem_u32(parts_in), 0u, abort, &g_mx4_status, kWaitLimitNs);
            if (!in) wait_drain(smem_u32(parts_in), 0u);
            ok = ok && in;
            for (int c = 0; c < share && ok; ++c) {
                const int64_t m = m0 + rank * share + c;
                if (m >= p.M || n >= p.N) break;
                float sum = 0.0f;
                for (int r = 0; r < p.split; ++r) sum += parts[(r * share + c) * kRows + row];
                if (p.dtype == QMM_F32) static_cast<float *>(p.y)[m * p.ldy + n] = sum;
                else if (p.dtype == QMM_F16) float_to_elem(sum, static_cast<__half *>(p.y)[m * p.ldy + n]);
                else float_to_elem(sum, static_cast<__nv_bfloat16 *>(p.y)[m * p.ldy + n]);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.cols) : "memory");
    }
}

template <int TN, typename XT = void>
cudaError_t launch_tn(Mx4Params p, const uint8_t *wc, int64_t K, const uint8_t *ac, cudaStream_t s) {
    using L = Plan<TN>;
    auto kern = mx4_gemm_kernel<TN, XT>;
    static int attr_done[4] = {0, 0, 0, 0};
    cudaError_t e = ensure_smem_limit(kern, L::kSmem, attr_done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.N + kRows - 1) / kRows;
    // K is shared while all CTAs are on the GPU at once, each with four stages at least (with two, one token through
    // 4096 x 4096 takes 6.3 us for 5.1)
    static_assert(L::kSmem <= 113 * 1024, "two CTAs do not fit on an SM");
    constexpr int64_t slots = 304;
    p.split = 1;
    while (p.split < kMaxSplit && 2 * p.split <= TN && 2 * tiles * p.split <= slots && p.nk >= 8 * p.split) p.split *= 2;
    p.sums = ((p.nk + p.split - 1) / p.split + kDrain - 1) / kDrain;
    p.cols = L::cols(p.sums);
    alignas(64) CUtensorMap wm, am;
    e = make_map_2d(&wm, CU_TENSOR_MAP_DATA_TYPE_UINT8, wc, (uint64_t)(K / 2), (uint64_t)p.N, (uint64_t)(K / 2), 128, kRows,
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    am = wm;                                                     // not read by a fused kernel
    if (ac)
        e = make_map_2d(&am, CU_TENSOR_MAP_DATA_TYPE_UINT8, ac, (uint64_t)(K / 2), (uint64_t)p.M, (uint64_t)(K / 2), 128, TN,
                        CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p, wm, am);
}

// ---------------------------------------------------------------------------------------------
// More than 32 tokens: pairs of CTAs (cta_group::2) share a tile of 256 weight rows x 256 tokens.  Each CTA holds
// 128 of the weight rows and 128 of the tokens, and the pair's instruction reads both halves of the
// tokens, so that a byte brought into shared memory takes part in twice the products of a single CTA's
// tile.  The pairs stay on their SMs and take tiles in turn.  The eight result warps of a CTA read a finished tile into registers, 128 sums a
// thread, which frees the accumulator for the next tile before the first result is stored.
// ---------------------------------------------------------------------------------------------
constexpr int kPairTok = 256;              // tokens of a pair's tile
struct Pair {
    static constexpr int kStages = 6;
    static constexpr int kW = 0;
    static constexpr int kA = kRows * 128;
    static constexpr int kWS = kA + kPairTok / 2 * 128;
    static constexpr int kAS = kWS + 2 * kMx4ScaleBlock;
    static constexpr int kStageBytes = kAS + 4 * kMx4ScaleBlock;         // both CTAs hold the scales of all tokens
    static constexpr int kSums = kPairTok;
    static constexpr int kHalfCols = 12;                                 // weight 4, tokens 8
    static constexpr int kBars = kStages * kStageBytes;
    static constexpr size_t kSmem = 1024 + kBars + (2 * kStages + 2) * 8 + 16;
    static constexpr int kThreads = 64 + 256;
    static_assert(kSums + kStages * 2 * kHalfCols <= 512 && kSmem <= 227 * 1024, "does not fit");
};

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_mxf4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa, uint32_t sb,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// An arrival on the barrier at this offset in both CTAs, once the products issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
        "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Eight columns, loaded by the time it returns.
__device__ __forceinline__ void tmem_ld8_wait(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}
// Completes the loads of r and keeps their uses behind it.
__device__ __forceinline__ void tmem_wait32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

struct PairParams {
    void *y;
    int64_t N, M, ldy;
    int n128, nk, last_steps;
    int m_tiles, n_tiles, tiles;
    // Tiles run through bands of 8 weight tiles, in a band through the tokens: the 76 tiles of a moment are some
    // 8 x 10, so that each byte of either operand is asked for by 8 or 10 pairs at about the same time.
    __device__ __forceinline__ void place(int tile, int &mt, int &nt) const {
        const int band = tile / (8 * m_tiles), in = tile - band * 8 * m_tiles, wide = min(8, n_tiles - 8 * band);
        mt = in / wide;
        nt = 8 * band + in - mt * wide;
    }
};

// LONG: more than kDrain stages.  The accumulator then starts anew after each kDrain, and the result warps add up.
template <typename T, bool LONG>
__global__ void __launch_bounds__(Pair::kThreads, 1)
mx4_pair_kernel(const PairParams p, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap a_map,
                const __grid_constant__ CUtensorMap ws_map, const __grid_constant__ CUtensorMap as_map) {
    using L = Pair;
    constexpr int S = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars), *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(acc_full), 1);
        mbar_init(smem_u32(acc_empty), 16);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");      // only now: as in the kernel for few tokens
            Ring<S> r;
            const uint32_t st0 = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
            const uint32_t lead0 = peer_addr(full0, 0u);                   // the leader's, for both CTAs' copies
            bool ok = true;
            int it = 0;
            for (int tile = pair; tile < p.tiles && ok; tile += pairs) {
                int mt, nt;
                p.place(tile, mt, nt);
                const int row0 = nt * 2 * kRows + rank * kRows, tok0 = mt * kPairTok + rank * (kPairTok / 2);
                const int wb = (nt * 2 + rank) * p.n128, ab = mt * 2 * p.n128;
                for (int k = 0; k < p.nk; ++k, ++it, r.next()) {
                    if (!wait_bounded(empty0 + 8 * r.s, r.phase ^ 1u, abort)) { ok = false; break; }
                    const uint32_t st = st0 + (uint32_t)(r.s * L::kStageBytes), bar = lead0 + 8 * r.s;
                    if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * r.s, 2 * L::kStageBytes);
                    tma_load_2d_pair(st + L::kW, &w_map, k * 128, row0, bar);
                    tma_load_2d_pair(st + L::kA, &a_map, k * 128, tok0, bar);
                    tma_load_2d_pair(st + L::kWS, &ws_map, 0, wb + 2 * k, bar);
                    tma_load_2d_pair(st + L::kAS, &as_map, 0, ab + 2 * k, bar);
                    tma_load_2d_pair(st + L::kAS + 2 * kMx4ScaleBlock, &as_map, 0, ab + p.n128 + 2 * k, bar);
                }
            }
            // every stage has been read, and the arrivals that say so have reached this CTA
            for (int i = it > S ? it - S : 0; i < it; ++i) wait_drain(smem_u32(&empty[i % S]), (uint32_t)((i / S) & 1));
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // the warp walks the stages together, so that addresses stay in uniform registers; one thread issues
            const bool lead = elect_one();
            const uint32_t st0 = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
            const uint64_t w_desc = smem_desc_sw128(st0 + L::kW), a_desc = smem_desc_sw128(st0 + L::kA);
            const uint64_t ws_desc = smem_desc_scales(st0 + L::kWS), as_desc = smem_desc_scales(st0 + L::kAS);
            constexpr uint32_t id0 = idesc_mxf4(kPairTok, 0) + ((uint32_t)(kRows >> 4) << 24);      // 256 rows
            constexpr uint32_t id1 = idesc_mxf4(kPairTok, 1) + ((uint32_t)(kRows >> 4) << 24);
            constexpr int kHalf = kMx4ScaleBlock >> 4;             // in units of a descriptor's address
            asm volatile("griddepcontrol.wait;" ::: "memory");     // before the first bounded wait
            bool ok = true;
            uint32_t acc_phase = 1;
            Ring<S> r;
            for (int tile = pair; tile < p.tiles && ok; tile += pairs) {
                for (int k = 0; k < p.nk; ++k, r.next()) {
                    if (!wait_warp(full0 + 8 * r.s, r.phase, abort)) { ok = false; break; }
                    const int in_sum = LONG ? k % kDrain : k;
                    if (in_sum == 0) {
                        if (!__all_sync(0xffffffffu, wait_cluster_bounded(smem_u32(acc_empty), acc_phase, abort, &g_mx4_status, kWaitLimitNs))) {
                            ok = false;
                            break;
                        }
                        acc_phase ^= 1u;
                    }
                    tc_fence_after();
                    const uint64_t off = (uint64_t)(uint32_t)(r.s * (L::kStageBytes >> 4));
                    const uint32_t cols = tmem + (uint32_t)(L::kSums + r.s * 2 * L::kHalfCols);
                    const int steps = k == p.nk - 1 ? p.last_steps : 4;
                    if (lead) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            copy_scales_pair(cols + h * L::kHalfCols, ws_desc + off + h * kHalf);
                            copy_scales_pair(cols + h * L::kHalfCols + 4, as_desc + off + h * kHalf);
                            copy_scales_pair(cols + h * L::kHalfCols + 8, as_desc + off + (2 + h) * kHalf);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t c = cols + (uint32_t)((q >> 1) * L::kHalfCols);
                            if (q < steps)
                                mma_mxf4_pair(tmem, w_desc + off + 2 * q, a_desc + off + 2 * q, (q & 1) ? id1 : id0, c, c + 4,
                                              q > 0 ? 1u : (in_sum > 0 ? 1u : 0u));
                        }
                        mma_commit_pair(empty0 + 8 * r.s);
                        if (k == p.nk - 1 || (LONG && in_sum == kDrain - 1)) mma_commit_pair(smem_u32(acc_full));
                    }
                    __syncwarp();
                }
            }
            if (!ok && lead) {
                // lets the products in flight finish and both CTAs go on to their end
                mma_commit_pair(smem_u32(acc_full));
                for (int s = 0; s < S; ++s) mma_commit_pair(smem_u32(&empty[s]));
            }
        }
        __syncwarp();
    } else {
        const int qd = warp & 3, half = (warp - 2) >> 2, row = 32 * qd + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)(half * (kPairTok / 2));
        const uint32_t free_bar = peer_addr(smem_u32(acc_empty), 0u);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        int done = 0;
        for (int tile = pair; tile < p.tiles; tile += pairs, ++done) {
            if (!wait_warp(smem_u32(acc_full), (uint32_t)(done & 1), abort)) break;
            tc_fence_after();
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(t_lane + 32 * c, v + 32 * c);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_wait32(v + 32 * c);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_peer(free_bar);
            if constexpr (LONG) {
                bool ok = true;
                for (int k = kDrain; k < p.nk; k += kDrain) {
                    ++done;
                    ok = wait_warp(smem_u32(acc_full), (uint32_t)(done & 1), abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        uint32_t u[8];
                        tmem_ld8_wait(t_lane + 8 * c, u);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[8 * c + i] = __float_as_uint(__uint_as_float(v[8 * c + i]) + __uint_as_float(u[i]));
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_peer(free_bar);
                }
                if (!ok) break;
            }
            int mt, nt;
            p.place(tile, mt, nt);
            const int64_t n = (int64_t)nt * 2 * kRows + rank * kRows + row, m0 = (int64_t)mt * kPairTok + half * (kPairTok / 2);
            const int have = (int)min((int64_t)(kPairTok / 2), p.M - m0);
            if (n < p.N && QMM_DCHECK(mt >= 0 && mt < p.m_tiles && nt >= 0 && nt < p.n_tiles && n < p.ldy)) {
                T *y = static_cast<T *>(p.y) + m0 * p.ldy + n;
#pragma unroll
                for (int c = 0; c < kPairTok / 2; ++c) {
                    if (c < have) float_to_elem(__uint_as_float(v[c]), *y);
                    y += p.ldy;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

cudaError_t launch_pairs(const Mx4Params &q, const uint8_t *wc, int64_t K, const uint8_t *ac, cudaStream_t s) {
    PairParams p = {q.y, q.N, q.M, q.ldy, q.n128, q.nk, q.last_steps, 0, 0, 0};
    const int64_t mt = (p.M + kPairTok - 1) / kPairTok, nt = (p.N + 2 * kRows - 1) / (2 * kRows);
    if (mt * nt > 0x3fffffff) return cudaErrorInvalidValue;
    p.m_tiles = (int)mt;
    p.n_tiles = (int)nt;
    p.tiles = (int)(mt * nt);
    alignas(64) CUtensorMap wm, am, wsm, asm_;
    cudaError_t e = make_map_2d(&wm, CU_TENSOR_MAP_DATA_TYPE_UINT8, wc, (uint64_t)(K / 2), (uint64_t)p.N, (uint64_t)(K / 2), 128, kRows,
                                CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = make_map_2d(&am, CU_TENSOR_MAP_DATA_TYPE_UINT8, ac, (uint64_t)(K / 2), (uint64_t)p.M, (uint64_t)(K / 2), 128, kPairTok / 2,
                        CU_TENSOR_MAP_SWIZZLE_128B);
    // the scales as rows of 512 bytes, two a copy
    if (e == cudaSuccess)
        e = make_map_2d(&wsm, CU_TENSOR_MAP_DATA_TYPE_UINT32, q.ws, 128, (uint64_t)((p.N + 127) / 128) * (uint64_t)p.n128, 512, 128, 2,
                        CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e == cudaSuccess)
        e = make_map_2d(&asm_, CU_TENSOR_MAP_DATA_TYPE_UINT32, q.as, 128, (uint64_t)((p.M + 127) / 128) * (uint64_t)p.n128, 512, 128, 2,
                        CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kern, int (&attr_done)[4]) {
        cudaError_t err = ensure_smem_limit(kern, Pair::kSmem, attr_done);
        if (err != cudaSuccess) return err;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(2 * (p.tiles < 76 ? p.tiles : 76)), 1, 1);
        cfg.blockDim = dim3(Pair::kThreads, 1, 1);
        cfg.dynamicSmemBytes = Pair::kSmem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kern, p, wm, am, wsm, asm_);
    };
    static int done[6][4] = {};
    const bool lng = p.nk > kDrain;
    if (q.dtype == QMM_F32) return lng ? go(mx4_pair_kernel<float, true>, done[0]) : go(mx4_pair_kernel<float, false>, done[1]);
    if (q.dtype == QMM_F16) return lng ? go(mx4_pair_kernel<__half, true>, done[2]) : go(mx4_pair_kernel<__half, false>, done[3]);
    return lng ? go(mx4_pair_kernel<__nv_bfloat16, true>, done[4]) : go(mx4_pair_kernel<__nv_bfloat16, false>, done[5]);
}

}  // namespace

static Mx4Params make_params(const uint8_t *ws, int64_t K, int64_t N, int64_t M, qmm_dtype t, void *y, int64_t ldy) {
    Mx4Params p = {};
    p.ws = ws;
    p.y = y;
    p.N = N;
    p.M = M;
    p.ldy = ldy;
    p.K = K;
    p.n128 = (int)((K + 127) / 128);
    p.nk = (int)((K + 255) / 256);
    p.last_steps = (int)((K - (int64_t)(p.nk - 1) * 256 + 63) / 64);
    p.dtype = (int)t;
    return p;
}

cudaError_t launch_mx4_matmul(const uint8_t *wc, const uint8_t *ws, int64_t K, int64_t N, const uint8_t *ac, const uint8_t *as,
                              int64_t M, qmm_dtype t, void *y, int64_t ldy, int early_weights, cudaStream_t s) {
    Mx4Params p = make_params(ws, K, N, M, t, y, ldy);
    p.as = as;
    p.early_weights = early_weights;
    if (M <= 16) return launch_tn<16>(p, wc, K, ac, s);
    if (M <= 32) return launch_tn<32>(p, wc, K, ac, s);
    return launch_pairs(p, wc, K, ac, s);
}

cudaError_t launch_mx4_linear_few(const uint8_t *wc, const uint8_t *ws, int64_t K, int64_t N, qmm_dtype xt, const void *x, int64_t ldx,
                                  int64_t M, qmm_dtype t, void *y, int64_t ldy, cudaStream_t s) {
    Mx4Params p = make_params(ws, K, N, M, t, y, ldy);
    p.early_weights = 1;
    p.x = x;
    p.ldx = ldx;
    p.x_vec = rows_aligned(x, ldx, dtype_bytes(xt));
    return with_dtype(xt, [&](auto z) { return launch_tn<16, decltype(z)>(p, wc, K, nullptr, s); });
}

cudaError_t read_and_clear_mx4_status(unsigned *out, cudaStream_t s) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_mx4_status, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbolAsync(g_mx4_status, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, s);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(s);
}

QMM_DCHECK_READER(read_dcheck_mx4_gemm)

}  // namespace qmm
