// attend.cu -- attention of a few new tokens of each sequence over the block-quantized cache (cache.cuh).
//
// For new token i of a sequence with n cached tokens, nq of them new, and query head hq (key/value head
// h = hq / G, G = Hq / H):
//   s_j = scale * sum_d q[i, hq, d] * k[j, h, d]  over the visible j,
//   out[i, hq] = sum_j exp(s_j - max s) v[j, h] / sum_j exp(s_j - max s),   lse = max s + ln(sum);
// j is visible when j < n - nq, or when bit j - (n - nq) of the token's tree word is set (without tree
// words: when j - (n - nq) <= i).  A row that sees nothing is 0 with lse -inf.
//
// How the products are taken and what bounds them: attend_mma.cuh (up to 32 rows a CTA), attend_tc.cu (128 rows).
#include "attend_mma.cuh"

namespace qmm {
namespace {

template <int TYPE, int DB, int NT, bool TWO>
__global__ void __launch_bounds__(Tile<TYPE, DB, NT>::kThreads, 2) attend_kernel(const __grid_constant__ AttendParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Rows w;
    if (!find_rows<Tile<TYPE, DB, NT>::kRowsTile>(p, reinterpret_cast<int *>(smem), Tile<TYPE, DB, NT>::kThreads, w)) return;
    attend_rows<TYPE, DB, NT, TWO, false>(p, w, smem);
}

// Joins the partial results of the sequences that were split.
template <int DB, int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Hq = p.H * p.group;
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
    join_row<DB, WPR>(p, at, tok, hq, used);
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
