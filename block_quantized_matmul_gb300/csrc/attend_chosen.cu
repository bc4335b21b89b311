// attend_chosen.cu -- attention of each new token over the pages of the block-quantized cache that were chosen for it
// (cache_select.cu), the products as in attend_mma.cuh.
//
// The tokens of a list of pages are taken as one sequence of keys, page after page; which of them the row sees follows from
// their places in the sequence, 16 at a time, and is the same for all query heads of the key/value head.  So a CTA takes one
// token and key/value head (up to 32 query heads of it), and where tokens and heads are fewer than the GPU has
// places for CTAs, a chunk of the list; a second kernel joins the chunks.
//
// What bounds it.  Decode steps: memory (31 tokens x 8 heads over up to 64 pages of 64 tokens, Q8_0: 53 us for 263 MB, 5.0 TB/s).  One
// token: latency (9 us with the join).  Pieces of prompts: the expansion of codes and the products, each token for itself, from L2
// (128 tokens x 8 heads over 32 pages of 64, Q4_0: 104 us, 60 % of the issue slots).
#include "attend_mma.cuh"

namespace qmm {
namespace {

// Entries of a list before its first negative one, by a warp.
__device__ __forceinline__ int list_length(const int32_t *list, int most) {
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < most; base += 128) {
        int v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = base + 32 * u + lane < most ? __ldcg(list + base + 32 * u + lane) : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const unsigned end = __ballot_sync(0xffffffffu, v[u] < 0);
            if (end) return min(most, base + 32 * u + __ffs(end) - 1);
        }
    }
    return most;
}

__device__ __forceinline__ int chunks_of(int64_t keys, uint32_t chunk) { return (int)max((int64_t)1, (keys + chunk - 1) / chunk); }

template <int ROWS>
__device__ __forceinline__ bool find_chosen(const AttendParams &p, Rows &w) {
    uint32_t at = blockIdx.x;
    const int rt = (int)(at % (uint32_t)p.row_tiles);
    at /= (uint32_t)p.row_tiles;
    w.h = (int)(at % (uint32_t)p.H);
    at /= (uint32_t)p.H;
    const int64_t row = at % (uint32_t)p.T;
    w.sp = (int)(at / (uint32_t)p.T);
    w.list = p.chosen + (row * p.H + w.h) * p.list_len;
    w.n = (int64_t)list_length(w.list, p.list_len) << p.log_p;
    w.used = chunks_of(w.n, p.chunk);
    if (w.sp >= w.used) return false;
    w.s = last_start(p.q_starts, p.n_seq, row);
    if (w.s < 0 || w.s >= p.n_seq) return false;                       // behind the last sequence
    const int64_t q0 = p.q_starts[w.s], q1 = p.q_starts[w.s + 1];
    const int len = p.kv_lens[w.s];
    if (q0 < 0 || q1 > p.T) return false;                              // not rows of q
    w.q0 = row;
    w.nq = 1;
    w.first = len - (q1 - q0);
    w.tree = p.tree != nullptr;
    w.word = w.tree ? p.tree[row] : 0;
    w.upto = w.tree ? cached(p, len) : min(w.first + (row - q0) + 1, cached(p, len));
    w.r0 = rt * ROWS;
    w.rows = min(ROWS, p.group - w.r0);
    w.k0 = (int64_t)w.sp * p.chunk;
    w.k1 = min(w.n, w.k0 + p.chunk);
    return true;
}

template <int TYPE, int DB, int NT, bool TWO>
__global__ void __launch_bounds__(Tile<TYPE, DB, NT>::kThreads, 2) attend_chosen_kernel(const __grid_constant__ AttendParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Rows w;
    if (!find_chosen<Tile<TYPE, DB, NT>::kRowsTile>(p, w)) return;
    attend_rows<TYPE, DB, NT, TWO, true>(p, w, smem);
}

// Joins the chunks' results.
template <int DB, int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_chosen_join_kernel(const AttendParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int Hq = p.H * p.group;
    const int64_t at = (int64_t)blockIdx.x * (kJoinWarps / WPR) + (threadIdx.x >> 5) / WPR;
    if (at >= p.T * Hq) return;                                        // (a row's warps together)
    const int64_t tok = (uint32_t)at / (uint32_t)Hq;
    const int hq = (int)(at - tok * Hq);
    const int64_t s = last_start(p.q_starts, p.n_seq, tok);
    if (s < 0 || s >= p.n_seq || p.q_starts[s] < 0 || p.q_starts[s + 1] > p.T) return;
    const int64_t n = (int64_t)list_length(p.chosen + (tok * p.H + hq / p.group) * p.list_len, p.list_len) << p.log_p;
    const int used = chunks_of(n, p.chunk);
    if (used <= 1 || !QMM_DCHECK(used <= p.splits)) return;
    join_row<DB, WPR>(p, at, tok, hq, used);
}

// Query rows of a CTA: as for the whole cache, but never more than one token's.
int chosen_rows_of(int group, int D) { return group <= kMmaRows ? kMmaRows : (group <= 2 * kMmaRows || D > 128 ? 2 * kMmaRows : 4 * kMmaRows); }

// Keys of a chunk, so that all chunks fill the GPU's 304 places for CTAs (two an SM) once; at least 128, four tiles of 32
// keys.
struct Chunks {
    int64_t units, chunk, splits;           // CTAs with whole lists; keys of a chunk; chunks of a list at most
};
Chunks chunks_for(int64_t T, int H, int group, int D, int P, int64_t budget) {
    const int rows = chosen_rows_of(group, D);
    Chunks c = {T * H * ((group + rows - 1) / rows), budget * P, 1};
    if (c.units >= 304) return c;
    const int64_t want = 304 / c.units, least = (budget * P + want - 1) / want;
    c.chunk = (least + 127) / 128 * 128;
    c.splits = (budget * P + c.chunk - 1) / c.chunk;
    return c;
}

template <int TYPE, int DB, int NT, bool TWO = true>
cudaError_t launch_chosen(const AttendParams &p, int64_t ctas, cudaStream_t s) {
    using L = Tile<TYPE, DB, NT>;
    auto kern = attend_chosen_kernel<TYPE, DB, NT, TWO>;
    static int attr_done[4] = {0, 0, 0, 0};
    const cudaError_t e = ensure_smem_limit(kern, L::kSmem, attr_done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)ctas), L::kThreads, L::kSmem, s, p);
}

template <int TYPE, int DB>
cudaError_t launch_chosen_rows(const AttendParams &p, int64_t ctas, cudaStream_t s) {
    if (p.tile_rows == kMmaRows) return launch_chosen<TYPE, DB, 1>(p, ctas, s);
    if constexpr (DB <= 4) {
        if (p.tile_rows == 4 * kMmaRows) return p.bf16 ? launch_chosen<TYPE, DB, 4, false>(p, ctas, s) : launch_chosen<TYPE, DB, 4>(p, ctas, s);
    }
    return launch_chosen<TYPE, DB, 2>(p, ctas, s);
}

template <int DB>
cudaError_t launch_chosen_blocks(qmm_type type, const AttendParams &p, int64_t ctas, cudaStream_t s) {
    const cudaError_t e = type == QMM_Q8_0 ? launch_chosen_rows<QMM_Q8_0, DB>(p, ctas, s) : launch_chosen_rows<QMM_Q4_0, DB>(p, ctas, s);
    if (e != cudaSuccess || p.splits == 1) return e;
    const int64_t rows = p.T * p.H * p.group;
    if (p.splits > kJoinWarps) return launch_pdl(attend_chosen_join_kernel<DB, kJoinWarps>, dim3((unsigned)rows), kJoinWarps * 32, 0, s, p);
    return launch_pdl(attend_chosen_join_kernel<DB, 1>, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), kJoinWarps * 32, 0, s, p);
}

}  // namespace

size_t attend_chosen_workspace_bytes(int64_t T, int H, int Hq, int D, int P, int64_t budget) {
    const Chunks c = chunks_for(T, H, Hq / H, D, P, budget);
    return c.splits == 1 ? 0 : (size_t)c.splits * split_bytes(T * Hq, D);
}

cudaError_t launch_cache_attend_chosen(qmm_type type, const uint8_t *k_cache, const uint8_t *v_cache, int64_t n_pages, int P, int H, int D,
                                       const int32_t *pages, int64_t ld_pages, const int32_t *q_starts, const int32_t *kv_lens,
                                       int64_t n_seq, qmm_dtype t, const void *q, int64_t ldq, int64_t T, int Hq, const uint64_t *tree,
                                       float scale, const int32_t *chosen, int64_t budget, void *out, int64_t ldo, float *lse, void *ws,
                                       size_t ws_bytes, cudaStream_t s) {
    AttendParams p = {};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.n_pages = n_pages;
    p.P = P;
    while ((1 << p.log_p) < P) ++p.log_p;
    p.H = H;
    p.group = Hq / H;
    p.tile_rows = chosen_rows_of(p.group, D);
    p.row_tiles = (p.group + p.tile_rows - 1) / p.tile_rows;
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
    p.chosen = chosen;
    p.list_len = (int)budget;
    const size_t per_split = split_bytes(T * Hq, D);
    Chunks c = chunks_for(T, H, p.group, D, P, budget);
    if (c.splits > 1 && (size_t)c.splits * per_split > ws_bytes) {
        // fewer and longer chunks, or none
        const int64_t fit = (int64_t)(ws_bytes / per_split);
        c.chunk = fit < 2 ? budget * P : ((budget * P + fit - 1) / fit + 127) / 128 * 128;
        c.splits = (budget * P + c.chunk - 1) / c.chunk;
    }
    p.splits = (int)c.splits;
    p.chunk = (uint32_t)c.chunk;
    if (p.splits > 1) {
        p.part_o = static_cast<float *>(ws);
        p.part_ml = p.part_o + (size_t)p.splits * (size_t)T * (size_t)Hq * (size_t)D;
    }
    const int64_t ctas = c.units * c.splits;
    if (ctas > 0x7fffffff || (p.splits > 1 && T * Hq > 0x7fffffff)) return cudaErrorInvalidValue;
    switch (D / 32) {
        case 1: return launch_chosen_blocks<1>(type, p, ctas, s);
        case 2: return launch_chosen_blocks<2>(type, p, ctas, s);
        case 3: return launch_chosen_blocks<3>(type, p, ctas, s);
        case 4: return launch_chosen_blocks<4>(type, p, ctas, s);
        case 5: return launch_chosen_blocks<5>(type, p, ctas, s);
        case 6: return launch_chosen_blocks<6>(type, p, ctas, s);
        case 7: return launch_chosen_blocks<7>(type, p, ctas, s);
        default: return launch_chosen_blocks<8>(type, p, ctas, s);
    }
}

QMM_DCHECK_READER(read_dcheck_attend_chosen)

}  // namespace qmm
