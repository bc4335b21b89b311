// cache_plan.cu -- the plan of a step over the paged cache: from each request's cached length and new tokens the
// pages it is given, the first row of each sequence, and the slot of every row.
//
// For sequence s with n cached tokens, m new ones and held(n) = ceil(n / P):
//   need = held(n + m) - held(n),   line = sum of need up to and including s (of those that fit their rows of the table),
//   it is run when it fits, and need = 0 or line <= free.
// Sums of need never fall, so once one waits for want of pages all later ones that need a page wait too: the pages of
// those that run are the ring's entries first + line - need ...
//
// Every CTA runs the same scan over the sequences (a tile of as many as it has threads at a time) and takes its share of the
// rows, the new pages and the pages given back that fall into it, so that no sum has to travel between CTAs.  A few
// CTAs do for a decode step; with 152 the rows of many prompts (412000 rows of 2048 sequences) take 12.7 us, with a cluster
// of eight they took 29; 64 sequences of a decode step take 3.5 us in a captured graph.  Where the new lengths or counters replace the old ones, which other CTAs may still read, a
// second kernel writes them.  What bounds it is latency: the loads of the lengths, three scans in one, a row's
// search for its sequence (8 or 10 steps in shared memory), and a load of the page.
#include <climits>

#include "qmm_internal.cuh"

namespace qmm {
namespace {

struct PlanParams {
    const int32_t *lens, *news;
    int64_t n_seq, ld_pages, n_ring, T;
    int log_p;
    int32_t *pages, *ring;
    const int64_t *ring_at;
    int32_t *q_starts, *kv_lens;
    int64_t *slots;
    int32_t *positions, *next_lens;
    int64_t *next_at;
    int later;                              // next_lens and next_at are cache_plan_next_kernel's
};

struct Sums {
    int64_t rows, need, back;               // new tokens, pages wanted, pages given back
};
__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) { return {a.rows + b.rows, a.need + b.need, a.back + b.back}; }

// Inclusive sums over the first `width` lanes of a warp.
__device__ __forceinline__ Sums warp_sums(Sums x, int width) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        if (m >= width) break;
        const Sums y = {__shfl_up_sync(0xffffffffu, x.rows, m), __shfl_up_sync(0xffffffffu, x.need, m), __shfl_up_sync(0xffffffffu, x.back, m)};
        if (lane >= m) x = x + y;
    }
    return x;
}

// Place number `at` of a ring of n, for at >= 0.
__device__ __forceinline__ int64_t around(int64_t at, int64_t n) { return at < n ? at : at % n; }

constexpr int kWaits = -1;                  // in place of the pages that a sequence holds (and for one that is done)

template <int THREADS>
__global__ void __launch_bounds__(THREADS) cache_plan_kernel(const PlanParams p) {
    constexpr int kWarps = THREADS / 32;
    __shared__ Sums part[kWarps];
    __shared__ int64_t s_start[THREADS], s_base[THREADS];             // first row; first new page in the ring
    __shared__ int s_len[THREADS], s_held[THREADS];
    __shared__ int64_t s_back[THREADS];                               // pages given back by the sequences before
    __shared__ unsigned long long s_taken;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ctas = (int)gridDim.x, cta = (int)blockIdx.x;
    if (threadIdx.x == 0) s_taken = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int P = 1 << p.log_p;
    const int64_t first = p.ring_at[0], last = p.ring_at[1], free = last - first, room = min(p.ld_pages << p.log_p, (int64_t)INT_MAX);
    const int64_t front = ((first % p.n_ring) + p.n_ring) % p.n_ring, behind = ((last % p.n_ring) + p.n_ring) % p.n_ring;
    Sums done = {0, 0, 0};
    for (int64_t base = 0; base < p.n_seq; base += THREADS) {
        const int64_t s = base + threadIdx.x;
        const bool have = s < p.n_seq;
        const int64_t len = have ? max((int64_t)0, min((int64_t)p.lens[s], room)) : 0, news = have ? p.news[s] : 0;
        const int64_t held = (len + P - 1) >> p.log_p, rows = max(news, (int64_t)0);
        bool run = news >= 0 && len + rows <= room;
        const Sums v = {rows, run ? ((len + rows + P - 1) >> p.log_p) - held : 0, news < 0 ? held : 0};
        // ---- sums of all before: over the warp, over the warps, over the tiles ----
        Sums x = warp_sums(v, 32);
        if (lane == 31) part[warp] = x;
        __syncthreads();
        if (warp == 0) {
            const Sums w = warp_sums(lane < kWarps ? part[lane] : Sums{0, 0, 0}, kWarps);
            if (lane < kWarps) part[lane] = w;
        }
        __syncthreads();
        const Sums all = part[kWarps - 1], before = warp ? part[warp - 1] : Sums{0, 0, 0};
        x = {done.rows + before.rows + x.rows - v.rows, done.need + before.need + x.need - v.need, done.back + before.back + x.back - v.back};
        run = run && x.rows + rows <= p.T && (v.need == 0 || x.need + v.need <= free);
        const unsigned takes = __ballot_sync(0xffffffffu, run && v.need > 0);
        if (takes && lane == 31 - __clz(takes)) atomicMax(&s_taken, (unsigned long long)(x.need + v.need));
        s_start[threadIdx.x] = x.rows;
        s_back[threadIdx.x] = x.back;
        s_len[threadIdx.x] = (int)len;
        s_held[threadIdx.x] = run ? (int)held : kWaits;
        s_base[threadIdx.x] = around(front + x.need, p.n_ring);
        __syncthreads();
        if (have && cta == (int)((base / THREADS) % ctas)) {
            p.q_starts[s] = (int32_t)min(x.rows, (int64_t)INT_MAX);
            p.kv_lens[s] = run ? (int32_t)(len + rows) : 0;
            if (p.next_lens && !p.later) p.next_lens[s] = news < 0 ? 0 : (int32_t)(run ? len + rows : len);
        }
        // the last sequence of the tile for which `first` is not above `at`
        auto find = [](const int64_t *first, int64_t at) {
            int lo = 0, hi = THREADS;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= at) lo = mid;
                else hi = mid;
            }
            return lo;
        };
        // ---- pages that go back, four of them under way at a time ----
        for (int64_t at = done.back + (int64_t)cta * THREADS + threadIdx.x; at < done.back + all.back; at += (int64_t)ctas * THREADS * 4) {
            int32_t page[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t i = at + (int64_t)u * ctas * THREADS;
                page[u] = 0;
                if (i >= done.back + all.back) continue;
                const int lo = find(s_back, i);
                const int64_t k = i - s_back[lo];
                if (QMM_DCHECK(k < p.ld_pages && base + lo < p.n_seq)) page[u] = p.pages[(base + lo) * p.ld_pages + k];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t i = at + (int64_t)u * ctas * THREADS, to = around(behind + i, p.n_ring);
                if (i < done.back + all.back && QMM_DCHECK(to >= 0 && to < p.n_ring)) p.ring[to] = page[u];
            }
        }
        // ---- the rows that fall into this tile ----
        const int64_t r1 = min(done.rows + all.rows, p.T);
        for (int64_t r = done.rows + (int64_t)cta * THREADS + threadIdx.x; r < r1; r += (int64_t)ctas * THREADS) {
            const int lo = find(s_start, r);
            int64_t slot = -1;
            int pos = -1;
            if (s_held[lo] >= 0) {
                pos = s_len[lo] + (int)(r - s_start[lo]);
                const int number = pos >> p.log_p, k = number - s_held[lo], place = pos & (P - 1);
                int64_t page = -1;
                if (QMM_DCHECK(number < p.ld_pages && base + lo < p.n_seq)) {
                    int32_t *entry = p.pages + (base + lo) * p.ld_pages + number;
                    if (k >= 0) {
                        page = p.ring[around(s_base[lo] + k, p.n_ring)];
                        if (place == 0) *entry = (int32_t)page;
                    } else {
                        page = *entry;
                    }
                }
                slot = page * P + place;
            }
            p.slots[r] = slot;
            if (p.positions) p.positions[r] = pos;
        }
        done = done + all;
        __syncthreads();                                              // the tile's arrays are free again
    }
    for (int64_t r = done.rows + (int64_t)cta * THREADS + threadIdx.x; r < p.T; r += (int64_t)ctas * THREADS) {
        p.slots[r] = -1;
        if (p.positions) p.positions[r] = -1;
    }
    if (cta == 0 && threadIdx.x == 0) {
        p.q_starts[p.n_seq] = (int32_t)min(done.rows, (int64_t)INT_MAX);
        if (p.next_at && !p.later) {
            p.next_at[0] = first + (int64_t)s_taken;
            p.next_at[1] = last + done.back;
        }
    }
}

// The lengths and the ring's counters after the step, from those before it and from kv_lens, by one CTA.
__global__ void __launch_bounds__(1024) cache_plan_next_kernel(const PlanParams p) {
    __shared__ unsigned long long s_taken, s_back;
    if (threadIdx.x == 0) s_taken = s_back = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int P = 1 << p.log_p;
    const int64_t room = min(p.ld_pages << p.log_p, (int64_t)INT_MAX);
    unsigned long long taken = 0, back = 0;
    for (int64_t s = threadIdx.x; s < p.n_seq; s += 1024) {
        const int64_t len = max((int64_t)0, min((int64_t)p.lens[s], room)), held = (len + P - 1) >> p.log_p, after = p.kv_lens[s];
        const int news = p.news[s];
        const bool runs = news > 0 && after > 0;
        if (runs) taken += ((after + P - 1) >> p.log_p) - held;
        if (news < 0) back += held;
        if (p.next_lens) p.next_lens[s] = news < 0 ? 0 : (int32_t)(runs ? after : len);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        taken += __shfl_xor_sync(0xffffffffu, taken, m);
        back += __shfl_xor_sync(0xffffffffu, back, m);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        atomicAdd(&s_taken, taken);
        atomicAdd(&s_back, back);
    }
    __syncthreads();
    if (threadIdx.x == 0 && p.next_at && QMM_DCHECK(p.n_ring > 0)) {
        const int64_t first = p.ring_at[0], last = p.ring_at[1];
        p.next_at[0] = first + (int64_t)s_taken;
        p.next_at[1] = last + (int64_t)s_back;
    }
}

}  // namespace

cudaError_t launch_cache_plan(const int32_t *lens, const int32_t *news, int64_t n_seq, int P, int32_t *pages, int64_t ld_pages,
                              int32_t *ring, int64_t n_ring, const int64_t *ring_at, int64_t T, int32_t *q_starts, int32_t *kv_lens,
                              int64_t *slots, int32_t *positions, int32_t *next_lens, int64_t *next_at, cudaStream_t s) {
    PlanParams p = {lens, news, n_seq, ld_pages, n_ring, T, 0, pages, ring, ring_at, q_starts, kv_lens, slots, positions, next_lens, next_at, 0};
    while ((1 << p.log_p) < P) ++p.log_p;
    if (n_seq <= 256 && T <= 1024) return launch_pdl(cache_plan_kernel<256>, dim3(1), 256, 0, s, p);
    // two rows a thread; a sequence that is done may give back many pages
    const int64_t want = (T + 16 * n_seq + 2047) / 2048;
    const unsigned ctas = (unsigned)(want < 152 ? want : 152);
    p.later = ctas > 1 && (next_lens == lens || next_at == ring_at);
    const cudaError_t e = launch_pdl(cache_plan_kernel<1024>, dim3(ctas), 1024, 0, s, p);
    return e != cudaSuccess || !p.later ? e : launch_pdl(cache_plan_next_kernel, dim3(1), 1024, 0, s, p);
}

QMM_DCHECK_READER(read_dcheck_cache_plan)

}  // namespace qmm
