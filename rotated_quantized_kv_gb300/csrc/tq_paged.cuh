// tq_paged.cuh -- the stage list of paged attention and the walk along it, shared by
// its kernels (tq_serve.h describes the list and its records).
//
// Lengths are on the device, so that the kernels lay out the list themselves: every
// CTA scans the sequences' stage counts once, which gives the total and its own first
// stage, and the first CTA leaves the scan for the merge.
#pragma once

#include "tq_serve.h"

namespace tqk {
namespace paged {

__device__ __forceinline__ int seg_tokens(const PagedList &l, int seg, int b) {
    return l.len[seg] ? min(max(l.len[seg][b], 0), l.limit[seg]) : l.limit[seg];
}
// Stages of the class's i-th segment.
__device__ __forceinline__ int seg_stages(const PagedList &l, const PagedClass &c, int i, int b) {
    const int n = seg_tokens(l, c.seg[i], b);
    return n / c.unit + (n % c.unit ? 1 : 0);
}
// Stages of (b, h, any rb).
__device__ __forceinline__ int head_stages(const PagedList &l, const PagedClass &c, int b, int h) {
    int n = 0;
    for (int i = 0; i < c.n; i++)
        if ((c.heads[i] >> h) & 1) n += seg_stages(l, c, i, b);
    return n;
}
// Stages of sequence b (below 2^31 over all sequences: the host checks it for the limits).
__device__ __forceinline__ int sequence_stages(const PagedList &l, const PagedClass &c, int b) {
    int n = 0;
    for (int i = 0; i < c.n; i++) n += __popc(c.heads[i]) * seg_stages(l, c, i, b);
    return n * l.n_rb;
}

// Workers that have a stage: those of a launch are sized for the segments' limits.
__device__ __forceinline__ int workers_of(const PagedClass &c, int total) { return max(min(c.workers, total), 1); }

__device__ __forceinline__ int worker_begin(int total, int w, int workers) {
    return static_cast<int>(static_cast<long long>(total) * w / workers);
}
// The worker whose range holds stage s.
__device__ __forceinline__ int worker_of(int total, int s, int workers) {
    return static_cast<int>(((s + 1LL) * workers - 1) / max(total, 1));
}

// Place in the list (the same in every thread that walks).  Every step ends and every place lies
// inside the call's segments even if the lengths change under the walk (nothing else may be
// expected of such a call): a place that is not found is a stage without tokens.
struct Walk {
    int b, h, rb;
    int i;               // segment of the class
    int st, n_st;        // stage, and stages of the segment
    int tokens;          // of the segment
};

__device__ __forceinline__ void lost(Walk &w) { w.h = w.rb = w.i = w.st = w.tokens = 0, w.n_st = 1; }

__device__ __forceinline__ void bind(const PagedList &l, const PagedClass &c, Walk &w) {
    w.tokens = seg_tokens(l, c.seg[w.i], w.b);
    w.n_st = w.tokens / c.unit + (w.tokens % c.unit ? 1 : 0);
}

// Stage `at` of sequence b.
__device__ __forceinline__ Walk seek(const PagedList &l, const PagedClass &c, int b, int at) {
    Walk w;
    w.b = b;
    for (w.h = 0; w.h < l.H; w.h++) {
        const int n = head_stages(l, c, b, w.h);
        if (at >= n * l.n_rb) {
            at -= n * l.n_rb;
            continue;
        }
        w.rb = at / n;
        at -= w.rb * n;
        for (w.i = 0; w.i < c.n; w.i++) {
            if (!((c.heads[w.i] >> w.h) & 1)) continue;
            bind(l, c, w);
            if (at < w.n_st) {
                w.st = at;
                return w;
            }
            at -= w.n_st;
        }
        break;
    }
    lost(w);
    return w;
}

// The next stage (whole warps; there is one).  True: of another (b, h, rb).
__device__ __forceinline__ bool next(const PagedList &l, const PagedClass &c, Walk &w) {
    if (++w.st < w.n_st) return false;
    w.st = 0;
    bool other = false;
    for (;;) {
        while (++w.i < c.n) {
            if (!((c.heads[w.i] >> w.h) & 1)) continue;
            bind(l, c, w);
            if (w.n_st > 0) return other;
        }
        w.i = -1;
        other = true;
        if (++w.rb < l.n_rb) continue;
        w.rb = 0;
        if (++w.h < l.H) continue;
        w.h = 0;
        // the next sequence that has a stage, 32 at a time
        unsigned some = 0;
        int b0 = w.b + 1;
        for (; b0 < l.B; b0 += 32) {
            const int b = b0 + static_cast<int>(threadIdx.x & 31);
            some = __ballot_sync(0xffffffffu, b < l.B && sequence_stages(l, c, b) > 0);
            if (some) break;
        }
        if (!some) {
            lost(w);
            return true;
        }
        w.b = b0 + __ffs(some) - 1;
    }
}

// Ranges of a CTA's TEAMS workers, worker t * step + first_worker for team t (THREADS threads, all of the CTA;
// synchronises).  buf: THREADS / 32 + 2 TEAMS ints of shared memory; team t's first sequence and the stages of it before
// its range are at THREADS / 32 + 2 t.  Returns the total.
template <int THREADS, int TEAMS>
__device__ __forceinline__ int ranges_of(const PagedList &l, const PagedClass &c, int first_worker, int step, int *first, int *buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = (l.B + THREADS - 1) / THREADS, b0 = min(static_cast<int>(threadIdx.x) * chunk, l.B), b1 = min(b0 + chunk, l.B);
    int sum = 0;
    for (int b = b0; b < b1; b++) sum += sequence_stages(l, c, b);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) buf[warp] = incl;
    __syncthreads();
    int before = incl - sum, total = 0;
    for (int w = 0; w < THREADS / 32; w++) {
        if (w < warp) before += buf[w];
        total += buf[w];
    }
    if (first_worker == 0) {
        int at = before;
        for (int b = b0; b < b1; b++) {
            first[b] = at;
            at += sequence_stages(l, c, b);
        }
        if (threadIdx.x == 0) first[l.B] = total;
    }
    const int workers = workers_of(c, total);
#pragma unroll
    for (int t = 0; t < TEAMS; t++) {
        const int worker = t * step + first_worker;
        if (worker >= workers) break;
        const int begin = worker_begin(total, worker, workers);
        if (sum > 0 && before <= begin && begin < before + sum) {
            int at = before, b = b0;
            for (int n; b + 1 < b1 && begin >= at + (n = sequence_stages(l, c, b)); b++) at += n;
            buf[THREADS / 32 + 2 * t] = b;
            buf[THREADS / 32 + 2 * t + 1] = begin - at;
        }
    }
    __syncthreads();
    return total;
}
// The range [begin, end) of a worker.
__device__ __forceinline__ void worker_range(const PagedClass &c, int total, int worker, int &begin, int &end) {
    const int workers = workers_of(c, total);
    begin = worker < workers ? worker_begin(total, worker, workers) : total;
    end = worker < workers ? worker_begin(total, worker + 1, workers) : total;
}

// The index of the page that holds token t.
__device__ __forceinline__ int page_index(const PagedSeg &s, int t) {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(t)) * s.magic) >> s.shift);
}
// The index-th page of sequence b in the pool, or -1.
__device__ __forceinline__ int page_at(const PagedSeg &s, int b, int index) {
    const int page = s.table ? s.table[b * s.table_stride + index] : b;
    return page >= 0 && page < s.n_pages ? page : -1;
}

__device__ __forceinline__ size_t group_slot(const PagedList &l, const PagedClass &c, int worker, int b, int h, int rb) {
    return static_cast<size_t>(c.slot0 + worker + (static_cast<long long>(b) * l.H + h) * l.n_rb + rb);
}

}  // namespace paged
}  // namespace tqk
