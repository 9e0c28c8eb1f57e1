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

__host__ __device__ __forceinline__ int seg_tokens(const PagedList &l, int seg, int b) {
    return l.len[seg] ? min(max(l.len[seg][b], 0), l.limit[seg]) : l.limit[seg];
}
// Stages of the class's i-th segment.
__host__ __device__ __forceinline__ int seg_stages(const PagedList &l, const PagedClass &c, int i, int b) {
    const int n = seg_tokens(l, c.seg[i], b);
    return n / c.unit + (n % c.unit ? 1 : 0);
}
// Stages of (b, h, any rb).
__host__ __device__ __forceinline__ int head_stages(const PagedList &l, const PagedClass &c, int b, int h) {
    int n = 0;
#pragma unroll 1
    for (int i = 0; i < c.n; i++)
        if ((c.heads[i] >> h) & 1) n += seg_stages(l, c, i, b);
    return n;
}
// Stages of sequence b (below 2^31 over all sequences: the host checks it for the limits).
__device__ __forceinline__ int sequence_stages(const PagedList &l, const PagedClass &c, int b) {
    int n = 0;
#pragma unroll 1
    for (int i = 0; i < c.n; i++) n += __popc(c.heads[i]) * seg_stages(l, c, i, b);
    return n * c.n_rb;
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
    bool fresh;          // begins a (b, h, rb)
};

__host__ __device__ __forceinline__ void lost(Walk &w) { w.h = w.rb = w.i = w.st = w.tokens = 0, w.n_st = 1; }

__host__ __device__ __forceinline__ void bind(const PagedList &l, const PagedClass &c, Walk &w) {
    w.tokens = seg_tokens(l, c.seg[w.i], w.b);
    w.n_st = w.tokens / c.unit + (w.tokens % c.unit ? 1 : 0);
}

// The n-th head of a set (from 0), or -1.
__host__ __device__ __forceinline__ int head_of(unsigned heads, int n) {
#pragma unroll 1
    for (int h = 0; h < kMaxH; h++)
        if (((heads >> h) & 1) && n-- == 0) return h;
    return -1;
}

// Stage `at` of sequence b.  (This and what follows are no part of a kernel's loop and would be most of its code, a
// quarter of a megabyte, if they were inlined: warps then waited for instructions.)
static __host__ __device__ __noinline__ Walk seek(const PagedList &l, const PagedClass &c, int b, int at) {
    Walk w;
    w.b = b;
    w.fresh = true;
    if (c.n == 1) {  // one segment: all its heads have as many stages
        w.i = 0;
        bind(l, c, w);
        if (w.n_st > 0) {
            const int block = at / w.n_st, head = block / c.n_rb;
            w.st = at - block * w.n_st;
            w.rb = block - head * c.n_rb;
            w.h = head_of(c.heads[0], head);
            if (w.h >= 0) return w;  // (a length that has become shorter: there is no such head)
        }
        lost(w);
        return w;
    }
#pragma unroll 1
    for (w.h = 0; w.h < l.H; w.h++) {
        const int n = head_stages(l, c, b, w.h);
        if (at >= n * c.n_rb) {
            at -= n * c.n_rb;
            continue;
        }
        w.rb = at / n;
        at -= w.rb * n;
#pragma unroll 1
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

// The first stage behind the segment's last one (whole warps; there is one).  fresh: it is of another (b, h, rb).
static __device__ __noinline__ Walk next(const PagedList &l, const PagedClass &c, Walk w) {
    w.st = 0;
    bool other = false, moved = false;
    for (;;) {
        while (++w.i < c.n) {
            if (!((c.heads[w.i] >> w.h) & 1)) continue;
            if (c.n > 1 || moved) bind(l, c, w);  // (one segment: as the head before)
            if (w.n_st > 0) {
                w.fresh = other;
                return w;
            }
        }
        w.i = -1;
        other = true;
        if (++w.rb < c.n_rb) continue;
        w.rb = 0;
        if (++w.h < l.H) continue;
        w.h = 0;
        moved = true;
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
            w.fresh = true;
            return w;
        }
        w.b = b0 + __ffs(some) - 1;
    }
}

// The stages of the thread's share of the sequences [b0, b1) (THREADS threads).
template <int THREADS>
struct Share {
    int b0, b1, sum;
    __device__ __forceinline__ Share(const PagedList &l, const PagedClass &c) {
        const int chunk = (l.B + THREADS - 1) / THREADS;
        b0 = min(static_cast<int>(threadIdx.x) * chunk, l.B);
        b1 = min(b0 + chunk, l.B);
        sum = 0;
#pragma unroll 1
        for (int b = b0; b < b1; b++) sum += sequence_stages(l, c, b);
    }
};
// Ranges of a CTA's TEAMS workers, worker t * step + first_worker for team t (all of the CTA's threads with their
// shares; synchronises).  buf: THREADS / 32 + 4 TEAMS ints of shared memory; team t's first sequence and the stages of it
// before its range, and the range [begin, end), are at THREADS / 32 + 4 t.  (A division of 64 bits for each bound, by a
// thread of its own: all threads doing all of them were 3 us of 32 with 8 sequences of up to 4096 tokens, fp16.)
template <int THREADS, int TEAMS>
__device__ __forceinline__ void ranges_of(const PagedList &l, const PagedClass &c, const Share<THREADS> &own, int first_worker, int step,
                                         int *first, int *buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = own.sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) buf[warp] = incl;
    __syncthreads();
    int before = incl - own.sum, total = 0;
    for (int w = 0; w < THREADS / 32; w++) {
        if (w < warp) before += buf[w];
        total += buf[w];
    }
    if (first_worker == 0) {
        int at = before;
#pragma unroll 1
        for (int b = own.b0; b < own.b1; b++) {
            first[b] = at;
            at += sequence_stages(l, c, b);
        }
        if (threadIdx.x == 0) first[l.B] = total;
    }
    buf += THREADS / 32;
    if (threadIdx.x < 2 * TEAMS) {
        const int workers = workers_of(c, total), t = threadIdx.x >> 1, worker = t * step + first_worker;
        buf[4 * t + 2 + (threadIdx.x & 1)] = worker < workers ? worker_begin(total, worker + (threadIdx.x & 1), workers) : total;
    }
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < TEAMS; t++) {
        const int begin = buf[4 * t + 2];
        if (own.sum > 0 && before <= begin && begin < before + own.sum) {
            int at = before, b = own.b0;
#pragma unroll 1
            for (int n; b + 1 < own.b1 && begin >= at + (n = sequence_stages(l, c, b)); b++) at += n;
            buf[4 * t] = b;
            buf[4 * t + 1] = begin - at;
        }
    }
    __syncthreads();
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

// A warp's view of a sequence's row of the table: two windows of 32 entries, so that a walk along the
// sequence reads the table once every 32 pages, and ahead.
struct Pages {
    int now, then;       // the lane's entries of the windows at `base` and behind it
    int base;
    __device__ __forceinline__ int entry(const PagedSeg &s, int b, int last, int index) const {
        return index > last ? -1 : s.table ? s.table[b * s.table_stride + index] : 0;
    }
    // The row of sequence b from page `index` on; `last`: its last page.
    __device__ __forceinline__ void open(const PagedSeg &s, int b, int last, int index, int lane) {
        base = index & ~31;
        now = entry(s, b, last, base + lane);
        then = entry(s, b, last, base + 32 + lane);
    }
    // Moves on to a place at page `index` (not before base).
    __device__ __forceinline__ void move(const PagedSeg &s, int b, int last, int index, int lane) {
        if (index < base + 32) return;
        if (index >= base + 64) return open(s, b, last, index, lane);
        base += 32;
        now = then;
        then = entry(s, b, last, base + 32 + lane);
    }
    // Entry `index` (in the windows; its own for each lane, all lanes).
    __device__ __forceinline__ int at(int index) const {
        const int x = __shfl_sync(0xffffffffu, now, index & 31), y = __shfl_sync(0xffffffffu, then, index & 31);
        return index < base + 32 ? x : y;
    }
};

__device__ __forceinline__ size_t group_slot(const PagedList &l, const PagedClass &c, int worker, int b, int h, int rb) {
    return static_cast<size_t>(worker + (static_cast<long long>(b) * l.H + h) * c.n_rb + rb);
}

}  // namespace paged
}  // namespace tqk
