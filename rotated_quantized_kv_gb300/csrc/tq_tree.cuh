// tq_tree.cuh -- the tile list of tree attention and the walk along it, shared
// by its kernels (tq_serve.h describes the list, its parts and their records).
#pragma once

#include "tq_serve.h"

namespace tqk {
namespace tree {

template <typename P>
__device__ __forceinline__ int seg_tokens(const P &p, int i, int b) {
    const auto &s = p.seg[i];
    return s.len ? min(max(s.len[b], 0), s.n_tokens) : s.n_tokens;
}

// Tiles of sequence b's packed segments, and of its fp16 ones.
template <typename P>
__device__ __forceinline__ void seq_tiles(const P &p, int b, int &tp, int &tf) {
    tp = 0;
    tf = 0;
    for (int i = 0; i < p.n_seg; i++) {
        const int n = (seg_tokens(p, i, b) + kTreeTile - 1) / kTreeTile;
        if (i < p.n_packed) tp += n;
        else tf += n;
    }
}

// Tiles of the whole call (below 2^31, which the host checks for the segments'
// n_tokens).  A warp takes 32 sequences at a time; all lanes return the sum.
template <typename P>
__device__ __forceinline__ unsigned total_tiles(const P &p) {
    const unsigned per = p.H * p.n_rb;
    int tp, tf;
    if (!p.ragged) {
        seq_tiles(p, 0, tp, tf);
        return per * p.B * (tp + tf);
    }
    unsigned sum = 0;
    for (int b = threadIdx.x & 31; b < p.B; b += 32) {
        seq_tiles(p, b, tp, tf);
        sum += tp + tf;
    }
    return per * __reduce_add_sync(0xffffffffu, sum);
}

// Tiles of a worker: worker c has [c n, (c + 1) n) of the T, n = ceil(T / workers)
// (every worker that starts below T has a tile; the launch is sized for the
// segments' n_tokens, the lengths on the device may be shorter).
template <typename P>
__device__ __forceinline__ unsigned worker_tiles(const P &p, unsigned T) {
    return max((T + p.workers - 1) / p.workers, 1u);
}

struct Pos {
    int b, h, rb;   // sequence, KV head, block of query rows
    int k;          // tile of (b, h, rb)
    int tp, tf;     // its packed tiles and the others
};

// The place of tile `at` < total_tiles in the list (whole warp, `at` uniform).
__device__ __forceinline__ Pos seek(const TreeParams &p, unsigned at) {
    Pos x;
    const unsigned per = p.H * p.n_rb;
    x.b = 0;
    if (!p.ragged) {
        seq_tiles(p, 0, x.tp, x.tf);
        const unsigned each = per * (x.tp + x.tf);
        x.b = at / each;
        at -= x.b * each;
    } else {
        const int lane = threadIdx.x & 31;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            int tp = 0, tf = 0;
            if (b0 + lane < p.B) seq_tiles(p, b0 + lane, tp, tf);
            unsigned end = per * (tp + tf);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, end > at);
            const int l = past ? __ffs(past) - 1 : 31;
            const unsigned upto = __shfl_sync(0xffffffffu, end, l);
            x.b = b0 + l;
            x.tp = __shfl_sync(0xffffffffu, tp, l);
            x.tf = __shfl_sync(0xffffffffu, tf, l);
            if (past) {
                at -= upto - per * (x.tp + x.tf);
                break;
            }
            at -= upto;
        }
    }
    const unsigned tiles = x.tp + x.tf, hr = at / tiles;
    x.k = at - hr * tiles;
    x.h = hr / p.n_rb;
    x.rb = hr - x.h * p.n_rb;
    return x;
}

__device__ __forceinline__ void advance(const TreeParams &p, Pos &x) {
    if (++x.k < x.tp + x.tf) return;
    x.k = 0;
    if (++x.rb < p.n_rb) return;
    x.rb = 0;
    if (++x.h < p.H) return;
    x.h = 0;
    ++x.b;
    if (p.ragged) {
        for (; x.b < p.B; ++x.b) {
            seq_tiles(p, x.b, x.tp, x.tf);
            if (x.tp + x.tf > 0) break;
        }
    }
}

__device__ __forceinline__ int group_of(const TreeParams &p, const Pos &x) { return (x.b * p.H + x.h) * p.n_rb + x.rb; }

// Index of the part that tile k of group `group` belongs to.
template <typename P>
__device__ __forceinline__ int part_of(const P &p, int group, int tp, int k) {
    return group * p.parts + (k < tp ? k / kTreePart : p.parts_packed + (k - tp) / kTreePart);
}

// A walk along the list: the current tile holds tokens [128 t, min(128 (t + 1), n))
// of segment `seg`, tile k of its (b, h, rb), and belongs to part `part`.
struct Walk {
    Pos x;
    int seg, t, tiles, n;  // tiles, n: of the segment, for sequence b
    int part;
    bool fresh;            // first tile of its (group, segment)
    bool first;            // first tile of its part
};

// Segment and part of tile w.x.k.
__device__ __forceinline__ void walk_locate(const TreeParams &p, Walk &w) {
    const bool packed = w.x.k < w.x.tp;
    int k = packed ? w.x.k : w.x.k - w.x.tp;
    w.part = part_of(p, group_of(p, w.x), w.x.tp, w.x.k);
    w.seg = packed ? 0 : p.n_packed;
    for (;; w.seg++) {  // (ends: k counts the tiles of these segments)
        w.n = seg_tokens(p, w.seg, w.x.b);
        w.tiles = (w.n + kTreeTile - 1) / kTreeTile;
        if (k < w.tiles || w.seg + 1 >= p.n_seg) break;
        k -= w.tiles;
    }
    w.t = k;
    w.fresh = true;
}
__device__ __forceinline__ Walk walk_begin(const TreeParams &p, unsigned at) {
    Walk w;
    w.x = seek(p, at);
    walk_locate(p, w);
    w.first = true;
    return w;
}
__device__ __forceinline__ void walk_next(const TreeParams &p, Walk &w) {
    if (w.t + 1 < w.tiles) {
        w.t++;
        w.x.k++;
        const int k = w.x.k < w.x.tp ? w.x.k : w.x.k - w.x.tp;
        w.first = k % kTreePart == 0;
        w.part += w.first;
        w.fresh = false;
        return;
    }
    advance(p, w.x);
    if (w.x.b >= p.B) return;  // behind the last tile
    const int part = w.part;
    walk_locate(p, w);
    w.first = w.part != part;
}

// Word w of the drafts that draft i of sequence b sees.
template <typename P>
__device__ __forceinline__ uint32_t seen_word(const P &p, int N, int b, int i, int w) {
    const int left = N - 32 * w;
    const uint32_t real = left >= 32 ? 0xffffffffu : (1u << left) - 1u;  // bits behind the last draft mean nothing
    if (p.mask) return p.mask[b * p.mask_stride + static_cast<int64_t>(i) * p.mask_words + w] & real;
    return (i >= 32 * w + 31 ? 0xffffffffu : i < 32 * w ? 0u : (2u << (i - 32 * w)) - 1u) & real;
}

}  // namespace tree
}  // namespace tqk
