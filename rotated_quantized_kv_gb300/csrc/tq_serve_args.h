// tq_serve_args.h -- argument checks and kernel views that the serving calls' host sides
// share.
#pragma once

#include <cstdlib>
#include <cstring>

#include <cuda_runtime.h>

#include "tq_serve.h"

namespace tqk {
namespace {

inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline tq_status launched(cudaError_t e) { return e == cudaSuccess ? TQ_OK : record_cuda_error(e); }

inline tq_status check_rope_view(const tq_rope_view *v, int head_dim) {
    if (v->rotary_dim < 2 || v->rotary_dim % 2 || v->rotary_dim > head_dim) return TQ_ERR_ARG;
    if (v->layout != TQ_ROPE_HALF && v->layout != TQ_ROPE_INTERLEAVED) return TQ_ERR_ARG;
    if (v->n_pos < 0 || (v->n_pos > 0 && !v->table)) return TQ_ERR_ARG;
    if (!aligned(v->table, 16)) return TQ_ERR_ALIGN;
    return TQ_OK;
}

inline RopeView rope_view(const tq_rope_view *v) {
    RopeView r;
    r.table = v->table;
    r.half = v->rotary_dim / 2;
    r.interleaved = v->layout == TQ_ROPE_INTERLEAVED;
    r.n_pos = v->n_pos;
    return r;
}

// no two rows of d elements at the same place: every axis longer than one steps
// over at least a row
inline bool rows_apart(const int64_t *st, int B, int H, int T, int64_t d) {
    const int n[3] = {B, H, T};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && std::llabs(st[i]) < d) return false;
    return true;
}

// A segment of `B` sequences and `d` dims; `packed_ptrs` false: sizes only.
inline tq_status check_segment(const tq_segment *sg, bool check_ptrs) {
    if (!sg || (sg->kind != TQ_SEG_PACKED && sg->kind != TQ_SEG_FP16)) return TQ_ERR_ARG;
    const tq_segment_layout &L = sg->layout;
    const bool packed = sg->kind == TQ_SEG_PACKED;
    const tq_status st = layout_status(&L, packed);
    if (st != TQ_OK) return st;
    if (!check_ptrs || L.capacity == 0) return TQ_OK;
    if (packed) {
        const tq_packed_bufs &b = sg->packed;
        if (!b.kcodes || !b.vcodes || !b.kscale || !b.vscale) return TQ_ERR_ARG;
        if (!aligned(b.kcodes, 16) || !aligned(b.vcodes, 16) || !aligned(b.kscale, 16) || !aligned(b.vscale, 16))
            return TQ_ERR_ALIGN;
    } else {
        if (!sg->k16 || !sg->v16) return TQ_ERR_ARG;
        if (!aligned(sg->k16, 16) || !aligned(sg->v16, 16)) return TQ_ERR_ALIGN;
    }
    return TQ_OK;
}

inline bool sphere_elsewhere(const tq_segment_layout &L) {
    return L.value_law == TQ_VALUE_LAW_SPHERE && L.head_dim != kD;
}

inline SegView seg_view(const tq_segment *sg) {
    SegView v;
    std::memset(&v, 0, sizeof(v));
    const tq_segment_layout &L = sg->layout;
    v.fp16 = sg->kind == TQ_SEG_FP16;
    v.capacity = L.capacity;
    const uint64_t cap = static_cast<uint64_t>(L.capacity);
    if (v.fp16) {
        v.k = static_cast<const uint8_t *>(sg->k16);
        v.v = static_cast<const uint8_t *>(sg->v16);
        for (int h = 0; h < L.n_heads; ++h) v.koff[h] = v.voff[h] = h * cap * L.head_dim * 2;
        v.kblock = v.vblock = L.n_heads * cap * L.head_dim * 2;
    } else {
        v.k = static_cast<const uint8_t *>(sg->packed.kcodes);
        v.v = static_cast<const uint8_t *>(sg->packed.vcodes);
        v.ks = sg->packed.kscale;
        v.vs = sg->packed.vscale;
        for (int h = 0; h < L.n_heads; ++h) {
            v.koff[h] = v.kblock;
            v.voff[h] = v.vblock;
            v.kbits[h] = L.kbits[h];
            v.vbits[h] = L.vbits[h];
            v.kblock += cap * L.head_dim * L.kbits[h] / 8;
            v.vblock += cap * L.head_dim * L.vbits[h] / 8;
        }
    }
    return v;
}

inline bool any_sketch(const tq_segment_layout &L) {
    for (int h = 0; h < L.n_heads; ++h)
        if (L.qjl[h] || L.qjl_v[h]) return true;
    return false;
}

}  // namespace
}  // namespace tqk
