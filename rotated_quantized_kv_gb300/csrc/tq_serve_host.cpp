// tq_serve_host.cpp -- host side of the serving calls of include/tq.h (rotary
// positions, ragged writes and reads, tree attention): argument checks, kernel
// parameters, launches.  Nothing is allocated and no device value is read here.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "tq_serve.h"

using namespace tqk;

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

tq_status launched(cudaError_t e) { return e == cudaSuccess ? TQ_OK : record_cuda_error(e); }

bool finite_positive(double x) { return std::isfinite(x) && x > 0.0; }

tq_status check_rope_spec(const tq_rope_spec *s) {
    if (!s || s->rotary_dim < 2 || s->rotary_dim > TQ_MAX_HEAD_DIM || s->rotary_dim % 2) return TQ_ERR_ARG;
    if (s->scaling < TQ_ROPE_SCALE_NONE || s->scaling > TQ_ROPE_SCALE_INDEX) return TQ_ERR_ARG;
    if (!std::isfinite(s->base) || s->base <= 1.0 || !finite_positive(s->amplitude)) return TQ_ERR_ARG;
    if (s->scaling != TQ_ROPE_SCALE_NONE && !finite_positive(s->factor)) return TQ_ERR_ARG;
    if (s->scaling == TQ_ROPE_SCALE_BASE && s->rotary_dim == 2) return TQ_ERR_ARG;
    if (s->scaling == TQ_ROPE_SCALE_TURNS || s->scaling == TQ_ROPE_SCALE_INDEX)
        if (!finite_positive(s->original_len) || !finite_positive(s->slow) || !std::isfinite(s->fast) ||
            s->fast <= s->slow)
            return TQ_ERR_ARG;
    return TQ_OK;
}

void frequencies(const tq_rope_spec &s, double *freq) {
    const int r = s.rotary_dim;
    const double two_pi = 6.283185307179586476925;
    double base = s.base;
    if (s.scaling == TQ_ROPE_SCALE_BASE) base *= std::pow(s.factor, static_cast<double>(r) / (r - 2));
    double lo = 0.0, hi = 0.0;
    if (s.scaling == TQ_ROPE_SCALE_INDEX) {
        auto index_of = [&](double turns) {
            return r * std::log(s.original_len / (two_pi * turns)) / (2.0 * std::log(s.base));
        };
        lo = std::fmax(std::floor(index_of(s.fast)), 0.0);
        hi = std::fmin(std::ceil(index_of(s.slow)), r - 1.0);
        if (hi == lo) hi = lo + 0.001;
    }
    for (int m = 0; m < r / 2; ++m) {
        const double w = std::pow(base, -2.0 * m / r);
        double u = 1.0;  // share of the unscaled frequency
        if (s.scaling == TQ_ROPE_SCALE_LINEAR) u = 0.0;
        if (s.scaling == TQ_ROPE_SCALE_TURNS)
            u = std::fmin(std::fmax((s.original_len * w / two_pi - s.slow) / (s.fast - s.slow), 0.0), 1.0);
        if (s.scaling == TQ_ROPE_SCALE_INDEX) u = 1.0 - std::fmin(std::fmax((m - lo) / (hi - lo), 0.0), 1.0);
        freq[m] = u == 1.0 ? w : w * (u + (1.0 - u) / s.factor);
    }
}

tq_status check_rope_view(const tq_rope_view *v, int head_dim) {
    if (v->rotary_dim < 2 || v->rotary_dim % 2 || v->rotary_dim > head_dim) return TQ_ERR_ARG;
    if (v->layout != TQ_ROPE_HALF && v->layout != TQ_ROPE_INTERLEAVED) return TQ_ERR_ARG;
    if (v->n_pos < 0 || (v->n_pos > 0 && !v->table)) return TQ_ERR_ARG;
    if (!aligned(v->table, 16)) return TQ_ERR_ALIGN;
    return TQ_OK;
}

RopeView rope_view(const tq_rope_view *v) {
    RopeView r;
    r.table = v->table;
    r.half = v->rotary_dim / 2;
    r.interleaved = v->layout == TQ_ROPE_INTERLEAVED;
    r.n_pos = v->n_pos;
    return r;
}

// no two rows of d elements at the same place: every axis longer than one steps
// over at least a row
bool rows_apart(const int64_t *st, int B, int H, int T, int64_t d) {
    const int n[3] = {B, H, T};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && std::llabs(st[i]) < d) return false;
    return true;
}

// A segment of `B` sequences and `d` dims; `packed_ptrs` false: sizes only.
tq_status check_segment(const tq_segment *sg, bool check_ptrs) {
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

bool sphere_elsewhere(const tq_segment_layout &L) {
    return L.value_law == TQ_VALUE_LAW_SPHERE && L.head_dim != kD;
}

SegView seg_view(const tq_segment *sg) {
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

bool any_sketch(const tq_segment_layout &L) {
    for (int h = 0; h < L.n_heads; ++h)
        if (L.qjl[h] || L.qjl_v[h]) return true;
    return false;
}

// ---------------------------------------------------------------- tree attention
tq_status check_tree_view(const tq_layer_view *lv, int B, int H, int Hq, int d, int N, bool check_ptrs) {
    if (!lv || B < 1 || H < 1 || H > TQ_MAX_HEADS || Hq < H || Hq % H) return TQ_ERR_ARG;
    if (d < 16 || d > TQ_MAX_HEAD_DIM || (d & (d - 1))) return TQ_ERR_ARG;
    if (N < 1 || N > TQ_MAX_DRAFTS) return TQ_ERR_ARG;
    if (lv->n_segments < 0 || lv->n_segments > TQ_MAX_SEGMENTS || lv->rot.head_dim != d) return TQ_ERR_ARG;
    if (lv->rot.dense) return TQ_ERR_UNSUPPORTED;
    for (int i = 0; i < lv->n_segments; ++i) {
        const tq_segment &sg = lv->seg[i];
        const tq_status st = check_segment(&sg, check_ptrs);
        if (st != TQ_OK) return st;
        const tq_segment_layout &L = sg.layout;
        if (L.batch != B || L.n_heads != H || L.head_dim != d) return TQ_ERR_ARG;
        if (sg.n_tokens < 0 || sg.n_tokens > L.capacity) return TQ_ERR_SIZE;
        if (sg.n_tokens > 0x7fffffff - (kTreeTile - 1)) return TQ_ERR_UNSUPPORTED;  // rounded up to tiles in 32 bits
        if (sg.attn_mass) return TQ_ERR_UNSUPPORTED;
        if (sg.kind == TQ_SEG_PACKED) {
            if (any_sketch(L) || sphere_elsewhere(L)) return TQ_ERR_UNSUPPORTED;
            if (L.capacity % 16) return TQ_ERR_ALIGN;
        }
    }
    // query rows are counted in 32 bits
    if (static_cast<int64_t>(N) * Hq > 0x7fffffff / B) return TQ_ERR_UNSUPPORTED;
    return TQ_OK;
}

int tiles_of(int n) { return n / kTreeTile + (n % kTreeTile ? 1 : 0); }

// counts, parts and the record area of a shape
struct TreeLayout {
    TreeShape shape;
    int parts_packed, parts;
    int n_var;
    uint8_t var[TQ_MAX_SEGMENTS][kMaxH], var_bits[TQ_MAX_SEGMENTS][kMaxH];  // packed segments first
    size_t image_off, part_off, total;
};

tq_status tree_layout(const tq_layer_view *lv, int B, int H, int Hq, int d, int N, TreeLayout &o) {
    int64_t tp = 0, tf = 0;
    for (int i = 0; i < lv->n_segments; ++i)
        (lv->seg[i].kind == TQ_SEG_PACKED ? tp : tf) += tiles_of(lv->seg[i].n_tokens);
    o.shape = tree_shape(B, H, Hq / H, N, d, tp + tf);
    const int64_t pp = (tp + kTreePart - 1) / kTreePart, pf = (tf + kTreePart - 1) / kTreePart;
    const int64_t slots = o.shape.workers + static_cast<int64_t>(B) * H * o.shape.n_rb * (pp + pf);
    if (slots > 0x7fffffff || static_cast<int64_t>(B) * H * o.shape.n_rb * (tp + tf) > 0x7fffffff)
        return TQ_ERR_UNSUPPORTED;  // tiles and slots are counted in 32 bits
    o.parts_packed = static_cast<int>(pp);
    o.parts = static_cast<int>(pp + pf);
    // distinct key widths among each head's segments (fp16: 0)
    o.n_var = 0;
    std::memset(o.var, 0, sizeof(o.var));
    std::memset(o.var_bits, 0, sizeof(o.var_bits));
    for (int h = 0; h < H; ++h) {
        int n = 0, at = 0;
        for (int pass = 0; pass < 2; ++pass)
            for (int i = 0; i < lv->n_segments; ++i) {
                const tq_segment &sg = lv->seg[i];
                if ((sg.kind == TQ_SEG_FP16) != (pass == 1)) continue;
                const uint8_t kb = pass ? 0 : sg.layout.kbits[h];
                int v = 0;
                while (v < n && o.var_bits[v][h] != kb) ++v;
                if (v == n) o.var_bits[n++][h] = kb;
                o.var[at++][h] = static_cast<uint8_t>(v);
            }
        o.n_var = std::max(o.n_var, n);
    }
    o.image_off = 256;  // the error flag has the first 256 bytes
    o.part_off = o.image_off;
    if (tree_on_tensor_cores(d))
        o.part_off += static_cast<size_t>(B) * H * o.shape.n_rb * o.n_var * tree_image_bytes(d, o.shape.R);
    o.total = o.part_off + static_cast<size_t>(slots) * o.shape.R * (d + 4) * sizeof(float);
    return TQ_OK;
}

}  // namespace

extern "C" {

tq_status tq_rope_frequencies(const tq_rope_spec *spec, double *freq) {
    const tq_status st = check_rope_spec(spec);
    if (st != TQ_OK) return st;
    if (!freq) return TQ_ERR_ARG;
    frequencies(*spec, freq);
    return TQ_OK;
}

tq_status tq_rope_table(const tq_rope_spec *spec, int first_pos, int n_pos, float *table, void *stream) {
    const tq_status st = check_rope_spec(spec);
    if (st != TQ_OK) return st;
    if (first_pos < 0 || n_pos < 0 || static_cast<int64_t>(first_pos) + n_pos > 0x7fffffff) return TQ_ERR_ARG;
    if (n_pos == 0) return TQ_OK;
    if (!table) return TQ_ERR_ARG;
    if (!aligned(table, 16)) return TQ_ERR_ALIGN;
    RopeTable p;
    std::memset(&p, 0, sizeof(p));
    frequencies(*spec, p.freq);
    p.amplitude = spec->amplitude;
    p.half = spec->rotary_dim / 2;
    p.first = first_pos;
    p.n = n_pos;
    p.table = table;
    return launched(launch_rope_table(p, static_cast<cudaStream_t>(stream)));
}

tq_status tq_rope(const tq_rope_view *rope, int dtype, int batch, int n_tokens, int head_dim, const int *positions,
                  int64_t pos_stride_b, const tq_rope_tensor *x, int n_tensors, int inverse, void *stream) {
    if (!rope || dtype < TQ_DTYPE_F16 || dtype > TQ_DTYPE_F32) return TQ_ERR_ARG;
    if (batch < 0 || n_tokens < 0 || head_dim < 1 || head_dim > TQ_MAX_HEAD_DIM) return TQ_ERR_ARG;
    if (n_tensors < 0 || n_tensors > TQ_MAX_ROPE_TENSORS || (n_tensors > 0 && !x)) return TQ_ERR_ARG;
    const tq_status st = check_rope_view(rope, head_dim);
    if (st != TQ_OK) return st;
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    int64_t heads = 0;
    for (int i = 0; i < n_tensors; ++i) {
        if (x[i].n_heads < 0) return TQ_ERR_ARG;
        if (x[i].n_heads == 0) continue;
        if (batch > 0 && n_tokens > 0) {
            if (!x[i].in || !x[i].out) return TQ_ERR_ARG;
            const size_t elem = dtype == TQ_DTYPE_F32 ? 4 : 2;
            if (!aligned(x[i].in, elem) || !aligned(x[i].out, elem)) return TQ_ERR_ALIGN;
            if (!rows_apart(x[i].out_stride, batch, x[i].n_heads, n_tokens, head_dim)) return TQ_ERR_ARG;
            if (x[i].in == x[i].out && std::memcmp(x[i].in_stride, x[i].out_stride, sizeof(x[i].in_stride)))
                return TQ_ERR_ARG;
        }
        RopeTensorParams &t = p.x[p.n_tensors++];
        t.in = x[i].in;
        t.out = x[i].out;
        for (int j = 0; j < 3; ++j) {
            t.is[j] = x[i].in_stride[j];
            t.os[j] = x[i].out_stride[j];
        }
        t.head0 = static_cast<int>(heads);
        heads += x[i].n_heads;
    }
    if (heads > 65535) return TQ_ERR_UNSUPPORTED;
    if (batch == 0 || n_tokens == 0 || heads == 0) return TQ_OK;
    if (!positions) return TQ_ERR_ARG;
    if (!aligned(positions, 4)) return TQ_ERR_ALIGN;
    p.rope = rope_view(rope);
    p.positions = positions;
    p.pos_stride = pos_stride_b;
    p.B = batch;
    p.T = n_tokens;
    p.d = head_dim;
    p.inverse = inverse != 0;
    p.heads = static_cast<int>(heads);
    return launched(launch_rope(p, dtype, static_cast<cudaStream_t>(stream)));
}

tq_status tq_append(const tq_segment *dst, const tq_rotation *rot, const tq_rope_view *rope, const int *positions,
                    int64_t pos_stride_b, const void *K, const int64_t *k_stride, const void *V,
                    const int64_t *v_stride, int n_source, int n_max, const int *t_begin, const int *n_new,
                    const int *index, int64_t index_stride_b, void *stream) {
    tq_status st = check_segment(dst, true);
    if (st != TQ_OK) return st;
    const tq_segment_layout &L = dst->layout;
    const bool packed = dst->kind == TQ_SEG_PACKED;
    if (n_source < 0 || n_max < 0 || !k_stride || !v_stride) return TQ_ERR_ARG;
    if (packed) {
        if (!rot || rot->head_dim != L.head_dim) return TQ_ERR_ARG;
        if (rot->dense || any_sketch(L) || sphere_elsewhere(L)) return TQ_ERR_UNSUPPORTED;
    }
    if (rope) {
        st = check_rope_view(rope, L.head_dim);
        if (st != TQ_OK) return st;
    }
    if (n_max == 0 || n_source == 0 || L.capacity == 0) return TQ_OK;
    if (!K || !V || !t_begin || (rope && !positions)) return TQ_ERR_ARG;
    if (!aligned(K, 2) || !aligned(V, 2) || !aligned(t_begin, 4) || !aligned(n_new, 4) || !aligned(index, 4) ||
        (rope && !aligned(positions, 4)))
        return TQ_ERR_ALIGN;
    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.seg = seg_view(dst);
    p.rows.t_begin = t_begin;
    p.rows.n_rows = n_new;
    p.rows.index = index;
    p.rows.index_stride = index_stride_b;
    p.rows.n_max = index ? n_max : std::min(n_max, n_source);  // (row j is source row j)
    p.rows.n_source = n_source;
    if (rope) {
        p.rope = rope_view(rope);
        p.positions = positions;
        p.pos_stride = pos_stride_b;
    }
    p.K = static_cast<const uint16_t *>(K);
    p.V = static_cast<const uint16_t *>(V);
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = k_stride[i];
        p.vs[i] = v_stride[i];
    }
    p.B = L.batch;
    p.H = L.n_heads;
    p.d = L.head_dim;
    if (packed) {
        std::memcpy(p.sign_bits, rot->sign_bits, sizeof(p.sign_bits));
        p.inv_sqrt_d = rotation_scale(p.d);
        p.law = L.value_law;
        try {
            value_thresholds(p.thr, L.vbits, p.H, L.value_law);
        } catch (...) {
            return TQ_ERR_SIZE;  // no host memory for the codebook fit
        }
    }
    return launched(launch_append(p, static_cast<cudaStream_t>(stream)));
}

tq_status tq_read(const tq_segment *src, const tq_rotation *rot, int n_max, const int *t_begin, const int *n_read,
                  int dtype, void *K, const int64_t *k_stride, void *V, const int64_t *v_stride, void *stream) {
    const tq_status st = check_segment(src, true);
    if (st != TQ_OK) return st;
    const tq_segment_layout &L = src->layout;
    const bool packed = src->kind == TQ_SEG_PACKED;
    if (dtype < TQ_DTYPE_F16 || dtype > TQ_DTYPE_F32 || n_max < 0) return TQ_ERR_ARG;
    if (packed) {
        if (rot && rot->head_dim != L.head_dim) return TQ_ERR_ARG;
        if ((rot && rot->dense) || sphere_elsewhere(L)) return TQ_ERR_UNSUPPORTED;
    }
    if ((K && !k_stride) || (V && !v_stride)) return TQ_ERR_ARG;
    if (n_max == 0 || L.capacity == 0 || (!K && !V)) return TQ_OK;
    if (!t_begin) return TQ_ERR_ARG;
    const size_t elem = dtype == TQ_DTYPE_F32 ? 4 : 2;
    if (!aligned(K, elem) || !aligned(V, elem) || !aligned(t_begin, 4) || !aligned(n_read, 4)) return TQ_ERR_ALIGN;
    ReadParams p;
    std::memset(&p, 0, sizeof(p));
    p.seg = seg_view(src);
    p.rows.t_begin = t_begin;
    p.rows.n_rows = n_read;
    p.rows.n_max = n_max;
    p.K = K;
    p.V = V;
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = K ? k_stride[i] : 0;
        p.vs[i] = V ? v_stride[i] : 0;
    }
    p.B = L.batch;
    p.H = L.n_heads;
    p.d = L.head_dim;
    if ((K && !rows_apart(p.ks, p.B, p.H, n_max, p.d)) || (V && !rows_apart(p.vs, p.B, p.H, n_max, p.d)))
        return TQ_ERR_ARG;
    if (packed) {
        p.rotate = rot != nullptr;
        if (rot) std::memcpy(p.sign_bits, rot->sign_bits, sizeof(p.sign_bits));
        p.inv_sqrt_d = rotation_scale(p.d);
        try {
            value_centroids(p.centroid, L.vbits, p.H, L.value_law);
        } catch (...) {
            return TQ_ERR_SIZE;
        }
    }
    return launched(launch_read(p, dtype, static_cast<cudaStream_t>(stream)));
}

tq_status tq_tree_workspace_size(const tq_layer_view *layer, int batch, int n_heads, int q_heads, int head_dim,
                                 int n_drafts, size_t *bytes) {
    if (!bytes) return TQ_ERR_ARG;
    tq_status st = check_tree_view(layer, batch, n_heads, q_heads, head_dim, n_drafts, false);
    if (st != TQ_OK) return st;
    TreeLayout o;
    st = tree_layout(layer, batch, n_heads, q_heads, head_dim, n_drafts, o);
    if (st == TQ_OK) *bytes = o.total;
    return st;
}

tq_status tq_tree_attention(const tq_layer_view *layer, int batch, int n_heads, int q_heads, int head_dim,
                            const tq_tree *tree, void *workspace, size_t ws_bytes, void *stream) {
    if (!tree) return TQ_ERR_ARG;
    tq_status st = check_tree_view(layer, batch, n_heads, q_heads, head_dim, tree->n_drafts, true);
    if (st != TQ_OK) return st;
    if (!tree->q || !tree->k || !tree->v || !tree->out || !workspace) return TQ_ERR_ARG;
    if (tree->mask_stride_b < 0) return TQ_ERR_ARG;
    if (!aligned(tree->q, 2) || !aligned(tree->k, 2) || !aligned(tree->v, 2) || !aligned(tree->out, 16) ||
        !aligned(workspace, 16) || !aligned(tree->mask, 4))
        return TQ_ERR_ALIGN;
    for (int i = 0; i < layer->n_segments; ++i)
        if (!aligned(tree->seg_len[i], 4)) return TQ_ERR_ALIGN;
    TreeLayout o;
    st = tree_layout(layer, batch, n_heads, q_heads, head_dim, tree->n_drafts, o);
    if (st != TQ_OK) return st;
    if (ws_bytes < o.total) return TQ_ERR_SIZE;
    TreeParams p;
    std::memset(&p, 0, sizeof(p));
    p.B = batch;
    p.H = n_heads;
    p.g = q_heads / n_heads;
    p.N = tree->n_drafts;
    p.d = head_dim;
    p.R = o.shape.R;
    p.n_rb = o.shape.n_rb;
    p.workers = o.shape.workers;
    p.parts_packed = o.parts_packed;
    p.parts = o.parts;
    try {
        for (int pass = 0; pass < 2; ++pass)  // packed segments first
            for (int i = 0; i < layer->n_segments; ++i) {
                const tq_segment &sg = layer->seg[i];
                if ((sg.kind == TQ_SEG_FP16) != (pass == 1)) continue;
                TreeSeg &t = p.seg[p.n_seg++];
                t.seg = seg_view(&sg);
                t.len = tree->seg_len[i];
                t.n_tokens = sg.n_tokens;
                p.ragged |= t.len != nullptr;
                if (pass == 0) {
                    t.law = sg.layout.value_law;
                    ++p.n_packed;
                    value_centroids(p.centroid[t.law], sg.layout.vbits, n_heads, t.law);
                }
            }
    } catch (...) {
        return TQ_ERR_SIZE;  // no host memory for the codebook fit
    }
    p.q = static_cast<const uint16_t *>(tree->q);
    p.k = static_cast<const uint16_t *>(tree->k);
    p.v = static_cast<const uint16_t *>(tree->v);
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = tree->q_stride[i];
        p.ks[i] = tree->k_stride[i];
        p.vs[i] = tree->v_stride[i];
    }
    p.mask = tree->mask;
    p.mask_stride = tree->mask_stride_b;
    p.mask_words = (p.N + 31) / 32;
    p.out = static_cast<uint16_t *>(tree->out);
    p.error = static_cast<int *>(workspace);
    p.images = static_cast<uint8_t *>(workspace) + o.image_off;
    p.n_var = o.n_var;
    std::memcpy(p.var, o.var, sizeof(p.var));
    std::memcpy(p.var_bits, o.var_bits, sizeof(p.var_bits));
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + o.part_off);
    p.wait_polls = decode_wait_polls();
    std::memcpy(p.sign_bits, layer->rot.sign_bits, sizeof(p.sign_bits));
    p.inv_sqrt_d = rotation_scale(head_dim);
    p.qk_scale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(head_dim)));
    return launched(launch_tree(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
