// tq_paged_host.cpp -- host side of the page tables, of paged attention and of the
// verification of drafts (include/tq.h): argument checks, kernel parameters, launches.
// Nothing is allocated and no device value is read here.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "tq_serve.h"
#include "tq_serve_args.h"

using namespace tqk;

namespace {

tq_status check_pages(int batch, int page_size, int max_pages, int n_pages, const int *table, int64_t table_stride,
                      const int *length, const int *count, const int *free_pages, const int *n_free) {
    if (batch < 0 || page_size < 1 || max_pages < 0 || n_pages < 0 || table_stride < 0) return TQ_ERR_ARG;
    // tokens of a sequence, slots of the pool and sequences (rounded up to a CTA's) are counted in 32 bits
    if (max_pages > 0x7fffffff / page_size || n_pages > 0x7fffffff / page_size || batch > 1 << 30) return TQ_ERR_UNSUPPORTED;
    if (batch == 0) return TQ_OK;
    if (batch > 1 && table_stride < max_pages) return TQ_ERR_ARG;
    if (!length || !count || !n_free || (max_pages > 0 && !table) || (n_pages > 0 && !free_pages)) return TQ_ERR_ARG;
    if (!aligned(table, 4) || !aligned(length, 4) || !aligned(count, 4) || !aligned(free_pages, 4) || !aligned(n_free, 4))
        return TQ_ERR_ALIGN;
    return TQ_OK;
}

// The classes of a view's heads, their workers and the workspace's areas.
struct PagedLayout {
    int n_classes;
    PagedClass cls[kPagedClasses];
    size_t first_off, part_off, total;
};

tq_status check_paged_view(const tq_layer_view *lv, int B, int H, int Hq, int d, bool check_ptrs) {
    if (!lv || B < 1 || H < 1 || H > TQ_MAX_HEADS || Hq < H || Hq % H) return TQ_ERR_ARG;
    if (d < 16 || d > TQ_MAX_HEAD_DIM || (d & (d - 1))) return TQ_ERR_ARG;
    if (lv->n_segments < 0 || lv->n_segments > TQ_MAX_SEGMENTS || lv->rot.head_dim != d) return TQ_ERR_ARG;
    if (lv->rot.dense) return TQ_ERR_UNSUPPORTED;
    for (int i = 0; i < lv->n_segments; ++i) {
        const tq_segment &sg = lv->seg[i];
        const tq_status st = check_segment(&sg, check_ptrs);
        if (st != TQ_OK) return st;
        const tq_segment_layout &L = sg.layout;
        if (L.n_heads != H || L.head_dim != d) return TQ_ERR_ARG;
        if (sg.attn_mass) return TQ_ERR_UNSUPPORTED;
        if (sg.kind == TQ_SEG_PACKED) {
            if (any_sketch(L) || sphere_elsewhere(L)) return TQ_ERR_UNSUPPORTED;
            if (L.capacity % 16) return TQ_ERR_ALIGN;
        }
    }
    // query rows are counted in 32 bits (rounded up to a CTA's)
    return Hq > (0x7fffffff - 64) / B ? TQ_ERR_UNSUPPORTED : TQ_OK;
}

tq_status paged_layout(const tq_layer_view *lv, int B, int H, int Hq, int d, PagedLayout &o) {
    const int g = Hq / H;
    o.n_classes = 0;
    for (int i = 0; i < lv->n_segments; ++i) {
        const tq_segment &sg = lv->seg[i];
        const bool packed = sg.kind == TQ_SEG_PACKED;
        for (int h = 0; h < H; ++h) {
            const int kb = packed ? sg.layout.kbits[h] : 0, vb = packed ? sg.layout.vbits[h] : 0;
            const int law = packed ? sg.layout.value_law : 0;
            int k = 0;
            while (k < o.n_classes && (o.cls[k].kb != kb || o.cls[k].vb != vb || o.cls[k].law != law)) ++k;
            PagedClass &c = o.cls[k];
            if (k == o.n_classes) {
                if (k == kPagedClasses) return TQ_ERR_UNSUPPORTED;
                std::memset(&c, 0, sizeof(c));
                c.kb = kb, c.vb = vb, c.law = law;
                const PagedShape s = paged_shape(d, packed);
                c.R = s.rows;
                c.n_rb = (g + s.rows - 1) / s.rows;
                c.unit = s.unit;
                c.workers = s.workers;
                ++o.n_classes;
            }
            if (c.n == 0 || c.seg[c.n - 1] != i) {
                c.seg[c.n] = static_cast<uint8_t>(i);
                c.heads[c.n++] = 0;
            }
            c.heads[c.n - 1] |= static_cast<uint16_t>(1u << h);
        }
    }
    int64_t floats = 0;
    for (int k = 0; k < o.n_classes; ++k) {
        PagedClass &c = o.cls[k];
        c.part0 = floats;
        floats += (c.workers + static_cast<int64_t>(B) * H * c.n_rb) * c.R * (d + 4);
    }
    o.first_off = 256;  // the error flag has the first 256 bytes
    o.part_off = (o.first_off + sizeof(int) * o.n_classes * (static_cast<size_t>(B) + 1) + 255) / 256 * 256;
    o.total = o.part_off + static_cast<size_t>(floats) * sizeof(float);
    return TQ_OK;
}

}  // namespace

extern "C" {

tq_status tq_page_tables(int batch, int page_size, int max_pages, int n_pages, int *table, int64_t table_stride_b, int *length,
                         const int *n_new, int n_max, int *free_pages, int *n_free, int *slots, int *positions, int *granted,
                         void *stream) {
    if (n_max < 0) return TQ_ERR_ARG;
    const tq_status st = check_pages(batch, page_size, max_pages, n_pages, table, table_stride_b, length, n_new, free_pages, n_free);
    if (st != TQ_OK || batch == 0) return st;
    if (!granted) return TQ_ERR_ARG;
    if (!aligned(slots, 4) || !aligned(positions, 4) || !aligned(granted, 4)) return TQ_ERR_ALIGN;
    PageParams p;
    std::memset(&p, 0, sizeof(p));
    p.B = batch, p.page = page_size, p.width = max_pages, p.n_pages = n_pages, p.n_max = n_max;
    p.table = table, p.table_stride = table_stride_b;
    p.length = length, p.count = n_new;
    p.free_pages = free_pages, p.n_free = n_free;
    p.slots = slots, p.positions = positions, p.granted = granted;
    return launched(launch_page_tables(p, static_cast<cudaStream_t>(stream)));
}

tq_status tq_page_release(int batch, int page_size, int max_pages, int n_pages, const int *table, int64_t table_stride_b,
                          int *length, const int *keep, int *free_pages, int *n_free, void *stream) {
    const tq_status st = check_pages(batch, page_size, max_pages, n_pages, table, table_stride_b, length, keep, free_pages, n_free);
    if (st != TQ_OK || batch == 0) return st;
    PageParams p;
    std::memset(&p, 0, sizeof(p));
    p.B = batch, p.page = page_size, p.width = max_pages, p.n_pages = n_pages;
    p.table = const_cast<int *>(table), p.table_stride = table_stride_b;
    p.length = length, p.count = keep;
    p.free_pages = free_pages, p.n_free = n_free;
    return launched(launch_page_release(p, static_cast<cudaStream_t>(stream)));
}

tq_status tq_paged_workspace_size(const tq_layer_view *pools, int batch, int n_heads, int q_heads, int head_dim, size_t *bytes) {
    if (!bytes) return TQ_ERR_ARG;
    tq_status st = check_paged_view(pools, batch, n_heads, q_heads, head_dim, false);
    if (st != TQ_OK) return st;
    PagedLayout o;
    st = paged_layout(pools, batch, n_heads, q_heads, head_dim, o);
    if (st == TQ_OK) *bytes = o.total;
    return st;
}

tq_status tq_paged_attention(const tq_layer_view *pools, const tq_pages *pages, int batch, int n_heads, int q_heads, int head_dim,
                             const void *q, const int64_t *q_stride, void *out, void *workspace, size_t ws_bytes, void *stream) {
    tq_status st = check_paged_view(pools, batch, n_heads, q_heads, head_dim, true);
    if (st != TQ_OK) return st;
    if (!q || !q_stride || !out || !workspace || (pools->n_segments > 0 && !pages)) return TQ_ERR_ARG;
    if (!aligned(q, 2) || !aligned(out, 16) || !aligned(workspace, 16)) return TQ_ERR_ALIGN;
    PagedParams p;
    std::memset(&p, 0, sizeof(p));
    p.list.B = batch;
    p.list.H = n_heads;
    for (int i = 0; i < pools->n_segments; ++i) {
        const tq_segment &sg = pools->seg[i];
        const tq_pages &pg = pages[i];
        if (!aligned(pg.table, 4) || !aligned(pg.len, 4)) return TQ_ERR_ALIGN;
        PagedSeg &s = p.seg[i];
        s.seg = seg_view(&sg);
        s.n_pages = sg.layout.batch;
        s.page = sg.layout.capacity;
        int limit;  // most tokens a sequence can hold
        if (pg.table) {
            if (pg.max_pages < 0 || pg.table_stride_b < 0 || (batch > 1 && pg.table_stride_b < pg.max_pages) || !pg.len)
                return TQ_ERR_ARG;
            if (s.page > 0 && pg.max_pages > 0x7fffffff / s.page) return TQ_ERR_UNSUPPORTED;
            // bytes of a page in 32 bits
            if ((s.seg.kblock | s.seg.vblock | (static_cast<uint64_t>(n_heads) * s.page * 4)) >> 32) return TQ_ERR_UNSUPPORTED;
            s.table = pg.table;
            s.table_stride = pg.table_stride_b;
            limit = pg.max_pages * s.page;
        } else {  // a page a sequence
            if (sg.layout.batch != batch) return TQ_ERR_ARG;
            if (sg.n_tokens < 0 || sg.n_tokens > sg.layout.capacity) return TQ_ERR_SIZE;
            limit = sg.n_tokens;
        }
        // 2^shift / page rounded up, shift = 31 + ceil(log2 page): the excess times t stays below 2^shift / page
        s.shift = 31;
        while (s.page > 1 && (1LL << (s.shift - 31)) < s.page) ++s.shift;
        if (s.page > 0) s.magic = static_cast<uint32_t>(((1ULL << s.shift) + s.page - 1) / s.page);
        if (limit > 0x7fffffff - 1024) return TQ_ERR_UNSUPPORTED;  // rounded up to stages in 32 bits
        p.list.len[i] = pg.len;
        p.list.limit[i] = limit;
    }
    PagedLayout o;
    st = paged_layout(pools, batch, n_heads, q_heads, head_dim, o);
    if (st != TQ_OK) return st;
    if (ws_bytes < o.total) return TQ_ERR_SIZE;
    int64_t most[kPagedClasses];  // stages at the limits
    for (int k = 0; k < o.n_classes; ++k) {
        PagedClass &c = o.cls[k];
        most[k] = 0;
        for (int i = 0; i < c.n; ++i)
            most[k] += static_cast<int64_t>(__builtin_popcount(c.heads[i])) * ((p.list.limit[c.seg[i]] + c.unit - 1) / c.unit);
        if (most[k] > 0x7fffffff / (static_cast<int64_t>(batch) * c.n_rb)) return TQ_ERR_UNSUPPORTED;
        most[k] *= static_cast<int64_t>(batch) * c.n_rb;
        c.workers = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(c.workers, most[k])));
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.g = q_heads / n_heads;
    p.d = head_dim;
    p.q = static_cast<const uint16_t *>(q);
    p.qs[0] = q_stride[0], p.qs[1] = q_stride[1];
    p.part = reinterpret_cast<float *>(ws + o.part_off);
    std::memcpy(p.sign_bits, pools->rot.sign_bits, sizeof(p.sign_bits));
    p.inv_sqrt_d = rotation_scale(head_dim);
    p.qk_scale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(head_dim)));
    PagedMergeParams m;
    std::memset(&m, 0, sizeof(m));
    m.list = p.list;
    m.n_classes = o.n_classes;
    m.g = p.g, m.d = head_dim;
    m.out = static_cast<uint16_t *>(out);
    m.part = p.part;
    m.first = reinterpret_cast<int *>(ws + o.first_off);
    m.error = reinterpret_cast<int *>(ws);
    std::memcpy(m.sign_bits, p.sign_bits, sizeof(m.sign_bits));
    m.inv_sqrt_d = p.inv_sqrt_d;
    std::copy(o.cls, o.cls + o.n_classes, m.cls);
    try {  // the codebooks before anything is launched
        for (int k = 0; k < o.n_classes; ++k) {
            const uint8_t vb = static_cast<uint8_t>(o.cls[k].vb);
            if (vb) value_centroids(p.centroid, &vb, 1, o.cls[k].law);
        }
    } catch (...) {
        return TQ_ERR_SIZE;  // no host memory for the codebook fit
    }
    for (int k = 0; k < o.n_classes; ++k) {
        p.cls = o.cls[k];
        const uint8_t vb = static_cast<uint8_t>(p.cls.vb);
        if (vb) value_centroids(p.centroid, &vb, 1, p.cls.law);
        p.first = const_cast<int *>(m.first) + static_cast<size_t>(k) * (batch + 1);
        p.first_class = k == 0;
        st = launched(launch_paged(p, static_cast<cudaStream_t>(stream)));
        if (st != TQ_OK) return st;
    }
    return launched(launch_paged_merge(m, static_cast<cudaStream_t>(stream)));
}

tq_status tq_verify(const tq_verification *v, void *stream) {
    if (!v || v->batch < 0 || v->n_drafts < 0 || v->n_drafts > TQ_MAX_DRAFTS || v->vocab < 1 || v->dtype < TQ_DTYPE_F16 ||
        v->dtype > TQ_DTYPE_F32)
        return TQ_ERR_ARG;
    if (v->vocab > 1 << 30 || v->batch > 1 << 24) return TQ_ERR_UNSUPPORTED;  // (vectors and blocks in 32 bits)
    if (v->batch == 0) return TQ_OK;
    if (!v->target || !v->uniform || !v->n_accepted || !v->token || (v->n_drafts > 0 && (!v->tokens || !v->accepted)))
        return TQ_ERR_ARG;
    const size_t elem = v->dtype == TQ_DTYPE_F32 ? 4 : 2;
    if (!aligned(v->target, elem) || !aligned(v->draft, elem) || !aligned(v->tokens, 4) || !aligned(v->parents, 4) ||
        !aligned(v->uniform, 4) || !aligned(v->accepted, 4) || !aligned(v->n_accepted, 4) || !aligned(v->token, 4))
        return TQ_ERR_ALIGN;
    VerifyParams p;
    std::memset(&p, 0, sizeof(p));
    p.B = v->batch, p.N = v->n_drafts, p.V = v->vocab;
    p.tokens = v->tokens, p.tokens_stride = v->tokens_stride_b;
    p.parents = v->parents, p.parents_stride = v->parents_stride_b;
    p.target = v->target, p.draft = v->draft;
    for (int i = 0; i < 2; ++i) p.ts[i] = v->target_stride[i], p.ds[i] = v->draft_stride[i];
    p.uniform = v->uniform, p.uniform_stride = v->uniform_stride_b;
    p.accepted = v->accepted, p.n_accepted = v->n_accepted, p.token = v->token;
    return launched(launch_verify(p, v->dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
