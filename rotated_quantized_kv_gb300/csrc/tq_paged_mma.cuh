// tq_paged_mma.cuh -- attention of one new token over paged segments at head dims 64 and 128: the
// kernel, and its form for packed pages, specialised by (key bits, value bits).
//
// The arithmetic of a tile is that of decode attention (tq_decode_packed.cuh: raw key codes as
// fp16 subnormals against the query's hi and lo parts, values by table into the P.V product,
// mma.m16n8k16).  What differs:
//   - the eight columns of the P.V product are four query heads' weights as fp16 hi + 2^-11 lo (22 bits, down to
//     2^-36 of the row's largest);
//   - head_dim 64: a tile row is a pair of tokens read as one record of 128 dims, and the four columns
//     are two heads times two parities, a query with zeros in the other token's half, so that a (head, parity) is a
//     head of its own until the record;
//   - weights are relative to the row's largest weighted value, as in tq_tree_mma.cu: the running
//     maximum is that of S + log2 sigma (sigma from 2^-64 up, its logarithm read off the bits: at most 0.09 below), so
//     that fp16 holds the weights that count whatever the values' sizes;
//   - value levels are fp16 operands, scaled together so that they round closely (value_levels): beside the result's own
//     fp16 rounding (2.07e-4 of it) the error against 64 bits is 2.09, 2.12, 2.13, 2.27, 2.38, 2.53 and 2.7e-4 at 2 to
//     8 bits, 3000 tokens; a second part of the levels would double the products and the tables;
//   - sums leave the tensor cores every kFold tiles: mma.sync adds with truncation, relative to the largest
//     of what it adds.  They go to the warp's copy in shared memory, by binary32 additions.
//
// Every warp is a worker of its own: a range of the stage list (tq_paged.cuh), a ring of stages that it fills
// itself by cp.async, its queries, its sums, its records; warps meet nowhere behind the prologue, and nothing waits but for
// its own copies.  (Measured against it: CTAs of four warps that share a stage, the warps issuing bulk copies in turn, then
// teams of four warps with a loader warp each by bulk copies and by cp.async: the loader's serial instructions, some
// 2000 cycles a stage, and the barriers bounded all of these, 145 us on the first case below.)  Twelve
// warps an SM are what 168 registers leave (14 and 16 with fewer registers: no faster); they share one value table, a
// column a lane.
//
// Bound by instruction issue and the latency of dependent instructions at K1 to K8, by memory at fp16: whole calls, 4
// query heads a KV head, 64-token pages, 8 KV heads, a copy being 6677 GB/s: 32 x 16384 K4V4 118 us (4.82 TB/s; pages
// of 48 and 16 tokens, whose stages come from several pages: 125 and 135 us), 32 x 32768 K4V4 211 us (5.42), K3V3 248 us
// (3.53), 32 x 16384 fp16 336 us (6.40), 32 x 9000 at d = 64, two heads a KV head, K8V3 57 us (3.88; pages of 16: 62 us).
#pragma once

#include <algorithm>
#include <type_traits>

#include "tq_decode_packed.cuh"
#include "tq_paged.cuh"

namespace tqk {
namespace pmma {

using namespace dec;

constexpr int kWarps = kPagedWarps;
constexpr int kPagedThreads = 32 * kWarps;
constexpr int kFold = 16;               // tiles of 16 rows between folds
constexpr int kMaxRing = 6;
// Floats of a head's copy of the sums (heads apart in banks), and bytes of a warp's four.
__host__ __device__ constexpr int copy_stride(int d) { return d + 4; }
__host__ __device__ constexpr int copy_bytes(int d) { return 4 * copy_stride(d) * 4; }
constexpr int kSmemMax = 232448;

// Value levels of the class: fp16(s c_k), 1/s, and level 1 of a 1-bit codebook.
struct Levels {
    unsigned short half[256];
    float inv, c1;
};

// 16 bytes into shared memory; a cache that is read once streams through L2: evicted first.
__device__ __forceinline__ void copy16(unsigned dst, const void *src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ uint64_t policy_for(bool once) {
    uint64_t first, normal;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
    return once ? first : normal;
}

// What a special stage of the ring is.
struct alignas(16) Stage {
    int word;            // tokens, and kFresh (another sequence, head or block of rows), kPart (not whole)
    int b, block;        // sequence; KV head and block of rows as h n_rb + rb
    unsigned bad;        // kPart: bit i: the i-th page of it is outside the pool
    int page, skip;      // kPart: tokens a page, and tokens of the first page before the stage
    int pad[2];
};
constexpr int kFresh = 1 << 16, kPart = 1 << 17;

// A warp's running state: lane (g, c) has head c of its four; columns 2c, 2c + 1 of the
// accumulator are that head's hi and lo parts.
template <int MT>
struct Run {
    float m, mt;         // reference of the weights; the maximum of S + log2 sigma (+ 127)
    float l, w;          // sums of p, and of p sigma since the last fold (of the lane's rows: even or odd ones)
    float m_ref;         // reference of the copy
    float acc[MT][4];
    int tiles;           // since the last fold
    bool some;           // the copy holds something
    __device__ __forceinline__ float sum(int mt_, int k) const { return fmaf(acc[mt_][2 * k + 1], 0x1p-11f, acc[mt_][2 * k]); }
    __device__ __forceinline__ void clear() {
        w = 0.f;
        tiles = 0;
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int k = 0; k < 4; k++) acc[i][k] = 0.f;
    }
    // The reference, or that there is none yet: no score, or only scores of minus infinity, whose weights are 0 at
    // any finite m (against a reference of minus infinity they would be NaN).
    __device__ __forceinline__ float reference() const { return mt == kNegInf ? kNegInf : m; }
    __device__ __forceinline__ void start() {
        m = 0.f;
        mt = m_ref = kNegInf;
        l = 0.f;
        some = false;
        clear();
    }
};

// Online softmax of T tiles of 16 rows: s (base-2 scores) and v (value scales) of rows g, g + 8 of each for
// head c, and the B fragments of the weights: column n is head n / 2, the hi part (n even) or 2^11 times the lo one.
template <bool FULL, int T, int MT>
__device__ __forceinline__ void softmax(Run<MT> &r, const float (&s)[2 * T], const bool (&ok)[2 * T], const float (&v)[2 * T], int g,
                                        int c, uint32_t sel, uint32_t (&b)[2 * T]) {
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < 2 * T; i++) {
        // log2 v + 127, less up to 0.09: the exponent, and the mantissa as its fraction
        const float lg = static_cast<float>(__float_as_int(fmaxf(v[i], 0x1p-64f)));
        const float t = fmaf(lg, 0x1p-23f, s[i]);
        top = fmaxf(top, FULL || ok[i] ? t : kNegInf);
    }
    if (__any_sync(0xffffffffu, top > r.mt + 8.0f)) {
        const float now = fmaxf(r.mt, warp_max_g(top));
        const float f = now == kNegInf ? 1.f : ex2(r.mt - now);
        r.mt = now;
        r.m = now == kNegInf ? 0.f : now - 127.f;
        r.l *= f;
        r.w *= f;
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int k = 0; k < 4; k++) r.acc[i][k] *= f;
    }
    const int src = 8 * c + (g >> 1);
#pragma unroll
    for (int t = 0; t < T; t++) {
        float w[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int i = 2 * t + k;
            const float p = FULL || ok[i] ? ex2(s[i] - r.m) : 0.f;
            r.l += p;
            w[k] = FULL || ok[i] ? p * v[i] : 0.f;  // (a select: the scales of what is masked may be anything)
        }
        r.w += w[0] + w[1];
        const __half2 hi = __floats2half2_rn(w[0], w[1]);
        const float2 f = __half22float2(hi);
        const __half2 lo = __floats2half2_rn((w[0] - f.x) * 2048.f, (w[1] - f.y) * 2048.f);
        const uint32_t h = *reinterpret_cast<const uint32_t *>(&hi), o = *reinterpret_cast<const uint32_t *>(&lo);
        const uint32_t x0 = prmt(h, o, 0x5410u), x1 = prmt(h, o, 0x7632u);  // (hi, lo) of rows g, g + 8
        b[2 * t] = prmt(__shfl_sync(0xffffffffu, x0, src), __shfl_sync(0xffffffffu, x0, src + 4), sel);
        b[2 * t + 1] = prmt(__shfl_sync(0xffffffffu, x1, src), __shfl_sync(0xffffffffu, x1, src + 4), sel);
    }
}

// Four query rows of a block (those behind the last head: zeros), as fp16 hi and lo parts [row][part][D] of R q 2^-e, and
// in lane i of the warp row i's sum and 2^e (the largest coordinate in [0.5, 1)).  Four at once: their shuffles overlap.
template <int D>
__device__ __forceinline__ void rotate_queries(const PagedParams &p, __half *to, int b, int h, int rb, int lane, float &qsum, float &qexp) {
    constexpr int J = D / 32;
    float x[4][J], sum[4], top[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int row = rb * p.cls.R + i;
        const uint16_t *q = p.q + b * p.qs[0] + (static_cast<int64_t>(h) * p.g + row) * p.qs[1] + lane;
#pragma unroll
        for (int j = 0; j < J; j++) x[i][j] = i < p.cls.R && row < p.g ? __half2float(__ushort_as_half(q[32 * j])) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < J; j++)
        if ((p.sign_bits[j] >> lane) & 1u) {
#pragma unroll
            for (int i = 0; i < 4; i++) x[i][j] = -x[i][j];
        }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int j = 0; j < J; j++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float y = __shfl_xor_sync(0xffffffffu, x[i][j], o);
                x[i][j] = up ? y - x[i][j] : x[i][j] + y;
            }
    }
#pragma unroll
    for (int o = 1; o < J; o <<= 1)
#pragma unroll
        for (int j = 0; j < J; j++)
            if (!(j & o)) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float a = x[i][j], y = x[i][j + o];
                    x[i][j] = a + y;
                    x[i][j + o] = a - y;
                }
            }
#pragma unroll
    for (int i = 0; i < 4; i++) sum[i] = top[i] = 0.f;
#pragma unroll
    for (int j = 0; j < J; j++) {
        const float f = ((p.sign_bits[j] >> lane) & 1u) ? -p.inv_sqrt_d : p.inv_sqrt_d;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[i][j] *= f;
            sum[i] += x[i][j];
            top[i] = fmaxf(top[i], fabsf(x[i][j]));
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
        }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        // (rotated fp16 coordinates reach 2^21, the least is 2^-28; a row of zeros or of what is no number: e = 0)
        int e = 0;
        if (top[i] > 0.f && top[i] < 0x1p100f) e = static_cast<int>(__float_as_uint(top[i]) >> 23) - 126;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int j = 0; j < J; j++) {
            const float y = x[i][j] * down;
            const __half hi = __float2half_rn(y);
            to[2 * i * D + lane + 32 * j] = hi;
            to[(2 * i + 1) * D + lane + 32 * j] = __float2half_rn(y - __half2float(hi));
        }
        if (lane == i) {
            qsum = sum[i];
            qexp = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        }
    }
}

// The pages of a segment, sequence and head, and the place of the next stage in them.
struct Source {
    const uint8_t *k, *v;
    const char *s;                         // scales: keys' for the first half of the warp, values' for the second
    uint32_t kblock, vblock, sblock;       // bytes a page (below 2^32: the host checks; without a table: 0)
    int page, n_pages, last;               // tokens a page; pages of the pool; the sequence's last page (-1: none)
    int index, left;                       // page of the stage's first token, and tokens of it from there on
    bool good;                             // that page is in the pool
    const uint8_t *ka, *va;                // the lane's 16 bytes of the stage
    const char *sa;
    paged::Pages pages;
    template <class F>
    static __device__ __noinline__ Source open(const PagedParams &p, paged::Walk w, int lane) {
        Source o;
        const PagedSeg &g = p.seg[p.cls.seg[w.i]];
        const SegView &x = g.seg;
        const size_t sc = static_cast<size_t>(w.h) * x.capacity * 4, sb = static_cast<size_t>(p.list.H) * x.capacity * 4;
        o.k = x.k + x.koff[w.h] + 16 * lane, o.v = x.v + x.voff[w.h] + 16 * lane;
        o.s = reinterpret_cast<const char *>(lane < 16 ? x.ks : x.vs) + sc + 16 * (lane & 15);
        if (g.table) {
            o.kblock = static_cast<uint32_t>(x.kblock), o.vblock = static_cast<uint32_t>(x.vblock), o.sblock = static_cast<uint32_t>(sb);
            o.n_pages = g.n_pages;
        } else {  // (no pages: entry 0 of them)
            o.k += w.b * x.kblock, o.v += w.b * x.vblock, o.s += w.b * sb;
            o.kblock = o.vblock = o.sblock = 0;
            o.n_pages = p.list.B;
        }
        o.page = g.page;
        o.last = w.tokens > 0 ? paged::page_index(g, w.tokens - 1) : -1;
        o.index = paged::page_index(g, w.st * F::PT);
        o.pages.open(g, w.b, o.last, o.index, lane);
        o.point<F>(w);
        return o;
    }
    // The addresses of page `page_` from its token `skip` on.  (In 64 bits: a segment without a table is one page of any size.)
    template <class F>
    __device__ __forceinline__ void aim(uint32_t page_, uint32_t skip, const uint8_t *&ka_, const uint8_t *&va_, const char *&sa_) const {
        ka_ = k + static_cast<uint64_t>(page_) * kblock + static_cast<uint64_t>(skip) * F::kTokenK;
        va_ = v + static_cast<uint64_t>(page_) * vblock + static_cast<uint64_t>(skip) * F::kTokenV;
        sa_ = s + static_cast<uint64_t>(page_) * sblock + static_cast<uint64_t>(skip) * 4u;
    }
    // At page `index`, for the stage at w.
    template <class F>
    __device__ __forceinline__ void point(const paged::Walk &w) {
        const int skip = w.st * F::PT - index * page;
        const uint32_t at = static_cast<uint32_t>(pages.at(index));
        left = page - skip;
        good = at < static_cast<uint32_t>(n_pages);
        aim<F>(at, static_cast<uint32_t>(skip), ka, va, sa);
    }
    // On to the next stage of the same.
    template <class F>
    __device__ __forceinline__ void step(const PagedParams &p, const paged::Walk &w, int lane) {
        left -= F::PT;
        ka += F::PT * F::kTokenK;
        va += F::PT * F::kTokenV;
        sa += F::PT * 4;
        if (left > 0) return;
        const PagedSeg &g = p.seg[p.cls.seg[w.i]];
        index = paged::page_index(g, w.st * F::PT);
        pages.move(g, w.b, last, index, lane);
        point<F>(w);
    }
};

// A warp's attention over its range, in the form F:
//   D, R, MT                    dims, query rows, m-tiles of the sums
//   PT, kSlot, kTable           tokens and bytes of a stage, bytes of the CTA's table
//   kTokenK, kTokenV            bytes of a token's rows
//   fill_all(...), fill(...)    a whole stage, a run of tokens of a page into the slot; clear(...): a slot that will not be full
//   fill_blocks(...)            a whole stage from several pages, where the form has a way of its own
//   queries(...), stage(...)    a block's queries; the tiles of a stage
//   fold(...), record(...)      the sums into the copy, the copy into the record
// What a stage costs beside its tiles is kept short: addresses move by constants inside a page, and only stages that
// begin a block or are not whole (special) have a description in shared memory.
template <class F, int NS>
__device__ __forceinline__ void attend(const PagedParams &p, F &f, int worker, int n_st, int b0, int rest, uint8_t *mine, float *copy, int lane) {
    const PagedList &l = p.list;
    const uint32_t sel = (lane & 4) ? 0x7632u : 0x5410u;
    const uint64_t pol = policy_for(p.cls.n_rb == 1);
    Stage *stages = reinterpret_cast<Stage *>(mine + NS * F::kSlot);
    paged::Walk w = paged::seek(l, p.cls, b0, rest);
    Source src = Source::open<F>(p, w, lane);
    unsigned special = 0;                // bit i: the i-th last of the stages sent for
    int to = 0;                          // slot of the next stage to fill
    auto fill = [&](int j) {             // stage j, the one at `w`
        const unsigned slot = smem_u32(mine + to * F::kSlot);
        const int n = max(min(F::PT, w.tokens - w.st * F::PT), 0);
        bool whole = n == F::PT;
        if (__builtin_expect(whole && src.left >= F::PT && src.good, 1)) {
            F::fill_all(src, slot, pol, lane);
        } else if (whole && F::fill_blocks(p, src, w, slot, pol, lane)) {
        } else {                         // its end, or several pages: page i to lane i
            const uint32_t pages = static_cast<uint32_t>(src.pages.at(src.index + lane));
            const bool used = lane == 0 ? n > 0 : src.left + (lane - 1) * min(src.page, F::PT) < n;
            const unsigned bad = __ballot_sync(0xffffffffu, used && pages >= static_cast<uint32_t>(src.n_pages));
            whole = whole && bad == 0;
            if (!whole) F::clear(mine + to * F::kSlot, lane);
            int skip = src.page - src.left;
#pragma unroll 1
            for (int from = 0, i = 0; from < n; i++) {
                const int run = min(src.page - skip, n - from);
                const uint32_t page = __shfl_sync(0xffffffffu, pages, i);
                const uint8_t *ka, *va;
                const char *sa;
                src.aim<F>(page, static_cast<uint32_t>(skip), ka, va, sa);
                if (!((bad >> i) & 1u)) F::fill(ka, va, sa, slot, from, run, pol, lane);
                from += run;
                skip = 0;
            }
            if (!whole && lane == 0) {
                stages[to].bad = bad;
                stages[to].page = src.page;
                stages[to].skip = src.page - src.left;
            }
        }
        if (w.fresh || !whole) {
            special |= 1u;
            if (lane == 0) {
                stages[to].word = n | (w.fresh ? kFresh : 0) | (whole ? 0 : kPart);
                stages[to].b = w.b;
                stages[to].block = w.h * p.cls.n_rb + w.rb;
            }
        }
        if (++to == NS) to = 0;
        w.fresh = false;
        if (++w.st < w.n_st) {
            src.step<F>(p, w, lane);
        } else if (j + 1 < n_st) {
            w = paged::next(l, p.cls, w);
            src = Source::open<F>(p, w, lane);
            if (w.fresh) {  // its queries into the cache
                const int row = w.rb * p.cls.R + (lane >> 1);
                if (lane < 2 * p.cls.R && row < p.g)
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + w.b * p.qs[0] + (static_cast<int64_t>(w.h) * p.g + row) * p.qs[1] + (lane & 1) * (F::D / 2)));
            }
        }
    };
    Run<F::MT> r;
    auto fold = [&]() {
        const float W = F::kLinear ? warp_sum_g(lane & 4 ? -r.w : r.w) : 0.f;  // even rows' less odd rows'
        const float scale = r.m_ref == r.m ? 1.f : ex2(r.m_ref - r.m);
        f.fold(r, copy, W, scale, lane);
        r.m_ref = r.reference();
        r.some = true;
        r.clear();
    };
    int now_b = 0, now_block = 0, at = 0;
    // one pass more than stages (k = n_st), so that a block ends in one place
#pragma unroll 1
    for (int k = 1 - NS; k <= n_st; k++) {  // (below 0: stages on their way first)
        special <<= 1;
        if (k + NS - 1 < n_st) fill(k + NS - 1);
        cp_async_commit();
        if (k < 0) continue;
        cp_async_wait<NS - 1>();
        __syncwarp();
        int word = F::PT;
        if (__builtin_expect(((special >> (NS - 1)) & 1u) || k == n_st, 0)) {
            word = k < n_st ? stages[at].word : kFresh;
            if (word & kFresh) {
                if (k > 0) {
                    fold();
                    const float sum = warp_sum_g(r.l);
                    __syncwarp();
                    F::record(p.part + p.cls.part0 + paged::group_slot(l, p.cls, worker, now_b, 0, now_block) * F::R * (F::D + 4), copy,
                              r.reference(), sum, lane);
                    __syncwarp();
                }
                if (k == n_st) break;
                now_b = stages[at].b;
                now_block = stages[at].block;
                const int h = now_block / p.cls.n_rb;
                f.queries(p, reinterpret_cast<__half *>(copy), now_b, h, now_block - h * p.cls.n_rb, lane);
                __syncwarp();
                r.start();
            }
        }
        const uint8_t *buf = mine + at * F::kSlot;
        if (!(word & kPart)) f.stage(r, buf, F::PT, stages[at], sel, lane, std::true_type{});
        else f.stage(r, buf, word & (kFresh - 1), stages[at], sel, lane, std::false_type{});
        __syncwarp();
        if (++at == NS) at = 0;
        if (__builtin_expect(r.tiles >= kFold, 0)) fold();
    }
}

// Whether token `tok` of a stage is there.
__device__ __forceinline__ bool have_token(const Stage &sg, int tok, int n) {
    return tok < n && !(sg.bad && ((sg.bad >> ((sg.skip + tok) / sg.page)) & 1u));
}

template <class F>
struct Ring {
    static constexpr int slot = F::kSlot + static_cast<int>(sizeof(Stage));
    static constexpr int fit = ((kSmemMax - 256 - F::kTable) / kWarps - copy_bytes(F::D)) / slot;
    static constexpr int NS = fit > kMaxRing ? kMaxRing : fit;
    static constexpr int warp_bytes = NS * slot + copy_bytes(F::D);
    static constexpr int smem = F::kTable + kWarps * warp_bytes;
    static_assert(NS >= 2, "a stage on its way beside the one at work");
};

template <class F, int NS>
__global__ void __launch_bounds__(kPagedThreads, 1) paged_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ Levels lv) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int bufs[kWarps + 4 * kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int worker = warp * gridDim.x + blockIdx.x;  // (few stages go to as many SMs)
    const paged::Share<kPagedThreads> share(p.list, p.cls);
    pdl_launch_dependents();
    F::fill_table(smem, lv);
    paged::ranges_of<kPagedThreads, kWarps>(p.list, p.cls, share, blockIdx.x, gridDim.x, p.first, bufs);  // (synchronises)
    const int *range = bufs + kWarps + 4 * warp;
    const int begin = range[2], end = range[3];
    if (begin < end) {
        uint8_t *mine = smem + F::kTable + warp * Ring<F>::warp_bytes;
        F f(smem, lv, lane);
        attend<F, NS>(p, f, worker, end - begin, range[0], range[1], mine,
                      reinterpret_cast<float *>(mine + NS * Ring<F>::slot), lane);
    }
    pdl_wait();  // the call's last launch ends behind its first
}

template <class F>
cudaError_t launch(const PagedParams &p, const Levels &lv, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(paged_kernel<F, Ring<F>::NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<F>::smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(p.cls.workers, current_sm_count())));
    cfg.blockDim = dim3(kPagedThreads);
    cfg.dynamicSmemBytes = Ring<F>::smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.first_class ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, paged_kernel<F, Ring<F>::NS>, p, lv);
}

// ------------------------------------------------------------------- packed
// 1-bit values: a set bit of fp16's exponent field (bits 10 to 14) is a normal number by itself, so that a code is one mask
// away from its word.  Even rows enter as b, odd rows as b - 1 (1 - b against negative weights): what is left to add is the even
// rows' weights less the odd rows', and the sums are no larger than what they are the sums of.  (As subnormals, bits 0
// to 9, the tensor cores align products by the exponent that all subnormals share, up to 10 bits off: weights that
// differ had errors of 3.3e-4 of the result, 30000 tokens, on top of fp16's own 2.1e-4, at 104 us for the 108 us of 32
// x 16384 tokens K4V1 here; +-1 by the sign bit takes a shift a code: 122 us.)
struct Bits1 {
    static constexpr bool kLinear = true;
    static constexpr __host__ __device__ int dim(int mt, int r) { return mt + 8 * r; }
    // the place of code j in its word
    static constexpr __host__ __device__ int place(int j) { return j < 5 ? j + 10 : j < 10 ? j + 5 : j < 15 ? j : 14; }
    static __device__ __forceinline__ void pair(const uint8_t *p, int RV, const VCtx &cx, uint32_t (&ra)[8], uint32_t (&rb)[8]) {
        const uint32_t x = *reinterpret_cast<const uint32_t *>(p + cx.off), y = *reinterpret_cast<const uint32_t *>(p + cx.off + RV);
        const uint32_t z = prmt(x, y, static_cast<uint32_t>(cx.sh)) ^ 0xFFFF0000u;  // the even row's 16 codes | the odd row's, inverted
        const uint32_t word[4] = {z << 10, z << 5, z, z >> 1};
#pragma unroll
        for (int mt = 0; mt < 8; mt++) {
            ra[mt] = word[mt / 5] & (0x00010001u << place(mt));
            rb[mt] = word[(mt + 8) / 5] & (0x00010001u << place(mt + 8));
        }
    }
    // 1 / the value of a set bit
    static __device__ __forceinline__ float unscale(int mt, int r) {
        return __uint_as_float(static_cast<uint32_t>(127 + 15 - (1 << (place(dim(mt, r)) - 10))) << 23);
    }
};

// 4-bit values: pair table of 256 entries; E/O fields of 8 bits: dims (2mt, 2mt+1)
struct Pairs4 {
    static constexpr bool kLinear = false;
    static constexpr __host__ __device__ int dim(int mt, int r) { return 2 * mt + r; }
    // address of the entry of field K: 128 bytes an entry, the byte's product and the sum in one instruction
    template <int K>
    static __device__ __forceinline__ uint32_t at(uint32_t F, uint32_t tab) { return __dp4a(F, 128u << (8 * K), tab); }
    static __device__ __forceinline__ void pair(const uint8_t *p, int RV, const VCtx &cx, uint32_t (&ra)[8], uint32_t (&rb)[8]) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p + cx.off), y = *reinterpret_cast<const uint2 *>(p + cx.off + RV);
        constexpr uint32_t M = 0x0F0F0F0Fu;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t wx = i ? x.y : x.x, wy = i ? y.y : y.x;
            const uint32_t E = (wx & M) | ((wy << 4) & ~M), O = ((wx >> 4) & M) | (wy & ~M);
            ra[4 * i] = lds32(at<0>(E, cx.tab));
            ra[4 * i + 1] = lds32(at<1>(E, cx.tab));
            ra[4 * i + 2] = lds32(at<2>(E, cx.tab));
            ra[4 * i + 3] = lds32(at<3>(E, cx.tab));
            rb[4 * i] = lds32(at<0>(O, cx.tab));
            rb[4 * i + 1] = lds32(at<1>(O, cx.tab));
            rb[4 * i + 2] = lds32(at<2>(O, cx.tab));
            rb[4 * i + 3] = lds32(at<3>(O, cx.tab));
        }
    }
};

template <int KB, int VB, int NP>
struct Packed {
    static constexpr int D = 128 / NP, R = 4 / NP, MT = 8;
    static constexpr int ROWS = 32, PT = ROWS * NP;              // rows and tokens of a stage
    static constexpr int RK = 16 * KB, RV = 16 * VB;             // bytes of a row
    static constexpr int kKs = ROWS * (RK + RV), kVs = kKs + PT * 4, kSlot = kVs + PT * 4;
    static constexpr int entries = VB >= 2 && VB <= 4 ? 1 << (2 * VB) : 0;
    static constexpr int kTable = entries * 128 + (VB >= 5 ? 512 : 0);  // pair table: a column a lane
    using KU = KUnpack<KB>;
    using VD = typename std::conditional<VB == 1, Bits1, typename std::conditional<VB == 4, Pairs4, VDec<VB, 7>>::type>::type;
    static constexpr bool kLinear = VD::kLinear;

    VCtx vx;
    int koff;
    float inv, c1;
    uint32_t bq[16];
    float aq, bqs;

    static __device__ __forceinline__ void fill_table(uint8_t *tab, const Levels &lv) {
        if constexpr (VB >= 5)
            for (int i = threadIdx.x; i < (1 << VB); i += kPagedThreads) reinterpret_cast<unsigned short *>(tab)[i] = lv.half[i];
        if constexpr (entries > 0)
            for (int i = threadIdx.x; i < entries * 32; i += kPagedThreads) {
                const int e = i / 32;
                reinterpret_cast<uint32_t *>(tab)[i] = static_cast<uint32_t>(lv.half[e & ((1 << VB) - 1)]) |
                                                       (static_cast<uint32_t>(lv.half[e >> VB]) << 16);
            }
    }
    __device__ __forceinline__ Packed(const uint8_t *tab, const Levels &lv, int lane) : inv(lv.inv), c1(lv.c1) {
        const int g = lane >> 2, c = lane & 3;
        vx.ctab = reinterpret_cast<const unsigned short *>(tab);
        vx.tab = smem_u32(tab) + 4 * lane;
        if constexpr (VB == 1) {
            vx.off = 2 * c * RV + 4 * (g >> 1);
            vx.sh = (g & 1) ? 0x7632 : 0x5410;
        } else if constexpr (VB == 3) {
            vx.off = 2 * c * RV + 4 * ((3 * g) >> 1);
            vx.sh = (g & 1) * 16;
        } else if constexpr (VB == 4) {
            vx.off = 2 * c * RV + 16 * ((g >> 1) ^ c) + 8 * (g & 1);
        } else {
            vx.off = 2 * c * RV + ((2 * VB * g) & ~3);
            vx.sh = ((2 * VB * g) & 3) * 8;
        }
        koff = g * RK + 4 * KB * c;
    }
    static constexpr uint32_t kTokenK = RK / NP, kTokenV = RV / NP;
    static __device__ __forceinline__ void clear(uint8_t *, int) {}
    // 16-byte chunk i of a value row of 4 bits lies at i ^ (row / 2 & 3): the four row pairs that a load takes at once share
    // two bank groups instead of one (the keys' rows, and the others', meet in fewer).
    static __device__ __forceinline__ unsigned value_at(int i) { return VB == 4 ? i ^ ((i >> 3) & 3) : i; }
    static __device__ __forceinline__ unsigned value_chunk(int lane) { return 16 * value_at(lane); }
    static __device__ __forceinline__ void fill_all(const Source &s, unsigned slot, uint64_t pol, int lane) {
        const unsigned dk = slot + 16 * lane, dv = slot + ROWS * RK + value_chunk(lane);
#pragma unroll
        for (int i = 0; i < KB; i++) copy16(dk + 512 * i, s.ka + 512 * i, pol);
#pragma unroll
        for (int i = 0; i < VB; i++) copy16(dv + 512 * i, s.va + 512 * i, pol);
        if ((lane & 15) < PT / 4) copy16(slot + (lane >= 16 ? kVs : kKs) + 16 * (lane & 15), s.sa, pol);
    }
    // A whole stage from several pages: they are multiples of 16 tokens, so LB lanes take a block of 16 each, wherever it lies
    // (32 x 16384 tokens K4V4 in pages of 16: 159 us page by page).  False: not all of them are in the pool.
    static __device__ __forceinline__ bool fill_blocks(const PagedParams &p, const Source &s, const paged::Walk &w, unsigned slot, uint64_t pol,
                                                       int lane) {
        constexpr int LB = 32 * 16 / PT;
        const PagedSeg &g = p.seg[p.cls.seg[w.i]];
        const int t0 = w.st * PT;
        auto place = [&](int block, uint32_t &page, uint32_t &skip) {
            const int t = t0 + 16 * block, i = paged::page_index(g, t);
            page = static_cast<uint32_t>(s.pages.at(i));
            skip = static_cast<uint32_t>(t - i * s.page);
        };
        uint32_t page, skip;
        const uint8_t *ka, *va;
        const char *sa;
        const int block = lane / LB, l = lane % LB;
        place(block, page, skip);
        if (__any_sync(0xffffffffu, page >= static_cast<uint32_t>(s.n_pages))) return false;
        s.aim<Packed>(page, skip, ka, va, sa);
        ka -= 16 * (lane - l);
        va -= 16 * (lane - l);
        const unsigned dk = slot + block * 16 * kTokenK + 16 * l, dv = slot + ROWS * RK + block * 16 * kTokenV;
#pragma unroll
        for (int i = 0; i < KB; i++) copy16(dk + 16 * LB * i, ka + 16 * LB * i, pol);
#pragma unroll
        for (int i = 0; i < VB; i++) copy16(dv + 16 * value_at(l + LB * i), va + 16 * LB * i, pol);
        const int sl = lane & 15;        // four scales a lane
        place(min(sl / 4, PT / 16 - 1), page, skip);
        s.aim<Packed>(page, skip, ka, va, sa);
        if (sl < PT / 4) copy16(slot + (lane >= 16 ? kVs : kKs) + 16 * sl, sa - 16 * (sl & ~3), pol);
        return true;
    }
    // (runs start at multiples of 16 tokens, eight rows at least; an odd end rounds up inside the page)
    static __device__ __forceinline__ void fill(const uint8_t *k, const uint8_t *v, const char *sc, unsigned slot, int from, int run,
                                                uint64_t pol, int lane) {
        const unsigned dk = slot + from * kTokenK + 16 * lane, dv = slot + ROWS * RK + from * kTokenV + value_chunk(lane);
        const int nk = run * static_cast<int>(kTokenK) - 16 * lane, nv = run * static_cast<int>(kTokenV) - 16 * lane;
#pragma unroll 1
        for (int o = 0; o < nk; o += 512) copy16(dk + o, k + o, pol);
#pragma unroll 1
        for (int o = 0; o < nv; o += 512) copy16(dv + o, v + o, pol);
        if (4 * (lane & 15) < run) copy16(slot + (lane >= 16 ? kVs : kKs) + from * 4 + 16 * (lane & 15), sc, pol);
    }
    __device__ __forceinline__ void queries(const PagedParams &p, __half *q, int b, int h, int rb, int lane) {
        constexpr float alpha = static_cast<float>(1 << (24 - KU::kA)) * 2.0f / static_cast<float>(1 << KB);
        constexpr float beta = 1.0f / static_cast<float>(1 << KB) - 1.0f;
        float qsum = 0.f, qexp = 0.f;
        rotate_queries<D>(p, q, b, h, rb, lane, qsum, qexp);
        __syncwarp();
        const int g = lane >> 2, c = lane & 3, v = g >> 1, part = g & 1;
        const int own = NP == 2 ? c & 1 : c;
        aq = alpha * __shfl_sync(0xffffffffu, qexp, own) * p.qk_scale;
        bqs = beta * __shfl_sync(0xffffffffu, qsum, own) * p.qk_scale;
        uint32_t x[16];
        const uint4 *from = reinterpret_cast<const uint4 *>(q + (2 * (NP == 2 ? v & 1 : v) + part) * D + 32 * (NP == 2 ? c & 1 : c));
        const bool zero = NP == 2 && (v >> 1) != (c >> 1);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint4 y = from[i];
            x[4 * i] = zero ? 0u : y.x, x[4 * i + 1] = zero ? 0u : y.y, x[4 * i + 2] = zero ? 0u : y.z, x[4 * i + 3] = zero ? 0u : y.w;
        }
        gather_b<KU>(x, bq);
    }
    template <bool FULL>
    __device__ __forceinline__ void stage(Run<MT> &r, const uint8_t *buf, int n, const Stage &sg, uint32_t sel, int lane,
                                          std::integral_constant<bool, FULL>) {
        const int g = lane >> 2, c = lane & 3;
        const float *kss = reinterpret_cast<const float *>(buf + kKs), *vss = reinterpret_cast<const float *>(buf + kVs);
        float s[4], v[4];
        bool have[4];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            float raw0, raw1;
            qk_raw<KU, KB, false>(buf + 16 * t * RK + koff, buf + (16 * t + 8) * RK + koff, bq, raw0, raw1);
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int tok = NP * (16 * t + g + 8 * k) + (NP == 2 ? c >> 1 : 0), i = 2 * t + k;
                s[i] = kss[tok] * fmaf(aq, k ? raw1 : raw0, bqs);
                v[i] = vss[tok];
                have[i] = FULL || have_token(sg, tok, n);
            }
        }
        uint32_t bp[4];
        softmax<FULL, 2>(r, s, have, v, g, c, sel, bp);
        if constexpr (VB == 1) {
#pragma unroll
            for (int i = 0; i < 4; i++) bp[i] ^= 0x80000000u;  // (odd rows')
        }
        const uint8_t *vst = buf + ROWS * RK;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const uint8_t *vrow = vst + 16 * t * RV;
            uint32_t ra[8], rb[8], rc[8], rd[8];
            VD::pair(vrow, RV, vx, ra, rb);
            VD::pair(vrow + 8 * RV, RV, vx, rc, rd);
#pragma unroll
            for (int mt = 0; mt < 8; mt++)
                mma16816(r.acc[mt], ra[mt], rb[mt], rc[mt], rd[mt], bp[2 * t], bp[2 * t + 1]);
        }
        r.tiles += 2;
    }
    // head c's coordinates 16 g .. of the copy; NP = 2: (head, parity) c's, the lanes of its half
    __device__ __forceinline__ void fold(const Run<MT> &r, float *copy, float W, float scale, int lane) const {
        const int g = lane >> 2, c = lane & 3;
        if (NP == 2 && (g >> 2) != (c >> 1)) return;
        copy += c * copy_stride(D) + 16 * (NP == 2 ? g & 3 : g);
        float x[16];
#pragma unroll
        for (int mt = 0; mt < 8; mt++)
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const float a = r.sum(mt, k);
                if constexpr (kLinear) x[VD::dim(mt, k)] = c1 * (2.0f * a * VD::unscale(mt, k) - W);
                else x[VD::dim(mt, k)] = a * inv;
            }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float4 y = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            float4 *at = reinterpret_cast<float4 *>(copy) + i;
            if (r.some) {
                const float4 z = *at;
                y.x = fmaf(z.x, scale, y.x), y.y = fmaf(z.y, scale, y.y), y.z = fmaf(z.z, scale, y.z), y.w = fmaf(z.w, scale, y.w);
            }
            *at = y;
        }
    }
    // The record from the copy; m and l of head c in lane c.  NP = 2: head i's even and odd tokens are heads i and i + 2 of the
    // copy.
    static __device__ __forceinline__ void record(float *rec, const float *copy, float m, float l, int lane) {
#pragma unroll
        for (int i = 0; i < R; i++) {
            float *to = rec + i * (D + 4);
            const float m0 = __shfl_sync(0xffffffffu, m, i), l0 = __shfl_sync(0xffffffffu, l, i);
            if constexpr (NP == 1) {
                if (lane == 0) *reinterpret_cast<float2 *>(to) = make_float2(m0, l0);
                *reinterpret_cast<float4 *>(to + 4 + 4 * lane) = *reinterpret_cast<const float4 *>(copy + i * copy_stride(D) + 4 * lane);
            } else {
                const float m1 = __shfl_sync(0xffffffffu, m, i + 2), l1 = __shfl_sync(0xffffffffu, l, i + 2);
                const float M = fmaxf(m0, m1), f0 = m0 == M ? 1.f : ex2(m0 - M), f1 = m1 == M ? 1.f : ex2(m1 - M);
                if (lane == 0) *reinterpret_cast<float2 *>(to) = make_float2(M, l0 * f0 + l1 * f1);
                const float2 x = *reinterpret_cast<const float2 *>(copy + i * copy_stride(D) + 2 * lane);
                const float2 y = *reinterpret_cast<const float2 *>(copy + (i + 2) * copy_stride(D) + 2 * lane);
                *reinterpret_cast<float2 *>(to + 4 + 2 * lane) = make_float2(x.x * f0 + y.x * f1, x.y * f0 + y.y * f1);
            }
        }
    }
};

template <int KB, int VB, int NP>
cudaError_t launch_packed(const PagedParams &p, cudaStream_t s) {
    Levels lv;
    value_levels(p.cls.law, VB, p.centroid + cb_off(VB), lv.half, &lv.inv);
    lv.c1 = p.centroid[cb_off(VB) + 1];
    return launch<Packed<KB, VB, NP>>(p, lv, s);
}

}  // namespace pmma
}  // namespace tqk

// One translation unit per key width and head dimension.
#define TQ_INSTANTIATE_PAGED(KB, NP)                                                              \
    namespace tqk {                                                                               \
    cudaError_t launch_paged_kb##KB##_np##NP(const PagedParams &p, cudaStream_t s) {              \
        switch (p.cls.vb) {                                                                       \
            case 1: return pmma::launch_packed<KB, 1, NP>(p, s);                                  \
            case 2: return pmma::launch_packed<KB, 2, NP>(p, s);                                  \
            case 3: return pmma::launch_packed<KB, 3, NP>(p, s);                                  \
            case 4: return pmma::launch_packed<KB, 4, NP>(p, s);                                  \
            case 5: return pmma::launch_packed<KB, 5, NP>(p, s);                                  \
            case 6: return pmma::launch_packed<KB, 6, NP>(p, s);                                  \
            case 7: return pmma::launch_packed<KB, 7, NP>(p, s);                                  \
            case 8: return pmma::launch_packed<KB, 8, NP>(p, s);                                  \
            default: return cudaErrorInvalidValue;                                                \
        }                                                                                         \
    }                                                                                             \
    }
