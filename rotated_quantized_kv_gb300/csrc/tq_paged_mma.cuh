// tq_paged_mma.cuh -- attention of one new token over paged segments at head dims 64 and 128:
// what the kernels of packed and of fp16 pages share, and the packed one, specialised by
// (key bits, value bits).
//
// The arithmetic of a tile is that of decode attention (tq_decode_packed.cuh: raw key codes as
// fp16 subnormals against the query's hi and lo parts, values by table into the P.V product,
// mma.m16n8k16).  What differs:
//   - a warp takes four query heads, and the eight columns of the P.V product hold the weights as fp16 hi + 2^-11 lo
//     (22 bits, down to 2^-36 of the row's largest);
//     more heads of a KV head go to other warps of the CTA, on the same rows in shared memory;
//   - head_dim 64: a tile row is a pair of tokens read as one record of 128 dims; the four columns
//     are two heads times two parities, a query with zeros in the other token's half, so that a (head, parity) is a
//     head of its own until the CTA joins its parts;
//   - weights are relative to the row's largest weighted value, as in tq_tree_mma.cu: the running
//     maximum is that of S + log2 sigma (sigma in [2^-64, 2^64], its logarithm read off the bits: within 0.09 above), so
//     that fp16 holds the weights that count whatever the values' sizes;
//   - sums leave the tensor cores every kFold tiles: mma.sync adds with truncation, which drifts by some
//     2^-19 of the sum a tile.  They go to a copy in shared memory, by binary32 additions, and at the
//     end of a (sequence, head) the warps' copies join there into one record;
//   - nothing stops the CTA between stages: warps take turns at issuing the copies of a stage (so that no
//     scheduler of the SM has all of that work), lane i those of the i-th page of it, page numbers read
//     a turn ahead; buffers go round by full and empty barriers.  Every wait is bounded, and a warp that gives
//     up marks its worker, sees its own copies land and leaves; it waits for no one.
#pragma once

#include <algorithm>
#include <type_traits>

#include "tq_decode_packed.cuh"
#include "tq_paged.cuh"

namespace tqk {
namespace pmma {

using namespace dec;

constexpr int kWarps = kThreads / 32;
constexpr int kFold = 16;               // tiles of 16 rows between folds
constexpr int kHeadStride = 128 + 4;    // floats of a head's copy of the sums (apart in banks)
constexpr int kCopyBytes = kWarps * 4 * kHeadStride * 4;
constexpr int kMaxRows = 16;

// Value levels of the class: fp16(s c_k), 1/s, and level 1 of a 1-bit codebook.
struct Levels {
    unsigned short half[256];
    float inv, c1;
};

// A wait that ends early where another warp gave up.
__device__ __forceinline__ bool wait(uint64_t *bar, unsigned parity, int polls, const volatile int *dead) {
    for (int i = 0; i < polls; i++) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*dead) return false;
    }
    return false;
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// What the loader tells the others of a stage.
struct Stage {
    int word;            // tokens (none: 0), kFresh: another (sequence, head, block), kBad: some page outside the pool
    int b, h_rb;         // sequence; KV head and block of rows
    unsigned bad;        // bit i: the i-th page of it is outside the pool
    int page, skip;      // tokens a page, and tokens of the first page before the stage
};
constexpr int kFresh = 1 << 16, kBad = 1 << 17;

struct alignas(16) Small {  // a team's shared memory besides stages, tables and copies
    uint64_t full[8], empty[8], sync, head;
    Stage stage[8];
    float m[kWarps][4], l[kWarps][4];
    float qsum[kMaxRows], qexp[kMaxRows];
    int dead;
};

// Running state of a warp: lane (g, c) has head c of its four; columns 2c, 2c + 1 of the
// accumulator are that head's hi and lo parts.
template <int MT>
struct Run {
    float m, mt;         // reference of the weights; the maximum of S + log2 sigma (+ 127)
    float l, w;          // sums of p, and of p sigma since the last fold
    float m_ref;         // reference of the copy
    float acc[MT][4];
    __device__ __forceinline__ float sum(int mt, int k) const { return fmaf(acc[mt][2 * k + 1], 0x1p-11f, acc[mt][2 * k]); }
    int tiles;           // since the last fold
    bool some;           // the copy holds something
    __device__ __forceinline__ void clear() {
        w = 0.f;
        tiles = 0;
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int k = 0; k < 4; k++) acc[i][k] = 0.f;
    }
    __device__ __forceinline__ void start() {
        m = mt = m_ref = kNegInf;
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
        // log2 v + 127 within [0, 0.09]: the exponent, and the mantissa as its fraction
        const float lg = static_cast<float>(__float_as_int(fminf(fmaxf(v[i], 0x1p-64f), 0x1p64f)));
        const float t = fmaf(lg, 0x1p-23f, s[i]);
        top = fmaxf(top, FULL || ok[i] ? t : kNegInf);
    }
    if (__any_sync(0xffffffffu, top > r.mt + 8.0f)) {
        const float now = fmaxf(r.mt, warp_max_g(top));
        const float f = now == kNegInf ? 1.f : ex2(r.mt - now);
        r.mt = now;
        r.m = now - 127.f;
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

// A team's four warps meet (bounded).
__device__ __forceinline__ bool meet(Small &sm, unsigned &phase, int polls, int lane) {
    __syncwarp();
    if (lane == 0) arrive(&sm.sync);
    const bool ok = wait(&sm.sync, phase & 1u, polls, &sm.dead);
    phase++;
    return ok;
}

// The block's queries, rotated or not, as fp16 hi and lo parts [row][part][D] of q 2^-e, e their sum's
// and the row's exponent (the largest coordinate in [0.5, 1)).
template <int D, bool ROTATE>
__device__ __forceinline__ void stage_queries(const PagedParams &p, Small &sm, __half *q, int b, int h, int rb, int rows, int warp, int lane) {
    constexpr int J = D / 32;
    for (int i = warp; i < rows; i += kWarps) {
        const int row = rb * rows + i;
        float x[J];
#pragma unroll
        for (int j = 0; j < J; j++)
            x[j] = row < p.g ? __half2float(__ushort_as_half(p.q[b * p.qs[0] + (static_cast<int64_t>(h) * p.g + row) * p.qs[1] + lane + 32 * j])) : 0.f;
        if constexpr (ROTATE) {
#pragma unroll
            for (int j = 0; j < J; j++)
                if ((p.sign_bits[j] >> lane) & 1u) x[j] = -x[j];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const bool up = (lane & o) != 0;
#pragma unroll
                for (int j = 0; j < J; j++) {
                    const float y = __shfl_xor_sync(0xffffffffu, x[j], o);
                    x[j] = up ? y - x[j] : x[j] + y;
                }
            }
#pragma unroll
            for (int o = 1; o < J; o <<= 1)
#pragma unroll
                for (int j = 0; j < J; j++)
                    if (!(j & o)) {
                        const float a = x[j], y = x[j + o];
                        x[j] = a + y;
                        x[j + o] = a - y;
                    }
#pragma unroll
            for (int j = 0; j < J; j++) x[j] *= ((p.sign_bits[j] >> lane) & 1u) ? -p.inv_sqrt_d : p.inv_sqrt_d;
        }
        float sum = 0.f, top = 0.f;
#pragma unroll
        for (int j = 0; j < J; j++) {
            sum += x[j];
            top = fmaxf(top, fabsf(x[j]));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        // 2^e: rotated fp16 coordinates reach 2^21, the least is 2^-28; a row of zeros or of what is no number keeps e = 0
        int e = 0;
        if (ROTATE && top > 0.f && top < 0x1p100f) e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 126;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int j = 0; j < J; j++) {
            const float y = x[j] * down;
            const __half hi = __float2half_rn(y);
            q[(2 * i) * D + lane + 32 * j] = hi;
            q[(2 * i + 1) * D + lane + 32 * j] = ROTATE ? __float2half_rn(y - __half2float(hi)) : __float2half_rn(0.f);
        }
        if (lane == 0) {
            sm.qsum[i] = sum;
            sm.qexp[i] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        }
    }
}

// The joined record of the CTA's warps: row i, coordinates [0, D).  NP = 2: rows' even and odd tokens
// (heads c and c + 2 of a warp, halves of 128 coordinates).  Warp tp nhb + hb has part tp of the rows of block hb.
template <int D, int NP>
__device__ __forceinline__ void write_record(const Small &sm, const float *copies, float *rec, int rows, int nhb) {
    constexpr int HPW = 4 / NP;
    const int parts = kWarps / nhb, dim = threadIdx.x % D;
    for (int i = static_cast<int>(threadIdx.x % kThreads) / D; i < rows; i += kThreads / D) {
        const int hb = i / HPW, c0 = i % HPW;
        float M = kNegInf;
        for (int tp = 0; tp < parts; tp++)
#pragma unroll
            for (int par = 0; par < NP; par++) M = fmaxf(M, sm.m[tp * nhb + hb][c0 + HPW * par]);
        float L = 0.f, sum = 0.f;
        if (M != kNegInf)
            for (int tp = 0; tp < parts; tp++)
#pragma unroll
                for (int par = 0; par < NP; par++) {
                    const int w = tp * nhb + hb, c = c0 + HPW * par;
                    const float f = ex2(sm.m[w][c] - M);
                    L = fmaf(sm.l[w][c], f, L);
                    sum = fmaf(copies[(w * 4 + c) * kHeadStride + D * par + dim], f, sum);
                }
        float *to = rec + static_cast<size_t>(i) * (D + 4);
        to[4 + dim] = sum;
        if (dim == 0) to[0] = M, to[1] = L;
    }
}

// ------------------------------------------------------------------- packed
constexpr int kTeams = 3;
constexpr int kTeamThreads = 512;       // three teams of four warps, and a warp that loads for each
constexpr int kSmemMax = 232448 - 1024;
constexpr int kBufBytes = 128;           // of ranges_of
static_assert(kBufBytes >= 4 * (kTeamThreads / 32 + 2 * kTeams), "ranges");

template <int KB, int VB, int NP>
struct Geom {
    static constexpr int ROWS = 128, PT = ROWS * NP;             // rows and tokens of a stage
    static constexpr int RK = 16 * KB, RV = 16 * VB;             // bytes of a row
    static constexpr int offV = ROWS * RK, offKS = offV + ROWS * RV, offVS = offKS + PT * 4, stage = offVS + PT * 4;
    static constexpr int entries = VB >= 2 && VB <= 4 ? 1 << (2 * VB) : 0;
    static constexpr int TS = 7;                                 // a column of the pair table a lane
    static constexpr int table = entries * 128 + (VB >= 5 ? 512 : 0);
    static constexpr int team = kCopyBytes + static_cast<int>(sizeof(Small));
    static constexpr int fit(int teams) { return (kSmemMax - table - kBufBytes - teams * team) / (teams * stage); }
    static constexpr int TEAMS = fit(kTeams) >= 2 ? kTeams : kTeams - 1;  // (the widest at head_dim 64: two)
    static constexpr int NS = fit(TEAMS) > 6 ? 6 : fit(TEAMS);
    static constexpr int smem = table + kBufBytes + TEAMS * (team + NS * stage);
    static_assert(NS >= 2 && NS <= 8, "stages");
};

// 4-bit values: pair table of 256 entries; E/O fields of 8 bits: dims (2mt, 2mt+1)
struct Pairs4 {
    static constexpr bool kLinear = false;
    static constexpr __host__ __device__ int dim(int mt, int r) { return 2 * mt + r; }
    template <int K>
    static __device__ __forceinline__ uint32_t at(uint32_t F) { return pair_off<8 * K, 8, 7>(F); }
    static __device__ __forceinline__ void pair(const uint8_t *p, int RV, const VCtx &cx, uint32_t (&ra)[8], uint32_t (&rb)[8]) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p + cx.off), y = *reinterpret_cast<const uint2 *>(p + cx.off + RV);
        constexpr uint32_t M = 0x0F0F0F0Fu;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t wx = i ? x.y : x.x, wy = i ? y.y : y.x;
            const uint32_t E = (wx & M) | ((wy << 4) & ~M), O = ((wx >> 4) & M) | (wy & ~M);
            ra[4 * i] = lds32(cx.tab + at<0>(E));
            ra[4 * i + 1] = lds32(cx.tab + at<1>(E));
            ra[4 * i + 2] = lds32(cx.tab + at<2>(E));
            ra[4 * i + 3] = lds32(cx.tab + at<3>(E));
            rb[4 * i] = lds32(cx.tab + at<0>(O));
            rb[4 * i + 1] = lds32(cx.tab + at<1>(O));
            rb[4 * i + 2] = lds32(cx.tab + at<2>(O));
            rb[4 * i + 3] = lds32(cx.tab + at<3>(O));
        }
    }
};

template <int KB, int VB, int NP>
__global__ void __launch_bounds__(kTeamThreads, 1)
    paged_packed_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ Levels lv, const int nhb) {
    using G = Geom<KB, VB, NP>;
    using KU = KUnpack<KB>;
    using VD = typename std::conditional<VB == 4, Pairs4, VDec<VB, G::TS>>::type;
    constexpr int NS = G::NS, D = 128 / NP, HPW = 4 / NP;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *tab = smem;
    int *bufs = reinterpret_cast<int *>(smem + G::table);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool loads = warp >= kTeams * kWarps;                  // a team's loader
    const int team = loads ? warp - kTeams * kWarps : warp / kWarps;  // (from TEAMS on: no work)
    uint8_t *mine = smem + G::table + kBufBytes + team * (G::team + NS * G::stage);
    float *copies = reinterpret_cast<float *>(mine + NS * G::stage);
    Small &sm = *reinterpret_cast<Small *>(mine + NS * G::stage + kCopyBytes);
    const int worker = team * gridDim.x + blockIdx.x;
    const PagedList &l = p.list;
    pdl_launch_dependents();
    if (loads && lane == 0 && team < G::TEAMS) {
#pragma unroll
        for (int i = 0; i < NS; i++) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], kWarps);
        }
        mbar_init(&sm.sync, kWarps);
        mbar_init(&sm.head, 1);
        mbar_init_fence();
        sm.dead = 0;
        if (worker < p.cls.workers) p.state[worker] = 0;
    }
    // ---- value tables
    if constexpr (VB >= 5)
        for (int i = threadIdx.x; i < (1 << VB); i += kTeamThreads) reinterpret_cast<unsigned short *>(tab)[i] = lv.half[i];
    if constexpr (G::entries > 0)
        for (int i = threadIdx.x; i < G::entries * 32; i += kTeamThreads) {
            const int e = i / 32;
            reinterpret_cast<uint32_t *>(tab)[i] = static_cast<uint32_t>(lv.half[e & ((1 << VB) - 1)]) |
                                                   (static_cast<uint32_t>(lv.half[e >> VB]) << 16);
        }
    const int total = paged::ranges_of<kTeamThreads, kTeams>(l, p.cls, blockIdx.x, gridDim.x, p.first, bufs);  // (synchronises)
    int begin, end;
    paged::worker_range(p.cls, total, worker, begin, end);
    const int n_st = team < G::TEAMS ? end - begin : 0;
    if (loads) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (n_st > 0) {
            paged::Walk w = paged::seek(l, p.cls, bufs[kTeamThreads / 32 + 2 * team], bufs[kTeamThreads / 32 + 2 * team + 1]);
            if (lane == 0) {
                sm.stage[0].b = w.b;
                sm.stage[0].h_rb = w.h | (w.rb << 8);
                arrive(&sm.head);
            }
            const uint64_t pol = policy_evict_first();
            int pid = -1, n = 0, skipped = 0, runs = 0;
            auto look = [&]() {  // the stage at `w`: n tokens on `runs` pages, the first page's tokens before it, the lane's page
                const PagedSeg &s = p.seg[p.cls.seg[w.i]];
                const int t0 = w.st * G::PT, page = paged::page_index(s, t0);
                n = max(min(G::PT, w.tokens - t0), 0);
                skipped = t0 - page * s.page;
                runs = n > 0 ? paged::page_index(s, t0 + n - 1) - page + 1 : 0;
                pid = lane < runs ? paged::page_at(s, w.b, page + lane) : -1;
            };
            look();
            int at = 0, round = 0, issued = -1;
            bool fresh = true;
            for (int j = 0; j < n_st; j++) {
                if (round > 0 && !wait(&sm.empty[at], (round - 1) & 1, p.wait_polls, &sm.dead)) break;
                const PagedSeg &s = p.seg[p.cls.seg[w.i]];
                const SegView &v = s.seg;
                uint8_t *dst = mine + at * G::stage;
                uint64_t *bar = &sm.full[at];
                const bool some = lane < runs;
                const int from = lane == 0 || !some ? 0 : lane * s.page - skipped;  // the run's first token in the stage
                const int in_page = lane == 0 ? skipped : 0;
                const int run = some ? min(s.page - in_page, n - from) : 0;
                const bool bad = some && pid < 0;
                // (runs start at multiples of 16 tokens; an odd end rounds up inside the page)
                const unsigned nk = some && !bad ? (run * (G::RK / NP) + 15) & ~15u : 0u;
                const unsigned nv = (run * (G::RV / NP) + 15) & ~15u, ns = (run * 4 + 15) & ~15u;
                const unsigned bytes = __reduce_add_sync(0xffffffffu, nk ? nk + nv + 2 * ns : 0u);
                const unsigned bads = __ballot_sync(0xffffffffu, bad);
                if (lane == 0) {
                    sm.stage[at] = {n | (fresh ? kFresh : 0) | (bads ? kBad : 0), w.b, w.h | (w.rb << 8), bads, s.page, skipped};
                    fence_proxy_async();
                    mbar_expect_tx(bar, bytes);
                }
                issued = j;
                __syncwarp();
                if (nk) {
                    const size_t sc = (static_cast<size_t>(pid) * l.H + w.h) * v.capacity + in_page;
                    fence_proxy_async();
                    bulk_g2s_hint(dst + from * (G::RK / NP), v.k + pid * v.kblock + v.koff[w.h] + static_cast<size_t>(in_page) * (G::RK / NP), nk, bar, pol);
                    bulk_g2s_hint(dst + G::offV + from * (G::RV / NP), v.v + pid * v.vblock + v.voff[w.h] + static_cast<size_t>(in_page) * (G::RV / NP), nv, bar, pol);
                    bulk_g2s_hint(dst + G::offKS + from * 4, v.ks + sc, ns, bar, pol);
                    bulk_g2s_hint(dst + G::offVS + from * 4, v.vs + sc, ns, bar, pol);
                }
                if (j + 1 < n_st) {
                    fresh = paged::next(l, p.cls, w);
                    look();
                }
                if (++at == NS) at = 0, ++round;
            }
            if (issued + 1 < n_st && lane == 0) {
                *const_cast<volatile int *>(&sm.dead) = 1;
                p.state[worker] = 1;
            }
            // no copy outlives its warp: the last fill of each buffer
            for (int j = max(issued - NS + 1, 0); j <= issued; j++) mbar_wait(&sm.full[j % NS], (j / NS) & 1);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        const int tw = warp % kWarps, g = lane >> 2, c = lane & 3;
        VCtx vx;
        vx.ctab = reinterpret_cast<const unsigned short *>(tab);
        vx.tab = smem_u32(tab) + 4 * lane;
        if constexpr (VB == 1) {
            vx.off = 2 * c * G::RV + 4 * (g >> 1);
            vx.sh = (g & 1) ? 0x7632 : 0x5410;
        } else if constexpr (VB == 3) {
            vx.off = 2 * c * G::RV + 4 * ((3 * g) >> 1);
            vx.sh = (g & 1) * 16;
        } else {
            vx.off = 2 * c * G::RV + ((2 * VB * g) & ~3);
            vx.sh = ((2 * VB * g) & 3) * 8;
        }
        const int hb = tw % nhb, tp = tw / nhb, parts = kWarps / nhb;
        const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
        constexpr float alpha = static_cast<float>(1 << (24 - KU::kA)) * 2.0f / static_cast<float>(1 << KB);
        constexpr float beta = 1.0f / static_cast<float>(1 << KB) - 1.0f;
        const int koff = g * G::RK + 4 * KB * c;
        uint32_t bq[16];
        float aq = 0.f, bqs = 0.f;
        Run<8> r;
        unsigned phase = 0;
        int now_b = 0, now_h = 0;
        bool ok = true;

        auto tile_pair = [&](const uint8_t *buf, int tA, int tokens, const Stage &sg, auto full_tag) {
            constexpr bool FULL = decltype(full_tag)::value;
            const float *kss = reinterpret_cast<const float *>(buf + G::offKS), *vss = reinterpret_cast<const float *>(buf + G::offVS);
            float s[4], v[4];
            bool have[4];
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const int t0r = tA + 16 * t;
                float raw0, raw1;
                qk_raw<KU, KB, false>(buf + t0r * G::RK + koff, buf + (t0r + 8) * G::RK + koff, bq, raw0, raw1);
#pragma unroll
                for (int k2 = 0; k2 < 2; k2++) {
                    const int tok = NP * (t0r + g + 8 * k2) + (NP == 2 ? c >> 1 : 0), i = 2 * t + k2;
                    s[i] = kss[tok] * fmaf(aq, k2 ? raw1 : raw0, bqs);
                    v[i] = vss[tok];
                    have[i] = true;
                    if constexpr (!FULL) {
                        have[i] = tok < tokens;
                        if (sg.bad) have[i] = have[i] && !((sg.bad >> ((sg.skip + tok) / sg.page)) & 1u);
                    }
                }
            }
            uint32_t bp[4];
            softmax<FULL, 2>(r, s, have, v, g, c, sel, bp);
            const uint8_t *vst = buf + G::offV;
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const uint8_t *vrow = vst + (tA + 16 * t) * G::RV;
                uint32_t ra[8], rb[8], rc[8], rd[8];
                VD::pair(vrow, G::RV, vx, ra, rb);
                VD::pair(vrow + 8 * G::RV, G::RV, vx, rc, rd);
#pragma unroll
                for (int mt = 0; mt < 8; mt++)
                    mma16816(r.acc[mt], ra[mt], rb[mt], rc[mt], rd[mt], bp[2 * t], bp[2 * t + 1]);
            }
            r.tiles += 2;
        };
        // the accumulators into the warp's copy: head c, coordinates 16 g ..
        auto fold = [&]() {
            float *to = copies + (tw * 4 + c) * kHeadStride + 16 * g;
            float W = 0.f;
            if constexpr (VD::kLinear) W = warp_sum_g(r.w);
            float x[16];
#pragma unroll
            for (int mt = 0; mt < 8; mt++)
#pragma unroll
                for (int k2 = 0; k2 < 2; k2++) {
                    const float a = r.sum(mt, k2);
                    if constexpr (VD::kLinear) x[VD::dim(mt, k2)] = lv.c1 * (2.0f * a * VDec<1, 7>::unscale(mt, k2) - W);
                    else x[VD::dim(mt, k2)] = a * lv.inv;
                }
            const float f = r.m_ref == r.m ? 1.f : ex2(r.m_ref - r.m);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float4 y = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                float4 *at = reinterpret_cast<float4 *>(to) + i;
                if (r.some) {
                    const float4 z = *at;
                    y.x = fmaf(z.x, f, y.x), y.y = fmaf(z.y, f, y.y), y.z = fmaf(z.z, f, y.z), y.w = fmaf(z.w, f, y.w);
                }
                *at = y;
            }
            r.m_ref = r.m;
            r.some = true;
            r.clear();
        };
        auto flush = [&]() {
            fold();
            const float sum = warp_sum_g(r.l);
            if (g == 0) sm.m[tw][c] = r.m, sm.l[tw][c] = sum;
            if (!meet(sm, phase, p.wait_polls, lane)) return false;
            write_record<D, NP>(sm, copies, p.part + paged::group_slot(l, p.cls, worker, now_b, now_h & 255, now_h >> 8) * l.R * (D + 4), l.R, nhb);
            return meet(sm, phase, p.wait_polls, lane);
        };
        auto start = [&]() {
            __half *q = reinterpret_cast<__half *>(copies);
            stage_queries<D, true>(p, sm, q, now_b, now_h & 255, now_h >> 8, l.R, tw, lane);
            if (!meet(sm, phase, p.wait_polls, lane)) return false;
            const int v = g >> 1, part = g & 1;
            const int head = hb * HPW + (NP == 2 ? v & 1 : v);
            uint32_t x[16];
            if (NP == 2 && (v >> 1) != (c >> 1)) {
#pragma unroll
                for (int i = 0; i < 16; i++) x[i] = 0u;
            } else {
                const uint4 *from = reinterpret_cast<const uint4 *>(q + (2 * head + part) * D + 32 * (NP == 2 ? c & 1 : c));
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint4 y = from[i];
                    x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
                }
            }
            gather_b<KU>(x, bq);
            const int own = hb * HPW + (NP == 2 ? c & 1 : c);
            aq = alpha * sm.qexp[own] * p.qk_scale;
            bqs = beta * sm.qsum[own] * p.qk_scale;
            r.start();
            return meet(sm, phase, p.wait_polls, lane);
        };

        if (n_st > 0) {
            ok = wait(&sm.head, 0, p.wait_polls, &sm.dead);
            if (ok) {
                now_b = sm.stage[0].b;
                now_h = sm.stage[0].h_rb;
                ok = start();  // (while the first stage is on its way)
            }
            int at = 0;
            unsigned parity = 0;
            for (int k = 0; k < n_st && ok; k++) {
                if (!(ok = wait(&sm.full[at], parity, p.wait_polls, &sm.dead))) break;
                const int word = sm.stage[at].word, n = word & (kFresh - 1);
                if (__builtin_expect((word & kFresh) && k > 0, 0)) {
                    if (!(ok = flush())) break;
                    now_b = sm.stage[at].b;
                    now_h = sm.stage[at].h_rb;
                    if (!(ok = start())) break;
                }
                const uint8_t *buf = mine + at * G::stage;
                for (int tA = tp * 32; NP * tA < n; tA += 32 * parts) {
                    if (NP * (tA + 32) <= n && !(word & kBad)) tile_pair(buf, tA, n, sm.stage[at], std::true_type{});
                    else tile_pair(buf, tA, n, sm.stage[at], std::false_type{});
                }
                __syncwarp();
                if (lane == 0) arrive(&sm.empty[at]);
                if (++at == NS) at = 0, parity ^= 1u;
                if (__builtin_expect(r.tiles >= kFold, 0)) fold();
            }
            if (ok) ok = flush();
            if (!ok && lane == 0) {
                *const_cast<volatile int *>(&sm.dead) = 1;
                p.state[worker] = 1;
            }
        }
    }
    pdl_wait();  // the call's last launch ends behind its first
}

// teams: workers of a CTA.
inline cudaError_t launch(const void *kernel, size_t smem, int threads, int teams, const PagedParams &p, void **args, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    // workers t, t + grid, t + 2 grid ... are one CTA's: few stages go to as many SMs
    const int ctas = std::max(1, p.cls.workers / teams);
    cfg.gridDim = dim3(static_cast<unsigned>(p.cls.workers < current_sm_count() * teams ? std::min(p.cls.workers, current_sm_count()) : ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.first_class ? 0 : 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

// Blocks of heads among a CTA's warps.
inline int head_blocks(int rows, int per_warp) { return rows <= per_warp ? 1 : rows <= 2 * per_warp ? 2 : 4; }

template <int KB, int VB, int NP>
cudaError_t launch_packed(const PagedParams &p, cudaStream_t s) {
    Levels lv;
    value_levels(p.cls.law, VB, p.centroid + cb_off(VB), lv.half, &lv.inv);
    lv.c1 = p.centroid[cb_off(VB) + 1];
    int nhb = head_blocks(p.list.R, 4 / NP);
    void *args[] = {const_cast<PagedParams *>(&p), &lv, &nhb};
    return launch(reinterpret_cast<const void *>(paged_packed_kernel<KB, VB, NP>), Geom<KB, VB, NP>::smem, kTeamThreads,
                  Geom<KB, VB, NP>::TEAMS, p, args, s);
}

template <int KB, int VB, int NP>
PagedShape shape_packed() {
    return {Geom<KB, VB, NP>::PT, Geom<KB, VB, NP>::TEAMS};
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
    PagedShape paged_shape_kb##KB##_np##NP(int vb) {                                              \
        switch (vb) {                                                                             \
            case 1: return pmma::shape_packed<KB, 1, NP>();                                       \
            case 2: return pmma::shape_packed<KB, 2, NP>();                                       \
            case 3: return pmma::shape_packed<KB, 3, NP>();                                       \
            case 4: return pmma::shape_packed<KB, 4, NP>();                                       \
            case 5: return pmma::shape_packed<KB, 5, NP>();                                       \
            case 6: return pmma::shape_packed<KB, 6, NP>();                                       \
            case 7: return pmma::shape_packed<KB, 7, NP>();                                       \
            default: return pmma::shape_packed<KB, 8, NP>();                                      \
        }                                                                                         \
    }                                                                                             \
    }
