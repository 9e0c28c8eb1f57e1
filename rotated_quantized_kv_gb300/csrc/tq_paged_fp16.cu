// tq_paged_fp16.cu -- attention of one new token over pages of fp16 rows, head dims 64 and 128.
//
// As the packed kernel (tq_paged_mma.cuh) without codes: a stage is 64 tokens, K rows by ldmatrix against
// the queries as they are (fp16, one part), V rows by ldmatrix.trans.  Pages of any size: rows arrive by
// cp.async, each from its own page (16-byte chunk i of row r at i ^ (r & 7): the eight rows of an
// ldmatrix in eight bank groups), V rows that are not there as zeros.  A warp has 16 of the 64 rows, and
// the warps issue the stages in turn.
#include "tq_paged_mma.cuh"

namespace tqk {
namespace pmma {
namespace {

template <int D>
struct Fp16 {
    static constexpr int PT = 64, row = 2 * D, offV = PT * row, stage = 2 * PT * row;
    static constexpr int fixed = kCopyBytes + static_cast<int>(sizeof(Small));
    static constexpr int CTAS = 3;
    static constexpr int fit = (232448 / CTAS - 1024 - fixed) / stage;
    static constexpr int NS = fit > 4 ? 4 : fit, AHEAD = NS - 1;
    static constexpr int smem = NS * stage + fixed;
    static_assert(NS >= 2, "stages");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&a)[4], unsigned at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&a)[4], unsigned at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(at));
}
__device__ __forceinline__ void arrive_when_copied(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, Fp16<D>::CTAS) paged_fp16_kernel(const __grid_constant__ PagedParams p, const int nhb) {
    using G = Fp16<D>;
    constexpr int NS = G::NS, MT = D / 16, CH = D / 8;  // m-tiles of the dims, chunks of a row
    extern __shared__ __align__(128) uint8_t smem[];
    float *copies = reinterpret_cast<float *>(smem + NS * G::stage);
    Small &sm = *reinterpret_cast<Small *>(smem + NS * G::stage + kCopyBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, worker = blockIdx.x;
    const PagedList &l = p.list;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < NS; i++) {
            mbar_init(&sm.full[i], 33);  // the loader's lanes when their copies are there, and its word on the stage
            mbar_init(&sm.empty[i], kWarps);
        }
        mbar_init(&sm.sync, kWarps);
        mbar_init_fence();
        sm.dead = 0;
        p.state[worker] = 0;
    }
    const paged::Range range = paged::range_of<kThreads>(l, p.cls, worker, p.first, sm.buf);  // (synchronises)
    const int n_st = range.end - range.begin;
    int k = 0;
    bool ok = true;

    paged::Walk w;
    int pid[2] = {-1, -1}, t0 = 0, n = 0;  // pages of rows lane, lane + 32
    auto look = [&]() {
        const PagedSeg &s = p.seg[p.cls.seg[w.i]];
        t0 = w.st * G::PT;
        n = min(G::PT, w.tokens - t0);
#pragma unroll
        for (int i = 0; i < 2; i++) pid[i] = lane + 32 * i < n ? paged::page_at(s, w.b, (t0 + lane + 32 * i) / s.page) : -1;
    };
    auto load = [&](int j) {
        const int at = j % NS;
        if (j >= NS && !wait(&sm.empty[at], (j / NS - 1) & 1, p.wait_polls, &sm.dead)) return false;
        const PagedSeg &s = p.seg[p.cls.seg[w.i]];
        const SegView &v = s.seg;
        long long off[2];
        unsigned miss[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int t = t0 + lane + 32 * i;
            off[i] = pid[i] < 0 ? -1 : static_cast<long long>(pid[i] * v.kblock + v.koff[w.h] + static_cast<size_t>(t % s.page) * G::row);
            miss[i] = __ballot_sync(0xffffffffu, lane + 32 * i < n && pid[i] < 0);
        }
        if (lane == 0) {  // (rows of the stage outside the pool: page and skip hold their bits)
            sm.stage[at] = {n, w.b, w.h | (w.rb << 8), miss[0] | miss[1], static_cast<int>(miss[0]), static_cast<int>(miss[1])};
            arrive(&sm.full[at]);
        }
        const int row0 = lane / CH, chunk = lane % CH;
        uint8_t *dst = smem + at * G::stage;
#pragma unroll 4
        for (int i = 0; i < G::PT; i += 32 / CH) {
            const int row = i + row0;
            const long long o = __shfl_sync(0xffffffffu, i < 32 ? off[0] : off[1], row & 31);
            const int to = row * G::row + 16 * (chunk ^ (row & 7));
            const size_t from = o < 0 ? 0 : static_cast<size_t>(o) + 16 * chunk;
            if (o >= 0) cp_async16_zfill(dst + to, v.k + from, 16);
            cp_async16_zfill(dst + G::offV + to, v.v + from, o < 0 ? 0 : 16);
        }
        arrive_when_copied(&sm.full[at]);
        if (j + kWarps < n_st) {
            skip(l, p.cls, w, kWarps);
            look();
        }
        return true;
    };

    if (n_st > 0) {
        w = paged::seek(l, p.cls, range.b, range.rest);
        if (warp < n_st) {
            if (warp > 0) skip(l, p.cls, w, warp);
            look();
        }
        for (int j = warp; j < G::AHEAD && j < n_st && ok; j += kWarps) ok = load(j);

        const int hb = warp % nhb, tp = warp / nhb, parts = kWarps / nhb;
        const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
        uint32_t bq[2 * MT];
        Run<MT> r;
        unsigned phase = 0;
        int now_b = -1, now_h = -1;
        // the lane's row address of an ldmatrix
        const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, kch = lane >> 4, vrow = (lane & 7) + (lane >> 4) * 8, vch = (lane >> 3) & 1;

        auto tile = [&](unsigned buf, int tA, const Stage &sg) {
            float e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < MT; kk++) {
                uint32_t a[4];
                ldmatrix4(a, buf + (tA + krow) * G::row + 16 * ((2 * kk + kch) ^ (krow & 7)));
                mma16816(e, a[0], a[1], a[2], a[3], bq[2 * kk], bq[2 * kk + 1]);
            }
            float s[2], v[2] = {1.f, 1.f};
            bool have[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int tok = tA + g + 8 * i;
                s[i] = e[2 * i] * p.qk_scale;
                have[i] = tok < sg.n && !(sg.bad && ((static_cast<unsigned>(tok < 32 ? sg.page : sg.skip) >> (tok & 31)) & 1u));
            }
            uint32_t bp[2];
            softmax<false, 1>(r, s, have, v, g, c, sel, bp);
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                uint32_t a[4];
                ldmatrix4_trans(a, buf + G::offV + (tA + vrow) * G::row + 16 * ((2 * mt + vch) ^ (vrow & 7)));
                mma16816(r.acc[mt], a[0], a[1], a[2], a[3], bp[0], bp[1]);
            }
            r.tiles++;
        };
        auto fold = [&]() {
            float *to = copies + (warp * 4 + c) * kHeadStride + g;
            const float f = r.m_ref == r.m ? 1.f : ex2(r.m_ref - r.m);
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float &at = to[16 * mt + 8 * i];
                    at = r.some ? fmaf(at, f, r.sum(mt, i)) : r.sum(mt, i);
                }
            r.m_ref = r.m;
            r.some = true;
            r.clear();
        };
        auto flush = [&]() {
            fold();
            const float sum = warp_sum_g(r.l);
            if (g == 0) sm.m[warp][c] = r.m, sm.l[warp][c] = sum;
            if (!meet(sm, phase, p.wait_polls, lane)) return false;
            write_record<D, 1>(sm, copies, p.part + paged::group_slot(l, p.cls, worker, now_b, now_h & 255, now_h >> 8) * l.R * (D + 4), l.R, nhb);
            return meet(sm, phase, p.wait_polls, lane);
        };
        auto start = [&]() {
            __half *q = reinterpret_cast<__half *>(copies);
            stage_queries<D, false>(p, sm, q, now_b, now_h & 255, now_h >> 8, l.R, warp, lane);
            if (!meet(sm, phase, p.wait_polls, lane)) return false;
            const int head = hb * 4 + (g >> 1);
            const uint32_t *from = reinterpret_cast<const uint32_t *>(q + 2 * head * D) + c;
#pragma unroll
            for (int i = 0; i < 2 * MT; i++) bq[i] = (g & 1) || head >= l.R ? 0u : from[8 * (i >> 1) + 4 * (i & 1)];
            r.start();
            return meet(sm, phase, p.wait_polls, lane);
        };

        for (; k < n_st && ok; k++) {
            const int at = k % NS, j = k + G::AHEAD;
            if (j < n_st && j % kWarps == warp && !(ok = load(j))) break;
            if (!(ok = wait(&sm.full[at], (k / NS) & 1, p.wait_polls, &sm.dead))) break;
            const Stage sg = sm.stage[at];
            if (sg.b != now_b || sg.h_rb != now_h) {
                if (k > 0 && !(ok = flush())) break;
                now_b = sg.b;
                now_h = sg.h_rb;
                if (!(ok = start())) break;
            }
            const unsigned buf = smem_u32(smem + at * G::stage);
            for (int tA = tp * 16; tA < sg.n; tA += 16 * parts) tile(buf, tA, sg);
            __syncwarp();
            if (lane == 0) arrive(&sm.empty[at]);
            if (__builtin_expect(r.tiles >= kFold, 0)) fold();
        }
        if (ok) ok = flush();
        if (!ok && lane == 0) {
            *const_cast<volatile int *>(&sm.dead) = 1;
            p.state[worker] = 1;
        }
        cp_async_wait<0>();  // no copy outlives its warp
    }
    pdl_wait();
}

}  // namespace
}  // namespace pmma

cudaError_t launch_paged_fp16(const PagedParams &p, cudaStream_t s) {
    int nhb = pmma::head_blocks(p.list.R, 4);
    void *args[] = {const_cast<PagedParams *>(&p), &nhb};
    return p.d == 128 ? pmma::launch(reinterpret_cast<const void *>(pmma::paged_fp16_kernel<128>), pmma::Fp16<128>::smem, p, args, s)
                      : pmma::launch(reinterpret_cast<const void *>(pmma::paged_fp16_kernel<64>), pmma::Fp16<64>::smem, p, args, s);
}

PagedShape paged_shape_fp16(int d) {
    return d == 128 ? PagedShape{pmma::Fp16<128>::PT, pmma::Fp16<128>::CTAS} : PagedShape{pmma::Fp16<64>::PT, pmma::Fp16<64>::CTAS};
}

}  // namespace tqk
