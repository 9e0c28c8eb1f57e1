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
    static constexpr int team = kCopyBytes + static_cast<int>(sizeof(Small));
    static constexpr int fit = (kSmemMax - kBufBytes - kTeams * team) / (kTeams * stage);
    static constexpr int NS = fit > 4 ? 4 : fit;
    static constexpr int smem = kBufBytes + kTeams * (team + NS * stage);
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
__global__ void __launch_bounds__(kTeamThreads, 1) paged_fp16_kernel(const __grid_constant__ PagedParams p, const int nhb) {
    using G = Fp16<D>;
    constexpr int NS = G::NS, MT = D / 16, CH = D / 8;  // m-tiles of the dims, chunks of a row
    extern __shared__ __align__(128) uint8_t smem[];
    int *bufs = reinterpret_cast<int *>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool loads = warp >= kTeams * kWarps;
    const int team = loads ? warp - kTeams * kWarps : warp / kWarps;  // (from kTeams on: no work)
    uint8_t *mine = smem + kBufBytes + team * (G::team + NS * G::stage);
    float *copies = reinterpret_cast<float *>(mine + NS * G::stage);
    Small &sm = *reinterpret_cast<Small *>(mine + NS * G::stage + kCopyBytes);
    const int worker = team * gridDim.x + blockIdx.x;
    const PagedList &l = p.list;
    pdl_launch_dependents();
    if (loads && lane == 0 && team < kTeams) {
#pragma unroll
        for (int i = 0; i < NS; i++) {
            mbar_init(&sm.full[i], 33);  // the loader's lanes when their copies are there, and its word on the stage
            mbar_init(&sm.empty[i], kWarps);
        }
        mbar_init(&sm.sync, kWarps);
        mbar_init(&sm.head, 1);
        mbar_init_fence();
        sm.dead = 0;
        if (worker < p.cls.workers) p.state[worker] = 0;
    }
    const int total = paged::ranges_of<kTeamThreads, kTeams>(l, p.cls, blockIdx.x, gridDim.x, p.first, bufs);  // (synchronises)
    int begin, end;
    paged::worker_range(p.cls, total, worker, begin, end);
    const int n_st = team < kTeams ? end - begin : 0;
    if (loads) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (n_st > 0) {
            paged::Walk w = paged::seek(l, p.cls, bufs[kTeamThreads / 32 + 2 * team], bufs[kTeamThreads / 32 + 2 * team + 1]);
            if (lane == 0) {
                sm.stage[0].b = w.b;
                sm.stage[0].h_rb = w.h | (w.rb << 8);
                arrive(&sm.head);
            }
            int pid[2], n = 0;  // pages of rows lane, lane + 32
            auto look = [&]() {
                const PagedSeg &s = p.seg[p.cls.seg[w.i]];
                const int t0 = w.st * G::PT;
                n = max(min(G::PT, w.tokens - t0), 0);
#pragma unroll
                for (int i = 0; i < 2; i++)
                    pid[i] = lane + 32 * i < n ? paged::page_at(s, w.b, paged::page_index(s, t0 + lane + 32 * i)) : -1;
            };
            look();
            int at = 0, round = 0, issued = -1;
            bool fresh = true;
            for (int j = 0; j < n_st; j++) {
                if (round > 0 && !wait(&sm.empty[at], (round - 1) & 1, p.wait_polls, &sm.dead)) break;
                const PagedSeg &s = p.seg[p.cls.seg[w.i]];
                const SegView &v = s.seg;
                long long off[2];
                unsigned miss[2];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int t = w.st * G::PT + lane + 32 * i;
                    off[i] = -1;
                    if (pid[i] >= 0)
                        off[i] = static_cast<long long>(pid[i] * v.kblock + v.koff[w.h] + static_cast<size_t>(t - paged::page_index(s, t) * s.page) * G::row);
                    miss[i] = __ballot_sync(0xffffffffu, lane + 32 * i < n && pid[i] < 0);
                }
                if (lane == 0) {  // (rows of the stage outside the pool: page and skip hold their bits)
                    sm.stage[at] = {n | (fresh ? kFresh : 0) | (miss[0] | miss[1] ? kBad : 0), w.b, w.h | (w.rb << 8), 0u,
                                    static_cast<int>(miss[0]), static_cast<int>(miss[1])};
                    arrive(&sm.full[at]);
                }
                issued = j;
                const int row0 = lane / CH, chunk = lane % CH;
                uint8_t *dst = mine + at * G::stage;
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
            cp_async_wait<0>();  // no copy outlives its warp
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        const int tw = warp % kWarps, g = lane >> 2, c = lane & 3;
        const int hb = tw % nhb, tp = tw / nhb, parts = kWarps / nhb;
        const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
        uint32_t bq[2 * MT];
        Run<MT> r;
        unsigned phase = 0;
        int now_b = 0, now_h = 0;
        bool ok = true;
        // the lane's row address of an ldmatrix
        const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, kch = lane >> 4, vrow = (lane & 7) + (lane >> 4) * 8, vch = (lane >> 3) & 1;

        auto tile = [&](unsigned buf, int tA, int n, bool bad, const Stage &sg) {
            float e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < MT; kk++) {
                uint32_t a[4];
                ldmatrix4(a, buf + (tA + krow) * G::row + 16 * ((2 * kk + kch) ^ (krow & 7)));
                mma16816(e, a[0], a[1], a[2], a[3], bq[2 * kk], bq[2 * kk + 1]);
            }
            float s[2];
            const float v[2] = {1.f, 1.f};
            bool have[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int tok = tA + g + 8 * i;
                s[i] = e[2 * i] * p.qk_scale;
                have[i] = tok < n;
                if (bad) have[i] = have[i] && !((static_cast<unsigned>(tok < 32 ? sg.page : sg.skip) >> (tok & 31)) & 1u);
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
            float *to = copies + (tw * 4 + c) * kHeadStride + g;
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
            if (g == 0) sm.m[tw][c] = r.m, sm.l[tw][c] = sum;
            if (!meet(sm, phase, p.wait_polls, lane)) return false;
            write_record<D, 1>(sm, copies, p.part + paged::group_slot(l, p.cls, worker, now_b, now_h & 255, now_h >> 8) * l.R * (D + 4), l.R, nhb);
            return meet(sm, phase, p.wait_polls, lane);
        };
        auto start = [&]() {
            __half *q = reinterpret_cast<__half *>(copies);
            stage_queries<D, false>(p, sm, q, now_b, now_h & 255, now_h >> 8, l.R, tw, lane);
            if (!meet(sm, phase, p.wait_polls, lane)) return false;
            const int head = hb * 4 + (g >> 1);
            const uint32_t *from = reinterpret_cast<const uint32_t *>(q + 2 * head * D) + c;
#pragma unroll
            for (int i = 0; i < 2 * MT; i++) bq[i] = (g & 1) || head >= l.R ? 0u : from[8 * (i >> 1) + 4 * (i & 1)];
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
                const unsigned buf = smem_u32(mine + at * G::stage);
                for (int tA = tp * 16; tA < n; tA += 16 * parts) tile(buf, tA, n, (word & kBad) != 0, sm.stage[at]);
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
    pdl_wait();
}

}  // namespace
}  // namespace pmma

cudaError_t launch_paged_fp16(const PagedParams &p, cudaStream_t s) {
    int nhb = pmma::head_blocks(p.list.R, 4);
    void *args[] = {const_cast<PagedParams *>(&p), &nhb};
    return p.d == 128 ? pmma::launch(reinterpret_cast<const void *>(pmma::paged_fp16_kernel<128>), pmma::Fp16<128>::smem,
                                     pmma::kTeamThreads, pmma::kTeams, p, args, s)
                      : pmma::launch(reinterpret_cast<const void *>(pmma::paged_fp16_kernel<64>), pmma::Fp16<64>::smem,
                                     pmma::kTeamThreads, pmma::kTeams, p, args, s);
}

PagedShape paged_shape_fp16(int) { return {64, pmma::kTeams}; }

}  // namespace tqk
