// tq_verify.cu -- verification of drafted tokens against the target's probabilities, from
// given random numbers (rejection sampling, so that the tokens that come out are distributed
// as the target's own).
//
// A sequence stands at a node of its draft tree (first the root) with weights r = p, the target's
// row there, and mass s = 1.  The node's children are tried in index order: child c with token t is
// accepted if u_c q(t) s < r(t), q the row that the children were drawn from (no such row: a draft
// that stands for itself, q(t) = 1), and the walk goes on from c.  A rejection leaves r <- max(r - s q, 0)
// (r(t) <- 0) and s = sum r; where nothing is left, p takes its place with its own sum.  Where no
// child is accepted, the next token is the first t whose cumulative r exceeds u sum r.
// (Weights are not divided by their mass: the comparisons carry it.)  Index order visits parents
// before children and siblings in turn, so that one pass over the drafts is the walk.
//
// What is read of the rows is what counts: the tests look up two numbers a draft, and only a
// rejection, or the end of the walk, takes a pass over the row of the node (a wave at the
// memory's rate: 32 sequences' two rows of 131072 bf16 are 16.8 MB, 2.5 us).  So a cluster of up to eight CTAs takes
// a sequence: every CTA has the drafts' numbers (one CTA fetches them and hands them to the others,
// so that all walk alike whatever happens to the inputs meanwhile), a pass splits the row, and
// the sums meet through shared memory of the cluster.
//
// Sums decide at borders between tokens: a row of 10^5 weights has as many borders, and sums with
// an error of 10^-8 draw another token once in 10^3 draws.  Lanes, warps and tiles keep their sums as two
// binary32 numbers (exact sums of two, 2^-48); CTAs' sums and prefixes are binary64, of which there are few (its
// rate is 1/64).  The difference r - s q takes s as two binary32 numbers, a rounding for each of them that is not 0.
//
// Bound by waits that follow one another: the drafts, their numbers, a pass for each rejection at the path's nodes
// (about 3 us: 20 instructions a weight, then the CTAs meet), the draw.  One chain of 4 drafts, 32000
// fp32: 13 us; 32 trees of 16 drafts, 131072 bf16, with their distributions: 33 us (clusters of four CTAs instead of
// eight: 6 us more; the walk by all warps, binary64 sums of tiles and bodies unrolled four times: 13 us more).
#include <algorithm>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tq_serve.h"

namespace tqk {
namespace {

namespace cg = cooperative_groups;

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerMaxCtas = 8;
constexpr int kUnroll = 4;           // 16-byte vectors a lane and tile
constexpr int kMaxTiles = 512;       // tile sums that a CTA keeps; longer slices take longer tiles

// A weight: what is not a positive number below 2^90 is none (so that sums of 2^30 of them are finite).
__device__ __forceinline__ float weight(float x) {
    x = fmaxf(x, 0.f);               // (and NaN)
    return x < 0x1p90f ? x : 0.f;
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// hi + lo += x (x >= 0, hi >= 0), the rounding of hi kept in lo.
__device__ __forceinline__ void add_exact(float &hi, float &lo, float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
}

// A row as 16-byte vectors of an aligned grid: vector i holds elements i VEC - skew ...
template <typename T>
struct Row {
    static constexpr int VEC = 16 / sizeof(T);
    const T *at;
    int skew, V;
    bool vec;
    __device__ __forceinline__ Row(const T *p, int V_, int skew_) : at(p), skew(skew_), V(V_) {
        vec = own_skew(p) == skew;
    }
    static __device__ __forceinline__ int own_skew(const T *p) {
        return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
    }
    // Vector i as it is; what is behind an end: zeros.
    __device__ __forceinline__ uint4 load(int i) const {
        const int e = i * VEC - skew;
        if (vec && e >= 0 && e + VEC <= V) return __ldg(reinterpret_cast<const uint4 *>(at + e));
        return ragged(at, e, V);
    }
    // (the code of a call runs once or twice: what is not on every vector's way is kept out of it)
    static __device__ __noinline__ uint4 ragged(const T *at, int e, int V) {
        union {
            T x[VEC];
            uint4 w;
        } v;
        v.w = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < VEC; k++)
            if (e + k >= 0 && e + k < V) v.x[k] = at[e + k];
        return v.w;
    }
};

struct Level {
    float hi, lo;                    // a mass s
};

struct Shared {
    // the drafts, the same in every CTA of the cluster
    int token[TQ_MAX_DRAFTS], parent[TQ_MAX_DRAFTS];
    float u[TQ_MAX_DRAFTS + 1], p[TQ_MAX_DRAFTS], q[TQ_MAX_DRAFTS];
    // rejections at the node: masses (with draft rows) or tokens (without)
    union {
        Level level[TQ_MAX_DRAFTS];
        int out[TQ_MAX_DRAFTS];
    };
    double total[2][kVerMaxCtas];    // a pass's sums of the CTAs, two passes in turn
    Level tile[kMaxTiles];
    int path[TQ_MAX_DRAFTS];
    int want, node;                  // what warp 0 asks for: rejections at the node (-1: the walk is over), the node
};

// r behind `gone` rejections of a vector (element e on) from its p and q, and its sum.
template <typename T>
__device__ __forceinline__ void residual(const Shared &sh, bool draft, uint4 pv, uint4 qv, int e, int gone, float (&r)[Row<T>::VEC]) {
    constexpr int VEC = Row<T>::VEC;
    const T *p = reinterpret_cast<const T *>(&pv), *qq = reinterpret_cast<const T *>(&qv);
#pragma unroll
    for (int k = 0; k < VEC; k++) r[k] = weight(to_float(p[k]));
    if (gone == 0) return;
    if (draft) {
        float q[VEC];
#pragma unroll
        for (int k = 0; k < VEC; k++) q[k] = weight(to_float(qq[k]));
#pragma unroll 1
        for (int j = 0; j < gone; j++) {
            const Level s = sh.level[j];
#pragma unroll
            for (int k = 0; k < VEC; k++) r[k] = fmaxf(__fmaf_rn(-s.lo, q[k], __fmaf_rn(-s.hi, q[k], r[k])), 0.f);
        }
    } else {
#pragma unroll 1
        for (int j = 0; j < gone; j++) {
            const int at = sh.out[j] - e;
#pragma unroll
            for (int k = 0; k < VEC; k++)
                if (at == k) r[k] = 0.f;
        }
    }
}
template <typename T>
__device__ __noinline__ Level vector_sum(const Shared &sh, bool draft, uint4 p, uint4 q, int e, int gone) {
    float r[Row<T>::VEC];
    residual<T>(sh, draft, p, q, e, gone, r);
    Level s = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < Row<T>::VEC; k++) add_exact(s.hi, s.lo, r[k]);
    return s;
}

// Sum over the warp (the same in every lane).
__device__ __forceinline__ Level warp_sum(Level s) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, s.hi, o), l = __shfl_xor_sync(0xffffffffu, s.lo, o);
        add_exact(s.hi, s.lo, h);
        s.lo = __fadd_rn(s.lo, l);
    }
    // (partners add their low parts in two orders; the CTAs of a cluster, to which lanes send it, have to agree on every bit)
    s.hi = __shfl_sync(0xffffffffu, s.hi, 0);
    s.lo = __shfl_sync(0xffffffffu, s.lo, 0);
    return s;
}
__device__ __forceinline__ double to_double(Level s) { return static_cast<double>(s.hi) + static_cast<double>(s.lo); }

// The lane where `before` and the inclusive prefix of x pass the goal (found), else the last with x > 0 (none: -1), and the
// sum before it; `before` moves on by all of x.
__device__ __noinline__ int find_lane(double x, double goal, double &before, double &at_sum, bool &found) {
    const int lane = threadIdx.x & 31;
    double y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    const unsigned some = __ballot_sync(0xffffffffu, x > 0.0), over = __ballot_sync(0xffffffffu, x > 0.0 && before + y > goal);
    const int at = over ? __ffs(over) - 1 : 31 - __clz(some);
    if (some) at_sum = before + __shfl_sync(0xffffffffu, y - x, at);
    before += __shfl_sync(0xffffffffu, y, 31);
    found = over != 0;
    return at;
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
    constexpr int VEC = Row<T>::VEC;
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int n_cta = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / n_cta, N = p.N, V = p.V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *target = static_cast<const T *>(p.target) + b * p.ts[0];
    const T *draft = p.draft ? static_cast<const T *>(p.draft) + b * p.ds[0] : nullptr;
    cluster.sync();                  // all CTAs are there (their shared memory is written next)
    if (rank == 0) {
        for (int i = threadIdx.x; i <= N; i += kVerThreads) {
            const float u = p.uniform[b * p.uniform_stride + i];
            int token = 0, parent = -2;  // -2: no candidate
            float pt = 0.f, qt = 1.f;
            if (i < N) {
                token = p.tokens[b * p.tokens_stride + i];
                parent = p.parents ? p.parents[b * p.parents_stride + i] : i - 1;
                if (parent < -1 || parent >= i || token < 0 || token >= V) {
                    parent = -2;
                } else {
                    pt = weight(to_float(target[(parent + 1) * p.ts[1] + token]));
                    if (draft) qt = weight(to_float(draft[(parent + 1) * p.ds[1] + token]));
                }
            }
            for (int c = 0; c < n_cta; c++) {
                Shared *to = cluster.map_shared_rank(&sh, c);
                to->u[i] = u;
                if (i < N) to->token[i] = token, to->parent[i] = parent, to->p[i] = pt, to->q[i] = qt;
            }
        }
    }
    cluster.sync();

    // ---- passes: sums of the weights r of a node's row behind `gone` rejections
    int passes = 0;
    // vectors of this CTA's slice, and of a tile
    int v0 = 0, v1 = 0, per_tile = 32 * kUnroll;
    auto rows = [&](int node, auto fn) {
        const T *pr = target + (node + 1) * p.ts[1];
        const int skew = Row<T>::own_skew(pr);
        const T *qr = draft ? draft + (node + 1) * p.ds[1] : pr;
        const int n_vec = (V + skew + VEC - 1) / VEC;
        const int each = (n_vec + n_cta - 1) / n_cta;
        v0 = min(rank * each, n_vec);
        v1 = min(v0 + each, n_vec);
        per_tile = 32 * kUnroll;
        while (static_cast<long long>(per_tile) * kMaxTiles < each) per_tile *= 2;
        fn(Row<T>(pr, V, skew), Row<T>(qr, V, skew));
    };
    // (warp 0 of every CTA gets the sum; the CTA keeps its tiles')
    auto pass = [&](int node, int gone) {
        rows(node, [&](const Row<T> &P, const Row<T> &Q) {
#pragma unroll 1
            for (int t = warp; v0 + t * per_tile < v1; t += kVerWarps) {
                const int to = min(v0 + (t + 1) * per_tile, v1);
                uint4 pv[3], qv[3];  // the vector at work and the two behind it
                auto fetch = [&](int i, uint4 &x, uint4 &y) {
                    x = y = make_uint4(0u, 0u, 0u, 0u);
                    if (i < to) {
                        x = P.load(i);
                        if (draft && gone) y = Q.load(i);
                    }
                };
                int i = v0 + t * per_tile + lane;
                fetch(i, pv[0], qv[0]);
                fetch(i + 32, pv[1], qv[1]);
                Level sum = {0.f, 0.f};
#pragma unroll 1
                for (; i - lane < to; i += 32) {
                    fetch(i + 64, pv[2], qv[2]);
                    const Level x = vector_sum<T>(sh, draft != nullptr, pv[0], qv[0], i * VEC - P.skew, gone);
                    add_exact(sum.hi, sum.lo, x.hi);
                    sum.lo = __fadd_rn(sum.lo, x.lo);
                    pv[0] = pv[1], qv[0] = qv[1], pv[1] = pv[2], qv[1] = qv[2];
                }
                sum = warp_sum(sum);
                if (lane == 0) sh.tile[t] = sum;
            }
        });
        __syncthreads();
        const int at = passes++ & 1;
        if (warp == 0) {
            const int n_tiles = (v1 - v0 + per_tile - 1) / per_tile;
            Level sum = {0.f, 0.f};
            for (int t = lane; t < n_tiles; t += 32) {
                add_exact(sum.hi, sum.lo, sh.tile[t].hi);
                sum.lo = __fadd_rn(sum.lo, sh.tile[t].lo);
            }
            sum = warp_sum(sum);
            if (lane < n_cta) cluster.map_shared_rank(&sh, lane)->total[at][rank] = to_double(sum);
        }
        cluster.sync();
        double total = 0.0;
        if (warp == 0) {
            total = (lane & 7) < n_cta ? sh.total[at][lane & 7] : 0.0;
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        return total;
    };

    // ---- the walk, by warp 0 of every CTA alike (sixteen warps take sixteen times as long for its binary64 products);
    // it stops at what needs a pass of the CTA
    int node = -1, count = 0, gone = 0;
    int next = 0;                    // the first draft that has not been looked at
    double mass = 1.0, sum = 0.0;
    bool summed = false;             // the tiles' sums are those of r
    for (;;) {
        if (warp == 0) {
            // (nothing is left behind a rejection: the target's own row takes the rest's place)
            bool rejected = summed && gone > 0 && !(sum > 0.0);
            if (rejected) gone = 0;
            while (next < N && !rejected) {
                const int from = next & ~31;
                const unsigned child = __ballot_sync(0xffffffffu, from + lane >= next && from + lane < N && sh.parent[from + lane] == node);
                if (child == 0) {
                    next = from + 32;
                    continue;
                }
                const int i = from + __ffs(child) - 1, t = sh.token[i];
                next = i + 1;
                const float qt = sh.q[i];
                float r = sh.p[i];       // r(t)
                for (int j = 0; j < gone; j++) {
                    if (draft) r = fmaxf(__fmaf_rn(-sh.level[j].lo, qt, __fmaf_rn(-sh.level[j].hi, qt, r)), 0.f);
                    else if (sh.out[j] == t) r = 0.f;
                }
                if (static_cast<double>(sh.u[i]) * static_cast<double>(qt) * mass < static_cast<double>(r)) {
                    if (lane == 0) sh.path[count] = i;
                    ++count;
                    node = i;
                    gone = 0;
                    mass = 1.0;
                    summed = false;
                    continue;
                }
                rejected = true;
                if (lane == 0) {
                    if (draft) {
                        const float hi = static_cast<float>(mass);
                        sh.level[gone] = {hi, static_cast<float>(mass - static_cast<double>(hi))};
                    } else {
                        sh.out[gone] = t;
                    }
                }
                ++gone;
            }
            if (lane == 0) sh.want = rejected || !summed ? gone : -1, sh.node = node;
        }
        __syncthreads();
        const int want = sh.want;    // (the node does not change in a pass)
        if (want < 0) break;
        mass = sum = pass(sh.node, want);
        summed = true;
    }

    // ---- results: the token's CTA draws it
    if (warp != 0) return;
    node = sh.node;
    if (rank == 0) {
        for (int i = lane; i < N; i += 32) p.accepted[static_cast<size_t>(b) * N + i] = i < count ? sh.path[i] : -1;
        if (lane == 0) {
            p.n_accepted[b] = count;
            if (!(sum > 0.0)) p.token[b] = -1;
        }
    }
    if (!(sum > 0.0)) return;
    const double goal = static_cast<double>(sh.u[N]) * sum;
    // the CTA where the sum passes the goal (or the last that has weights: the goal is the sum itself, by rounding)
    double before = 0.0, at_sum = 0.0;
    bool found;
    if (find_lane(lane < n_cta ? sh.total[(passes - 1) & 1][lane] : 0.0, goal, before, at_sum, found) != rank) return;
    before = at_sum;
    // its tile, likewise
    const int n_tiles = (v1 - v0 + per_tile - 1) / per_tile;
    int tile = 0;
    found = false;
    double tile_sum = before;
#pragma unroll 1
    for (int t0 = 0; t0 < n_tiles && !found; t0 += 32) {
        const int at = find_lane(t0 + lane < n_tiles ? to_double(sh.tile[t0 + lane]) : 0.0, goal, before, tile_sum, found);
        if (at >= 0) tile = t0 + at;
    }
    rows(node, [&](const Row<T> &P, const Row<T> &Q) {
        // its vector
        const int from = v0 + tile * per_tile, to = min(from + per_tile, v1);
        int vec = -1;
        uint4 pv, qv, pn, qn;        // the lane's vector, the one behind it
        auto fetch = [&](int i, uint4 &x, uint4 &y) {
            x = y = make_uint4(0u, 0u, 0u, 0u);
            if (i < to) {
                x = P.load(i);
                if (draft && gone) y = Q.load(i);
            }
        };
        uint4 pa, qa;                // that vector
        pa = qa = make_uint4(0u, 0u, 0u, 0u);
        found = false;
        before = tile_sum;
        fetch(from + lane, pv, qv);
#pragma unroll 1
        for (int i0 = from; i0 < to && !found; i0 += 32) {
            fetch(i0 + 32 + lane, pn, qn);
            const int at = find_lane(to_double(vector_sum<T>(sh, draft != nullptr, pv, qv, (i0 + lane) * VEC - P.skew, gone)), goal, before,
                                     at_sum, found);
            if (at >= 0) vec = i0 + at, pa = pv, qa = qv;
            pv = pn, qv = qn;
        }
        if (vec < 0 || lane != ((vec - from) & 31)) return;
        // its element
        float r[VEC];
        residual<T>(sh, draft != nullptr, pa, qa, vec * VEC - P.skew, gone, r);
        int token = -1;
#pragma unroll
        for (int k = 0; k < VEC; k++) {
            if (r[k] > 0.f && (token < 0 || !(at_sum > goal))) token = vec * VEC - P.skew + k;
            at_sum += static_cast<double>(r[k]);
        }
        p.token[b] = token;
    });
}

template <typename T>
cudaError_t verify(const VerifyParams &p, cudaStream_t s) {
    // a slice of 4096 elements or more a CTA (32000 fp32, before the walk was one warp's: 4 CTAs 15.3 us, 2 CTAs 16.8, 8
    // no less; now 12.8 us with 4)
    int ctas = 1;
    while (ctas < kVerMaxCtas && p.V / (2 * ctas) >= 4096) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B) * ctas);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams &p, int dtype, cudaStream_t s) {
    switch (dtype) {
        case TQ_DTYPE_F16: return verify<__half>(p, s);
        case TQ_DTYPE_BF16: return verify<__nv_bfloat16>(p, s);
        default: return verify<float>(p, s);
    }
}

}  // namespace tqk
