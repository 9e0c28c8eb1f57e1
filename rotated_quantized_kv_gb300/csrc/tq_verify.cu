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
// an error of 10^-8 draw another token once in 10^3 draws.  A lane keeps its sum as two binary32
// numbers (exact sums of two, 2^-48), tiles and prefixes are binary64, of which there are few (its
// rate is 1/64).  The difference r - s q takes s as two binary32 numbers, one rounding of the result.
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
    __device__ __forceinline__ void load(int i, float (&x)[VEC]) const {
        const int e = i * VEC - skew;
        if (vec && e >= 0 && e + VEC <= V) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(at + e));
            const T *v = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int k = 0; k < VEC; k++) x[k] = to_float(v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; k++) x[k] = e + k >= 0 && e + k < V ? to_float(at[e + k]) : 0.f;
        }
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
    double tile[kMaxTiles];
    int path[TQ_MAX_DRAFTS];
};

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

    // ---- passes: weights r of a node's row behind `gone` rejections
    // r of a vector's elements from p and q
    auto residual = [&](const Row<T> &P, const Row<T> &Q, int i, int gone, float (&r)[VEC]) {
        P.load(i, r);
#pragma unroll
        for (int k = 0; k < VEC; k++) r[k] = weight(r[k]);
        if (gone == 0) return;
        if (draft) {
            float q[VEC];
            Q.load(i, q);
#pragma unroll
            for (int k = 0; k < VEC; k++) q[k] = weight(q[k]);
            for (int j = 0; j < gone; j++) {
                const Level s = sh.level[j];
#pragma unroll
                for (int k = 0; k < VEC; k++) r[k] = fmaxf(__fmaf_rn(-s.lo, q[k], __fmaf_rn(-s.hi, q[k], r[k])), 0.f);
            }
        } else {
            const int e = i * VEC - P.skew;
            for (int j = 0; j < gone; j++) {
                const int at = sh.out[j] - e;
#pragma unroll
                for (int k = 0; k < VEC; k++)
                    if (at == k) r[k] = 0.f;
            }
        }
    };
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
    // sum of the weights (every thread of the cluster gets it); the CTA keeps its tiles' sums
    auto pass = [&](int node, int gone) {
        rows(node, [&](const Row<T> &P, const Row<T> &Q) {
            for (int t = warp; v0 + t * per_tile < v1; t += kVerWarps) {
                const int from = v0 + t * per_tile, to = min(from + per_tile, v1);
                double sum = 0.0;
                for (int i0 = from; i0 < to; i0 += 32 * kUnroll) {
                    float hi = 0.f, lo = 0.f;
#pragma unroll
                    for (int u = 0; u < kUnroll; u++) {
                        const int i = i0 + 32 * u + lane;
                        if (i < to) {
                            float r[VEC];
                            residual(P, Q, i, gone, r);
#pragma unroll
                            for (int k = 0; k < VEC; k++) add_exact(hi, lo, r[k]);
                        }
                    }
                    sum += static_cast<double>(hi) + static_cast<double>(lo);
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) sh.tile[t] = sum;
            }
        });
        __syncthreads();
        const int at = passes++ & 1;
        if (warp == 0) {
            const int n_tiles = (v1 - v0 + per_tile - 1) / per_tile;
            double sum = 0.0;
            for (int t = lane; t < n_tiles; t += 32) sum += sh.tile[t];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane < n_cta) cluster.map_shared_rank(&sh, lane)->total[at][rank] = sum;
        }
        cluster.sync();
        double total = 0.0;
        for (int c = 0; c < n_cta; c++) total += sh.total[at][c];
        return total;
    };

    // ---- the walk, by every thread alike
    int node = -1, count = 0, gone = 0;
    double mass = 1.0, sum = 0.0;
    bool summed = false;             // the tiles' sums are those of r
    for (int i = 0; i < N; i++) {
        if (sh.parent[i] != node) continue;
        const int t = sh.token[i];
        const float pt = sh.p[i], qt = sh.q[i];
        float r = pt;                // r(t)
        for (int j = 0; j < gone; j++) {
            if (draft) r = fmaxf(__fmaf_rn(-sh.level[j].lo, qt, __fmaf_rn(-sh.level[j].hi, qt, r)), 0.f);
            else if (sh.out[j] == t) r = 0.f;
        }
        if (static_cast<double>(sh.u[i]) * static_cast<double>(qt) * mass < static_cast<double>(r)) {
            if (threadIdx.x == 0) sh.path[count] = i;
            ++count;
            node = i;
            gone = 0;
            mass = 1.0;
            summed = false;
            continue;
        }
        __syncthreads();             // the list has been read
        if (threadIdx.x == 0) {
            if (draft) {
                const float hi = static_cast<float>(mass);
                sh.level[gone] = {hi, static_cast<float>(mass - static_cast<double>(hi))};
            } else {
                sh.out[gone] = t;
            }
        }
        __syncthreads();
        sum = pass(node, ++gone);
        if (!(sum > 0.0)) sum = pass(node, gone = 0);
        mass = sum;
        summed = true;
    }
    if (!summed) sum = pass(node, gone);

    // ---- results: the token's CTA draws it
    if (rank == 0) {
        __syncthreads();
        for (int i = threadIdx.x; i < N; i += kVerThreads) p.accepted[static_cast<size_t>(b) * N + i] = i < count ? sh.path[i] : -1;
        if (threadIdx.x == 0) {
            p.n_accepted[b] = count;
            if (!(sum > 0.0)) p.token[b] = -1;
        }
    }
    if (!(sum > 0.0) || warp != 0) return;
    const double goal = static_cast<double>(sh.u[N]) * sum;
    const double *total = sh.total[(passes - 1) & 1];
    int last = 0, mine = -1;         // the last CTA that has weights; the one where the sum passes the goal
    double before = 0.0, prefix = 0.0;
    for (int c = 0; c < n_cta; c++) {
        if (total[c] > 0.0) {
            last = c;
            if (c == rank) before = prefix;
        }
        prefix += total[c];
        if (mine < 0 && prefix > goal) mine = c;
    }
    if ((mine < 0 ? last : mine) != rank) return;  // (none: the goal is the sum itself, by rounding)
    // the tile, likewise
    const int n_tiles = (v1 - v0 + per_tile - 1) / per_tile;
    int tile = -1, last_tile = 0;
    double tile_before = before, last_before = before;
    for (int t0 = 0; t0 < n_tiles && tile < 0; t0 += 32) {
        const double x = t0 + lane < n_tiles ? sh.tile[t0 + lane] : 0.0;
        double y = x;                // inclusive prefix
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        const unsigned some = __ballot_sync(0xffffffffu, x > 0.0), over = __ballot_sync(0xffffffffu, x > 0.0 && before + y > goal);
        const int at = over ? __ffs(over) - 1 : (some ? 31 - __clz(some) : 0);
        const double at_before = before + __shfl_sync(0xffffffffu, y - x, at);
        if (over) tile = t0 + at, tile_before = at_before;
        else if (some) last_tile = t0 + at, last_before = at_before;
        before += __shfl_sync(0xffffffffu, y, 31);
    }
    if (tile < 0) tile = last_tile, tile_before = last_before;
    rows(node, [&](const Row<T> &P, const Row<T> &Q) {
        const int from = v0 + tile * per_tile, to = min(from + per_tile, v1);
        double run = tile_before;
        int token = -1;              // the last one with a weight, until one passes the goal
        for (int i0 = from; i0 < to; i0 += 32) {
            float r[VEC];
#pragma unroll
            for (int k = 0; k < VEC; k++) r[k] = 0.f;
            if (i0 + lane < to) residual(P, Q, i0 + lane, gone, r);
            double x = 0.0;
#pragma unroll
            for (int k = 0; k < VEC; k++) x += static_cast<double>(r[k]);
            double y = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double z = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y += z;
            }
            const unsigned some = __ballot_sync(0xffffffffu, x > 0.0), over = __ballot_sync(0xffffffffu, x > 0.0 && run + y > goal);
            const int at = over ? __ffs(over) - 1 : (some ? 31 - __clz(some) : -1);
            if (at >= 0) {
                int e = -1;
                double s = run + y - x;
#pragma unroll
                for (int k = 0; k < VEC; k++) {
                    if (r[k] > 0.f && !(s > goal)) e = k;
                    s += static_cast<double>(r[k]);
                }
                token = __shfl_sync(0xffffffffu, (i0 + lane) * VEC - P.skew + e, at);
                if (over) break;
            }
            run += __shfl_sync(0xffffffffu, y, 31);
        }
        if (lane == 0) p.token[b] = token;
    });
}

template <typename T>
cudaError_t verify(const VerifyParams &p, cudaStream_t s) {
    // a slice of 8192 elements or more a CTA: 16 a thread
    int ctas = 1;
    while (ctas < kVerMaxCtas && p.V / (2 * ctas) >= 8192) ctas *= 2;
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
