// tq_tree.cu -- attention of a tree of drafted tokens over the compressed cache.
//
// For query row r (draft i, head j of the KV head's group) and token t with key
// k_t, value v_t: x_t = q_r . k_t log2(e) / sqrt(d), m = max x_t, l = sum 2^(x_t -
// m), o = sum 2^(x_t - m) v_t / l.  Packed tokens have k_t = R y_t, so x_t = (R q) .
// y_t and their share of o is R sum 2^(x_t - m) z_t: scores and sums run in the
// rotated space, one R follows the merge.
//
// This file holds the form for every head dimension and the merge.  A CTA takes an equal
// range of the tile list (tq_serve.h), stages 8 to 32 tokens at a time as
// binary32 rows in shared memory and keeps the running max, sum and values of up to
// 16 query rows: CUDA cores in binary32, the simplest form, for head dimensions that models
// rarely have (256: 16 drafts of 4 heads over 4096 tokens of 8 heads 610 us, 2 drafts 169).
#include <algorithm>

#include <cuda_fp16.h>

#include "tq_serve.h"
#include "tq_team.cuh"
#include "tq_tree.cuh"

namespace tqk {
namespace {

using namespace tree;

constexpr int kTreeThreads = 128;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D>
struct Plain {
    static constexpr int R = D <= 256 ? 16 : 8;                    // query rows
    static constexpr int TT = D <= 256 ? 32 : 8192 / D;            // tokens staged
    static constexpr int DPT = (D + kTreeThreads - 1) / kTreeThreads;
    static constexpr int LD = D + 1;                               // row stride: columns in different banks
    static constexpr size_t smem = (2 * R * LD + TT * LD + R * TT + 3 * R) * sizeof(float);
};

// Element e of token t of K or V in binary32, rotated space for packed segments.
template <int D>
__device__ __forceinline__ float tile_value(const TreeParams &p, const Walk &w, int kv, int t, int e) {
    const Pos &x = w.x;
    const SegView &s = p.seg[w.seg].seg;
    const uint8_t *base = (kv ? s.v : s.k) + x.b * (kv ? s.vblock : s.kblock) + (kv ? s.voff[x.h] : s.koff[x.h]);
    if (s.fp16) return __half2float(reinterpret_cast<const __half *>(base)[static_cast<size_t>(t) * D + e]);
    const int bits = kv ? s.vbits[x.h] : s.kbits[x.h];
    const uint32_t c = code_at(base + static_cast<size_t>(t) * (D * bits / 8), e, bits);
    const float sc = (kv ? s.vs : s.ks)[(static_cast<size_t>(x.b) * p.H + x.h) * s.capacity + t];
    if (kv) return sc * p.centroid[p.seg[w.seg].law][cb_off(bits) + c];
    return sc * (static_cast<float>(2 * c + 1) * __uint_as_float(static_cast<uint32_t>(127 - bits) << 23) - 1.0f);
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads) tree_plain_kernel(const __grid_constant__ TreeParams p) {
    using C = Plain<D>;
    constexpr int R = C::R, TT = C::TT, LD = C::LD, DPT = C::DPT;
    extern __shared__ float sm[];
    float *q0 = sm, *q1 = q0 + R * LD, *tok = q1 + R * LD, *S = tok + TT * LD;  // q, R q, tokens, scores
    float *row_m = S + R * TT, *row_l = row_m + R, *row_c = row_l + R;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.error = 0;
    asm volatile("griddepcontrol.launch_dependents;");
    const unsigned T = total_tiles(p), per = worker_tiles(p, T), c = blockIdx.x;
    unsigned at = c * per;
    if (at >= T) return;
    const unsigned end = min(at + per, T);
    Walk w = walk_begin(p, at);
    float acc[R][DPT];
    int part = -1;
    auto restart = [&] {
        __syncthreads();
        for (int r = threadIdx.x; r < R; r += kTreeThreads) row_m[r] = -kInf, row_l[r] = 0.f;
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int e = 0; e < DPT; e++) acc[r][e] = 0.f;
        __syncthreads();
    };
    auto flush = [&] {  // the record of `part`
        __syncthreads();
        float *rec = p.part + (static_cast<size_t>(c) + part) * R * (D + 4);
        for (int r = threadIdx.x; r < R; r += kTreeThreads) {
            rec[r * (D + 4)] = row_m[r];
            rec[r * (D + 4) + 1] = row_l[r];
        }
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int e = 0; e < DPT; e++) {
                const int i = threadIdx.x + e * kTreeThreads;
                if (i < D) rec[r * (D + 4) + 4 + i] = acc[r][e];
            }
    };
    for (; at < end; at++, walk_next(p, w)) {
        const Pos &x = w.x;
        if (w.first) {
            if (part >= 0) flush();
            part = w.part;
            restart();
        }
        if (w.fresh) {  // the block's query rows, as they are and rotated
            __syncthreads();
            for (int r = warp; r < R; r += kTreeWarps) {
                const int row = x.rb * R + r;
                float v[(D + 31) / 32];
#pragma unroll
                for (int j = 0; j < (D + 31) / 32; j++) {
                    const int e = lane + 32 * j;
                    v[j] = 0.f;
                    if (row < p.N * p.g && e < D)
                        v[j] = __half2float(__ushort_as_half(
                            p.q[x.b * p.qs[0] + (row / p.g) * p.qs[1] + (x.h * p.g + row % p.g) * p.qs[2] + e]));
                    if (e < D) q0[r * LD + e] = v[j];
                }
                warp_rotate_strided<D>(v, p.sign_bits, p.inv_sqrt_d, lane);
#pragma unroll
                for (int j = 0; j < (D + 31) / 32; j++)
                    if (lane + 32 * j < D) q1[r * LD + lane + 32 * j] = v[j];
            }
        }
        const float *q = x.k < x.tp ? q1 : q0;
        const int hi = min(w.n, (w.t + 1) * kTreeTile);
        for (int t0 = w.t * kTreeTile; t0 < hi; t0 += TT) {
            const int nt = min(TT, hi - t0);
            __syncthreads();
            for (int i = threadIdx.x; i < nt * D; i += kTreeThreads)
                tok[(i / D) * LD + i % D] = tile_value<D>(p, w, 0, t0 + i / D, i % D);
            __syncthreads();
            for (int i = threadIdx.x; i < R * TT; i += kTreeThreads) {
                const int r = i / TT, t = i % TT;
                float s = -kInf;
                if (t < nt) {
                    s = 0.f;
                    for (int e = 0; e < D; e++) s = fmaf(q[r * LD + e], tok[t * LD + e], s);
                    s *= p.qk_scale;
                }
                S[i] = s;
            }
            __syncthreads();
            for (int r = warp; r < R; r += kTreeWarps) {
                const float s = lane < TT ? S[r * TT + lane] : -kInf;
                float m = s;
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float old = row_m[r], now = fmaxf(old, m);
                const float pr = s == -kInf ? 0.f : ex2(s - now);  // (no NaN from -inf - -inf)
                float l = pr;
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                const float f = now == -kInf ? 1.f : ex2(old - now);
                if (lane < TT) S[r * TT + lane] = pr;
                __syncwarp();
                if (lane == 0) row_m[r] = now, row_l[r] = row_l[r] * f + l, row_c[r] = f;
            }
            for (int i = threadIdx.x; i < nt * D; i += kTreeThreads)
                tok[(i / D) * LD + i % D] = tile_value<D>(p, w, 1, t0 + i / D, i % D);
            __syncthreads();
#pragma unroll
            for (int e = 0; e < DPT; e++) {
                const int i = threadIdx.x + e * kTreeThreads;
                if (i < D) {
#pragma unroll
                    for (int r = 0; r < R; r++) acc[r][e] *= row_c[r];
                    for (int t = 0; t < nt; t++) {
                        const float v = tok[t * LD + i];
#pragma unroll
                        for (int r = 0; r < R; r++) acc[r][e] = fmaf(S[r * TT + t], v, acc[r][e]);
                    }
                }
            }
        }
    }
    flush();
}

// ---------------------------------------------------------------- merge
// A lane's J consecutive coordinates of a row (D < 32: lanes below D hold one); vec: by one
// load (J >= 8: of 16 bytes).
template <int D>
struct RowOf {
    static constexpr int J = D >= 32 ? D / 32 : 1;
};
template <int D>
__device__ __forceinline__ void load_row(const uint16_t *row, int lane, bool vec, uint16_t (&x)[RowOf<D>::J]) {
    constexpr int J = RowOf<D>::J;
    row += lane * J;
    if constexpr (J == 1) {
        x[0] = lane < D ? __ldg(row) : 0;
    } else if (!vec) {
#pragma unroll
        for (int j = 0; j < J; j++) x[j] = __ldg(row + j);
    } else if constexpr (J == 2) {
        *reinterpret_cast<uint32_t *>(x) = __ldg(reinterpret_cast<const uint32_t *>(row));
    } else if constexpr (J == 4) {
        *reinterpret_cast<uint2 *>(x) = __ldg(reinterpret_cast<const uint2 *>(row));
    } else {
#pragma unroll
        for (int j = 0; j < J; j += 8)
            *reinterpret_cast<uint4 *>(x + j) = __ldg(reinterpret_cast<const uint4 *>(row + j));
    }
}
template <int D>
__device__ __forceinline__ void load_sums(const float *row, int lane, bool valid, float (&x)[RowOf<D>::J]) {
    constexpr int J = RowOf<D>::J;
    row += lane * J;
    if constexpr (J == 1) {
        x[0] = valid && lane < D ? __ldcg(row) : 0.f;
    } else if constexpr (J == 2) {
        const float2 v = valid ? __ldcg(reinterpret_cast<const float2 *>(row)) : make_float2(0.f, 0.f);
        x[0] = v.x, x[1] = v.y;
    } else {
#pragma unroll
        for (int j = 0; j < J; j += 4) {
            const float4 v = valid ? __ldcg(reinterpret_cast<const float4 *>(row + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
        }
    }
}
// R x of a row held like that (any order of the sums: attention arithmetic).
template <int D>
__device__ __forceinline__ void rotate_row(float (&x)[RowOf<D>::J], const uint32_t *sb, float c, int lane) {
    constexpr int J = RowOf<D>::J;
    const uint32_t neg = lane * J < D ? sb[lane * J >> 5] >> (lane * J & 31) : 0u;
#pragma unroll
    for (int j = 0; j < J; j++)
        if ((neg >> j) & 1u) x[j] = -x[j];
#pragma unroll
    for (int h = 1; h < J; h <<= 1)
#pragma unroll
        for (int j = 0; j < J; j++)
            if ((j & h) == 0) {
                const float u = x[j], v = x[j + h];
                x[j] = u + v, x[j + h] = u - v;
            }
#pragma unroll
    for (int h = J; h < D; h <<= 1) {
        const float sg = (lane & (h / J)) ? -1.f : 1.f;
#pragma unroll
        for (int j = 0; j < J; j++) x[j] = fmaf(x[j], sg, __shfl_xor_sync(0xffffffffu, x[j], h / J));
    }
#pragma unroll
    for (int j = 0; j < J; j++) x[j] *= ((neg >> j) & 1u) ? -c : c;
}

// A warp per query row: the drafted tokens that the row sees, in binary32 (few tokens
// per row, so that neither the mask nor a non-finite value of an unseen draft can
// reach the row), every record of its group in order, R on the packed share, the
// quotient, and the fp16 row.  The call's bytes here are few; what counts is the
// chain of loads, so F drafts' keys and values or U records are in flight at a time, and the
// drafts come before the wait for the records (the grid may start while the last
// CTAs of the main kernel run).
// U: 16 where the rows are too few to fill the GPU anyway (up to 4096), else 8, with
// which twice the warps fit.  8192 rows of 3 records: 31 us alone, 512 of 24: 12 us.
template <int D, int U>
__global__ void __launch_bounds__(kTreeThreads) tree_merge_kernel(const __grid_constant__ TreeMergeParams p) {
    constexpr int J = RowOf<D>::J;
    constexpr int F = J <= 8 ? 4 : 32 / J;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.t.N * p.t.g;
    const unsigned id = blockIdx.x * kTreeWarps + warp;  // (b, h, row)
    if (id >= static_cast<unsigned>(rows) * p.t.B * p.t.H) return;
    const int bh = id / rows, row = id - bh * rows;
    const int b = bh / p.t.H, h = bh - b * p.t.H, rb = row / p.t.R, r = row - rb * p.t.R;
    const int draft = row / p.t.g, head = h * p.t.g + row - draft * p.t.g;
    float M = -kInf, L = 0.f, a[2][J];
    bool nan = false;  // fmaxf passes over NaN: a row that sees only NaN scores is NaN, not empty
#pragma unroll
    for (int j = 0; j < J; j++) a[0][j] = a[1][j] = 0.f;
    {
        float q[J];
        __align__(16) uint16_t q16[J];
        load_row<D>(p.q + b * p.qs[0] + draft * p.qs[1] + head * p.qs[2], lane, p.vec, q16);
#pragma unroll
        for (int j = 0; j < J; j++) q[j] = __half2float(__ushort_as_half(q16[j]));
        const uint16_t *K = p.k + b * p.ks[0] + h * p.ks[1], *V = p.v + b * p.vs[0] + h * p.vs[1];
#pragma unroll 1
        for (int w = 0; w < p.mask_words; w++) {
#pragma unroll 1
            for (uint32_t m = seen_word(p, p.t.N, b, draft, w); m;) {
                const int some = min(__popc(m), F);
                __align__(16) uint16_t k16[F][J], v16[F][J];
                float s[F];
#pragma unroll
                for (int i = 0; i < F; i++) {
                    if (i < some) {
                        const int t = 32 * w + __ffs(m) - 1;
                        m &= m - 1;
                        load_row<D>(K + t * p.ks[2], lane, p.vec, k16[i]);
                        load_row<D>(V + t * p.vs[2], lane, p.vec, v16[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < F; i++) {
                    s[i] = 0.f;
                    if (i < some)
#pragma unroll
                        for (int j = 0; j < J; j++) s[i] = fmaf(q[j], __half2float(__ushort_as_half(k16[i][j])), s[i]);
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
                    for (int i = 0; i < F; i++) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
                float now = M;
#pragma unroll
                for (int i = 0; i < F; i++)
                    if (i < some) {
                        s[i] *= p.qk_scale;
                        now = fmaxf(now, s[i]);
                        nan |= s[i] != s[i];
                    }
                if (now == -kInf) continue;
                const float old = M == -kInf ? 0.f : ex2(M - now);
                M = now;
                L *= old;
#pragma unroll
                for (int j = 0; j < J; j++) a[1][j] *= old;
#pragma unroll
                for (int i = 0; i < F; i++)
                    if (i < some) {
                        const float f = ex2(s[i] - now);
                        L += f;
#pragma unroll
                        for (int j = 0; j < J; j++) a[1][j] = fmaf(f, __half2float(__ushort_as_half(v16[i][j])), a[1][j]);
                    }
            }
        }
    }
    // where the group's tiles lie in the list
    const unsigned T = total_tiles(p.t), per = worker_tiles(p.t, T);
    int tp, tf;
    seq_tiles(p.t, b, tp, tf);
    unsigned first = 0;
    if (p.t.ragged) {
        for (int i = lane; i < b; i += 32) {
            int x, y;
            seq_tiles(p.t, i, x, y);
            first += x + y;
        }
        first = __reduce_add_sync(0xffffffffu, first);
    } else {
        first = b * (tp + tf);
    }
    first = first * p.t.H * p.t.n_rb + (h * p.t.n_rb + rb) * (tp + tf);
    const int group = bh * p.t.n_rb + rb;
    const int np = (tp + kTreePart - 1) / kTreePart, nf = (tf + kTreePart - 1) / kTreePart;
    // part i (packed ones, then the others): workers lo..hi hold its records
    // Record `at` of the group (in order: the parts', within one its workers'): its slot, or -1;
    // kind: packed or not; n: the group's records
    auto locate = [&](int at, int &kind, int &n) {
        int slot = -1;
        n = 0;
#pragma unroll 1
        for (int i = 0; i < np + nf; i++) {
            const int k0 = i < np ? i * kTreePart : tp + (i - np) * kTreePart;
            const int k1 = min(k0 + kTreePart, i < np ? tp : tp + tf);
            const int lo = (first + k0) / per, hi = (first + k1 - 1) / per;
            if (at >= n && at - n <= hi - lo) slot = lo + at - n + part_of(p.t, group, tp, k0), kind = i >= np;
            n += hi - lo + 1;
        }
        return slot;
    };
    int kind = 0, records, slot = locate(lane, kind, records);
    const float *rows_at = p.part + static_cast<size_t>(r) * (D + 4);
    const size_t stride = static_cast<size_t>(p.t.R) * (D + 4);
    asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 1
    for (int base = 0; base < records; base += 32) {  // a record per lane, then U of them at a time
        if (base) slot = locate(base + lane, kind, records);
        float2 ml = make_float2(-kInf, 0.f);
        if (slot >= 0) ml = __ldcg(reinterpret_cast<const float2 *>(rows_at + slot * stride));
        const int count = min(32, records - base);
        float f = 0.f;
#pragma unroll 1
        for (int u0 = 0; u0 < count; u0 += U) {
            float v[U][J];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int s = __shfl_sync(0xffffffffu, slot, u0 + u);
                load_sums<D>(rows_at + max(s, 0) * stride + 4, lane, s >= 0, v[u]);
            }
            if (u0 == 0) {  // (the first loads are on their way) the new largest m
                float now = fmaxf(M, ml.x);
                nan |= ml.y != ml.y;
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
                if (now == -kInf) break;
                const float old = M == -kInf ? 0.f : ex2(M - now);
                f = ex2(ml.x - now);
                M = now;
                L *= old;
#pragma unroll
                for (int j = 0; j < J; j++) a[0][j] *= old, a[1][j] *= old;
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                const float fu = __shfl_sync(0xffffffffu, f, u0 + u);
                const bool raw = __shfl_sync(0xffffffffu, kind, u0 + u);
                L = fmaf(__shfl_sync(0xffffffffu, ml.y, u0 + u), fu, L);
                // (left out, not weighted by zero, of the sum that R spreads: an infinity among unrotated
                // values stays in its coordinate)
#pragma unroll
                for (int j = 0; j < J; j++) {
                    a[0][j] = fmaf(fu, raw ? 0.f : v[u][j], a[0][j]);
                    a[1][j] = fmaf(raw ? fu : 0.f, v[u][j], a[1][j]);
                }
            }
        }
    }
    nan = __any_sync(0xffffffffu, nan);
    rotate_row<D>(a[0], p.sign_bits, p.inv_sqrt_d, lane);
    const float inv = nan ? __int_as_float(0x7fffffff) : L == 0.f ? 0.f : 1.0f / L;  // nothing seen: zeros
    uint16_t *out = p.out + ((static_cast<size_t>(b) * p.t.N + draft) * p.t.H * p.t.g + head) * D;
    __align__(16) uint16_t o16[J];
#pragma unroll
    for (int j = 0; j < J; j++) o16[j] = __half_as_ushort(__float2half_rn((a[0][j] + a[1][j]) * inv));
    out += lane * J;
    if constexpr (J == 1) {
        if (lane < D) *out = o16[0];
    } else if constexpr (J == 2) {
        *reinterpret_cast<uint32_t *>(out) = *reinterpret_cast<const uint32_t *>(o16);
    } else if constexpr (J == 4) {
        *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<const uint2 *>(o16);
    } else {
#pragma unroll
        for (int j = 0; j < J; j += 8) *reinterpret_cast<uint4 *>(out + j) = *reinterpret_cast<const uint4 *>(o16 + j);
    }
}

template <int D>
cudaError_t tree_dim(const TreeParams &p, cudaStream_t s) {
    cudaError_t e;
    if (p.n_seg == 0) {  // drafts alone
        e = cudaMemsetAsync(p.error, 0, sizeof(int), s);
        if (e != cudaSuccess) return e;
    } else if constexpr (D == 64 || D == 128) {
        e = launch_tree_mma(p, s);
        if (e != cudaSuccess) return e;
    } else {
        e = cudaFuncSetAttribute(tree_plain_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(Plain<D>::smem));
        if (e != cudaSuccess) return e;
        tree_plain_kernel<D><<<p.workers, kTreeThreads, Plain<D>::smem, s>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    TreeMergeParams m;
    m.t.B = p.B, m.t.H = p.H, m.t.g = p.g, m.t.N = p.N, m.t.R = p.R, m.t.n_rb = p.n_rb;
    m.t.n_seg = p.n_seg, m.t.n_packed = p.n_packed, m.t.ragged = p.ragged;
    m.t.parts_packed = p.parts_packed, m.t.parts = p.parts, m.t.workers = p.workers;
    for (int i = 0; i < TQ_MAX_SEGMENTS; i++) m.t.seg[i].len = p.seg[i].len, m.t.seg[i].n_tokens = p.seg[i].n_tokens;
    m.q = p.q, m.k = p.k, m.v = p.v, m.mask = p.mask, m.out = p.out, m.part = p.part;
    m.mask_stride = p.mask_stride, m.mask_words = p.mask_words;
    for (int i = 0; i < 3; i++) m.qs[i] = p.qs[i], m.ks[i] = p.ks[i], m.vs[i] = p.vs[i];
    std::copy(p.sign_bits, p.sign_bits + kMaxD / 32, m.sign_bits);
    m.inv_sqrt_d = p.inv_sqrt_d, m.qk_scale = p.qk_scale;
    const int unit = std::min(8, RowOf<D>::J);  // elements of a lane's load
    uintptr_t odd = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v);
    for (int i = 0; i < 3; i++) odd |= static_cast<uintptr_t>((p.qs[i] | p.ks[i] | p.vs[i]) * 2);
    m.vec = odd % (2 * unit) == 0;
    const long long rows = static_cast<long long>(p.N) * p.g * p.B * p.H;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows + kTreeWarps - 1) / kTreeWarps));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.n_seg > 0 ? 1 : 0;  // (behind a kernel)
    if constexpr (D <= 128) {
        if (rows <= 4096) return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 16>, m);
        return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 8>, m);
    } else {
        return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 1024 / D>, m);
    }
}

}  // namespace

TreeShape tree_shape(int B, int H, int g, int N, int d, long long tiles_per_head) {
    TreeShape t;
    const int rows = N * g;
    // tensor cores: one CTA per SM
    if (tree_on_tensor_cores(d)) t.R = tree_mma_rows(rows);
    else t.R = d <= 256 ? 16 : 8;
    t.n_rb = (rows + t.R - 1) / t.R;
    const long long tiles = static_cast<long long>(B) * H * t.n_rb * tiles_per_head;
    const long long ctas = static_cast<long long>(current_sm_count()) * (tree_on_tensor_cores(d) ? 1 : 4);
    t.workers = static_cast<int>(std::min<long long>(std::max<long long>(tiles, 1), ctas));
    return t;
}

cudaError_t launch_tree(const TreeParams &p, cudaStream_t s) {
    switch (p.d) {
        case 16: return tree_dim<16>(p, s);
        case 32: return tree_dim<32>(p, s);
        case 64: return tree_dim<64>(p, s);
        case 128: return tree_dim<128>(p, s);
        case 256: return tree_dim<256>(p, s);
        case 512: return tree_dim<512>(p, s);
        case 1024: return tree_dim<1024>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tqk
