// tq_paged.cu -- attention of one new token of each sequence over paged segments: the
// form for every head dimension, and the merge of the records.
//
// The plain form works in binary32 on the CUDA cores: a CTA takes a range of the stage
// list (tq_paged.cuh), dequantizes some tokens at a time into shared memory, scores them
// against the block's rotated queries (fp16 segments: the queries as they are) with an
// online softmax, and sums the values.  Head dimensions 64 and 128 take tq_paged_mma.cuh
// (32 sequences of up to 16384 tokens of 8 heads, K4V4 and fp16 sinks: 102 to 114 us there by the lengths drawn, 8202 us in this form;
// 8 x 4096 tokens K4V4 of head_dim 256, bound by its scalar reads of codes: 1474 us).
#include <algorithm>
#include <cstring>

#include <cuda_fp16.h>

#include "tq_paged.cuh"
#include "tq_serve.h"
#include "tq_team.cuh"

namespace tqk {
namespace {

using namespace paged;

constexpr float kInf = __builtin_huge_valf();
constexpr int kPlainThreads = 256;
constexpr int kPlainWarps = kPlainThreads / 32;
constexpr int kPlainRows = 4;
constexpr int kPlainUnit = 64;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D>
struct Plain {
    static constexpr int R = kPlainRows, TT = D >= 512 ? 16 : 32, LD = D + 1;
    static constexpr int DPT = (D + kPlainThreads - 1) / kPlainThreads;
    static constexpr size_t smem = (R * LD + TT * LD + R * TT + 3 * R) * sizeof(float);
};

// Coordinate i of a token's key (kv 0) or value, in the rotated space.
template <int D>
__device__ __forceinline__ float token_value(const PagedParams &p, const PagedSeg &s, int kv, int page, int h, int t, int i) {
    const SegView &v = s.seg;
    const uint8_t *head = (kv ? v.v : v.k) + page * (kv ? v.vblock : v.kblock) + (kv ? v.voff[h] : v.koff[h]);
    if (v.fp16) return __half2float(__ushort_as_half(reinterpret_cast<const uint16_t *>(head)[static_cast<size_t>(t) * D + i]));
    const int bits = kv ? p.cls.vb : p.cls.kb;
    const uint32_t code = code_at(head + static_cast<size_t>(t) * (D * bits / 8), i, bits);
    const float scale = (kv ? v.vs : v.ks)[(static_cast<size_t>(page) * p.list.H + h) * v.capacity + t];
    if (kv) return scale * p.centroid[cb_off(bits) + code];
    return scale * (static_cast<float>(2 * code + 1) / static_cast<float>(1 << bits) - 1.0f);
}

template <int D>
__global__ void __launch_bounds__(kPlainThreads) paged_plain_kernel(const __grid_constant__ PagedParams p) {
    using C = Plain<D>;
    constexpr int R = C::R, TT = C::TT, LD = C::LD, DPT = C::DPT;
    extern __shared__ float sm[];
    __shared__ int buf[kPlainWarps + 4];
    float *q = sm, *tok = q + R * LD, *S = tok + TT * LD;  // queries in the segment's space; tokens; scores
    float *row_m = S + R * TT, *row_l = row_m + R, *row_c = row_l + R;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, worker = blockIdx.x;
    asm volatile("griddepcontrol.launch_dependents;");
    const PagedList &l = p.list;
    ranges_of<kPlainThreads, 1>(l, p.cls, Share<kPlainThreads>(l, p.cls), worker, 0, p.first, buf);
    const int begin = buf[kPlainWarps + 2], end = buf[kPlainWarps + 3];
    if (begin < end) {
        Walk w = seek(l, p.cls, buf[kPlainWarps], buf[kPlainWarps + 1]);
        float acc[R][DPT];
        bool fresh = true;
        for (int at = begin; at < end; at++) {
            if (fresh) {
                __syncthreads();
                for (int i = threadIdx.x; i < R; i += kPlainThreads) row_m[i] = -kInf, row_l[i] = 0.f;
#pragma unroll
                for (int i = 0; i < R; i++)
#pragma unroll
                    for (int e = 0; e < DPT; e++) acc[i][e] = 0.f;
                for (int i = warp; i < R; i += kPlainWarps) {
                    const int row = w.rb * R + i;
                    float v[(D + 31) / 32];
#pragma unroll
                    for (int j = 0; j < (D + 31) / 32; j++) {
                        const int e = lane + 32 * j;
                        v[j] = row < p.g && e < D ? __half2float(__ushort_as_half(p.q[w.b * p.qs[0] + (w.h * p.g + row) * p.qs[1] + e])) : 0.f;
                    }
                    if (p.cls.kb) warp_rotate_strided<D>(v, p.sign_bits, p.inv_sqrt_d, lane);
#pragma unroll
                    for (int j = 0; j < (D + 31) / 32; j++)
                        if (lane + 32 * j < D) q[i * LD + lane + 32 * j] = v[j];
                }
                __syncthreads();
            }
            const PagedSeg &s = p.seg[p.cls.seg[w.i]];
            const int hi = min(w.tokens, (w.st + 1) * kPlainUnit);
            for (int t0 = w.st * kPlainUnit; t0 < hi; t0 += TT) {
                const int nt = min(TT, hi - t0);
                __syncthreads();
                for (int i = threadIdx.x; i < nt * D; i += kPlainThreads) {
                    const int t = t0 + i / D, page = page_at(s, w.b, t / s.page);
                    tok[(i / D) * LD + i % D] = page < 0 ? 0.f : token_value<D>(p, s, 0, page, w.h, t % s.page, i % D);
                }
                __syncthreads();
                for (int i = threadIdx.x; i < R * TT; i += kPlainThreads) {
                    const int row = i / TT, t = i % TT;
                    float x = -kInf;
                    if (t < nt && page_at(s, w.b, (t0 + t) / s.page) >= 0) {
                        x = 0.f;
                        for (int e = 0; e < D; e++) x = fmaf(q[row * LD + e], tok[t * LD + e], x);
                        x *= p.qk_scale;
                    }
                    S[i] = x;
                }
                __syncthreads();
                for (int row = warp; row < R; row += kPlainWarps) {
                    const float x = lane < TT ? S[row * TT + lane] : -kInf;
                    float m = x;
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float old = row_m[row], now = fmaxf(old, m);
                    const float pr = x == -kInf ? 0.f : ex2(x - now);
                    float sum = pr;
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float f = now == -kInf ? 1.f : ex2(old - now);
                    if (lane < TT) S[row * TT + lane] = pr;
                    __syncwarp();
                    if (lane == 0) row_m[row] = now, row_l[row] = row_l[row] * f + sum, row_c[row] = f;
                }
                for (int i = threadIdx.x; i < nt * D; i += kPlainThreads) {
                    const int t = t0 + i / D, page = page_at(s, w.b, t / s.page);
                    tok[(i / D) * LD + i % D] = page < 0 ? 0.f : token_value<D>(p, s, 1, page, w.h, t % s.page, i % D);
                }
                __syncthreads();
#pragma unroll
                for (int e = 0; e < DPT; e++) {
                    const int i = threadIdx.x + e * kPlainThreads;
                    if (i < D) {
#pragma unroll
                        for (int row = 0; row < R; row++) acc[row][e] *= row_c[row];
                        for (int t = 0; t < nt; t++) {
                            const float v = tok[t * LD + i];
#pragma unroll
                            for (int row = 0; row < R; row++) acc[row][e] = fmaf(S[row * TT + t], v, acc[row][e]);
                        }
                    }
                }
            }
            const Walk x = w;
            const bool last = at + 1 == end;
            fresh = false;
            if (!last && ++w.st == w.n_st) {
                w = next(l, p.cls, w);
                fresh = w.fresh;
            }
            if (!fresh && !last) continue;
            __syncthreads();
            float *rec = p.part + p.cls.part0 + group_slot(l, p.cls, worker, x.b, x.h, x.rb) * R * (D + 4);
            for (int i = threadIdx.x; i < R; i += kPlainThreads) {
                rec[i * (D + 4)] = row_m[i];
                rec[i * (D + 4) + 1] = row_l[i];
            }
#pragma unroll
            for (int i = 0; i < R; i++)
#pragma unroll
                for (int e = 0; e < DPT; e++) {
                    const int k = threadIdx.x + e * kPlainThreads;
                    if (k < D) rec[i * (D + 4) + 4 + k] = acc[i][e];
                }
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the call's last launch ends behind its first
}

// ------------------------------------------------------------------- merge
// A CTA for each row (sequence, query head): the records of its (b, h, rb), class by class, with
// the weights 2^(m - M); packed classes' sums turn back from the rotated space together.  Threads: quads of
// coordinates times records in flight.
constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ PagedMergeParams p) {
    __shared__ __align__(16) float sum[2][kMergeThreads * 4];  // [space][record lane][d]
    __shared__ float red[kMergeThreads / 32];
    __shared__ int span[kPagedClasses][2];                    // first and last worker of the row's group
    const int d = p.d, B = p.list.B, H = p.list.H;
    const int row = blockIdx.x, b = row / (H * p.g), h = row / p.g % H, j = row % p.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x < p.n_classes) {
        const PagedClass &c = p.cls[threadIdx.x];
        const int *first = p.first + static_cast<size_t>(threadIdx.x) * (B + 1);
        const int n = head_stages(p.list, c, b, h);
        int w0 = 0, w1 = -1;
        if (n > 0) {
            int s = first[b] + j / c.R * n;
            for (int i = 0; i < h; i++) s += c.n_rb * head_stages(p.list, c, b, i);
            const int workers = workers_of(c, first[B]);
            w0 = max(worker_of(first[B], s, workers), 0);
            w1 = min(worker_of(first[B], s + n - 1, workers), workers - 1);
        }
        span[threadIdx.x][0] = w0;
        span[threadIdx.x][1] = w1;
    }
    if (row == 0 && threadIdx.x == 0) *p.error = 0;
    __syncthreads();
    auto record = [&](int c, int w) {
        const PagedClass &k = p.cls[c];
        return p.part + k.part0 + (group_slot(p.list, k, w, b, h, j / k.R) * k.R + j % k.R) * (d + 4);
    };
    // the largest m
    float M = -kInf;
    for (int c = 0; c < p.n_classes; c++)
        for (int w = span[c][0] + threadIdx.x; w <= span[c][1]; w += kMergeThreads) M = fmaxf(M, record(c, w)[0]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) red[warp] = M;
    __syncthreads();
    for (int i = 0; i < kMergeThreads / 32; i++) M = fmaxf(M, red[i]);
    const int quads = d / 4, lanes = kMergeThreads / quads, quad = threadIdx.x % quads, rl = threadIdx.x / quads;
    float L = 0.f;  // (of the record lane)
    float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (M != -kInf) {
        for (int c = 0; c < p.n_classes; c++) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = span[c][0] + rl; w <= span[c][1]; w += lanes) {
                const float *rec = record(c, w);
                const float2 ml = *reinterpret_cast<const float2 *>(rec);
                const float4 x = *reinterpret_cast<const float4 *>(rec + 4 + 4 * quad);
                const float f = ex2(ml.x - M);
                L = fmaf(ml.y, f, L);
                a.x = fmaf(x.x, f, a.x);
                a.y = fmaf(x.y, f, a.y);
                a.z = fmaf(x.z, f, a.z);
                a.w = fmaf(x.w, f, a.w);
            }
            float4 &to = s[p.cls[c].kb ? 1 : 0];
            to.x += a.x, to.y += a.y, to.z += a.z, to.w += a.w;
        }
    }
#pragma unroll
    for (int k = 0; k < 2; k++) *reinterpret_cast<float4 *>(&sum[k][rl * d + 4 * quad]) = s[k];
    __shared__ float lsum[kMergeThreads];  // [record lane]
    if (quad == 0) lsum[rl] = L;
    __syncthreads();
    L = 0.f;
    for (int i = 0; i < lanes; i++) L += lsum[i];
    for (int i = threadIdx.x; i < 2 * d; i += kMergeThreads) {
        float *x = sum[i >= d] + i % d;
        float a = x[0];
        for (int k = 1; k < lanes; k++) a += x[k * d];
        // the rotated sum's first sign flip
        x[0] = i >= d && ((p.sign_bits[(i - d) >> 5] >> ((i - d) & 31)) & 1u) ? -a : a;
    }
    __syncthreads();
    for (int o = 1; o < d; o <<= 1) {
        for (int i = threadIdx.x; i < d / 2; i += kMergeThreads) {
            const int at = 2 * o * (i / o) + i % o;
            const float x = sum[1][at], y = sum[1][at + o];
            sum[1][at] = x + y;
            sum[1][at + o] = x - y;
        }
        __syncthreads();
    }
    const float scale = L != 0.f ? 1.f / L : 0.f;  // (no token: zeros; a NaN stays one)
    for (int i = threadIdx.x; i < d; i += kMergeThreads) {
        const float y = ((p.sign_bits[i >> 5] >> (i & 31)) & 1u) ? -p.inv_sqrt_d : p.inv_sqrt_d;
        p.out[static_cast<size_t>(row) * d + i] = __half_as_ushort(__float2half_rn(fmaf(sum[1][i], y, sum[0][i]) * scale));
    }
}

// The merge at the head dims of the tensor-core forms: warps instead of a CTA for a row, W of them where the records
// are many, a lane four (two) coordinates of every record, four records in flight.  Where they lie is worked out from
// the lengths before the records are waited for (up to kScan sequences; behind that from the scan that the first CTA left).
constexpr int kRowWarps = 8;
constexpr int kScan = 256;

template <int D>
__global__ void __launch_bounds__(32 * kRowWarps) paged_merge_rows_kernel(const __grid_constant__ PagedMergeParams p, const int W) {
    constexpr int E = D / 32;
    struct alignas(16) Part {
        float x[2][D];
        float m, l, pad[2];
    };
    __shared__ Part parts[kRowWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, share = warp % W;
    const PagedList &l = p.list;
    const int rows = l.B * l.H * p.g, row = blockIdx.x * (kRowWarps / W) + warp / W;
    const int b = min(row, rows - 1) / (l.H * p.g), h = min(row, rows - 1) / p.g % l.H, j = min(row, rows - 1) % p.g;
    // the first and the last worker of the row's group in class k
    auto span = [&](int k, bool scan, int &w0, int &w1) {
        const PagedClass &c = p.cls[k];
        const int n = head_stages(l, c, b, h);
        int before = 0, total = 0;
        if (scan) {
            for (int i = lane; i < l.B; i += 32) {
                const int x = sequence_stages(l, c, i);
                total += x;
                if (i < b) before += x;
            }
            total = __reduce_add_sync(0xffffffffu, total);
            before = __reduce_add_sync(0xffffffffu, before);
        } else {
            before = p.first[static_cast<size_t>(k) * (l.B + 1) + b];
            total = p.first[static_cast<size_t>(k) * (l.B + 1) + l.B];
        }
        w0 = 0, w1 = -1;
        if (n == 0) return;
        int s = before + j / c.R * n;
        if (c.n == 1) s += __popc(c.heads[0] & ((1u << h) - 1u)) * c.n_rb * n;
        else
            for (int i = 0; i < h; i++) s += c.n_rb * head_stages(l, c, b, i);
        const int workers = workers_of(c, total);
        // (divisions of 64 bits: one lane's for the first, another's for the last)
        const int w = worker_of(total, lane & 1 ? s + n - 1 : s, workers);
        w0 = max(__shfl_sync(0xffffffffu, w, 0), 0);
        w1 = min(__shfl_sync(0xffffffffu, w, 1), workers - 1);
    };
    const bool scan = l.B <= kScan;
    int w0 = 0, w1 = -1;
    if (scan && p.n_classes > 0) span(0, true, w0, w1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.error = 0;
    float M = -kInf, L = 0.f, x[2][E];
#pragma unroll
    for (int e = 0; e < E; e++) x[0][e] = x[1][e] = 0.f;
    for (int k = 0; k < p.n_classes; k++) {
        if (k > 0 || !scan) span(k, scan, w0, w1);
        const PagedClass &c = p.cls[k];
        const float *rec = p.part + c.part0 + (group_slot(l, c, 0, b, h, j / c.R) * c.R + j % c.R) * (D + 4);
        const size_t step = static_cast<size_t>(c.R) * (D + 4);
        float a[E];
#pragma unroll
        for (int e = 0; e < E; e++) a[e] = 0.f;
        float was = M;  // the reference of a
        for (int w = w0 + share; w <= w1; w += 4 * W) {
            float2 ml[4];
            float y[4][E];
            float top = M;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const bool some = w + i * W <= w1;
                const float *r = rec + (some ? w + i * W : w) * step;
                ml[i] = *reinterpret_cast<const float2 *>(r);
                if constexpr (E == 4) *reinterpret_cast<float4 *>(y[i]) = *reinterpret_cast<const float4 *>(r + 4 + 4 * lane);
                else *reinterpret_cast<float2 *>(y[i]) = *reinterpret_cast<const float2 *>(r + 4 + 2 * lane);
                if (!some) ml[i] = make_float2(-kInf, 0.f);
                top = fmaxf(top, ml[i].x);
            }
            if (top == -kInf) continue;  // (records without a token)
            const float f = ex2(M - top), fa = ex2(was - top);
            L *= f;
#pragma unroll
            for (int e = 0; e < E; e++) a[e] *= fa;
#pragma unroll
            for (int s = 0; s < 2; s++)
#pragma unroll
                for (int e = 0; e < E; e++) x[s][e] *= f;
            M = was = top;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (ml[i].x == -kInf) continue;
                const float g = ex2(ml[i].x - M);
                L = fmaf(ml[i].y, g, L);
#pragma unroll
                for (int e = 0; e < E; e++) a[e] = fmaf(y[i][e], g, a[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < E; e++) {
            if (c.kb) x[1][e] += a[e];
            else x[0][e] += a[e];
        }
    }
    if (W > 1) {
        Part &mine = parts[warp];
#pragma unroll
        for (int e = 0; e < E; e++) mine.x[0][E * lane + e] = x[0][e], mine.x[1][E * lane + e] = x[1][e];
        if (lane == 0) mine.m = M, mine.l = L;
        __syncthreads();
        if (share != 0) return;
        float top = M;
        for (int i = 1; i < W; i++) top = fmaxf(top, parts[warp + i].m);
        const float f = M == top ? 1.f : ex2(M - top);
        L *= f;
#pragma unroll
        for (int e = 0; e < E; e++) x[0][e] *= f, x[1][e] *= f;
        for (int i = 1; i < W; i++) {
            const Part &o = parts[warp + i];
            if (o.m == -kInf) continue;
            const float g = ex2(o.m - top);
            L = fmaf(o.l, g, L);
#pragma unroll
            for (int e = 0; e < E; e++) {
                x[0][e] = fmaf(o.x[0][E * lane + e], g, x[0][e]);
                x[1][e] = fmaf(o.x[1][E * lane + e], g, x[1][e]);
            }
        }
    }
    if (row >= rows) return;
    // the rotated sum turns back: signs, butterflies in the lane and across lanes, signs
    const uint32_t neg = p.sign_bits[E * lane >> 5] >> (E * lane & 31);
#pragma unroll
    for (int e = 0; e < E; e++)
        if ((neg >> e) & 1u) x[1][e] = -x[1][e];
#pragma unroll
    for (int o = 1; o < E; o <<= 1)
#pragma unroll
        for (int e = 0; e < E; e++)
            if (!(e & o)) {
                const float u = x[1][e], v = x[1][e + o];
                x[1][e] = u + v;
                x[1][e + o] = u - v;
            }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int e = 0; e < E; e++) {
            const float v = __shfl_xor_sync(0xffffffffu, x[1][e], o);
            x[1][e] = up ? v - x[1][e] : x[1][e] + v;
        }
    }
    const float scale = L != 0.f ? 1.f / L : 0.f;  // (no token: zeros; a NaN stays one)
    __align__(8) __half out[E];
#pragma unroll
    for (int e = 0; e < E; e++)
        out[e] = __float2half_rn(fmaf(x[1][e], (neg >> e) & 1u ? -p.inv_sqrt_d : p.inv_sqrt_d, x[0][e]) * scale);
    uint16_t *to = p.out + static_cast<size_t>(row) * D + E * lane;
    if constexpr (E == 4) *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(out);
    else *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(out);
}

template <int D>
cudaError_t plain(const PagedParams &p, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(paged_plain_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(Plain<D>::smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.cls.workers));
    cfg.blockDim = dim3(kPlainThreads);
    cfg.dynamicSmemBytes = Plain<D>::smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.first_class ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, paged_plain_kernel<D>, p);
}

}  // namespace

#define TQ_PAGED_KB(KB)                                                       \
    cudaError_t launch_paged_kb##KB##_np1(const PagedParams &p, cudaStream_t s);  \
    cudaError_t launch_paged_kb##KB##_np2(const PagedParams &p, cudaStream_t s);
TQ_PAGED_KB(1)
TQ_PAGED_KB(2)
TQ_PAGED_KB(3)
TQ_PAGED_KB(4)
TQ_PAGED_KB(5)
TQ_PAGED_KB(6)
TQ_PAGED_KB(7)
TQ_PAGED_KB(8)
#undef TQ_PAGED_KB
cudaError_t launch_paged_fp16(const PagedParams &p, cudaStream_t s);

namespace {
using PackedLaunch = cudaError_t (*)(const PagedParams &, cudaStream_t);
#define TQ_PAGED_EACH(f, np) {f##1_np##np, f##2_np##np, f##3_np##np, f##4_np##np, f##5_np##np, f##6_np##np, f##7_np##np, f##8_np##np}
constexpr PackedLaunch kPackedLaunch[2][8] = {TQ_PAGED_EACH(launch_paged_kb, 1), TQ_PAGED_EACH(launch_paged_kb, 2)};
#undef TQ_PAGED_EACH

// Head dims that take the tensor cores.
bool on_tensor_cores(int d) { return d == 64 || d == 128; }
}  // namespace

// A warp of the tensor-core forms takes four rows, two of packed pages of head_dim 64.
PagedShape paged_shape(int d, bool packed) {
    if (!on_tensor_cores(d)) return {kPlainUnit, kPlainRows, 2 * current_sm_count()};
    const int workers = kPagedWarps * current_sm_count();
    if (!packed) return {16, 4, workers};
    return d == 64 ? PagedShape{64, 2, workers} : PagedShape{32, 4, workers};
}

cudaError_t launch_paged(const PagedParams &p, cudaStream_t s) {
    if (on_tensor_cores(p.d)) return p.cls.kb ? kPackedLaunch[p.d == 64][p.cls.kb - 1](p, s) : launch_paged_fp16(p, s);
    switch (p.d) {
        case 16: return plain<16>(p, s);
        case 32: return plain<32>(p, s);
        case 256: return plain<256>(p, s);
        case 512: return plain<512>(p, s);
        case 1024: return plain<1024>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_paged_merge(const PagedMergeParams &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.n_classes > 0 ? 1 : 0;  // (behind a kernel of the call)
    const long long rows = static_cast<long long>(p.list.B) * p.list.H * p.g;
    if (!on_tensor_cores(p.d)) {
        cfg.gridDim = dim3(static_cast<unsigned>(rows));
        cfg.blockDim = dim3(kMergeThreads);
        return cudaLaunchKernelEx(&cfg, paged_merge_kernel, p);
    }
    // warps a row: the records that a long row has, eight a warp (two rounds of loads).  (Of all workers, not of those
    // that the table's width leaves: a result does not depend on how wide the table is.)
    long long records = 0;
    for (int k = 0; k < p.n_classes; k++)
        records += 1 + paged_shape(p.d, p.cls[k].kb > 0).workers / (static_cast<long long>(p.list.B) * __builtin_popcount(p.cls[k].heads[0]) * p.cls[k].n_rb);
    int W = 1;
    while (W < kRowWarps && 8 * W < records) W *= 2;
    cfg.gridDim = dim3(static_cast<unsigned>((rows + kRowWarps / W - 1) / (kRowWarps / W)));
    cfg.blockDim = dim3(32 * kRowWarps);
    return p.d == 128 ? cudaLaunchKernelEx(&cfg, paged_merge_rows_kernel<128>, p, W) : cudaLaunchKernelEx(&cfg, paged_merge_rows_kernel<64>, p, W);
}

}  // namespace tqk
