// tq_append_rows.cuh -- ragged writes into a packed segment, one thread per vector
// (head_dim 128), instantiated for keys and values by tq_append_rows_*.cu.
//
// The compressor's layout and arithmetic (tq_compress_rows.cuh): a warp takes 32
// rows of one (sequence, head), staged in shared memory with cp.async (here each
// row from its own place), a thread holds its vector in registers.  Heads vary
// fastest, so that a CTA's four warps share the tokens' table rows (and, in a
// token-major source, their lines).  Keys with rotary positions are rotated in the
// staged rows first: 16 lanes a row, four pairs a lane, so that the table is read in
// whole lines, the lines of eight tokens at a time (two at a time: 17 us more on the
// launch below).  Bound by issue slots and by the latency of few warps (12 an SM, the
// registers' limit): 4 x 8192 tokens of 8 heads in 4 bits, keys rotated, 75 us for both
// launches (64 without the rotation), 172 MB moved.
#pragma once

#include "tq_compress_rows.cuh"
#include "tq_row_map.cuh"
#include "tq_serve.h"
#include "tq_team.cuh"

namespace tqk {
namespace {

struct RowBlock {
    int b, h, j;            // sequence, head, this lane's row
    int src, at, pos;       // its source row, batch element (or page) and position
    bool valid;
};

template <bool SLOTS>
__device__ __forceinline__ RowBlock row_block(const AppendRowsParams &p, int n_tblk, int blk, int lane) {
    RowBlock r;
    r.h = p.r.head[blk % p.r.n_heads];
    const int rest = blk / p.r.n_heads;
    r.j = (rest % n_tblk) * 32 + lane;
    r.b = rest / n_tblk;
    r.src = r.at = r.pos = 0;
    r.valid = map_row<SLOTS>(p.rows, r.b, r.j, p.r.capacity, r.src, r.at, r.pos);
    return r;
}

__device__ __forceinline__ void stage_mapped(const AppendRowsParams &p, const RowBlock &r, uint8_t *buf, int lane) {
    const uint16_t *base = p.r.X + r.b * p.r.sb + r.h * p.r.sh + 8 * (lane & 15);
    const int mine = r.valid ? r.src : -1;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int row = 2 * i + (lane >> 4), c = lane & 15, src = __shfl_sync(0xffffffffu, mine, row);
        if (src >= 0) cp_async16(buf + row * kRowBytes + 16 * (c ^ (row & 7)), base + src * p.r.st);
    }
}

// Rotary positions of the staged key rows: products and sums in binary32, rounded to fp16.
__device__ __forceinline__ void rope_rows(const AppendRowsParams &p, const RowBlock &r, uint8_t *buf, int lane) {
    int at = -1;
    if (r.valid) {
        at = p.positions[r.b * p.pos_stride + r.src];
        if (at >= p.rope.n_pos) at = -1;
    }
    const int half = p.rope.half, l16 = lane & 15;
    auto turn = [](__half &lo, __half &hi, float c, float s) {
        const float x = __half2float(lo), y = __half2float(hi);
        lo = __float2half_rn(__fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)));
        hi = __float2half_rn(__fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s)));
    };
    auto elem = [&](int row, int dim) {
        return reinterpret_cast<__half *>(buf + row * kRowBytes + 16 * ((dim >> 3) ^ (row & 7)) + 2 * (dim & 7));
    };
    if (half % 4 == 0) {  // four pairs a lane (half <= 64), the table's rows of eight tokens on their way at once
        const int m = 4 * l16;
#pragma unroll 1
        for (int i = 0; i < 16; i += 4) {
            float4 c[4], s[4];
            bool on[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int pos = __shfl_sync(0xffffffffu, at, 2 * (i + k) + (lane >> 4));
                on[k] = pos >= 0 && m < half;
                if (on[k]) {
                    const float *cs = p.rope.table + static_cast<size_t>(pos) * 2 * half + m;
                    c[k] = __ldg(reinterpret_cast<const float4 *>(cs));
                    s[k] = __ldg(reinterpret_cast<const float4 *>(cs + half));
                }
            }
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if (!on[k]) continue;
                const int row = 2 * (i + k) + (lane >> 4);
                if (p.rope.interleaved) {
                    uint4 *w = reinterpret_cast<uint4 *>(elem(row, 2 * m));
                    uint4 v = *w;
                    __half *x = reinterpret_cast<__half *>(&v);
                    turn(x[0], x[1], c[k].x, s[k].x);
                    turn(x[2], x[3], c[k].y, s[k].y);
                    turn(x[4], x[5], c[k].z, s[k].z);
                    turn(x[6], x[7], c[k].w, s[k].w);
                    *w = v;
                } else {
                    uint2 *wa = reinterpret_cast<uint2 *>(elem(row, m)), *wb = reinterpret_cast<uint2 *>(elem(row, half + m));
                    uint2 a = *wa, b = *wb;
                    __half *x = reinterpret_cast<__half *>(&a), *y = reinterpret_cast<__half *>(&b);
                    turn(x[0], y[0], c[k].x, s[k].x);
                    turn(x[1], y[1], c[k].y, s[k].y);
                    turn(x[2], y[2], c[k].z, s[k].z);
                    turn(x[3], y[3], c[k].w, s[k].w);
                    *wa = a;
                    *wb = b;
                }
            }
        }
        return;
    }
#pragma unroll 1
    for (int i = 0; i < 16; i++) {
        const int row = 2 * i + (lane >> 4), pos = __shfl_sync(0xffffffffu, at, row);
        if (pos < 0) continue;
        const float *cs = p.rope.table + static_cast<size_t>(pos) * 2 * half;
        for (int m = l16; m < half; m += 16)
            turn(*elem(row, p.rope.interleaved ? 2 * m : m), *elem(row, p.rope.interleaved ? 2 * m + 1 : half + m), cs[m],
                 cs[half + m]);
    }
}

template <int BITS, bool VAL, bool SLOTS>
__global__ void __launch_bounds__(kThreads, 3) append_rows_kernel(const __grid_constant__ AppendRowsParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t *in_mask = reinterpret_cast<uint32_t *>(smem + kWarps * 2 * kWarpBuf);
    float *out_pair = reinterpret_cast<float *>(in_mask + kMaskStride);
    float *thr = out_pair + kPairStride;
    uint2 *vtab = reinterpret_cast<uint2 *>(thr + 256);
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const RowsParams &t = *param_table(&p.r);
    for (int i = threadIdx.x; i < 64; i += kThreads) in_mask[i] = t.in_mask[i];
    for (int i = threadIdx.x; i < kD; i += kThreads) out_pair[i] = t.out_scale[(i >> 1) + 64 * (i & 1)];
    if constexpr (VAL) {
        for (int i = threadIdx.x; i < (1 << BITS) - 1; i += kThreads) thr[i] = t.thr[i];
        if constexpr (BITS <= 3)
            for (int i = threadIdx.x; i < kRowsBuckets; i += kThreads) vtab[i] = make_uint2(t.bucket[i].t, t.bucket[i].k);
        if constexpr (BITS == 4)
            if (p.r.bucket4_ok)
                for (int i = threadIdx.x; i < kRowsBuckets; i += kThreads)
                    vtab[i] = make_uint2(t.bucket4[2 * i], t.bucket4[2 * i + 1]);
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *bufs = smem + warp * 2 * kWarpBuf;
    const int n_tblk = (p.r.T + 31) / 32, n_blk = n_tblk * p.r.n_heads * p.r.B;
    const int gw = blockIdx.x * kWarps + warp, nw = gridDim.x * kWarps;
    if (gw < n_blk) stage_mapped(p, row_block<SLOTS>(p, n_tblk, gw, lane), bufs, lane);
    asm volatile("cp.async.commit_group;\n" ::);
    for (int blk = gw, it = 0; blk < n_blk; blk += nw, it++) {
        if (blk + nw < n_blk) stage_mapped(p, row_block<SLOTS>(p, n_tblk, blk + nw, lane), bufs + ((it + 1) & 1) * kWarpBuf, lane);
        asm volatile("cp.async.commit_group;\n" ::);
        asm volatile("cp.async.wait_group 1;\n" ::: "memory");
        __syncwarp();
        const RowBlock r = row_block<SLOTS>(p, n_tblk, blk, lane);
        uint8_t *buf = bufs + (it & 1) * kWarpBuf;
        if (!__any_sync(0xffffffffu, r.valid)) continue;  // (its buffer holds nothing new)
        if constexpr (!VAL) {
            if (p.rope.table) {
                rope_rows(p, r, buf, lane);
                __syncwarp();
            }
        }
        uint32_t w[4 * BITS];
        float scale, scale_b;
        rows_vector<BITS, VAL, 1, 1>(buf + lane * kRowBytes, in_mask, out_pair, thr, vtab, p.r.bucket4_ok != 0, lane, 0, w,
                                     scale, scale_b);
        if (r.valid) {
            const int at = SLOTS ? r.at : r.b;
            uint4 *dst = reinterpret_cast<uint4 *>(p.r.codes + static_cast<size_t>(at) * p.r.block + p.r.off[r.h] +
                                                   static_cast<size_t>(r.pos) * (16 * BITS));
#pragma unroll
            for (int j = 0; j < BITS; j++) dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            p.r.scale[(static_cast<size_t>(at) * p.r.H + r.h) * p.r.capacity + r.pos] = scale;
        }
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the call's last launch ends behind its first
}

template <int BITS, bool VAL, bool SLOTS>
cudaError_t append_rows_launch(const AppendRowsParams &p, bool beside, cudaStream_t s) {
    constexpr size_t smem = rows_smem_bytes<1>(VAL && BITS <= 4);
    const cudaError_t e = cudaFuncSetAttribute(append_rows_kernel<BITS, VAL, SLOTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const long long blocks = (static_cast<long long>((p.r.T + 31) / 32) * p.r.n_heads * p.r.B + kWarps - 1) / kWarps;
    const long long grid = std::min<long long>(blocks, static_cast<long long>(current_sm_count()) * 3);
    return launch_beside(append_rows_kernel<BITS, VAL, SLOTS>, static_cast<unsigned>(grid), kThreads, smem, s, beside, p);
}

template <bool VAL, bool SLOTS>
cudaError_t append_rows_dispatch(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s) {
    switch (bits) {
        case 1: return append_rows_launch<1, VAL, SLOTS>(p, beside, s);
        case 2: return append_rows_launch<2, VAL, SLOTS>(p, beside, s);
        case 3: return append_rows_launch<3, VAL, SLOTS>(p, beside, s);
        case 4: return append_rows_launch<4, VAL, SLOTS>(p, beside, s);
        case 5: return append_rows_launch<5, VAL, SLOTS>(p, beside, s);
        case 6: return append_rows_launch<6, VAL, SLOTS>(p, beside, s);
        case 7: return append_rows_launch<7, VAL, SLOTS>(p, beside, s);
        case 8: return append_rows_launch<8, VAL, SLOTS>(p, beside, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace tqk
