// tq_append.cu -- ragged writes into a segment: gathered source rows, rotary
// positions, then the format's compression (or a verbatim copy) at each
// sequence's own position.
//
// Method and format: as tq_compress ("turboquant-mlx", "Walsh-Hadamard
// Rotation"; "TurboMOQ", "Architecture"): every rounding step is the format's
// binary32 operation, so the stored bits are those tq_compress gives the same
// rows.  A key is rotated by its position first (products and sums in binary32,
// rounded to fp16: the bits tq_rope writes).
//
// A team of lanes takes a vector (tq_team.cuh); small calls are bound by the latency of
// one pass: 64 rows of 8 heads, keys rotated, 4.2 us, 32 x 16 gathered rows 7.2 us.
#include <algorithm>
#include <cstring>

#include <cuda_fp16.h>

#include "tq_row_map.cuh"
#include "tq_serve.h"
#include "tq_team.cuh"

namespace tqk {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;

// Coordinate i of a row, rotated by its position (cs: the table's row, null:
// none) and rounded to fp16.
__device__ __forceinline__ __half load_coord(const uint16_t *row, int i, const RopeView &r, const float *cs) {
    const __half x = __ushort_as_half(row[i]);
    if (!cs || i >= 2 * r.half) return x;
    const int m = r.interleaved ? i >> 1 : (i < r.half ? i : i - r.half);
    const bool second = r.interleaved ? (i & 1) : i >= r.half;
    const int other = r.interleaved ? i ^ 1 : (second ? i - r.half : i + r.half);
    const float own = __half2float(x), o = __half2float(__ushort_as_half(row[other]));
    const float c = cs[m], s = cs[r.half + m];
    const float y = second ? __fadd_rn(__fmul_rn(own, c), __fmul_rn(o, s)) : __fsub_rn(__fmul_rn(own, c), __fmul_rn(o, s));
    return __float2half_rn(y);
}

__device__ __forceinline__ const float *table_row(const AppendParams &p, int kv, int b, int src) {
    if (kv || !p.rope.table) return nullptr;
    const int at = p.positions[b * p.pos_stride + src];
    return at >= 0 && at < p.rope.n_pos ? p.rope.table + static_cast<size_t>(at) * 2 * p.rope.half : nullptr;
}

// Coordinates i0..i0 + 3 (i0 a multiple of four) likewise; VEC: by 8-byte loads, the
// rotary half a multiple of four (a group is then rotated as a whole, or not at all).
__device__ __forceinline__ void load_coords4(const uint16_t *row, int i0, const RopeView &r, const float *cs, bool vec,
                                             __half (&x)[4]) {
    if (!vec) {
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = load_coord(row, i0 + e, r, cs);
        return;
    }
    const uint2 w = *reinterpret_cast<const uint2 *>(row + i0);
    const __half *own = reinterpret_cast<const __half *>(&w);
    if (!cs || i0 >= 2 * r.half) {
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = own[e];
        return;
    }
    if (r.interleaved) {
        const float2 c = *reinterpret_cast<const float2 *>(cs + (i0 >> 1));
        const float2 s = *reinterpret_cast<const float2 *>(cs + r.half + (i0 >> 1));
        const float a0 = __half2float(own[0]), b0 = __half2float(own[1]), a1 = __half2float(own[2]), b1 = __half2float(own[3]);
        x[0] = __float2half_rn(__fsub_rn(__fmul_rn(a0, c.x), __fmul_rn(b0, s.x)));
        x[1] = __float2half_rn(__fadd_rn(__fmul_rn(b0, c.x), __fmul_rn(a0, s.x)));
        x[2] = __float2half_rn(__fsub_rn(__fmul_rn(a1, c.y), __fmul_rn(b1, s.y)));
        x[3] = __float2half_rn(__fadd_rn(__fmul_rn(b1, c.y), __fmul_rn(a1, s.y)));
        return;
    }
    const bool second = i0 >= r.half;
    const int m = second ? i0 - r.half : i0;
    const uint2 v = *reinterpret_cast<const uint2 *>(row + (second ? m : i0 + r.half));
    const __half *oth = reinterpret_cast<const __half *>(&v);
    const float4 c4 = *reinterpret_cast<const float4 *>(cs + m), s4 = *reinterpret_cast<const float4 *>(cs + r.half + m);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float y = __fmul_rn(__half2float(own[e]), c[e]), z = __fmul_rn(__half2float(oth[e]), s[e]);
        x[e] = __float2half_rn(second ? __fadd_rn(y, z) : __fsub_rn(y, z));
    }
}

// One team of lanes per vector (kv, b, h, j); heads vary fastest, so that the
// rows of a token-major source lie next to each other.
template <int D>
__global__ void __launch_bounds__(kAppThreads) append_team_kernel(const __grid_constant__ AppendParams p) {
    using TM = Team<D>;
    constexpr int E = TM::E, T = TM::T, VPW = TM::VPW;
    __shared__ float thr[kCbTotal];
    __shared__ __align__(16) float stage[TM::STAGE ? kAppWarps * D : 4];
    __shared__ __align__(16) uint8_t codes[kAppWarps][E == 4 ? 4 : D];
    stage_widths(thr, p.thr, p.vwidths, 1);
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int v = lane / T, lt = lane % T;
    uint32_t in_neg, out_neg;
    lane_sign_masks<D>(p.sign_bits, lt, in_neg, out_neg);
    const long long n = 2LL * p.B * p.rows.n_max * p.H;
    const long long step = static_cast<long long>(gridDim.x) * kAppWarps * VPW;
    for (long long base = (static_cast<long long>(blockIdx.x) * kAppWarps + warp) * VPW; base < n; base += step) {
        const long long f = base + v;
        unsigned long long r = f < n ? f : 0;
        const int h = split_index(r, p.H), j = split_index(r, p.rows.n_max), b = split_index(r, p.B), kv = static_cast<int>(r);
        int src = 0, at = 0, pos = 0;
        const bool valid = f < n && map_row(p.rows, b, j, p.seg.capacity, src, at, pos);
        if (!__any_sync(0xffffffffu, valid)) continue;  // (n_max may be far above the sequences' counts)
        float a[E];
        if (valid) {
            const int64_t *st = kv ? p.vs : p.ks;
            const uint16_t *row = (kv ? p.V : p.K) + b * st[0] + h * st[1] + src * st[2];
            const float *cs = table_row(p, kv, b, src);
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                __half x[4];
                load_coords4(row, lt * E + e, p.rope, cs, p.vec != 0, x);
#pragma unroll
                for (int i = 0; i < 4; i++) a[e + i] = __half2float(x[i]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; e++) a[e] = 0.0f;
        }
        rotate_exact<D>(a, lt, in_neg, out_neg, p.inv_sqrt_d, stage + (TM::STAGE ? warp * D : 0));
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e++) m = fmaxf(m, fabsf(a[e]));
#pragma unroll
        for (int x = 1; x < T; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        const float S = tree_sum_squares<D>(a, lt, stage + (TM::STAGE ? warp * D : 0));
        const int bits = kv ? p.seg.vbits[h] : p.seg.kbits[h];
        uint8_t *dst = const_cast<uint8_t *>(kv ? p.seg.v : p.seg.k) + at * (kv ? p.seg.vblock : p.seg.kblock) +
                       (kv ? p.seg.voff[h] : p.seg.koff[h]) + static_cast<size_t>(pos) * (D * bits / 8);
        float scale;
        if constexpr (E == 4) {
            uint32_t k[4];
            scale = team_codes<D>(a, m, S, bits, kv != 0, thr + cb_off(bits), k);
            store_fields<D>(k, bits, dst, lt, valid);
        } else {
            scale = quantize_team<D>(a, m, S, bits, kv != 0, thr + cb_off(bits), codes[warp], lt);
            __syncwarp();
            if (valid) store_record<D>(codes[warp], bits, dst, lt);
        }
        if (valid && lt == 0)
            const_cast<float *>(kv ? p.seg.vs : p.seg.ks)[(static_cast<size_t>(at) * p.H + h) * p.seg.capacity + pos] = scale;
        __syncwarp();
    }
}

// fp16 segments: 8 coordinates per thread.
__global__ void __launch_bounds__(kAppThreads) append_copy_kernel(const __grid_constant__ AppendParams p) {
    const int units = p.d / 8;
    const long long n = 2LL * p.B * p.rows.n_max * p.H * units;
    for (long long f = blockIdx.x * static_cast<long long>(kAppThreads) + threadIdx.x; f < n;
         f += gridDim.x * static_cast<long long>(kAppThreads)) {
        unsigned long long r = f;
        const int u = split_index(r, units), h = split_index(r, p.H), j = split_index(r, p.rows.n_max);
        const int b = split_index(r, p.B), kv = static_cast<int>(r);
        int src, at, pos;
        if (!map_row(p.rows, b, j, p.seg.capacity, src, at, pos)) continue;
        const int64_t *st = kv ? p.vs : p.ks;
        const uint16_t *row = (kv ? p.V : p.K) + b * st[0] + h * st[1] + src * st[2];
        const float *cs = table_row(p, kv, b, src);
        __half lo[4], hi[4];
        load_coords4(row, 8 * u, p.rope, cs, p.vec != 0, lo);
        load_coords4(row, 8 * u + 4, p.rope, cs, p.vec != 0, hi);
        __align__(16) const __half x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        uint8_t *dst = const_cast<uint8_t *>(kv ? p.seg.v : p.seg.k) + at * (kv ? p.seg.vblock : p.seg.kblock) +
                       (kv ? p.seg.voff[h] : p.seg.koff[h]) + (static_cast<size_t>(pos) * p.d + 8 * u) * 2;
        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(x);
    }
}

unsigned grid_for(long long blocks, int per_sm) {
    return static_cast<unsigned>(
        std::max<long long>(1, std::min<long long>(blocks, static_cast<long long>(current_sm_count()) * per_sm)));
}

template <int D>
cudaError_t append_team(const AppendParams &p, cudaStream_t s) {
    const long long vec = 2LL * p.B * p.rows.n_max * p.H;
    const int per = kAppWarps * Team<D>::VPW;
    append_team_kernel<D><<<grid_for((vec + per - 1) / per, 8), kAppThreads, 0, s>>>(p);
    return cudaGetLastError();
}

// Head_dim 128 and many rows: one thread per vector, a launch per width
// (tq_append_rows.cuh).  Small writes take the team kernel: one launch, 32 lanes a
// vector, no cold start of 2000 straight instructions.  So the rows that make up for the
// launches grow with their number.  One sequence of 8 heads, keys rotated, team / rows, us:
//   tokens               512         768         1024        1536        2048        4096        8192
//   1 + 1 widths      7.5 / 10.2  10.3 / 10.2  13.3 / 10.4  17.8 / 10.6  23.5 / 11.2  43.2 / 18.4  87.6 / 26.9
//   2 + 2             7.6 / 13.9  10.5 / 14.1  13.4 / 14.1  18.0 / 14.7  23.6 / 15.0  43.5 / 20.8  87.9 / 33.4
//   4 + 4             8.0 / 18.7  10.8 / 19.0  13.9 / 19.6  18.5 / 19.8  24.2 / 20.1  44.5 / 26.8  89.6 / 40.9
//   8 + 8             9.2 / 37.3  12.0 / 37.5  15.2 / 38.5  20.0 / 39.1  25.9 / 40.4  47.1 / 42.7  94.2 / 61.3
// (16 vectors a token: they cross at about 12300, 17300, 26000 and 59000 vectors)
constexpr long long rows_vectors(int launches) { return 5700 + 3300LL * launches; }

bool rows_fit(const AppendParams &p) {
    uint32_t kwidths = 0;
    for (int h = 0; h < p.H; h++) kwidths |= 1u << p.seg.kbits[h];
    const int launches = __builtin_popcount(kwidths) + __builtin_popcount(p.vwidths);
    if (p.d != kD || 2LL * p.B * p.H * p.rows.n_max < rows_vectors(launches) || !blocks_fit(p.B, p.H, p.rows.n_max, 1))
        return false;
    if (p.seg.kblock >> 32 || p.seg.vblock >> 32) return false;
    if ((reinterpret_cast<uintptr_t>(p.K) | reinterpret_cast<uintptr_t>(p.V)) & 15u) return false;
    for (int i = 0; i < 3; i++)
        if (p.ks[i] % 8 || p.vs[i] % 8) return false;
    return true;
}

cudaError_t append_rows(const AppendParams &p, cudaStream_t s) {
    AppendRowsParams q;
    std::memset(&q, 0, sizeof(q));
    q.rows = p.rows;
    q.r.B = p.B, q.r.H = p.H, q.r.T = p.rows.n_max, q.r.capacity = p.seg.capacity;
    q.r.nh = q.r.np = 1;
    fill_rows_rotation(q.r, p.sign_bits, kD);
    for (int bits = 1; bits <= 8; bits++)  // before anything is launched
        if (((p.vwidths >> bits) & 1u) && !fill_rows_values(q.r, bits, p.law)) return cudaErrorNotSupported;
    bool beside = false;  // the first launch waits for the stream, the others need not wait for it
    for (int kv = 0; kv < 2; kv++) {
        const int64_t *st = kv ? p.vs : p.ks;
        q.r.X = kv ? p.V : p.K;
        q.r.sb = st[0], q.r.sh = st[1], q.r.st = st[2];
        q.r.codes = const_cast<uint8_t *>(kv ? p.seg.v : p.seg.k);
        q.r.scale = const_cast<float *>(kv ? p.seg.vs : p.seg.ks);
        q.r.block = static_cast<uint32_t>(kv ? p.seg.vblock : p.seg.kblock);
        for (int h = 0; h < p.H; h++) q.r.off[h] = static_cast<uint32_t>(kv ? p.seg.voff[h] : p.seg.koff[h]);
        if (!kv) q.rope = p.rope, q.positions = p.positions, q.pos_stride = p.pos_stride;
        for (int bits = 1; bits <= 8; bits++) {
            q.r.n_heads = 0;
            for (int h = 0; h < p.H; h++)
                if ((kv ? p.seg.vbits[h] : p.seg.kbits[h]) == bits) q.r.head[q.r.n_heads++] = static_cast<uint8_t>(h);
            if (q.r.n_heads == 0) continue;
            if (kv) fill_rows_values(q.r, bits, p.law);
            const cudaError_t e = kv ? launch_append_values(q, bits, beside, s) : launch_append_keys(q, bits, beside, s);
            if (e != cudaSuccess) return e;
            beside = true;
        }
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_append(const AppendParams &params, cudaStream_t s) {
    AppendParams p = params;
    p.vwidths = 0;
    for (int h = 0; h < p.H; h++) p.vwidths |= 1u << p.seg.vbits[h];
    p.vec = ((reinterpret_cast<uintptr_t>(p.K) | reinterpret_cast<uintptr_t>(p.V)) & 7u) == 0 && p.rope.half % 4 == 0;
    for (int i = 0; i < 3; i++) p.vec &= p.ks[i] % 4 == 0 && p.vs[i] % 4 == 0;
    if (!p.seg.fp16 && rows_fit(p)) {
        const cudaError_t e = append_rows(p, s);
        if (e != cudaErrorNotSupported) return e;
    }
    if (p.seg.fp16) {
        const long long n = 2LL * p.B * p.rows.n_max * p.H * (p.d / 8);
        append_copy_kernel<<<grid_for((n + kAppThreads - 1) / kAppThreads, 16), kAppThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    switch (p.d) {
        case 16: return append_team<16>(p, s);
        case 32: return append_team<32>(p, s);
        case 64: return append_team<64>(p, s);
        case 128: return append_team<128>(p, s);
        case 256: return append_team<256>(p, s);
        case 512: return append_team<512>(p, s);
        case 1024: return append_team<1024>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tqk
