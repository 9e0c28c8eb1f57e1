// tq_append.cu -- ragged writes into a segment: gathered source rows, rotary
// positions, then the format's compression (or a verbatim copy) at each
// sequence's own position.
//
// Method and format: as tq_compress ("turboquant-mlx", "Walsh-Hadamard
// Rotation"; "TurboMOQ", "Architecture"): every rounding step is the format's
// binary32 operation, so the stored bits are those tq_compress gives the same
// rows.  A key is rotated by its position first (products and sums in binary32,
// rounded to fp16: the bits tq_rope writes).
#include <algorithm>

#include <cuda_fp16.h>

#include "tq_serve.h"
#include "tq_team.cuh"

namespace tqk {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;

// Source row and target position of row j of sequence b; false: not written.
__device__ __forceinline__ bool map_row(const RowMap &m, int b, int j, int capacity, int &src, int &pos) {
    const int n = m.n_rows ? min(m.n_rows[b], m.n_max) : m.n_max;
    if (j >= n) return false;
    src = m.index ? m.index[b * m.index_stride + j] : j;
    const long long t = static_cast<long long>(m.t_begin[b]) + j;
    pos = static_cast<int>(t);
    return src >= 0 && src < m.n_source && t >= 0 && t < capacity;
}

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

// One team of lanes per vector (kv, b, h, j); heads vary fastest, so that the
// rows of a token-major source lie next to each other.
template <int D>
__global__ void __launch_bounds__(kAppThreads) append_team_kernel(const __grid_constant__ AppendParams p) {
    using TM = Team<D>;
    constexpr int E = TM::E, T = TM::T, VPW = TM::VPW;
    __shared__ float thr[kCbTotal];
    __shared__ __align__(16) float stage[TM::STAGE ? kAppWarps * D : 4];
    __shared__ __align__(16) uint8_t codes[kAppWarps][VPW * D];
    for (int j = threadIdx.x; j < kCbTotal; j += kAppThreads) thr[j] = p.thr[j];
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int v = lane / T, lt = lane % T;
    uint32_t in_neg, out_neg;
    lane_sign_masks<D>(p.sign_bits, lt, in_neg, out_neg);
    const long long n = 2LL * p.B * p.rows.n_max * p.H;
    const long long step = static_cast<long long>(gridDim.x) * kAppWarps * VPW;
    for (long long base = (static_cast<long long>(blockIdx.x) * kAppWarps + warp) * VPW; base < n; base += step) {
        const long long f = base + v;
        long long r = f < n ? f : 0;
        const int h = static_cast<int>(r % p.H);
        r /= p.H;
        const int j = static_cast<int>(r % p.rows.n_max);
        r /= p.rows.n_max;
        const int b = static_cast<int>(r % p.B), kv = static_cast<int>(r / p.B);
        int src = 0, pos = 0;
        const bool valid = f < n && map_row(p.rows, b, j, p.seg.capacity, src, pos);
        float a[E];
        if (valid) {
            const int64_t *st = kv ? p.vs : p.ks;
            const uint16_t *row = (kv ? p.V : p.K) + b * st[0] + h * st[1] + src * st[2];
            const float *cs = table_row(p, kv, b, src);
#pragma unroll
            for (int e = 0; e < E; e++) a[e] = __half2float(load_coord(row, lt * E + e, p.rope, cs));
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
        uint8_t *cw = codes[warp] + v * D;
        const float scale = quantize_team<D>(a, m, S, bits, kv != 0, thr + cb_off(bits), cw, lt);
        __syncwarp();
        if (valid) {
            uint8_t *dst = const_cast<uint8_t *>(kv ? p.seg.v : p.seg.k) + b * (kv ? p.seg.vblock : p.seg.kblock) +
                           (kv ? p.seg.voff[h] : p.seg.koff[h]) + static_cast<size_t>(pos) * (D * bits / 8);
            store_record<D>(cw, bits, dst, lt);
            if (lt == 0)
                const_cast<float *>(kv ? p.seg.vs : p.seg.ks)[(static_cast<size_t>(b) * p.H + h) * p.seg.capacity + pos] = scale;
        }
        __syncwarp();
    }
}

// fp16 segments: 8 coordinates per thread.
__global__ void __launch_bounds__(kAppThreads) append_copy_kernel(const __grid_constant__ AppendParams p) {
    const int units = p.d / 8;
    const long long n = 2LL * p.B * p.rows.n_max * p.H * units;
    for (long long f = blockIdx.x * static_cast<long long>(kAppThreads) + threadIdx.x; f < n;
         f += gridDim.x * static_cast<long long>(kAppThreads)) {
        long long r = f;
        const int u = static_cast<int>(r % units);
        r /= units;
        const int h = static_cast<int>(r % p.H);
        r /= p.H;
        const int j = static_cast<int>(r % p.rows.n_max);
        r /= p.rows.n_max;
        const int b = static_cast<int>(r % p.B), kv = static_cast<int>(r / p.B);
        int src, pos;
        if (!map_row(p.rows, b, j, p.seg.capacity, src, pos)) continue;
        const int64_t *st = kv ? p.vs : p.ks;
        const uint16_t *row = (kv ? p.V : p.K) + b * st[0] + h * st[1] + src * st[2];
        const float *cs = table_row(p, kv, b, src);
        __align__(16) __half x[8];
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = load_coord(row, 8 * u + e, p.rope, cs);
        uint8_t *dst = const_cast<uint8_t *>(kv ? p.seg.v : p.seg.k) + b * (kv ? p.seg.vblock : p.seg.kblock) +
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

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t s) {
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
