// tq_read.cu -- rows of a segment read back into the caller's type: codes and
// scales to rotated vectors, then the inverse rotation (R is its own inverse).
// The binary32 steps are those of tq_dequantize, the result is rounded once.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tq_serve.h"
#include "tq_team.cuh"

namespace tqk {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadWarps = kReadThreads / 32;

__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__half *p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Position of row j of sequence b; false: not read.
__device__ __forceinline__ bool read_row(const RowMap &m, int b, int j, int capacity, int &pos) {
    const int n = m.n_rows ? min(m.n_rows[b], m.n_max) : m.n_max;
    const long long t = static_cast<long long>(m.t_begin[b]) + j;
    pos = static_cast<int>(t);
    return j < n && t >= 0 && t < capacity;
}

// One team of lanes per vector (kv, b, h, j), rows of a head consecutive.
template <int D, typename T>
__global__ void __launch_bounds__(kReadThreads) read_team_kernel(const __grid_constant__ ReadParams p) {
    using TM = Team<D>;
    constexpr int E = TM::E, TL = TM::T, VPW = TM::VPW;
    __shared__ float cent[kCbTotal];
    __shared__ __align__(16) float stage[TM::STAGE ? kReadWarps * D : 4];
    for (int j = threadIdx.x; j < kCbTotal; j += kReadThreads) cent[j] = p.centroid[j];
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int v = lane / TL, lt = lane % TL;
    uint32_t in_neg, out_neg;
    lane_sign_masks<D>(p.sign_bits, lt, in_neg, out_neg);
    const int kv0 = p.K ? 0 : 1, nkv = (p.K ? 1 : 0) + (p.V ? 1 : 0);
    const long long n = static_cast<long long>(nkv) * p.B * p.H * p.rows.n_max;
    const long long step = static_cast<long long>(gridDim.x) * kReadWarps * VPW;
    for (long long base = (static_cast<long long>(blockIdx.x) * kReadWarps + warp) * VPW; base < n; base += step) {
        const long long f = base + v;
        long long r = f < n ? f : 0;
        const int j = static_cast<int>(r % p.rows.n_max);
        r /= p.rows.n_max;
        const int h = static_cast<int>(r % p.H);
        r /= p.H;
        const int b = static_cast<int>(r % p.B), kv = kv0 + static_cast<int>(r / p.B);
        int pos = 0;
        const bool valid = f < n && read_row(p.rows, b, j, p.seg.capacity, pos);
        float a[E];
        if (valid) {
            const int bits = kv ? p.seg.vbits[h] : p.seg.kbits[h];
            const uint8_t *rec = (kv ? p.seg.v : p.seg.k) + b * (kv ? p.seg.vblock : p.seg.kblock) +
                                 (kv ? p.seg.voff[h] : p.seg.koff[h]) + static_cast<size_t>(pos) * (D * bits / 8);
            const float sc = (kv ? p.seg.vs : p.seg.ks)[(static_cast<size_t>(b) * p.H + h) * p.seg.capacity + pos];
            const float inv_cells = __uint_as_float(static_cast<uint32_t>(127 - bits) << 23);  // 2^-b
#pragma unroll
            for (int e = 0; e < E; e++) {
                const uint32_t k = code_at(rec, lt * E + e, bits);
                a[e] = kv ? __fmul_rn(sc, cent[cb_off(bits) + k])
                          : __fmul_rn(sc, __fadd_rn(__fmul_rn(static_cast<float>(2 * k + 1), inv_cells), -1.0f));
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; e++) a[e] = 0.0f;
        }
        if (p.rotate) rotate_exact<D>(a, lt, in_neg, out_neg, p.inv_sqrt_d, stage + (TM::STAGE ? warp * D : 0));
        if (valid) {
            const int64_t *st = kv ? p.vs : p.ks;
            T *out = static_cast<T *>(kv ? p.V : p.K) + b * st[0] + h * st[1] + j * st[2];
#pragma unroll
            for (int e = 0; e < E; e++) put(out + (p.rotate ? coord<D>(lt, e) : lt * E + e), a[e]);
        }
    }
}

// fp16 segments: 8 coordinates per thread.
template <typename T>
__global__ void __launch_bounds__(kReadThreads) read_copy_kernel(const __grid_constant__ ReadParams p) {
    const int units = p.d / 8;
    const int kv0 = p.K ? 0 : 1, nkv = (p.K ? 1 : 0) + (p.V ? 1 : 0);
    const long long n = static_cast<long long>(nkv) * p.B * p.H * p.rows.n_max * units;
    for (long long f = blockIdx.x * static_cast<long long>(kReadThreads) + threadIdx.x; f < n;
         f += gridDim.x * static_cast<long long>(kReadThreads)) {
        long long r = f;
        const int u = static_cast<int>(r % units);
        r /= units;
        const int j = static_cast<int>(r % p.rows.n_max);
        r /= p.rows.n_max;
        const int h = static_cast<int>(r % p.H);
        r /= p.H;
        const int b = static_cast<int>(r % p.B), kv = kv0 + static_cast<int>(r / p.B);
        int pos;
        if (!read_row(p.rows, b, j, p.seg.capacity, pos)) continue;
        const uint8_t *src = (kv ? p.seg.v : p.seg.k) + b * (kv ? p.seg.vblock : p.seg.kblock) +
                             (kv ? p.seg.voff[h] : p.seg.koff[h]) + (static_cast<size_t>(pos) * p.d + 8 * u) * 2;
        const uint4 w = *reinterpret_cast<const uint4 *>(src);
        const __half *x = reinterpret_cast<const __half *>(&w);
        const int64_t *st = kv ? p.vs : p.ks;
        T *out = static_cast<T *>(kv ? p.V : p.K) + b * st[0] + h * st[1] + j * st[2] + 8 * u;
#pragma unroll
        for (int e = 0; e < 8; e++) put(out + e, __half2float(x[e]));
    }
}

unsigned grid_for(long long blocks, int per_sm) {
    return static_cast<unsigned>(
        std::max<long long>(1, std::min<long long>(blocks, static_cast<long long>(current_sm_count()) * per_sm)));
}

template <int D, typename T>
cudaError_t read_team(const ReadParams &p, cudaStream_t s) {
    const long long vec = ((p.K ? 1LL : 0) + (p.V ? 1 : 0)) * p.B * p.H * p.rows.n_max;
    const int per = kReadWarps * Team<D>::VPW;
    read_team_kernel<D, T><<<grid_for((vec + per - 1) / per, 8), kReadThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t read_typed(const ReadParams &p, cudaStream_t s) {
    if (p.seg.fp16) {
        const long long n = ((p.K ? 1LL : 0) + (p.V ? 1 : 0)) * p.B * p.H * p.rows.n_max * (p.d / 8);
        read_copy_kernel<T><<<grid_for((n + kReadThreads - 1) / kReadThreads, 16), kReadThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    switch (p.d) {
        case 16: return read_team<16, T>(p, s);
        case 32: return read_team<32, T>(p, s);
        case 64: return read_team<64, T>(p, s);
        case 128: return read_team<128, T>(p, s);
        case 256: return read_team<256, T>(p, s);
        case 512: return read_team<512, T>(p, s);
        case 1024: return read_team<1024, T>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_read(const ReadParams &p, int dtype, cudaStream_t s) {
    switch (dtype) {
        case TQ_DTYPE_F16: return read_typed<__half>(p, s);
        case TQ_DTYPE_BF16: return read_typed<__nv_bfloat16>(p, s);
        default: return read_typed<float>(p, s);
    }
}

}  // namespace tqk
