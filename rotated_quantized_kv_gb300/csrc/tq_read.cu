// tq_read.cu -- rows of a segment read back into the caller's type: codes and
// scales to rotated vectors, then the inverse rotation (R is its own inverse).
// The binary32 steps are those of tq_dequantize, the result is rounded once.
// Small calls are bound by latency: 64 rows of 8 heads 3.0 us.
#include <algorithm>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tq_row_map.cuh"
#include "tq_serve.h"
#include "tq_team.cuh"

namespace tqk {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadWarps = kReadThreads / 32;

__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__half *p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Four coordinates by one store.
__device__ __forceinline__ void put4(float *p, const float *x) { *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void put4(__half *p, const float *x) {
    __half2 v[2] = {__floats2half2_rn(x[0], x[1]), __floats2half2_rn(x[2], x[3])};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(v);
}
__device__ __forceinline__ void put4(__nv_bfloat16 *p, const float *x) {
    __nv_bfloat162 v[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(v);
}

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
    stage_widths(cent, p.centroid, p.vwidths, 0);
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
        unsigned long long r = f < n ? f : 0;
        const int j = split_index(r, p.rows.n_max), h = split_index(r, p.H), b = split_index(r, p.B);
        const int kv = kv0 + static_cast<int>(r);
        int pos = 0;
        const bool valid = f < n && read_row(p.rows, b, j, p.seg.capacity, pos);
        if (!__any_sync(0xffffffffu, valid)) continue;  // (n_max may be far above the sequences' counts)
        float a[E];
        if (valid) {
            const int bits = kv ? p.seg.vbits[h] : p.seg.kbits[h];
            const uint8_t *rec = (kv ? p.seg.v : p.seg.k) + b * (kv ? p.seg.vblock : p.seg.kblock) +
                                 (kv ? p.seg.voff[h] : p.seg.koff[h]) + static_cast<size_t>(pos) * (D * bits / 8);
            const float sc = (kv ? p.seg.vs : p.seg.ks)[(static_cast<size_t>(b) * p.H + h) * p.seg.capacity + pos];
            const float inv_cells = __uint_as_float(static_cast<uint32_t>(127 - bits) << 23);  // 2^-b
            const int rk = D * bits / 8;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                uint32_t k[4];
                if (whole_words<D>(rec, rk)) {
                    load_codes4(rec, rk / 4, lt * E + e, bits, k);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++) k[i] = code_at(rec, lt * E + e + i, bits);
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
                    a[e + i] = kv ? __fmul_rn(sc, cent[cb_off(bits) + k[i]])
                                  : __fmul_rn(sc, __fadd_rn(__fmul_rn(static_cast<float>(2 * k[i] + 1), inv_cells), -1.0f));
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; e++) a[e] = 0.0f;
        }
        if (p.rotate) rotate_exact<D>(a, lt, in_neg, out_neg, p.inv_sqrt_d, stage + (TM::STAGE ? warp * D : 0));
        if (valid) {
            const int64_t *st = kv ? p.vs : p.ks;
            T *out = static_cast<T *>(kv ? p.V : p.K) + b * st[0] + h * st[1] + j * st[2];
            if (p.vec && (!TM::STAGE || !p.rotate)) {
#pragma unroll
                for (int e = 0; e < E; e += 4) put4(out + lt * E + e, a + e);
                continue;
            }
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
        unsigned long long r = f;
        const int u = split_index(r, units), j = split_index(r, p.rows.n_max), h = split_index(r, p.H);
        const int b = split_index(r, p.B), kv = kv0 + static_cast<int>(r);
        int pos;
        if (!read_row(p.rows, b, j, p.seg.capacity, pos)) continue;
        const uint8_t *src = (kv ? p.seg.v : p.seg.k) + b * (kv ? p.seg.vblock : p.seg.kblock) +
                             (kv ? p.seg.voff[h] : p.seg.koff[h]) + (static_cast<size_t>(pos) * p.d + 8 * u) * 2;
        const uint4 w = *reinterpret_cast<const uint4 *>(src);
        const __half *x = reinterpret_cast<const __half *>(&w);
        const int64_t *st = kv ? p.vs : p.ks;
        T *out = static_cast<T *>(kv ? p.V : p.K) + b * st[0] + h * st[1] + j * st[2] + 8 * u;
        float f8[8];
#pragma unroll
        for (int e = 0; e < 8; e++) f8[e] = __half2float(x[e]);
        if (p.vec) {
            put4(out, f8);
            put4(out + 4, f8 + 4);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) put(out + e, f8[e]);
        }
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

// Head_dim 128 or 64 and many rows: 128 coordinates a thread, a launch per width
// (tq_read_rows.cuh).  Small reads take the team kernel: one launch, up to 32 lanes a vector.
// One sequence of 8 heads, team / rows, us (head_dim 128; at 64 twice the tokens take about the same):
//   tokens               512         768         1024        1536        2048        4096        8192
//   1 + 1 widths      5.4 /  6.0   7.0 /  6.0   8.7 /  6.1  11.5 /  6.9  14.6 /  7.3  26.3 / 10.8  52.9 / 17.2
//   2 + 2             5.4 /  8.1   7.1 /  8.1   8.8 /  8.1  11.6 /  9.9  14.7 / 11.0  26.5 / 13.7  53.0 / 19.6
//   4 + 4             5.7 / 12.7   7.4 / 13.5   9.1 / 13.8  11.9 / 13.9  15.1 / 14.7  26.7 / 17.3  53.5 / 25.2
//   8 + 8             6.4 / 21.8   8.1 / 22.1   9.8 / 19.9  12.6 / 23.8  15.8 / 25.0  27.5 / 30.6  53.9 / 36.7
// Counted in vectors of 128 (two of 64 make one): 16 a token here.
constexpr long long rows_vectors(int launches) { return 1600 + 3800LL * launches; }

// Whether every value codebook in use is odd (the Gaussian one is, by construction).
bool odd_levels(const ReadParams &p) {
    for (int b = 1; b <= 8; b++) {
        if (!((p.vwidths >> b) & 1u)) continue;
        const float *c = p.centroid + cb_off(b);
        for (int i = 0; i < 1 << (b - 1); i++)
            if (c[i] != -c[(1 << b) - 1 - i]) return false;
    }
    return true;
}

cudaError_t read_rows(const ReadParams &p, int dtype, cudaStream_t s) {
    ReadRowsParams q;
    std::memset(&q, 0, sizeof(q));
    q.rows = p.rows;
    q.B = p.B, q.H = p.H, q.capacity = p.seg.capacity;
    q.dtype = dtype, q.rotate = p.rotate;
    auto *keys = p.d == kD ? launch_read_keys : launch_read_keys_d64;
    auto *values = p.d == kD ? launch_read_values : launch_read_values_d64;
    for (int i = 0; i < kD; i++) {
        const bool n = (p.sign_bits[(i & (p.d - 1)) >> 5] >> (i & 31)) & 1u;
        q.out_scale[i] = n ? -p.inv_sqrt_d : p.inv_sqrt_d;
    }
    bool beside = false;  // the first launch waits for the stream, the others need not wait for it
    for (int kv = 0; kv < 2; kv++) {
        q.out = kv ? p.V : p.K;
        if (!q.out) continue;
        const int per16 = dtype == TQ_DTYPE_F32 ? 4 : 8;
        q.vec = (reinterpret_cast<uintptr_t>(q.out) & 15u) == 0;
        for (int i = 0; i < 3; i++) {
            q.st[i] = kv ? p.vs[i] : p.ks[i];
            q.vec &= q.st[i] % per16 == 0;
        }
        q.codes = kv ? p.seg.v : p.seg.k;
        q.scale = kv ? p.seg.vs : p.seg.ks;
        q.block = kv ? p.seg.vblock : p.seg.kblock;
        for (int h = 0; h < p.H; h++) q.off[h] = kv ? p.seg.voff[h] : p.seg.koff[h];
        for (int bits = 1; bits <= 8; bits++) {
            q.n_heads = 0;
            for (int h = 0; h < p.H; h++)
                if ((kv ? p.seg.vbits[h] : p.seg.kbits[h]) == bits) q.head[q.n_heads++] = static_cast<uint8_t>(h);
            if (q.n_heads == 0) continue;
            if (kv) std::memcpy(q.level, p.centroid + cb_off(bits), sizeof(float) << bits);
            std::memset(q.flip, 0, sizeof(q.flip));
            for (int i = 0, bit = 0; i < kD && p.rotate; i++, bit += bits) {
                if (!((p.sign_bits[(i & (p.d - 1)) >> 5] >> (i & 31)) & 1u)) continue;
                const uint64_t field = static_cast<uint64_t>((1u << bits) - 1u) << (bit & 31);
                q.flip[bit >> 5] |= static_cast<uint32_t>(field);
                if (field >> 32) q.flip[(bit >> 5) + 1] |= static_cast<uint32_t>(field >> 32);
            }
            const cudaError_t e = kv ? values(q, bits, beside, s) : keys(q, bits, beside, s);
            if (e != cudaSuccess) return e;
            beside = true;
        }
    }
    return cudaSuccess;
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

cudaError_t launch_read(const ReadParams &params, int dtype, cudaStream_t s) {
    ReadParams p = params;
    const uintptr_t align = dtype == TQ_DTYPE_F32 ? 15u : 7u;
    p.vwidths = 0;
    for (int h = 0; h < p.H; h++) p.vwidths |= 1u << p.seg.vbits[h];
    p.vec = ((reinterpret_cast<uintptr_t>(p.K) | reinterpret_cast<uintptr_t>(p.V)) & align) == 0;
    for (int i = 0; i < 3; i++) p.vec &= (!p.K || p.ks[i] % 4 == 0) && (!p.V || p.vs[i] % 4 == 0);
    const long long vec = ((p.K ? 1LL : 0) + (p.V ? 1 : 0)) * p.B * p.H * p.rows.n_max;
    uint32_t kwidths = 0;
    for (int h = 0; h < p.H; h++) kwidths |= 1u << p.seg.kbits[h];
    const int launches = (p.K ? __builtin_popcount(kwidths) : 0) + (p.V ? __builtin_popcount(p.vwidths) : 0);
    if (!p.seg.fp16 && (p.d == kD || p.d == 64) && vec * p.d >= rows_vectors(launches) * kD &&
        blocks_fit(p.B, p.H, p.rows.n_max, kD / p.d) && odd_levels(p))
        return read_rows(p, dtype, s);
    switch (dtype) {
        case TQ_DTYPE_F16: return read_typed<__half>(p, s);
        case TQ_DTYPE_BF16: return read_typed<__nv_bfloat16>(p, s);
        default: return read_typed<float>(p, s);
    }
}

}  // namespace tqk
