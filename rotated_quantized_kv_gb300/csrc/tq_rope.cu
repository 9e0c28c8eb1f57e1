// tq_rope.cu -- rotary positions: the cosine/sine table and its application to
// the rows of queries and keys.
//
// Pair (a, b) of a row at position p with angle p w_m: (a c - b s, b c + a s),
// c and s the table's binary32 cosine and sine.  Each product and sum is one
// binary32 operation (a fused multiply-add would round differently), the result
// is rounded once to the tensor's type: a pure function of x and the table.
//
// The kernel is bound by memory: x is read and written once, the table row
// of a token is read once per group of heads.  A thread owns one unit of a row
// (two 16-byte vectors: the two halves' partners, or 8 neighbouring pairs) and
// loops over heads with its cosines and sines in registers, because reading
// them per head would move twice the bytes of x through L1 (64 table bytes for
// 32 of x).  The heads of a token are spread over as many threads as the call
// needs to fill the GPU.  Rows that are not 16-byte aligned, or whose pairs do
// not fall into whole vectors, take one pair per thread.  Measured: 16384 tokens of 32 + 8
// heads of 128 in fp16 61.5 us (83% of the copy rate); one token 2.2 us.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tq_serve.h"

namespace tqk {
namespace {

constexpr int kRopeThreads = 256;

// ---------------------------------------------------------------- table
// The angle p w in binary64 is off by at most 2^-53 of itself (2e-7 at p = 2^31,
// 1e-10 at 1M positions); the binary64 cosine is then rounded once.
__global__ void __launch_bounds__(128) rope_table_kernel(const __grid_constant__ RopeTable p) {
    const long long n = static_cast<long long>(p.n) * p.half;
    for (long long i = blockIdx.x * 128LL + threadIdx.x; i < n; i += gridDim.x * 128LL) {
        const int row = static_cast<int>(i / p.half), m = static_cast<int>(i - static_cast<long long>(row) * p.half);
        double s, c;
        sincos((static_cast<double>(p.first) + row) * p.freq[m], &s, &c);
        float *t = p.table + static_cast<size_t>(row) * 2 * p.half;
        t[m] = static_cast<float>(c * p.amplitude);
        t[p.half + m] = static_cast<float>(s * p.amplitude);
    }
}

// ---------------------------------------------------------------- rows
template <typename T>
struct Elem;
template <>
struct Elem<__half> {
    static constexpr int kVec = 8;  // elements of 16 bytes
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};

template <typename T>
struct alignas(16) Vec {
    T e[Elem<T>::kVec];
};

__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

__device__ __forceinline__ const RopeTensorParams &tensor_of(const RopeParams &p, int head) {
    int i = p.n_tensors - 1;
    while (i > 0 && head < p.x[i].head0) --i;
    return p.x[i];
}

// Geometry of one launch: `units` threads per row, head_groups per token.
struct RopeGrid {
    long long threads;  // B T head_groups units
    int units, rot_units, head_groups;
};

// Vector path: unit u < rot_units holds the pairs [u V, (u + 1) V) (half layout:
// vectors u V and half + u V; interleaved: vectors 2 u V and (2 u + 1) V), the
// units behind copy two vectors of the unrotated rest each.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(const __grid_constant__ RopeParams p,
                                                               const RopeGrid g) {
    constexpr int V = Elem<T>::kVec;
    const long long id = blockIdx.x * static_cast<long long>(kRopeThreads) + threadIdx.x;
    if (id >= g.threads) return;
    long long r;
    int u, hs, t, b;
    if (g.threads <= 0x7fffffffLL) {  // 32-bit divisions where they do
        unsigned q = static_cast<unsigned>(id);
        u = q % g.units, q /= g.units;
        hs = q % g.head_groups, q /= g.head_groups;
        t = q % p.T, b = q / p.T;
    } else {
        r = id;
        u = static_cast<int>(r % g.units), r /= g.units;
        hs = static_cast<int>(r % g.head_groups), r /= g.head_groups;
        t = static_cast<int>(r % p.T), b = static_cast<int>(r / p.T);
    }
    const int pos = p.positions[b * p.pos_stride + t];
    const bool rot = u < g.rot_units && pos >= 0 && pos < p.rope.n_pos;
    int o0, o1;
    bool two = true;
    if (u < g.rot_units) {
        o0 = INTER ? 2 * u * V : u * V;
        o1 = INTER ? o0 + V : p.rope.half + o0;
    } else {
        o0 = 2 * p.rope.half + 2 * (u - g.rot_units) * V;
        o1 = o0 + V;
        two = o1 < p.d;
    }
    float c[V], s[V];
    if (rot) {
        const float *row = p.rope.table + static_cast<size_t>(pos) * 2 * p.rope.half + u * V;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(row + i));
            const float4 y = __ldg(reinterpret_cast<const float4 *>(row + p.rope.half + i));
            c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
            s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
        if (p.inverse) {
#pragma unroll
            for (int i = 0; i < V; i++) s[i] = -s[i];
        }
    }
#pragma unroll 4
    for (int h = hs; h < p.heads; h += g.head_groups) {
        const RopeTensorParams &x = tensor_of(p, h);
        const int hh = h - x.head0;
        const T *in = static_cast<const T *>(x.in) + b * x.is[0] + hh * x.is[1] + t * x.is[2];
        T *out = static_cast<T *>(x.out) + b * x.os[0] + hh * x.os[1] + t * x.os[2];
        Vec<T> a0 = *reinterpret_cast<const Vec<T> *>(in + o0), a1;
        if (two) a1 = *reinterpret_cast<const Vec<T> *>(in + o1);
        if (rot) {
#pragma unroll
            for (int i = 0; i < V; i++) {
                T &lo = INTER ? (2 * i < V ? a0.e[2 * i] : a1.e[2 * i - V]) : a0.e[i];
                T &hi = INTER ? (2 * i < V ? a0.e[2 * i + 1] : a1.e[2 * i + 1 - V]) : a1.e[i];
                float f = Elem<T>::get(lo), k = Elem<T>::get(hi);
                turn(f, k, c[i], s[i]);
                lo = Elem<T>::put(f);
                hi = Elem<T>::put(k);
            }
        } else if (in == out) {
            continue;  // in place: nothing to copy
        }
        *reinterpret_cast<Vec<T> *>(out + o0) = a0;
        if (two) *reinterpret_cast<Vec<T> *>(out + o1) = a1;
    }
}

// Any alignment and size: a thread holds one pair (or one element of the
// unrotated rest) of a row.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_pair_kernel(const __grid_constant__ RopeParams p,
                                                                const RopeGrid g) {
    for (long long id = blockIdx.x * static_cast<long long>(kRopeThreads) + threadIdx.x; id < g.threads;
         id += gridDim.x * static_cast<long long>(kRopeThreads)) {
        long long r = id;
        const int u = static_cast<int>(r % g.units);
        r /= g.units;
        const int h = static_cast<int>(r % p.heads);
        r /= p.heads;
        const int t = static_cast<int>(r % p.T), b = static_cast<int>(r / p.T);
        const RopeTensorParams &x = tensor_of(p, h);
        const int hh = h - x.head0;
        const T *in = static_cast<const T *>(x.in) + b * x.is[0] + hh * x.is[1] + t * x.is[2];
        T *out = static_cast<T *>(x.out) + b * x.os[0] + hh * x.os[1] + t * x.os[2];
        const int half = p.rope.half;
        if (u >= half) {
            out[u + half] = in[u + half];
            continue;
        }
        const int i = p.rope.interleaved ? 2 * u : u, j = p.rope.interleaved ? 2 * u + 1 : u + half;
        const int pos = p.positions[b * p.pos_stride + t];
        if (pos < 0 || pos >= p.rope.n_pos) {
            const T a = in[i], c = in[j];
            out[i] = a;
            out[j] = c;
            continue;
        }
        const float *row = p.rope.table + static_cast<size_t>(pos) * 2 * half;
        float a = Elem<T>::get(in[i]), c = Elem<T>::get(in[j]);
        const float s = row[half + u];
        turn(a, c, row[u], p.inverse ? -s : s);
        out[i] = Elem<T>::put(a);
        out[j] = Elem<T>::put(c);
    }
}

template <typename T>
bool vectors_fit(const RopeParams &p) {
    constexpr int V = Elem<T>::kVec;
    if (p.rope.half % V || p.d % V) return false;  // whole vectors of pairs (a half is a multiple of V, so is 2 half)
    for (int i = 0; i < p.n_tensors; i++) {
        const RopeTensorParams &x = p.x[i];
        if ((reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out)) & 15u) return false;
        for (int j = 0; j < 3; j++)
            if (x.is[j] % V || x.os[j] % V) return false;
    }
    return true;
}

template <typename T>
cudaError_t rope_typed(const RopeParams &p, cudaStream_t s) {
    constexpr int V = Elem<T>::kVec;
    const long long tokens = static_cast<long long>(p.B) * p.T;
    const long long fill = static_cast<long long>(current_sm_count()) * 2048;  // threads resident on the GPU
    RopeGrid g;
    if (vectors_fit<T>(p)) {
        g.rot_units = p.rope.half / V;
        g.units = g.rot_units + ((p.d - 2 * p.rope.half) / V + 1) / 2;
        // as many groups of heads as fill the GPU (small calls: one head per
        // thread), at least enough for a warp's accesses to share their lines
        const long long want = std::max<long long>((fill + tokens * g.units - 1) / (tokens * g.units), 1);
        g.head_groups = static_cast<int>(std::min<long long>(p.heads, std::max<long long>(want, (32 + g.units - 1) / g.units)));
        g.threads = tokens * g.units * g.head_groups;
        const long long blocks = (g.threads + kRopeThreads - 1) / kRopeThreads;
        if (blocks <= 0x7fffffffLL) {
            if (p.rope.interleaved)
                rope_vec_kernel<T, true><<<static_cast<unsigned>(blocks), kRopeThreads, 0, s>>>(p, g);
            else
                rope_vec_kernel<T, false><<<static_cast<unsigned>(blocks), kRopeThreads, 0, s>>>(p, g);
            return cudaGetLastError();
        }
    }
    g.rot_units = p.rope.half;
    g.units = p.d - p.rope.half;
    g.head_groups = p.heads;
    g.threads = tokens * g.units * p.heads;
    const long long blocks = std::min<long long>((g.threads + kRopeThreads - 1) / kRopeThreads, fill / kRopeThreads * 4);
    rope_pair_kernel<T><<<static_cast<unsigned>(blocks), kRopeThreads, 0, s>>>(p, g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(const RopeTable &p, cudaStream_t s) {
    const long long n = static_cast<long long>(p.n) * p.half;
    const long long blocks = std::min<long long>((n + 127) / 128, static_cast<long long>(current_sm_count()) * 16);
    rope_table_kernel<<<static_cast<unsigned>(blocks), 128, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_rope(const RopeParams &p, int dtype, cudaStream_t s) {
    switch (dtype) {
        case TQ_DTYPE_F16: return rope_typed<__half>(p, s);
        case TQ_DTYPE_BF16: return rope_typed<__nv_bfloat16>(p, s);
        default: return rope_typed<float>(p, s);
    }
}

}  // namespace tqk
