// tq_team.cuh -- a vector of any power-of-two head dimension (16..1024) held by
// a team of lanes: the format's rotation, sum of squares and record access.
// Shared by the kernels that take every head dimension.  The layout (T lanes,
// E contiguous coordinates each; a shared-memory transpose for d >= 256) and
// the order of the binary32 operations are described in tq_generic.cu.
#pragma once

#include <cuda_fp16.h>

#include "tq_internal.h"

namespace tqk {
namespace {

__device__ __forceinline__ bool neg_coord(const uint32_t *sb, int i) { return (sb[i >> 5] >> (i & 31)) & 1u; }

template <int D>
struct Team {
    static constexpr int T = D >= 128 ? 32 : D / 4;  // lanes per vector
    static constexpr int E = D / T;                  // coordinates per lane
    static constexpr int VPW = 32 / T;               // vectors per warp
    static constexpr bool STAGE = D >= 256;          // shared-memory stage between the in-lane stages
};

// Coordinate held in slot e of team lane lt once the rotation is done.
template <int D>
__device__ __forceinline__ int coord(int lt, int e) {
    return Team<D>::STAGE ? lt + 32 * e : lt * Team<D>::E + e;
}

// The signs a team lane applies, as bit masks over its E slots: in_neg bit e
// for coordinate lt * E + e (the input), out_neg bit e for coord<D>(lt, e).
template <int D>
__device__ __forceinline__ void lane_sign_masks(const uint32_t *sb, int lt, uint32_t &in_neg, uint32_t &out_neg) {
    constexpr int E = Team<D>::E;
    in_neg = (sb[lt * E >> 5] >> (lt * E & 31)) & (E == 32 ? 0xFFFFFFFFu : (1u << E % 32) - 1u);
    out_neg = in_neg;
    if constexpr (Team<D>::STAGE) {
        out_neg = 0u;
#pragma unroll
        for (int e = 0; e < E; e++) out_neg |= ((sb[e] >> lt) & 1u) << e;
    }
}

// y = c * D H D x in the format's binary32 order: input sign flip (exact),
// butterfly widths h = 1, 2, ..., D/2 ascending with each pair (i, i + h) ->
// (a + b, a - b), output sign flip (exact), one rounded multiply by c.  On
// entry a[e] is coordinate lt * E + e; on return slot e holds coord<D>(lt, e).
// stage: D floats of this warp's shared memory (d >= 256).
template <int D>
__device__ __forceinline__ void rotate_exact(float (&a)[Team<D>::E], int lt, uint32_t in_neg, uint32_t out_neg,
                                             float c, float *stage) {
    constexpr int E = Team<D>::E;
#pragma unroll
    for (int e = 0; e < E; e++)
        if ((in_neg >> e) & 1u) a[e] = -a[e];
#pragma unroll
    for (int h = 1; h < E; h <<= 1) {
#pragma unroll
        for (int i = 0; i < E; i++) {
            if ((i & h) == 0) {
                const float u = a[i], v = a[i + h];
                a[i] = __fadd_rn(u, v);
                a[i + h] = __fsub_rn(u, v);
            }
        }
    }
    if constexpr (!Team<D>::STAGE) {
        // stages h >= E: partner lane lt ^ (h / E) inside the team; the lower
        // lane keeps a + o, the upper one o - a
#pragma unroll
        for (int h = E; h < D; h <<= 1) {
            const int x = h / E;
            const bool up = (lt & x) != 0;
#pragma unroll
            for (int e = 0; e < E; e++) {
                const float o = __shfl_xor_sync(0xffffffffu, a[e], x);
                a[e] = up ? __fsub_rn(o, a[e]) : __fadd_rn(a[e], o);
            }
        }
    } else {
        // shared-memory stage: contiguous -> strided (lane l: coordinates l + 32 j)
#pragma unroll
        for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4 *>(stage + lt * E + e) = make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < E; j++) a[j] = stage[lt + 32 * j];
        __syncwarp();
#pragma unroll
        for (int h = E; h < 32; h <<= 1) {  // partner lane lt ^ h, same slot
            const bool up = (lt & h) != 0;
#pragma unroll
            for (int j = 0; j < E; j++) {
                const float o = __shfl_xor_sync(0xffffffffu, a[j], h);
                a[j] = up ? __fsub_rn(o, a[j]) : __fadd_rn(a[j], o);
            }
        }
#pragma unroll
        for (int h = 32; h < D; h <<= 1) {  // slots j, j + h / 32 of the lane
            const int hj = h / 32;
#pragma unroll
            for (int j = 0; j < E; j++) {
                if ((j & hj) == 0) {
                    const float u = a[j], v = a[j + hj];
                    a[j] = __fadd_rn(u, v);
                    a[j + hj] = __fsub_rn(u, v);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < E; e++) a[e] = __fmul_rn(c, ((out_neg >> e) & 1u) ? -a[e] : a[e]);
}

// sum_i y_i^2 as a pairwise binary tree in index order, each square and sum
// rounded once; every lane of the team returns the root.  The lane's squares
// of E consecutive indices lt * E + e (for d >= 256 the rotated vector is
// strided, so the squares go through the warp's stage first) sum in-lane for
// the blocks up to E, then across lanes (partner lt ^ x: the two add the same
// pair, and IEEE addition commutes).
template <int D>
__device__ __forceinline__ float tree_sum_squares(const float (&a)[Team<D>::E], int lt, float *stage) {
    constexpr int E = Team<D>::E, T = Team<D>::T;
    float p[E];
    if constexpr (!Team<D>::STAGE) {
#pragma unroll
        for (int e = 0; e < E; e++) p[e] = __fmul_rn(a[e], a[e]);
    } else {
#pragma unroll
        for (int j = 0; j < E; j++) stage[lt + 32 * j] = __fmul_rn(a[j], a[j]);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(stage + lt * E + e);
            p[e] = v.x;
            p[e + 1] = v.y;
            p[e + 2] = v.z;
            p[e + 3] = v.w;
        }
    }
#pragma unroll
    for (int len = E; len > 1; len >>= 1) {
#pragma unroll
        for (int j = 0; j < len / 2; j++) p[j] = __fadd_rn(p[2 * j], p[2 * j + 1]);
    }
    float s = p[0];
#pragma unroll
    for (int x = 1; x < T; x <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, x));
    return s;
}

// Bits [32 w, 32 w + 32) of a record from its code bytes (LSB-first stream).
__device__ __forceinline__ uint32_t record_word(const uint8_t *cw, int bits, int d, int w) {
    const int lo = 32 * w;
    uint32_t x = 0;
    for (int i = lo / bits; i < d && i * bits < lo + 32; i++) {
        const int off = i * bits - lo;
        const uint32_t k = cw[i];
        x |= off >= 0 ? (k << off) : (k >> -off);
    }
    return x;
}

// Whether a record of rk bytes is one of whole 32-bit words: records of d = 16 at an odd
// width are not, nor one of even width behind an odd number of 2-byte units (an odd capacity
// of a head of odd width); all other head dims have records of a multiple of four bytes.
template <int D>
__device__ __forceinline__ bool whole_words(const uint8_t *rec, int rk) {
    return D > 16 || (rk % 4 == 0 && (reinterpret_cast<uintptr_t>(rec) & 3u) == 0);
}

// Store the d*bits/8-byte record built from the code bytes: each team lane
// assembles whole 32-bit words (coalesced 4-byte stores), or 2-byte halves.
template <int D>
__device__ __forceinline__ void store_record(const uint8_t *cw, int bits, uint8_t *dst, int lt) {
    constexpr int T = Team<D>::T;
    const int rk = D * bits / 8;
    if (whole_words<D>(dst, rk)) {
        for (int c = lt; c < rk / 4; c += T) reinterpret_cast<uint32_t *>(dst)[c] = record_word(cw, bits, D, c);
    } else {
        for (int c = lt; c < rk / 2; c += T) {
            const uint32_t w = record_word(cw, bits, D, c >> 1);
            reinterpret_cast<uint16_t *>(dst)[c] = static_cast<uint16_t>((c & 1) ? (w >> 16) : (w & 0xFFFFu));
        }
    }
}

// Codes of the lane's rotated coordinates (slot by slot) and the vector's scale: keys on the midrise grid of [-m, m], values by #{k : thr_k < y / sigma}
// (S: the sum of squares; thr: the width's thresholds).
template <int D>
__device__ __forceinline__ float team_codes(const float (&a)[Team<D>::E], float m, float S, int bits, bool values,
                                            const float *thr, uint32_t (&k)[Team<D>::E]) {
    constexpr int E = Team<D>::E;
    float u[E];
    if (!values) {
        const float rr = m > 0.0f ? __frcp_rn(m) : 0.0f;
        const float hc = static_cast<float>(1 << (bits - 1)), top = static_cast<float>((1 << bits) - 1);
#pragma unroll
        for (int e = 0; e < E; e++) {
            // round(v + 1) 2^(b-1) as one FMA (scaling by a power of two commutes with the rounding)
            u[e] = __fmaf_rn(__fmul_rn(a[e], rr), hc, hc);
            u[e] = fminf(fmaxf(u[e], 0.0f), top);
            k[e] = __float_as_uint(__fadd_rd(u[e], 8388608.0f)) & 0xFFu;
        }
        return m;
    }
    const float sigma = __fsqrt_rn(__fmul_rn(S, 1.0f / D));  // / d exact (a power of two)
    const float rr = sigma > 0.0f ? __frcp_rn(sigma) : 0.0f;
#pragma unroll
    for (int e = 0; e < E; e++) {
        u[e] = __fmul_rn(a[e], rr);
        k[e] = 0;
    }
    for (int s = 1 << (bits - 1); s >= 1; s >>= 1) {
#pragma unroll
        for (int e = 0; e < E; e++)
            if (thr[k[e] + s - 1] < u[e]) k[e] += s;
    }
    return sigma;
}

// The same with the codes as bytes, cw[coordinate].
template <int D>
__device__ __forceinline__ float quantize_team(const float (&a)[Team<D>::E], float m, float S, int bits, bool values,
                                               const float *thr, uint8_t *cw, int lt) {
    uint32_t k[Team<D>::E];
    const float scale = team_codes<D>(a, m, S, bits, values, thr, k);
#pragma unroll
    for (int e = 0; e < Team<D>::E; e++) cw[coord<D>(lt, e)] = static_cast<uint8_t>(k[e]);
    return scale;
}

// The record of a team of four codes a lane (d <= 128), written without shared
// memory: the lane's codes as one field of 4 * bits bits, and lane c gathers the
// fields that reach into word c.  Every lane of the warp calls it; store: the
// team's vector is written.
template <int D>
__device__ __forceinline__ void store_fields(const uint32_t (&k)[4], int bits, uint8_t *dst, int lt, bool store) {
    constexpr int T = Team<D>::T;
    static_assert(Team<D>::E == 4, "four coordinates a lane");
    const int width = 4 * bits, first = 32 * lt / width;
    const uint32_t field = k[0] | (k[1] << bits) | (k[2] << (2 * bits)) | (k[3] << (3 * bits));
    const int n = T == 32 ? 8 / bits + 2 : 8;  // teams of a warp may differ in width
    uint32_t x = 0;
    for (int i = 0; i < n; i++) {
        const int from = first + i, off = width * from - 32 * lt;
        const uint32_t f = __shfl_sync(0xffffffffu, field, from < T ? from : 0, T);
        if (from < T && off < 32) x |= off >= 0 ? f << off : f >> -off;
    }
    if (!store) return;
    const int rk = D * bits / 8;
    if (whole_words<D>(dst, rk)) {
        if (lt < rk / 4) reinterpret_cast<uint32_t *>(dst)[lt] = x;
    } else {
        if (lt < (rk + 2) / 4) reinterpret_cast<uint16_t *>(dst)[2 * lt] = static_cast<uint16_t>(x);
        if (lt < rk / 4) reinterpret_cast<uint16_t *>(dst)[2 * lt + 1] = static_cast<uint16_t>(x >> 16);
    }
}

// Codes i0..i0 + 3 (i0 a multiple of four) of a record of a multiple of four bytes.
__device__ __forceinline__ void load_codes4(const uint8_t *rec, int words, int i0, int bits, uint32_t (&k)[4]) {
    const int bit = i0 * bits, w = bit >> 5;
    const uint32_t *r = reinterpret_cast<const uint32_t *>(rec);
    const uint32_t lo = r[w], hi = w + 1 < words ? r[w + 1] : 0u, mask = (1u << bits) - 1u;
    const uint32_t f = __funnelshift_r(lo, hi, bit & 31);
#pragma unroll
    for (int e = 0; e < 4; e++) k[e] = (f >> (e * bits)) & mask;
}

// A kernel parameter through its generic address: lanes that read different words of
// a table then share memory transactions (the constant path serves one word at a time).
template <class P>
__device__ __forceinline__ const P *param_table(const P *p) {
    asm("" : "+l"(p));
    return p;
}

// The tables of the widths in `used` (bit b: width b), flat by width.
__device__ __forceinline__ void stage_widths(float *to, const float *param, uint32_t used, int count_less) {
    const float *from = param_table(param);
    for (int b = 1; b <= 8; b++) {
        if (!((used >> b) & 1u)) continue;
        for (int j = threadIdx.x; j < (1 << b) - count_less; j += blockDim.x) to[cb_off(b) + j] = from[cb_off(b) + j];
    }
}

// vec / n and vec % n for the index of a vector: 32-bit arithmetic where it fits.
__device__ __forceinline__ int split_index(unsigned long long &r, int n) {
    if ((r >> 32) == 0) {
        const uint32_t x = static_cast<uint32_t>(r), q = x / static_cast<uint32_t>(n);
        r = q;
        return static_cast<int>(x - q * static_cast<uint32_t>(n));
    }
    const int m = static_cast<int>(r % static_cast<unsigned>(n));
    r /= static_cast<unsigned>(n);
    return m;
}

// Load the lane's E contiguous fp16 coordinates (16- or 8-byte loads).
template <int E>
__device__ __forceinline__ void load_coords(const uint16_t *src, float (&a)[E]) {
    if constexpr (E % 8 == 0) {
#pragma unroll
        for (int c = 0; c < E / 8; c++) {
            const uint4 v = reinterpret_cast<const uint4 *>(src)[c];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[q]));
                a[8 * c + 2 * q] = f.x;
                a[8 * c + 2 * q + 1] = f.y;
            }
        }
    } else {
        static_assert(E == 4, "four coordinates per lane below 256 dimensions");
        const uint2 v = *reinterpret_cast<const uint2 *>(src);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
        a[0] = f0.x;
        a[1] = f0.y;
        a[2] = f1.x;
        a[3] = f1.y;
    }
}

__device__ __forceinline__ uint32_t code_at(const uint8_t *rec, int i, int bits) {
    const int bit = i * bits, by = bit >> 3, sh = bit & 7;
    uint32_t v = rec[by];
    if (sh + bits > 8) v |= static_cast<uint32_t>(rec[by + 1]) << 8;
    return (v >> sh) & ((1u << bits) - 1u);
}

// R x for a vector held by one warp with lane l owning coordinates l + 32 j
// (j < ceil(D/32); for D < 32 lanes >= D hold zeros): sign flip, butterflies
// (shuffles for h < 32, in-lane for h >= 32), sign flip, scale.  Attention
// arithmetic: any order within its tolerance.
template <int D>
__device__ __forceinline__ void warp_rotate_strided(float (&x)[(D + 31) / 32], const uint32_t *sb, float c,
                                                    int lane) {
    constexpr int J = (D + 31) / 32;
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int i = lane + 32 * j;
        if (i < D && neg_coord(sb, i)) x[j] = -x[j];
    }
#pragma unroll
    for (int h = 1; h < (D < 32 ? D : 32); h <<= 1) {
        const bool up = (lane & h) != 0;
#pragma unroll
        for (int j = 0; j < J; j++) {
            const float o = __shfl_xor_sync(0xffffffffu, x[j], h);
            x[j] = up ? o - x[j] : x[j] + o;
        }
    }
#pragma unroll
    for (int h = 32; h < D; h <<= 1) {
        const int hj = h / 32;
#pragma unroll
        for (int j = 0; j < J; j++) {
            if ((j & hj) == 0) {
                const float u = x[j], v = x[j + hj];
                x[j] = u + v;
                x[j + hj] = u - v;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int i = lane + 32 * j;
        x[j] = (i < D && neg_coord(sb, i)) ? -c * x[j] : c * x[j];
    }
}

}  // namespace
}  // namespace tqk
