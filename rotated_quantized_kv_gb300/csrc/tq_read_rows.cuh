// tq_read_rows.cuh -- rows of a packed segment read back, one thread per vector of
// head_dim 128 or two consecutive vectors of head_dim 64, instantiated for keys and values
// by tq_read_rows_*.cu (NP: vectors a thread).
//
// The mirror of the compressor (tq_compress_rows.cuh): a thread loads its record
// (neighbouring threads' records are adjacent), holds the 128 coordinates as 64 packed
// pairs (m, m + 64), and runs the butterflies in registers.  A key level is read off
// the bits: the code placed at the top of the mantissa of 1.0 gives x = 1 + code 2^-b,
// and 2 x + (2^-b - 3) = (2 code + 1) 2^-b - 1 exactly.  Value levels come from a table
// with a column per lane.  The input signs of the rotation are applied to the codes:
// both grids are odd, level(2^b - 1 - code) = -level(code), so that one XOR per record
// word flips all its coordinates' signs.  The next block's records are on their way into shared memory
// meanwhile (cp.async).  The rows leave through shared memory in the caller's type
// (16-byte chunk q of row r at q ^ (r & 7)), so that global stores are whole lines.
// At head_dim 64 the two records are one stream of 128 codes, pair (m, m + 64) holds coordinate m
// of both vectors, and the stage that joins a pair's halves falls away.
// Every step is the operation of tq_dequantize, so the results are the same bits.
// Bound by issue slots and latency at 12 warps an SM: 65408 tokens of 8 heads from 3 bits
// into fp16, 113 us for both launches, 322 MB moved.  (Records by plain loads and rows
// staged as binary32: 135 us; sign flips on the coordinates: 127 us.)  5 x 777 tokens of 8 heads
// of 64 dims, K5V2, into bf16: 7.1 us for both (32 lanes on two vectors: 14.2 us).
#pragma once

#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>

#include "tq_compress_rows.cuh"
#include "tq_row_map.cuh"
#include "tq_serve.h"
#include "tq_team.cuh"

namespace tqk {
namespace {

// A warp's 32 rows in the caller's type, and two blocks of 32 records.
__host__ __device__ constexpr int read_rows_bytes(int dtype) { return dtype == TQ_DTYPE_F32 ? 32 * 512 : 32 * 256; }
template <int BITS>
__host__ __device__ constexpr int read_records_bytes() {
    return 32 * 16 * BITS;
}

template <int BITS>
__host__ __device__ constexpr int level_lanes() {  // columns of the level table
    return BITS <= 5 ? 32 : 1024 >> BITS;
}

template <int BITS, bool VAL>
__host__ __device__ constexpr size_t read_smem_bytes(int dtype) {
    return kWarps * (read_rows_bytes(dtype) + 2 * read_records_bytes<BITS>()) + 32 * 4 + 128 * 4 +
           (VAL ? (level_lanes<BITS>() << BITS) * 4 : 0);
}

// Code I placed with its top bit at bit 22.
template <int BITS, int I>
__device__ __forceinline__ uint32_t code_top(const uint32_t *w) {
    constexpr int bit = BITS * I, k = bit >> 5, o = bit & 31, up = 23 - BITS;
    if constexpr (o + BITS > 32) {
        return __funnelshift_r(w[k], w[k + 1], o) << up;
    } else {
        return o >= up ? w[k] >> (o - up) : w[k] << (up - o);
    }
}
template <int BITS, int I>
__device__ __forceinline__ float key_one(const uint32_t *w) {  // 1 + code 2^-b
    constexpr uint32_t mask = ((1u << BITS) - 1u) << (23 - BITS);
    return __uint_as_float((code_top<BITS, I>(w) & mask) | 0x3F800000u);
}
template <int BITS, int M>
__device__ __forceinline__ float2 key_levels(const uint32_t *w) {
    constexpr float c = 1.0f / (1 << BITS) - 3.0f;
    return ffma2(make_float2(key_one<BITS, M>(w), key_one<BITS, M + 64>(w)), make_float2(2.0f, 2.0f), make_float2(c, c));
}
template <int BITS, int I>
__device__ __forceinline__ float value_level(const uint32_t *w, const float *table) {
    constexpr int bit = BITS * I, k = bit >> 5, o = bit & 31;
    uint32_t c;
    if constexpr (o + BITS > 32) c = __funnelshift_r(w[k], w[k + 1], o);
    else c = w[k] >> o;
    return table[(c & ((1u << BITS) - 1u)) * level_lanes<BITS>()];
}
template <int BITS, bool VAL, int... M>
__device__ __forceinline__ void all_levels(const uint32_t *w, const float *table, float2 (&a)[64],
                                           std::integer_sequence<int, M...>) {
    if constexpr (VAL) ((a[M] = make_float2(value_level<BITS, M>(w, table), value_level<BITS, M + 64>(w, table))), ...);
    else ((a[M] = key_levels<BITS, M>(w)), ...);
}

struct ReadBlock {
    int b, h, tb;           // sequence, head, block of 32 threads' rows
    int at, t;              // this lane's (first) batch element (or page) and position
    int at2, t2;            // those of the second vector (head_dim 64)
    bool valid, valid2;
};

template <int NP, bool SLOTS>
__device__ __forceinline__ ReadBlock read_block(const ReadRowsParams &p, int n_tblk, int blk, int lane) {
    ReadBlock r;
    r.tb = blk % n_tblk;
    const int rest = blk / n_tblk;
    r.h = p.head[rest % p.n_heads];
    r.b = rest / p.n_heads;
    const int j = (32 * r.tb + lane) * NP;
    r.at = r.t = 0;
    r.valid = place_row<SLOTS>(p.rows, r.b, j, p.capacity, r.at, r.t);
    r.at2 = r.t2 = 0;
    r.valid2 = NP == 2 && place_row<SLOTS>(p.rows, r.b, j + 1, p.capacity, r.at2, r.t2);
    return r;
}

__device__ __forceinline__ void cp_async8(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(static_cast<unsigned>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

// The lane's records and scales on their way (records lie at the lane's place).
template <int BITS, int NP, bool SLOTS>
__device__ __forceinline__ float2 fetch_record(const ReadRowsParams &p, const ReadBlock &r, uint8_t *buf, int lane) {
    buf += lane * (16 * BITS);
    auto block = [&](int at) { return SLOTS ? at : r.b; };
    auto record = [&](int at, int t) { return p.codes + block(at) * p.block + p.off[r.h] + static_cast<size_t>(t) * (16 * BITS / NP); };
    auto scale = [&](int at, int t) { return p.scale + (static_cast<size_t>(block(at)) * p.H + r.h) * p.capacity + t; };
    float2 s = make_float2(0.f, 0.f);
    if constexpr (NP == 1) {
        if (r.valid) {
            const uint8_t *rec = record(r.at, r.t);
#pragma unroll
            for (int i = 0; i < BITS; i++) cp_async16(buf + 16 * i, rec + 16 * i);
            s.x = __ldg(scale(r.at, r.t));
        }
    } else {
        const uint8_t *rec = record(r.at, r.t);
        const float *sc = scale(r.at, r.t);
        if (r.valid) {
#pragma unroll
            for (int i = 0; i < BITS; i++) cp_async8(buf + 8 * i, rec + 8 * i);
            s.x = __ldg(sc);
        }
        if constexpr (SLOTS) rec = record(r.at2, r.t2) - 8 * BITS, sc = scale(r.at2, r.t2) - 1;  // (else they follow one another)
        if (r.valid2) {
#pragma unroll
            for (int i = BITS; i < 2 * BITS; i++) cp_async8(buf + 8 * i, rec + 8 * i);
            s.y = __ldg(sc + 1);
        }
    }
    return s;
}

template <class T2>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    T2 v;
    if constexpr (std::is_same<T2, __half2>::value) v = __floats2half2_rn(x, y);
    else v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t *>(&v);
}

// The thread's row into its warp's buffer, 16-bit types.
template <class T2>
__device__ __forceinline__ void put_row16(const float2 (&a)[64], uint8_t *row, int lane) {
#pragma unroll
    for (int q = 0; q < 8; q++) {
        *reinterpret_cast<uint4 *>(row + 16 * (q ^ (lane & 7))) =
            make_uint4(pack2<T2>(a[8 * q].x, a[8 * q + 1].x), pack2<T2>(a[8 * q + 2].x, a[8 * q + 3].x),
                       pack2<T2>(a[8 * q + 4].x, a[8 * q + 5].x), pack2<T2>(a[8 * q + 6].x, a[8 * q + 7].x));
        *reinterpret_cast<uint4 *>(row + 16 * ((8 + q) ^ (lane & 7))) =
            make_uint4(pack2<T2>(a[8 * q].y, a[8 * q + 1].y), pack2<T2>(a[8 * q + 2].y, a[8 * q + 3].y),
                       pack2<T2>(a[8 * q + 4].y, a[8 * q + 5].y), pack2<T2>(a[8 * q + 6].y, a[8 * q + 7].y));
    }
}

template <int BITS, bool VAL, int NP, bool SLOTS>
__global__ void __launch_bounds__(kThreads, 3) read_rows_kernel(const __grid_constant__ ReadRowsParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int rows_bytes = read_rows_bytes(p.dtype), per_warp = rows_bytes + 2 * read_records_bytes<BITS>();
    uint32_t *flip = reinterpret_cast<uint32_t *>(smem + kWarps * per_warp);
    float *op = reinterpret_cast<float *>(flip + 32);  // pairs (m, m + 64)
    float *table = op + 128;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const ReadRowsParams &g = *param_table(&p);
    for (int i = threadIdx.x; i < 4 * BITS; i += kThreads) flip[i] = g.flip[i];
    for (int i = threadIdx.x; i < kD; i += kThreads) op[i] = g.out_scale[(i >> 1) + 64 * (i & 1)];
    if constexpr (VAL)
        for (int i = threadIdx.x; i < (level_lanes<BITS>() << BITS); i += kThreads) table[i] = g.level[i / level_lanes<BITS>()];
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *buf = smem + warp * per_warp, *recs = buf + rows_bytes;
    const float *mine = table + (lane & (level_lanes<BITS>() - 1));
    const int n_tblk = (p.rows.n_max + 32 * NP - 1) / (32 * NP), n_blk = n_tblk * p.n_heads * p.B;
    const int gw = blockIdx.x * kWarps + warp, nw = gridDim.x * kWarps;
    float2 sc, sc_next = make_float2(0.f, 0.f);
    if (gw < n_blk) sc_next = fetch_record<BITS, NP, SLOTS>(p, read_block<NP, SLOTS>(p, n_tblk, gw, lane), recs, lane);
    asm volatile("cp.async.commit_group;\n" ::);
    for (int blk = gw, it = 0; blk < n_blk; blk += nw, it++) {
        sc = sc_next;
        if constexpr (NP == 1) sc.y = sc.x;
        if (blk + nw < n_blk)  // each lane reads its own place alone
            sc_next = fetch_record<BITS, NP, SLOTS>(p, read_block<NP, SLOTS>(p, n_tblk, blk + nw, lane),
                                         recs + ((it + 1) & 1) * read_records_bytes<BITS>(), lane);
        asm volatile("cp.async.commit_group;\n" ::);
        asm volatile("cp.async.wait_group 1;\n" ::: "memory");
        const ReadBlock r = read_block<NP, SLOTS>(p, n_tblk, blk, lane);
        const unsigned some = __ballot_sync(0xffffffffu, r.valid);
        const unsigned some2 = NP == 2 ? __ballot_sync(0xffffffffu, r.valid2) : 0u;
        if (!(some | some2)) continue;
        uint32_t w[4 * BITS];
        const uint4 *rec = reinterpret_cast<const uint4 *>(recs + (it & 1) * read_records_bytes<BITS>() + lane * (16 * BITS));
#pragma unroll
        for (int i = 0; i < BITS; i++) {
            const uint4 v = rec[i];
            const uint4 g = *reinterpret_cast<const uint4 *>(flip + 4 * i);
            w[4 * i] = v.x ^ g.x, w[4 * i + 1] = v.y ^ g.y, w[4 * i + 2] = v.z ^ g.z, w[4 * i + 3] = v.w ^ g.w;
        }
        float2 a[64];
        all_levels<BITS, VAL>(w, mine, a, std::make_integer_sequence<int, 64>{});
#pragma unroll
        for (int m = 0; m < 64; m++) a[m] = fmul2(a[m], sc);
        if (p.rotate) {
#pragma unroll
            for (int hh = 1; hh < 64; hh <<= 1) {
#pragma unroll
                for (int m = 0; m < 64; m++) {
                    if ((m & hh) == 0) {
                        const float2 u = a[m], v = a[m + hh];
                        a[m] = fadd2(u, v);
                        a[m + hh] = fsub2(u, v);
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < 64; m += 2) {
                const float4 o = *reinterpret_cast<const float4 *>(op + 2 * m);
                if constexpr (NP == 1) {
                    a[m] = make_float2(__fadd_rn(a[m].x, a[m].y), __fsub_rn(a[m].x, a[m].y));
                    a[m + 1] = make_float2(__fadd_rn(a[m + 1].x, a[m + 1].y), __fsub_rn(a[m + 1].x, a[m + 1].y));
                }
                a[m] = fmul2(a[m], make_float2(o.x, o.y));
                a[m + 1] = fmul2(a[m + 1], make_float2(o.z, o.w));
            }
        }
        __syncwarp();  // the last block's rows have left the buffer
        if (p.dtype == TQ_DTYPE_F32) {
            uint8_t *row = buf + lane * 512;
#pragma unroll
            for (int q = 0; q < 16; q++) {
                *reinterpret_cast<float4 *>(row + 16 * (q ^ (lane & 7))) =
                    make_float4(a[4 * q].x, a[4 * q + 1].x, a[4 * q + 2].x, a[4 * q + 3].x);
                *reinterpret_cast<float4 *>(row + 16 * ((16 + q) ^ (lane & 7))) =
                    make_float4(a[4 * q].y, a[4 * q + 1].y, a[4 * q + 2].y, a[4 * q + 3].y);
            }
        } else if (p.dtype == TQ_DTYPE_F16) {
            put_row16<__half2>(a, buf + lane * 256, lane);
        } else {
            put_row16<__nv_bfloat162>(a, buf + lane * 256, lane);
        }
        __syncwarp();
        const int64_t base = r.b * p.st[0] + r.h * p.st[1] + static_cast<int64_t>(32 * NP * r.tb) * p.st[2];
        if (p.dtype == TQ_DTYPE_F32) {  // four coordinates a lane, a thread's row(s) at a time
            const int second = NP == 2 ? lane >> 4 : 0;
#pragma unroll 4
            for (int i = 0; i < 32; i++) {
                if (!(((second ? some2 : some) >> i) & 1u)) continue;
                const float4 x = *reinterpret_cast<const float4 *>(buf + i * 512 + 16 * (lane ^ (i & 7)));
                float *o = static_cast<float *>(p.out) + base + (i * NP + second) * p.st[2] + 4 * (lane - 16 * second);
                if (p.vec) {
                    *reinterpret_cast<float4 *>(o) = x;
                } else {
                    o[0] = x.x, o[1] = x.y, o[2] = x.z, o[3] = x.w;
                }
            }
        } else {  // eight coordinates a lane, two threads' row(s) at a time
            const int c = lane & 15, second = NP == 2 ? c >> 3 : 0;
#pragma unroll 4
            for (int i = 0; i < 16; i++) {
                const int k = 2 * i + (lane >> 4);
                if (!(((second ? some2 : some) >> k) & 1u)) continue;
                const uint4 x = *reinterpret_cast<const uint4 *>(buf + k * 256 + 16 * (c ^ (k & 7)));
                uint16_t *o = static_cast<uint16_t *>(p.out) + base + (k * NP + second) * p.st[2] + 8 * (c - 8 * second);
                if (p.vec) {
                    *reinterpret_cast<uint4 *>(o) = x;
                } else {
                    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 8; e++) o[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the call's last launch ends behind its first
}

template <int BITS, bool VAL, int NP, bool SLOTS>
cudaError_t read_rows_launch(const ReadRowsParams &p, bool beside, cudaStream_t s) {
    const size_t smem = read_smem_bytes<BITS, VAL>(p.dtype);
    const cudaError_t e = cudaFuncSetAttribute(read_rows_kernel<BITS, VAL, NP, SLOTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(read_smem_bytes<BITS, VAL>(TQ_DTYPE_F32)));
    if (e != cudaSuccess) return e;
    const long long blocks = (static_cast<long long>((p.rows.n_max + 32 * NP - 1) / (32 * NP)) * p.n_heads * p.B + kWarps - 1) / kWarps;
    const long long grid = std::min<long long>(blocks, static_cast<long long>(current_sm_count()) * 3);
    return launch_beside(read_rows_kernel<BITS, VAL, NP, SLOTS>, static_cast<unsigned>(grid), kThreads, smem, s, beside, p);
}

template <bool VAL, int NP, bool SLOTS>
cudaError_t read_rows_dispatch(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s) {
    switch (bits) {
        case 1: return read_rows_launch<1, VAL, NP, SLOTS>(p, beside, s);
        case 2: return read_rows_launch<2, VAL, NP, SLOTS>(p, beside, s);
        case 3: return read_rows_launch<3, VAL, NP, SLOTS>(p, beside, s);
        case 4: return read_rows_launch<4, VAL, NP, SLOTS>(p, beside, s);
        case 5: return read_rows_launch<5, VAL, NP, SLOTS>(p, beside, s);
        case 6: return read_rows_launch<6, VAL, NP, SLOTS>(p, beside, s);
        case 7: return read_rows_launch<7, VAL, NP, SLOTS>(p, beside, s);
        case 8: return read_rows_launch<8, VAL, NP, SLOTS>(p, beside, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace tqk
