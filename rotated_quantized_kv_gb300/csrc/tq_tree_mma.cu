// tq_tree_mma.cu -- tree attention on the fifth-generation tensor cores
// (head_dim 64 and 128).
//
// A CTA takes a contiguous range of the list of 128-token tiles (tq_serve.h).
// Per tile, with R query rows (draft x head of the group) as MMA columns:
//
//   S^T[128 tokens][R] = K[128][d] (R q)^T      A = K in TMEM, B = q in shared memory
//   P^T = 2^(S^T - m) sigma                     softmax warps, one token per thread
//   O^T[d][R] += V^T[d][128] P^T[128][R]        A = V in shared memory, B = P
//
// The transposed products put the tokens (and then the dims) on the 128 MMA
// rows, so a small tree wastes no tensor rows, and a token's key scale is one
// number per thread.  Key codes enter the MMA as they lie in the record: one
// AND leaves a code at bit s of an fp16 half, the exact (sub)normal code 2^(s -
// 24); the query element that meets it carries 2^(13 - s), and the affine map of
// the level, the scale m_t and the row's power of two are applied to the sum:
//   x = m_t (A_r U + B_r).
// q enters as fp16 hi + lo (22 bits; the lo products run over the same TMEM
// operand), P as fp16 p sigma, value levels as fp16(s c_k) with s chosen on the
// host so that the levels round closely; 1/s is part of sigma.
//
// The running max is lazy: a row's m moves only when a score exceeds it by 8
// (log2 units), or a sigma outgrows its common power of two by 2^7, so that
// most tiles neither reduce over tokens nor touch the accumulator.
//
// Why K in TMEM and V in shared memory: shared-memory bandwidth (128 B a
// clock, which the MMA's operand reads share) bounds the tile, and a K tile in
// TMEM costs none of it: a thread unpacks its token's record into its own TMEM lane.
// V^T needs the dims on the lanes, so V goes through shared memory with tokens
// as the K dimension (MN-major operand).
//
// Roles (18 warps): 0-7 softmax (two groups of four warps, half the rows each),
// 8-11 keys, 12-15 values, 16 MMA issue, 17 record loads (cp.async into a ring).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include <cuda_fp16.h>

#include "tq_serve.h"
#include "tq_team.cuh"
#include "tq_tree.cuh"

namespace tqk {
namespace {

using namespace tree;

constexpr int kMmaThreads = 18 * 32;
constexpr int kKeyWarp = 8, kValueWarp = 12, kIssueWarp = 16, kLoadWarp = 17;
constexpr int kTableBytes = 8192;      // value levels
constexpr int kSmemMax = 227 * 1024;
constexpr float kInf = __builtin_huge_valf();
constexpr int kDrainPolls = 1 << 20;

__device__ __forceinline__ unsigned su32(const void *p) { return static_cast<unsigned>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// ---------------------------------------------------------------- packed binary32 pairs
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 ra, rb, rc, rr;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mov.b64 rc, {%6, %7};\n"
        " fma.rn.f32x2 rr, ra, rb, rc;\n mov.b64 {%0, %1}, rr;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// ---------------------------------------------------------------- barriers
__device__ __forceinline__ void bar_init(unsigned bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int threads, bool x) {
    unsigned r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(static_cast<unsigned>(x))
        : "memory");
    return r != 0;
}

// A wait that gave up marks the CTA dead: from then on nothing waits, every role
// walks its range to the end (all addresses come from the list, none from
// data), and the error flag tells the host that the output is incomplete.
struct Waiter {
    volatile int *dead;
    int *error;
    int polls;
    __device__ __forceinline__ void operator()(unsigned bar, unsigned parity) const {
        if (*dead) return;
        for (int i = 0; i < polls; i++)
            if (bar_try(bar, parity)) return;
        *dead = 1;
        atomicExch(error, 1);
    }
};

// ---------------------------------------------------------------- tensor cores
// K-major operand, 128-byte swizzle: rows of 64 elements (128 B), 8-row groups 1024 B apart.
__device__ __forceinline__ uint64_t desc_k(unsigned addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// MN-major operand, 128-byte swizzle: for each k a line of 64 mn elements (128 B),
// 8 of k 1024 B apart, the next 64 of mn `mn` bytes further.
__device__ __forceinline__ uint64_t desc_mn(unsigned addr, unsigned mn) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(mn >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16: f32 sums (bit 4), f16 operands, MN-major A and B (bits 15, 16), N / 8, M / 16
__host__ __device__ constexpr uint32_t idesc(int n, bool mn) {
    return (1u << 4) | (mn ? 3u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_ts(unsigned d, unsigned a, uint64_t b, uint32_t id, unsigned acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ss(unsigned d, uint64_t a, uint64_t b, uint32_t id, unsigned acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(unsigned bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_ld16(unsigned a, float *v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\ntcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld32(unsigned a, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}
// C columns (8, 16 or 32), waited for in the same statement so that no use is scheduled before
template <int C>
__device__ __forceinline__ void tmem_ld(unsigned a, float (&v)[C]) {
    if constexpr (C == 8) {
        uint32_t r[8];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
            : "r"(a)
            : "memory");
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __uint_as_float(r[i]);
    } else if constexpr (C == 16) {
        tmem_ld16(a, v);
    } else {
        tmem_ld32(a, v);
    }
}
__device__ __forceinline__ void tmem_st8(unsigned a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(unsigned a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- key codes
// 32 consecutive codes of B bits as 16 words: word i holds code i in its low
// half and code i + 16 in its high half, both at bit key_shift(B, i).  16 codes
// are B half-words of the record, so the word Z_k = (half-word k, half-word k +
// B) carries the same places of both sixteens; Z'_k is Z_k a byte later.
struct KeyPlace {
    bool later;    // taken from Z'
    int k, x, s;   // half-word, right shift, resulting bit
};
__host__ __device__ constexpr KeyPlace key_place(int B, int i) {
    const int p = B * i, k = p >> 4, pos = p & 15;
    if (pos + B <= 10) return KeyPlace{false, k, 0, pos};
    const int o = pos >= 8 ? pos - 8 : pos;  // (pos < 8: the code ends inside the half-word)
    const int x = o + B > 10 ? o + B - 10 : 0;
    return KeyPlace{pos >= 8, k, x, o - x};
}

template <int B, int I>
__device__ __forceinline__ uint32_t key_word(const uint32_t *z, const uint32_t *zl) {
    constexpr KeyPlace q = key_place(B, I);
    constexpr uint32_t m = ((1u << B) - 1u) << q.s;
    return ((q.later ? zl[q.k] : z[q.k]) >> q.x) & (m | m << 16);
}
template <int B, int... I>
__device__ __forceinline__ void key_words_impl(const uint32_t *z, const uint32_t *zl, uint32_t (&out)[16],
                                               std::integer_sequence<int, I...>) {
    ((out[I] = key_word<B, I>(z, zl)), ...);
}
template <int B>
__device__ __forceinline__ void key_words(const uint32_t *w, uint32_t (&out)[16]) {
    uint32_t z[B], zl[B];
#pragma unroll
    for (int k = 0; k < B; k++)
        z[k] = B == 1 ? w[0] : prmt(w[k >> 1], w[(k + B) >> 1], ((k & 1) ? 0x32u : 0x10u) | (((k + B) & 1) ? 0x7600u : 0x5400u));
#pragma unroll
    for (int k = 0; k < B; k++) zl[k] = k + 1 < B ? prmt(z[k], z[k + 1], 0x6341u) : z[k] >> 8;
    key_words_impl<B>(z, zl, out, std::make_integer_sequence<int, 16>{});
}

// The record of one token from the ring (16-byte chunks permuted within blocks
// of eight so that eight tokens' chunks fall in different banks).
__host__ __device__ constexpr int chunk_mask(int rec) { return rec == 32 ? 1 : rec == 64 ? 3 : rec == 128 ? 7 : 0; }

template <int WORDS>
__device__ __forceinline__ void load_record(unsigned base, int token, uint32_t (&w)[WORDS]) {
    constexpr int rec = 4 * WORDS, m = chunk_mask(rec);
    if constexpr (rec % 16 == 0) {
#pragma unroll
        for (int j = 0; j < rec / 16; j++) {
            const int c = token * (rec / 16) + j;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[4 * j]), "=r"(w[4 * j + 1]), "=r"(w[4 * j + 2]), "=r"(w[4 * j + 3])
                         : "r"(base + 16 * (c ^ ((c >> 3) & m))));
        }
    } else {
#pragma unroll
        for (int j = 0; j < rec / 8; j++)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(w[2 * j]), "=r"(w[2 * j + 1])
                         : "r"(base + token * rec + 8 * j));
    }
}

// ---------------------------------------------------------------- value levels
// Table of a width: entry e of lane column c.  1 bit: the halves of four codes
// (8 bytes); 2 to 4 bits: of two codes; wider: one code's in both halves.  Up to 3
// bits (and at 5 and 6) every lane has a column of its own.
__host__ __device__ constexpr int level_codes(int vb) { return vb == 1 ? 4 : vb <= 4 ? 2 : 1; }
__host__ __device__ constexpr int level_bytes(int vb) { return vb == 1 ? 8 : 4; }
__host__ __device__ constexpr int level_entries(int vb) { return 1 << (vb * level_codes(vb)); }
__host__ __device__ constexpr int level_columns(int vb) {
    return level_entries(vb) * level_bytes(vb) * 32 <= kTableBytes ? 32 : kTableBytes / (level_entries(vb) * level_bytes(vb));
}

template <int OFF, int N>
__device__ __forceinline__ uint32_t bits_at(const uint32_t *w, int shl) {
    // bits [OFF, OFF + N) of the record, shifted left by shl (>= 0), other bits around them
    constexpr int k = OFF >> 5, o = OFF & 31;
    if constexpr (o + N > 32) {
        const uint32_t x = __funnelshift_r(w[k], w[k + 1], o);
        return x << shl;
    } else {
        return o >= shl ? w[k] >> (o - shl) : w[k] << (shl - o);
    }
}

// 8 dims (one 16-byte chunk) of a record: chunk C
template <int VB, int C>
__device__ __forceinline__ uint4 level_chunk(const uint32_t *w, unsigned table, unsigned col) {
    uint32_t h[4];
    constexpr int kRow = level_columns(VB) * level_bytes(VB);  // bytes of an entry's columns
    constexpr int kLog = kRow == 256 ? 8 : kRow == 128 ? 7 : kRow == 64 ? 6 : 5;
    static_assert((1 << kLog) == kRow, "entry size");
    constexpr int n = VB * level_codes(VB);
    constexpr uint32_t mask = ((1u << n) - 1u) << kLog;
    if constexpr (VB == 1) {
        const unsigned a0 = table + ((bits_at<8 * C, 4>(w, kLog) & mask) | col);
        const unsigned a1 = table + ((bits_at<8 * C + 4, 4>(w, kLog) & mask) | col);
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(h[0]), "=r"(h[1]) : "r"(a0));
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(h[2]), "=r"(h[3]) : "r"(a1));
    } else if constexpr (VB <= 4) {
        const uint32_t f[4] = {bits_at<8 * VB * C, n>(w, kLog), bits_at<8 * VB * C + n, n>(w, kLog),
                               bits_at<8 * VB * C + 2 * n, n>(w, kLog), bits_at<8 * VB * C + 3 * n, n>(w, kLog)};
#pragma unroll
        for (int i = 0; i < 4; i++)
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(h[i]) : "r"(table + ((f[i] & mask) | col)));
    } else {
        const uint32_t f[8] = {bits_at<8 * VB * C, n>(w, kLog),          bits_at<8 * VB * C + n, n>(w, kLog),
                               bits_at<8 * VB * C + 2 * n, n>(w, kLog), bits_at<8 * VB * C + 3 * n, n>(w, kLog),
                               bits_at<8 * VB * C + 4 * n, n>(w, kLog), bits_at<8 * VB * C + 5 * n, n>(w, kLog),
                               bits_at<8 * VB * C + 6 * n, n>(w, kLog), bits_at<8 * VB * C + 7 * n, n>(w, kLog)};
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[i]) : "r"(table + ((f[i] & mask) | col)));
#pragma unroll
        for (int i = 0; i < 4; i++) h[i] = prmt(v[2 * i], v[2 * i + 1], 0x7610u);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// ---------------------------------------------------------------- shared memory
template <int D, int R>
struct Mma {
    static constexpr int CW = R / 2;                // rows per softmax group
    static constexpr int HALVES = D / 64;
    static constexpr int QPART = HALVES * R * 128;  // hi or lo of a block's queries
    static constexpr int QBUF = 2 * QPART;
    static constexpr int VBUF = HALVES * 128 * 128;
    static constexpr int PBUF = 128 * 128;
    static constexpr int KCOLS = D / 2;             // TMEM columns of a K tile
    static constexpr int T_K = 0, T_S = 2 * KCOLS, T_O = T_S + 2 * R;
    static constexpr int TCOLS = T_O + R <= 128 ? 128 : T_O + R <= 256 ? 256 : 512;
    static constexpr int O_Q = 0;
    static constexpr int O_V = O_Q + 2 * QBUF;
    static constexpr int O_P = O_V + 2 * VBUF;
    static constexpr int O_T = O_P + 2 * PBUF;
    static constexpr int O_A = O_T + kTableBytes;   // [4][R] A, [4][R] B
    static constexpr int O_M = O_A + 8 * R * 4;     // [R] m, [R] -m as used, [R] factors
    static constexpr int O_X = O_M + 3 * R * 4;     // [2][4][CW + 1] maxima of the warps
    static constexpr int O_B = (O_X + 2 * 4 * (CW + 1) * 4 + 15) / 16 * 16;
    static constexpr int kBars = 2 * 8 + 4 + 1 + 1 + 16;
    static constexpr int O_RING = (O_B + kBars * 8 + 16 + 127) / 128 * 128;
    static constexpr int kRing = kSmemMax - 1024 - O_RING;  // (1024: alignment)
};

struct RingGeo {
    int stage, stages;
};

template <int KB, int D>
__device__ __forceinline__ void keys_to_tmem(unsigned raw, int token, unsigned release, unsigned dst, const Waiter &wait,
                                             unsigned kempty, unsigned parity) {
    uint32_t w[D / 32 * KB];
    load_record<D / 32 * KB>(raw, token, w);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(release);
    wait(kempty, parity);
    __syncwarp();
    tc_after();
#pragma unroll
    for (int g = 0; g < D / 32; g++) {
        uint32_t out[16];
        key_words<KB>(w + g * KB, out);
        tmem_st16(dst + 16 * g, out);
    }
}

template <int VB, int D, int... C>
__device__ __forceinline__ void level_chunks(const uint32_t *w, unsigned table, unsigned col, unsigned dst, int token,
                                             std::integer_sequence<int, C...>) {
    (
        [&] {
            const uint4 x = level_chunk<VB, C>(w, table, col);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (C >> 3) * 16384 +
                                                                          (((C & 7) ^ (token & 7)) << 4)),
                         "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                         : "memory");
        }(),
        ...);
}
template <int VB, int D>
__device__ __forceinline__ void values_to_smem(unsigned raw, int token, unsigned release, unsigned table, unsigned dst,
                                               const Waiter &wait, unsigned vempty, unsigned parity) {
    uint32_t w[D / 32 * VB];
    load_record<D / 32 * VB>(raw, token, w);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(release);
    wait(vempty, parity);
    const unsigned col = (token & (level_columns(VB) - 1)) * level_bytes(VB);
    level_chunks<VB, D>(w, table, col, dst + token * 128, token, std::make_integer_sequence<int, D / 8>{});
}

// Fill the value table of a width (the four value warps together).
__device__ __forceinline__ void fill_levels(uint8_t *table, const uint16_t *half, int vb, int tid) {
    const int codes = level_codes(vb), entries = level_entries(vb), cols = level_columns(vb);
    const uint32_t m = (1u << vb) - 1u;
    for (int i = tid; i < entries * cols; i += 128) {
        const int e = i / cols;
        if (codes == 4) {
            uint32_t lo = half[e & 1] | static_cast<uint32_t>(half[(e >> 1) & 1]) << 16;
            uint32_t hi = half[(e >> 2) & 1] | static_cast<uint32_t>(half[(e >> 3) & 1]) << 16;
            reinterpret_cast<uint2 *>(table)[i] = make_uint2(lo, hi);
        } else if (codes == 2) {
            reinterpret_cast<uint32_t *>(table)[i] = half[e & m] | static_cast<uint32_t>(half[(e >> vb) & m]) << 16;
        } else {
            reinterpret_cast<uint32_t *>(table)[i] = half[e] * 0x10001u;
        }
    }
}

__device__ __forceinline__ void cp16(unsigned dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

// ---------------------------------------------------------------- kernel
template <int D, int R>
__global__ void __launch_bounds__(kMmaThreads, 1)
    tree_mma_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeLevels lv, const RingGeo ring) {
    using C = Mma<D, R>;
    constexpr int CW = C::CW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const unsigned sb = su32(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned bars = sb + C::O_B;
    auto k_full = [&](int i) { return bars + 8u * i; };
    auto k_empty = [&](int i) { return bars + 8u * (2 + i); };
    auto v_full = [&](int i) { return bars + 8u * (4 + i); };
    auto v_empty = [&](int i) { return bars + 8u * (6 + i); };
    auto s_full = [&](int i) { return bars + 8u * (8 + i); };
    auto s_empty = [&](int i) { return bars + 8u * (10 + i); };
    auto p_full = [&](int i) { return bars + 8u * (12 + i); };
    auto p_empty = [&](int i) { return bars + 8u * (14 + i); };
    auto c_full = [&](int i) { return bars + 8u * (16 + i); };
    const unsigned o_free = bars + 8u * 20, drain = bars + 8u * 21;
    auto r_full = [&](int i) { return bars + 8u * (22 + i); };
    auto r_empty = [&](int i) { return bars + 8u * (30 + i); };
    int *dead = reinterpret_cast<int *>(sm + C::O_B + C::kBars * 8);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(dead + 1);

    if (blockIdx.x == 0 && threadIdx.x == 0 && p.wait_polls > 0) *p.error = 0;
    const long long T = total_tiles(p), G = workers_of(p, T), worker = blockIdx.x;
    if (worker >= G) return;
    const long long at0 = worker * T / G;
    const int n_tiles = static_cast<int>((worker + 1) * T / G - at0);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; i++) {
            bar_init(k_full(i), 4);
            bar_init(k_empty(i), 1);
            bar_init(v_full(i), 4);
            bar_init(v_empty(i), 1);
            bar_init(s_full(i), 1);
            bar_init(s_empty(i), 8);
            bar_init(p_full(i), 8);
            bar_init(p_empty(i), 1);
        }
        for (int i = 0; i < 4; i++) bar_init(c_full(i), 4);
        bar_init(o_free, 8);
        bar_init(drain, 1);
        for (int i = 0; i < 8; i++) {
            bar_init(r_full(i), 32);
            bar_init(r_empty(i), 8);
        }
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)),
                     "r"(C::TCOLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const unsigned tbase = *tmem_slot;
    const Waiter wait{dead, p.error, p.wait_polls};
    Pos x = seek(p, at0);

    if (warp == kLoadWarp) {
        // ------------------------------------------------------ records into the ring
        int jp = 0;
        for (int j = 0; j < n_tiles; j++, advance(p, x)) {
            if (x.k >= x.tp) continue;
            const Tile w = tile_at(p, x);
            const SegView &s = p.seg[w.seg].seg;
            const int st = jp % ring.stages;
            wait(r_empty(st), ((jp / ring.stages) & 1) ^ 1);
            __syncwarp();
            const unsigned base = sb + C::O_RING + st * ring.stage;
#pragma unroll
            for (int kv = 0; kv < 2; kv++) {
                const int rec = D / 8 * (kv ? s.vbits[x.h] : s.kbits[x.h]);
                const uint8_t *src = (kv ? s.v : s.k) + x.b * (kv ? s.vblock : s.kblock) +
                                     (kv ? s.voff[x.h] : s.koff[x.h]) + static_cast<size_t>(w.t0) * rec;
                const unsigned dst = base + (kv ? 128 * (D / 8) * s.kbits[x.h] : 0);
                const int m = chunk_mask(rec), n = (w.n * rec + 15) / 16;
                for (int c = lane; c < n; c += 32) cp16(dst + 16 * (c ^ ((c >> 3) & m)), src + 16 * static_cast<size_t>(c));
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(r_full(st)) : "memory");
            jp++;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------------ MMA issue
        if (lane == 0) {
            constexpr uint32_t id_s = idesc(R, false), id_o = idesc(R, true);
            long long group = -1, part = -1;
            int seg = -1, ev = -1, parts = 0;
            bool first_prev = false;
            for (int j = 0; j <= n_tiles; j++) {
                bool first = false;
                if (j < n_tiles) {
                    const Tile w = tile_at(p, x);
                    const long long g = group_of(p, x), pt = part_of(p, g, x.tp, x.k);
                    if (g != group || w.seg != seg) ev++;
                    first = pt != part;
                    group = g;
                    seg = w.seg;
                    part = pt;
                    const int b = j & 1;
                    wait(k_full(b), (j >> 1) & 1);
                    wait(s_empty(b), ((j >> 1) & 1) ^ 1);
                    tc_after();
                    const unsigned q = sb + C::O_Q + (ev & 1) * C::QBUF, a = tbase + C::T_K + b * C::KCOLS,
                                   d = tbase + C::T_S + b * R;
                    const int halves = p.seg[w.seg].seg.fp16 ? 1 : 2;  // fp16 queries are exact: no lo part
                    for (int part2 = 0; part2 < halves; part2++)
#pragma unroll
                        for (int k = 0; k < D / 16; k++)
                            mma_ts(d, a + 8 * k, desc_k(q + part2 * C::QPART + (k >> 2) * R * 128 + 32 * (k & 3)), id_s,
                                   (part2 | k) != 0);
                    mma_commit(k_empty(b));
                    mma_commit(s_full(b));
                }
                if (j > 0) {
                    const int i = j - 1, b = i & 1;
                    wait(v_full(b), (i >> 1) & 1);
                    wait(p_full(b), (i >> 1) & 1);
                    if (first_prev) {
                        if (parts > 0) wait(o_free, (parts - 1) & 1);
                        parts++;
                    }
                    tc_after();
                    const unsigned v = sb + C::O_V + b * C::VBUF, pp = sb + C::O_P + b * C::PBUF, d = tbase + C::T_O;
#pragma unroll
                    for (int k = 0; k < 8; k++)
                        mma_ss(d, desc_mn(v + 2048 * k, C::HALVES == 2 ? 16384 : 0), desc_mn(pp + 2048 * k, 0), id_o,
                               !(first_prev && k == 0));
                    mma_commit(v_empty(b));
                    mma_commit(p_empty(b));
                }
                first_prev = first;
                if (j < n_tiles) advance(p, x);
            }
            // everything issued has completed before TMEM and shared memory go away
            mma_commit(drain);
            for (int i = 0; i < kDrainPolls; i++)
                if (bar_try(drain, 0)) break;
        }
    } else if (warp >= kValueWarp) {
        // ------------------------------------------------------ values into shared memory
        const int tid = threadIdx.x - kValueWarp * 32;
        int jp = 0, tvb = 0, tlaw = -1;
        for (int j = 0; j < n_tiles; j++, advance(p, x)) {
            const Tile w = tile_at(p, x);
            const SegView &s = p.seg[w.seg].seg;
            const int b = j & 1;
            const unsigned dst = sb + C::O_V + b * C::VBUF, par = ((j >> 1) & 1) ^ 1;
            if (s.fp16) {
                const uint8_t *src = s.v + x.b * s.vblock + s.voff[x.h] + static_cast<size_t>(w.t0) * (2 * D);
                wait(v_empty(b), par);
                // 16-byte chunks, a row's consecutive in a quarter warp (coalesced); rows behind the tokens are zeros
                for (int c = tid; c < 128 * D / 8; c += 128) {
                    const int t = c / (D / 8), e = c % (D / 8);
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (t < w.n) v = __ldg(reinterpret_cast<const uint4 *>(src) + c);
                    *reinterpret_cast<uint4 *>(sm + C::O_V + b * C::VBUF + (e >> 3) * 16384 + t * 128 +
                                               (((e & 7) ^ (t & 7)) << 4)) = v;
                }
            } else {
                const int vb = s.vbits[x.h], law = p.seg[w.seg].law;
                if (vb != tvb || law != tlaw) {
                    named_sync(4, 128);  // the other warps have done with the old table
                    fill_levels(sm + C::O_T, lv.half[law] + cb_off(vb), vb, tid);
                    named_sync(4, 128);
                    tvb = vb;
                    tlaw = law;
                }
                const int st = jp % ring.stages;
                const unsigned raw = sb + C::O_RING + st * ring.stage + 128 * (D / 8) * s.kbits[x.h];
                wait(r_full(st), (jp / ring.stages) & 1);
                __syncwarp();
                switch (vb) {
                    case 1: values_to_smem<1, D>(raw, tid, r_empty(st), sb + C::O_T, dst, wait, v_empty(b), par); break;
                    case 2: values_to_smem<2, D>(raw, tid, r_empty(st), sb + C::O_T, dst, wait, v_empty(b), par); break;
                    case 3: values_to_smem<3, D>(raw, tid, r_empty(st), sb + C::O_T, dst, wait, v_empty(b), par); break;
                    case 4: values_to_smem<4, D>(raw, tid, r_empty(st), sb + C::O_T, dst, wait, v_empty(b), par); break;
                    case 5: values_to_smem<5, D>(raw, tid, r_empty(st), sb + C::O_T, dst, wait, v_empty(b), par); break;
                    case 6: values_to_smem<6, D>(raw, tid, r_empty(st), sb + C::O_T, dst, wait, v_empty(b), par); break;
                    case 7: values_to_smem<7, D>(raw, tid, r_empty(st), sb + C::O_T, dst, wait, v_empty(b), par); break;
                    default: values_to_smem<8, D>(raw, tid, r_empty(st), sb + C::O_T, dst, wait, v_empty(b), par); break;
                }
                jp++;
            }
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(v_full(b));
        }
    } else if (warp >= kKeyWarp) {
        // ------------------------------------------------------ queries, and keys into TMEM
        const int kw = warp - kKeyWarp, tid = threadIdx.x - kKeyWarp * 32;
        const unsigned lanes = static_cast<unsigned>(32 * kw) << 16;
        long long group = -1;
        int seg = -1, ev = -1, jp = 0;
        for (int j = 0; j < n_tiles; j++, advance(p, x)) {
            const Tile w = tile_at(p, x);
            const SegView &s = p.seg[w.seg].seg;
            const long long g = group_of(p, x);
            const int b = j & 1;
            const unsigned dst = tbase + lanes + C::T_K + b * C::KCOLS, par = ((j >> 1) & 1) ^ 1;
            if (g != group || w.seg != seg) {
                // the block's queries for this segment: the buffer was last read two changes ago,
                // by products before those of tile j - 2
                ev++;
                group = g;
                seg = w.seg;
                wait(k_empty(b), par);
                __syncwarp();
                const int kb = s.fp16 ? 0 : s.kbits[x.h];
                uint8_t *q = sm + C::O_Q + (ev & 1) * C::QBUF;
                float *ab = reinterpret_cast<float *>(sm + C::O_A) + (ev & 3) * R;
                // place of this lane's coordinates and the power of two that meets the codes
                int place = 0;
                float pw = 1.f;
                if (kb) {
                    place = 2 * (lane & 15) + (lane >> 4);
                    const int p0 = kb * (lane & 15), pos = p0 & 15;
                    const int o = pos + kb <= 10 ? pos : (pos >= 8 ? pos - 8 : pos);
                    const int sh = o + kb > 10 ? 10 - kb : o;
                    pw = __uint_as_float(static_cast<uint32_t>(127 + 13 - sh) << 23);
                }
                for (int r = kw; r < R; r += 4) {
                    const int row = x.rb * R + r;
                    float v[D / 32];
#pragma unroll
                    for (int i = 0; i < D / 32; i++) v[i] = 0.f;
                    if (row < p.N * p.g) {
                        const uint16_t *src = p.q + x.b * p.qs[0] + (row / p.g) * p.qs[1] + (x.h * p.g + row % p.g) * p.qs[2];
#pragma unroll
                        for (int i = 0; i < D / 32; i++) v[i] = __half2float(__ushort_as_half(src[lane + 32 * i]));
                    }
                    float f = 1.f, A = p.qk_scale, B = 0.f;
                    if (kb) {
                        warp_rotate_strided<D>(v, p.sign_bits, p.inv_sqrt_d, lane);
                        float mx = 0.f, sum = 0.f;
#pragma unroll
                        for (int i = 0; i < D / 32; i++) mx = fmaxf(mx, fabsf(v[i])), sum += v[i];
#pragma unroll
                        for (int o = 16; o >= 1; o >>= 1) {
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                            sum += __shfl_xor_sync(0xffffffffu, sum, o);
                        }
                        int e = 0;  // f mx in [0.5, 1)
                        if (mx > 0.f && mx < kInf) e = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFFu) - 126;
                        e = max(-100, min(100, e));
                        f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                        // x = m_t qk_scale (2^(1-b) sum code q + (2^-b - 1) sum q), U = f 2^-11 sum code q
                        A = p.qk_scale * __uint_as_float(static_cast<uint32_t>(127 + 12 - kb + e) << 23);
                        B = p.qk_scale * (__uint_as_float(static_cast<uint32_t>(127 - kb) << 23) - 1.0f) * sum;
                    }
                    if (lane == 0) ab[r] = A, ab[4 * R + r] = B;
#pragma unroll
                    for (int i = 0; i < D / 32; i++) {
                        const float y = v[i] * f * pw;
                        const __half hi = __float2half_rn(y), lo = __float2half_rn(y - __half2float(hi));
                        const int k = kb ? 32 * i + place : lane + 32 * i;
                        const int off = (k >> 6) * R * 128 + r * 128 + ((((k & 63) >> 3) ^ (r & 7)) << 4) + (k & 7) * 2;
                        *reinterpret_cast<__half *>(q + off) = hi;
                        *reinterpret_cast<__half *>(q + C::QPART + off) = lo;
                    }
                }
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(c_full(ev & 3));
            }
            if (s.fp16) {
                const uint4 *src = reinterpret_cast<const uint4 *>(s.k + x.b * s.kblock + s.koff[x.h] +
                                                                  static_cast<size_t>(w.t0 + tid) * (2 * D));
                wait(k_empty(b), par);
                __syncwarp();
                tc_after();
#pragma unroll
                for (int i = 0; i < D / 32; i++) {
                    uint32_t out[16];
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (tid < w.n) v = __ldg(src + 4 * i + c);
                        out[4 * c] = v.x, out[4 * c + 1] = v.y, out[4 * c + 2] = v.z, out[4 * c + 3] = v.w;
                    }
                    tmem_st16(dst + 16 * i, out);
                }
            } else {
                const int st = jp % ring.stages;
                const unsigned raw = sb + C::O_RING + st * ring.stage;
                wait(r_full(st), (jp / ring.stages) & 1);
                __syncwarp();
                switch (s.kbits[x.h]) {
                    case 1: keys_to_tmem<1, D>(raw, tid, r_empty(st), dst, wait, k_empty(b), par); break;
                    case 2: keys_to_tmem<2, D>(raw, tid, r_empty(st), dst, wait, k_empty(b), par); break;
                    case 3: keys_to_tmem<3, D>(raw, tid, r_empty(st), dst, wait, k_empty(b), par); break;
                    case 4: keys_to_tmem<4, D>(raw, tid, r_empty(st), dst, wait, k_empty(b), par); break;
                    case 5: keys_to_tmem<5, D>(raw, tid, r_empty(st), dst, wait, k_empty(b), par); break;
                    case 6: keys_to_tmem<6, D>(raw, tid, r_empty(st), dst, wait, k_empty(b), par); break;
                    case 7: keys_to_tmem<7, D>(raw, tid, r_empty(st), dst, wait, k_empty(b), par); break;
                    default: keys_to_tmem<8, D>(raw, tid, r_empty(st), dst, wait, k_empty(b), par); break;
                }
                jp++;
            }
            tmem_wait_st();
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(k_full(b));
        }
    } else {
        // ------------------------------------------------------ softmax
        const int wg = warp >> 2, qw = warp & 3, tok = 32 * qw + lane;  // TMEM lane = token (or dim of O)
        const unsigned lanes = static_cast<unsigned>(32 * qw) << 16;
        float *m_row = reinterpret_cast<float *>(sm + C::O_M) + wg * CW;  // m; + R: -m as used; + 2R: factors
        float *maxima = reinterpret_cast<float *>(sm + C::O_X) + wg * 4 * (CW + 1);
        long long group = -1, part = -1;
        int seg = -1, ev = -1, E = 0;
        float l[CW];
#pragma unroll
        for (int c = 0; c < CW; c++) l[c] = 0.f;
        for (int j = 0; j < n_tiles; j++) {
            const Tile w = tile_at(p, x);
            const SegView &s = p.seg[w.seg].seg;
            const long long g = group_of(p, x), pt = part_of(p, g, x.tp, x.k);
            const int b = j & 1;
            const unsigned par = (j >> 1) & 1;
            const bool first = pt != part, valid = tok < w.n;
            float ks = 1.f, vs = 1.f;
            if (!s.fp16) {
                ks = vs = 0.f;
                if (valid) {
                    const size_t at = (static_cast<size_t>(x.b) * p.H + x.h) * s.capacity + w.t0 + tok;
                    ks = __ldg(s.ks + at);
                    vs = __ldg(s.vs + at) * lv.inv[p.seg[w.seg].law][s.vbits[x.h]];
                }
            } else if (!valid) {
                ks = vs = 0.f;
            }
            if (g != group || w.seg != seg) {
                ev++;
                wait(c_full(ev & 3), (ev >> 2) & 1);
            }
            group = g;
            seg = w.seg;
            part = pt;
            const float *ab = reinterpret_cast<const float *>(sm + C::O_A) + (ev & 3) * R + wg * CW;
            wait(s_full(b), par);
            __syncwarp();
            tc_after();
            float u[CW];
            const unsigned s_addr = tbase + lanes + C::T_S + b * R + wg * CW;
            // x = ks (A U + B), less m
            auto scores = [&](bool less) {
                tmem_ld<CW>(s_addr, u);
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    const float4 A = *reinterpret_cast<const float4 *>(ab + c), B = *reinterpret_cast<const float4 *>(ab + 4 * R + c);
                    float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (less) m = *reinterpret_cast<const float4 *>(m_row + R + c);
                    float2 y = ffma2(make_float2(u[c], u[c + 1]), make_float2(A.x, A.y), make_float2(B.x, B.y));
                    y = ffma2(y, make_float2(ks, ks), make_float2(m.x, m.y));
                    u[c] = y.x, u[c + 1] = y.y;
                    y = ffma2(make_float2(u[c + 2], u[c + 3]), make_float2(A.z, A.w), make_float2(B.z, B.w));
                    y = ffma2(y, make_float2(ks, ks), make_float2(m.z, m.w));
                    u[c + 2] = y.x, u[c + 3] = y.y;
                }
            };
            bool raise = first;
            float scale = 1.f;  // 2^-E
            if (!first) {
                scores(true);
                float top = u[0];
#pragma unroll
                for (int c = 1; c < CW; c++) top = fmaxf(top, u[c]);
                scale = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);
                raise = valid && (top > 8.0f || vs * scale > 128.0f);
            }
            if (named_or(1 + wg, 128, raise)) {
                scores(false);
                float mine = -kInf;
#pragma unroll
                for (int c = 0; c < CW; c++) {
                    float v = valid ? u[c] : -kInf;
                    asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
                    if (lane == c) mine = v;
                }
                float big = valid ? vs : 0.f;
                asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(big));
                if (lane < CW) maxima[qw * (CW + 1) + lane] = mine;
                if (lane == 0) maxima[qw * (CW + 1) + CW] = big;
                named_sync(1 + wg, 128);
                big = fmaxf(fmaxf(maxima[CW], maxima[2 * CW + 1]), fmaxf(maxima[3 * CW + 2], maxima[4 * CW + 3]));
                // E: the largest sigma times 2^-E in [0.5, 1)
                int e = 0;
                if (!s.fp16 && big > 0.f && big < kInf)
                    e = max(-100, min(100, static_cast<int>((__float_as_uint(big) >> 23) & 0xFFu) - 126));
                const int now = first ? e : max(E, e);
                if (tok < CW) {
                    const float old = first ? -kInf : m_row[tok];
                    float m = old;
#pragma unroll
                    for (int i = 0; i < 4; i++) m = fmaxf(m, maxima[i * (CW + 1) + tok]);
                    m_row[tok] = m;
                    m_row[R + tok] = m == -kInf ? 0.f : -m;
                    m_row[2 * R + tok] = old == -kInf ? 0.f : ex2(old - m);
                }
                named_sync(1 + wg, 128);
                if (!first) {
                    // earlier weights to the new max: the sums here, the accumulator in TMEM
                    wait(p_empty((j - 1) & 1), ((j - 1) >> 1) & 1);
                    __syncwarp();
                    tc_after();
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - min(now - E, 126)) << 23);
#pragma unroll
                    for (int c = 0; c < CW; c += 8) {
                        float o[8];
                        uint32_t r[8];
                        tmem_ld<8>(tbase + lanes + C::T_O + wg * CW + c, o);
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const float f = m_row[2 * R + c + i];
                            l[c + i] *= f;
                            r[i] = __float_as_uint(o[i] * (f * down));
                        }
                        tmem_st8(tbase + lanes + C::T_O + wg * CW + c, r);
                    }
                    tmem_wait_st();
                }
                E = now;
                scale = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);
                scores(true);
            }
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(s_empty(b));
            const float sv = vs * scale;
            if (j >= 2) wait(p_empty(b), par ^ 1);
            uint8_t *prow = sm + C::O_P + b * C::PBUF + tok * 128;
#pragma unroll
            for (int c = 0; c < CW; c += 8) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float p0 = valid ? ex2(u[c + 2 * i]) : 0.f, p1 = valid ? ex2(u[c + 2 * i + 1]) : 0.f;
                    l[c + 2 * i] += p0;
                    l[c + 2 * i + 1] += p1;
                    const __half2 q = __floats2half2_rn(p0 * sv, p1 * sv);
                    h[i] = *reinterpret_cast<const uint32_t *>(&q);
                }
                *reinterpret_cast<uint4 *>(prow + ((((wg * CW + c) >> 3) ^ (tok & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
            fence_async();
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_full(b));
            // the part's last tile: its record
            advance(p, x);
            if (j + 1 == n_tiles || part_of(p, group_of(p, x), x.tp, x.k) != part) {
                float *rec = p.part + static_cast<size_t>(worker + part) * R * (D + 4);
                // row sums over the tokens: lane c of each warp ends up with row c's
#pragma unroll
                for (int c = 0; c < CW; c++) {
                    float v = l[c];
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    if (lane == 0) maxima[qw * (CW + 1) + c] = v;
                    l[c] = 0.f;
                }
                named_sync(1 + wg, 128);
                if (tok < CW) {
                    float *row = rec + (wg * CW + tok) * (D + 4);
                    row[0] = m_row[tok];
                    row[1] = (maxima[tok] + maxima[CW + 1 + tok]) + (maxima[2 * (CW + 1) + tok] + maxima[3 * (CW + 1) + tok]);
                }
                wait(p_empty(b), par);
                __syncwarp();
                tc_after();
                const float up = __uint_as_float(static_cast<uint32_t>(127 + E) << 23);
#pragma unroll
                for (int c = 0; c < CW; c += 8) {
                    float o[8];
                    tmem_ld<8>(tbase + lanes + C::T_O + wg * CW + c, o);
                    if (tok < D)
#pragma unroll
                        for (int i = 0; i < 8; i++) rec[(wg * CW + c + i) * (D + 4) + 4 + tok] = o[i] * up;
                }
                tc_before();
                named_sync(1 + wg, 128);  // (also: `maxima` is free again)
                if (lane == 0) bar_arrive(o_free);
            }
        }
    }
    tc_before();
    __syncthreads();
    if (warp == kIssueWarp) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(C::TCOLS) : "memory");
    }
}

// ---------------------------------------------------------------- value levels (host)
// fp16(s c_k), s in [1, 2) chosen so that the levels' rounding errors, weighted as
// N(0, 1) weighs their cells, are smallest: 4096 candidates for up to 6 bits
// (wider codebooks have too many levels for a choice to matter).
struct HostLevels {
    std::once_flag once;
    uint16_t half[256];
    float inv;
};
HostLevels g_levels[2][9];

void fit_levels(HostLevels &h, const float *c, int bits) {
    const int n = 1 << bits;
    double best = HUGE_VAL;
    float s_best = 1.f;
    const int tries = bits <= 6 ? 4096 : 1;
    for (int i = 0; i < tries; i++) {
        const float s = 1.f + static_cast<float>(i) / 4096.f;
        double err = 0.0;
        for (int k = n / 2; k < n; k++) {
            const double a = k == n / 2 ? 0.0 : 0.5 * (static_cast<double>(c[k - 1]) + c[k]);
            const double b = k + 1 == n ? 1e9 : 0.5 * (static_cast<double>(c[k]) + c[k + 1]);
            const double mass = std::erfc(a * 0.70710678118654752) - std::erfc(b * 0.70710678118654752);
            const double d = static_cast<double>(__half2float(__float2half_rn(s * c[k]))) / s - c[k];
            err += mass * d * d;
        }
        if (err < best) best = err, s_best = s;
    }
    for (int k = 0; k < n; k++) h.half[k] = __half_as_ushort(__float2half_rn(s_best * c[k]));
    h.inv = 1.f / s_best;
}

template <int D, int R>
cudaError_t tree_mma(const TreeParams &p, const TreeLevels &lv, cudaStream_t s) {
    using C = Mma<D, R>;
    static_assert(C::T_O + R <= 512, "TMEM columns");
    int stage = 0;
    for (int i = 0; i < p.n_packed; i++)
        for (int h = 0; h < p.H; h++) stage = std::max(stage, 128 * (D / 8) * (p.seg[i].seg.kbits[h] + p.seg[i].seg.vbits[h]));
    RingGeo ring;
    ring.stage = std::max(stage, 128);
    ring.stages = std::min(8, C::kRing / ring.stage);
    if (ring.stages < 1) return cudaErrorInvalidConfiguration;
    const size_t smem = kSmemMax;
    cudaError_t e = cudaFuncSetAttribute(tree_mma_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    tree_mma_kernel<D, R><<<p.workers, kMmaThreads, smem, s>>>(p, lv, ring);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_mma(const TreeParams &p, cudaStream_t s) {
    TreeLevels lv;
    std::memset(&lv, 0, sizeof(lv));
    for (int i = 0; i < p.n_packed; i++)
        for (int h = 0; h < p.H; h++) {
            const int vb = p.seg[i].seg.vbits[h], law = p.seg[i].law;
            if (lv.inv[law][vb] != 0.f) continue;
            HostLevels &hl = g_levels[law][vb];
            std::call_once(hl.once, [&] { fit_levels(hl, p.centroid[law] + cb_off(vb), vb); });
            std::memcpy(lv.half[law] + cb_off(vb), hl.half, sizeof(uint16_t) << vb);
            lv.inv[law][vb] = hl.inv;
        }
    if (p.d == 128) {
        if (p.R == 16) return tree_mma<128, 16>(p, lv, s);
        if (p.R == 32) return tree_mma<128, 32>(p, lv, s);
        return tree_mma<128, 64>(p, lv, s);
    }
    if (p.R == 16) return tree_mma<64, 16>(p, lv, s);
    if (p.R == 32) return tree_mma<64, 32>(p, lv, s);
    return tree_mma<64, 64>(p, lv, s);
}

}  // namespace tqk
