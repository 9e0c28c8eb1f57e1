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
// 24); the query element that meets it carries 2^(13 - s).  The affine map of the
// level adds a constant per row, which one more 16-deep step (constant columns in TMEM)
// brings into the sum, so that x = m_t A U with one A for the block.
// q enters as fp16 hi + lo (22 bits; the lo products run over the same TMEM
// operand), P as fp16 hi + 2^-11 lo of p sigma (22 bits; the lo products in columns of their
// own: with hi alone the output's error was 1.4 times that of rounding it to fp16, and weights
// below 2^-25 of the row's largest were lost; now it is 1.0 up to 4 value bits, 1.1 at 5, 1.2 at 6
// and 1.3 at 8), value levels as fp16(s c_k), s chosen on the host so that the levels round
// closely (those of 6 bits and more do not: the rest of that error); 1/s is part of sigma.
//
// A row's m is the running max of S + e, 2^e the power of two below the token's sigma (e in
// [-64, 64]): it bounds the weights p sigma that fp16 has to hold, whatever the values' sizes,
// and p = 2^(S - m) <= 2^(64 + 8) itself stays in binary32 (weights relative to the largest
// score alone, times a power of two common to a record's sigmas, lost a row's precision to
// one large value that it gave no weight: 0.5% at 2^16 times the others, all of it at 2^24).
// The running max is lazy: m moves only when some S + e exceeds it by 8, so that most
// tiles neither reduce over tokens nor touch the accumulator.
//
// Why K in TMEM and V in shared memory: shared-memory bandwidth (128 B a
// clock, which the MMA's operand reads share) bounds the tile, and a K tile in
// TMEM costs none of it: a thread unpacks its token's record into its own TMEM lane.
// V^T needs the dims on the lanes, so V goes through shared memory with tokens
// as the K dimension (MN-major operand).
//
// Roles (32 warps, 24 with 16 rows): softmax in four groups of four warps (two), an
// equal share of the rows each, four warps of keys, two groups of four of values that
// take alternate tiles, two that issue the MMAs, two that walk the list and load
// records and scales (cp.async into a ring); the others learn from a descriptor
// what a tile is.
//
// What bounds it: a tile costs a worker 1.57 us with 64 rows, 1.28 with 32, 1.04 with 16
// (head_dim 64: 1.63, 1.14, 0.97), where the tensor pipe is busy for 0.6 us (64 rows); the 32
// warps unpack 128 x 128 codes twice and exponentiate 128 x 64 scores, and the value rows, P and
// the MMA's operands share shared memory.  Start and end of the three kernels are some 22 us
// (64 rows; latencies, code that is cold).  Measured, all three: 16 drafts of 4 heads a KV head
// over 64K tokens of 8 heads K3V3 67 us, 64 drafts over 4 x 32K 304 us, 13 drafts over 16 x 9K at
// head_dim 64 80 us.  The weights' lo half is 0.17 us of a tile of 64 rows.
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

constexpr int kTableBytes = 8192;      // value levels
// Tiles whose descriptor and scales are kept, and ring stages: the loader is at most
// kMaxStages tiles ahead of the key and value warps, and these, when they release
// tile a, have waited for the MMA and the softmax of tile a - 4; so slot j % 8 has been
// read by everyone when tile j + 8 overwrites it.
constexpr int kSlots = 8;
constexpr int kMaxStages = 4;
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

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// two independent binary32 operations
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 ra, rb, rr;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n add.rn.f32x2 rr, ra, rb;\n"
        " mov.b64 {%0, %1}, rr;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fmul2(float2 a, float b) {
    float2 r;
    asm("{.reg .b64 ra, rb, rr;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %4};\n mul.rn.f32x2 rr, ra, rb;\n"
        " mov.b64 {%0, %1}, rr;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b));
    return r;
}
__device__ __forceinline__ float2 ffma2(float2 a, float b, float2 c) {
    float2 r;
    asm("{.reg .b64 ra, rb, rc, rr;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %4};\n mov.b64 rc, {%5, %6};\n"
        " fma.rn.f32x2 rr, ra, rb, rc;\n mov.b64 {%0, %1}, rr;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

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
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000u)  // (may suspend for a microsecond)
        : "memory");
    return ok != 0;
}
// Whether the phase has completed, without waiting (asked early, the answer's
// latency hides behind other work).
__device__ __forceinline__ bool bar_test(unsigned bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void bar_expect_tx(unsigned bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load(unsigned dst, const void *src, unsigned bytes, unsigned bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
        "r"(bytes), "r"(bar)
        : "memory");
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

// A bounded wait, by whole warps.  A warp whose wait ran out sets the error flag (the
// output is incomplete) and leaves its role's loop: it reads no descriptor, touches no
// memory and signals nothing any more, so that no other warp is let past a barrier
// early; those time out in turn.  Roles that meet at named barriers leave together.
struct Waiter {
    int *error;
    int polls;
    bool gone;  // the same in all lanes
    // Two barriers at once: half of the warp's lanes poll each (a wait costs some 200
    // cycles even when there is nothing to wait for).
    __device__ __forceinline__ void both(unsigned bar0, unsigned parity0, unsigned bar1, unsigned parity1) {
        const bool low = (threadIdx.x & 31) < 16;
        (*this)(low ? bar0 : bar1, low ? parity0 : parity1);
    }
    // The wait behind an early bar_test.
    __device__ __forceinline__ void unless(bool done, unsigned bar, unsigned parity) {
        bool lost = gone;
        if (!done) lost = poll(bar, parity);
        gone = __any_sync(0xffffffffu, lost);
    }
    __device__ __forceinline__ void operator()(unsigned bar, unsigned parity) {
        gone = __any_sync(0xffffffffu, poll(bar, parity));
    }
    __device__ __forceinline__ bool poll(unsigned bar, unsigned parity) {
        if (gone) return true;
        unsigned ok = 0;
        if (polls > 0)
            asm volatile(
                "{\n .reg .pred p, q;\n .reg .s32 n;\n mov.s32 n, %3;\n mov.u32 %0, 1;\n"
                "POLL:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n @p bra DONE;\n"
                " sub.s32 n, n, 1;\n setp.gt.s32 q, n, 0;\n @q bra POLL;\n mov.u32 %0, 0;\nDONE:\n}"
                : "=r"(ok)
                : "r"(bar), "r"(parity), "r"(polls), "r"(1000u)
                : "memory");
        if (!ok) atomicExch(error, 1);
        return !ok;
    }
};

// ---------------------------------------------------------------- tensor cores
// K-major operand without swizzle, 16 of k: 8 rows of 16 bytes, the second 8 of k 128 B
// further, the next 8 rows 256 B further.
__device__ __forceinline__ uint64_t desc_k16(unsigned addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
           (static_cast<uint64_t>(256 >> 4) << 32) | (1ull << 46);
}
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
__device__ __forceinline__ bool elect_one() {
    unsigned r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void mma_commit(unsigned bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// C columns (8, 16 or 32) of this thread's TMEM lane: the load, and the wait for it, which
// passes every register through so that no use is scheduled before.
template <int C>
__device__ __forceinline__ void tmem_issue(unsigned a, float (&v)[C]) {
    static_assert(C == 8 || C == 16 || C == 32, "8, 16 or 32 columns");
    if constexpr (C == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "r"(a)
                     : "memory");
    } else if constexpr (C == 16) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                     : "r"(a)
                     : "memory");
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
                     : "r"(a)
                     : "memory");
    }
}
template <int C>
__device__ __forceinline__ void tmem_wait(float (&v)[C]) {
    if constexpr (C == 8) {
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
                     :
                     : "memory");
    } else if constexpr (C == 16) {
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                     :
                     : "memory");
    } else {
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                     :
                     : "memory");
    }
}
template <int C>
__device__ __forceinline__ void tmem_ld(unsigned a, float (&v)[C]) {
    tmem_issue<C>(a, v);
    tmem_wait<C>(v);
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
__device__ __forceinline__ uint4 level_chunk(const uint32_t *w, const uint8_t *table) {
    uint32_t h[4];
    constexpr int kRow = level_columns(VB) * level_bytes(VB);  // bytes of an entry's columns
    constexpr int kLog = kRow == 256 ? 8 : kRow == 128 ? 7 : kRow == 64 ? 6 : 5;
    static_assert((1 << kLog) == kRow, "entry size");
    constexpr int n = VB * level_codes(VB);
    constexpr uint32_t mask = ((1u << n) - 1u) << kLog;
    if constexpr (VB == 1) {
        const uint2 a = *reinterpret_cast<const uint2 *>(table + (bits_at<8 * C, 4>(w, kLog) & mask));
        const uint2 b = *reinterpret_cast<const uint2 *>(table + (bits_at<8 * C + 4, 4>(w, kLog) & mask));
        h[0] = a.x, h[1] = a.y, h[2] = b.x, h[3] = b.y;
    } else if constexpr (VB <= 4) {
        const uint32_t f[4] = {bits_at<8 * VB * C, n>(w, kLog), bits_at<8 * VB * C + n, n>(w, kLog),
                               bits_at<8 * VB * C + 2 * n, n>(w, kLog), bits_at<8 * VB * C + 3 * n, n>(w, kLog)};
#pragma unroll
        for (int i = 0; i < 4; i++) h[i] = *reinterpret_cast<const uint32_t *>(table + (f[i] & mask));
    } else {
        const uint32_t f[8] = {bits_at<8 * VB * C, n>(w, kLog),          bits_at<8 * VB * C + n, n>(w, kLog),
                               bits_at<8 * VB * C + 2 * n, n>(w, kLog), bits_at<8 * VB * C + 3 * n, n>(w, kLog),
                               bits_at<8 * VB * C + 4 * n, n>(w, kLog), bits_at<8 * VB * C + 5 * n, n>(w, kLog),
                               bits_at<8 * VB * C + 6 * n, n>(w, kLog), bits_at<8 * VB * C + 7 * n, n>(w, kLog)};
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = *reinterpret_cast<const uint32_t *>(table + (f[i] & mask));
#pragma unroll
        for (int i = 0; i < 4; i++) h[i] = prmt(v[2 * i], v[2 * i + 1], 0x7610u);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// ---------------------------------------------------------------- tile descriptors
// What the loader tells the other roles about a tile.
struct TileDesc {
    int flags;     // kFirst.. | key bits << 8 | value bits << 16 | law << 20
    int left;      // tokens from the tile's first to the sequence's last in this segment
    int part;
    float inv;     // 1 / s of the value levels
    int b, h, seg, t;
    float A;       // of the query image
    int pad[7];
};
static_assert(sizeof(TileDesc) == 64, "slot size");
constexpr int kFirst = 1, kLast = 2;  // of its part
constexpr int kFresh = 4;             // first of its (group, segment)
constexpr int kFp16 = 8;
constexpr int kTurn = 16;             // the next tile is fresh

// ---------------------------------------------------------------- shared memory
template <int D, int R>
struct Mma {
    static constexpr int PC = 2 * R;                // columns of the P operand and of the sums: hi, lo
    static constexpr int NWG = R == 16 ? 2 : 4;     // softmax groups of four warps
    static constexpr int CW = R / NWG;              // rows per group
    static constexpr int kKeyWarp = 4 * NWG, kValueWarp = kKeyWarp + 4, kIssueWarp = kValueWarp + 8,
                         kLoadWarp = kIssueWarp + 2;
    static constexpr int kThreads = 32 * (kLoadWarp + 2);
    static constexpr int HALVES = D / 64;
    static constexpr int QPART = HALVES * R * 128;  // hi or lo of a block's queries
    static constexpr int QIMG = 2 * QPART + R * 32;  // hi, lo, and the 16-deep step that adds the rows' constants
    static constexpr int QBUF = (QIMG + 1023) / 1024 * 1024;
    static constexpr int VBUF = HALVES * 128 * 128;
    static constexpr int PLO = R == 64 ? 16384 : 0; // lo: lines of their own, or behind hi in the same ones
    static constexpr int PBUF = 128 * 128 + PLO;
    static constexpr int KCOLS = D / 2;             // TMEM columns of a K tile
    static constexpr int T_K = 0, T_S = 2 * KCOLS, T_O = T_S + 2 * R, T_C = T_O + PC;  // (T_C: 8 constant columns)
    static constexpr int TCOLS = 512;               // all of TMEM, so that its base is column 0
    static constexpr int O_Q = 0;
    static constexpr int O_V = O_Q + QBUF;
    static constexpr int O_P = O_V + 2 * VBUF;
    static constexpr int O_T = O_P + PBUF;
    static constexpr int O_S = O_T + 2 * kTableBytes;   // [kSlots][2][128] scales
    static constexpr int O_D = O_S + kSlots * 1024; // [kSlots] descriptors
    static constexpr int O_M = O_D + kSlots * 64;   // [R] m, [R] -m as used, [R] factors
    static constexpr int O_X = O_M + 3 * R * 4;     // [NWG][4][CW] maxima of the warps
    static constexpr int O_B = (O_X + NWG * 4 * CW * 4 + 15) / 16 * 16;
    static constexpr int kBars = 2 * 8 + 2 * 2 + 1 + 2 + 2 * kMaxStages + 2;
    static constexpr int O_RING = (O_B + kBars * 8 + 32 + 127) / 128 * 128;
    // the ring, and behind it the second buffer of queries where two tiles of records leave
    // room for one (1024: alignment)
    static constexpr int kRing = kSmemMax - 1024 - O_RING;
    static constexpr int O_Q2 = kSmemMax - 1024 - QBUF;
    static_assert(QBUF % 1024 == 0 && O_Q2 % 1024 == 0, "swizzled operands");
    static_assert(kRing >= 2 * 128 * (D / 8) * 16, "two tiles of the widest records");
};

template <int D, int R>
__host__ __device__ constexpr int tree_image_stride() {
    return (Mma<D, R>::QIMG + 16 + 127) / 128 * 128;
}

struct RingGeo {
    int stage, stages;
    int q_log;  // log2 of the query buffers
};

// The queries as the MMA's B operand, one image per (b, h, rb) and key width kb (0:
// fp16 keys, unrotated queries).  A CTA writes up to 32 rows of an image, a warp a row at a
// time, D / 32 neighbouring coordinates a lane.  A power of two 2^-e common to the block
// brings every rotated coordinate below 1: |(R q)_i| <= |q|_2 <= sqrt(d) max |q_i|.  (A
// row a thousand times smaller than the block's largest still has the precision of
// fp16, 22 bits being carried.)  The main kernel may start meanwhile: it waits for this grid
// before it touches the images.
constexpr int kPrepWarps = 8, kPrepRows = 32;
template <int D, int R>
__global__ void __launch_bounds__(32 * kPrepWarps) tree_queries_kernel(const __grid_constant__ TreeQueryParams p) {
    using C = Mma<D, R>;
    constexpr int EL = D / 32, ROWS = R < kPrepRows ? R : kPrepRows, SPLIT = R / ROWS;
    __shared__ unsigned red[kPrepWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.error = 0;
    asm volatile("griddepcontrol.launch_dependents;");
    const int part = blockIdx.x % SPLIT, img = blockIdx.x / SPLIT, v = img % p.n_var, group = img / p.n_var;
    const int bh = group / p.n_rb, rb = group - bh * p.n_rb, b = bh / p.H, h = bh - b * p.H, kb = p.var_bits[v][h];
    uint8_t *image = p.images + static_cast<size_t>(img) * tree_image_stride<D, R>();
    const bool vec = ((reinterpret_cast<uintptr_t>(p.q) | (p.qs[0] * 2) | (p.qs[1] * 2) | (p.qs[2] * 2)) & 7) == 0;
    auto load = [&](int r, uint32_t (&w)[EL / 2]) {
        const int row = rb * R + r;
        const uint16_t *src = p.q + b * p.qs[0] + (row / p.g) * p.qs[1] + (h * p.g + row % p.g) * p.qs[2] + EL * lane;
#pragma unroll
        for (int i = 0; i < EL / 2; i++) {
            w[i] = 0;
            if (row < p.rows)
                w[i] = vec ? __ldg(reinterpret_cast<const unsigned *>(src) + i)
                           : __ldg(src + 2 * i) | static_cast<uint32_t>(__ldg(src + 2 * i + 1)) << 16;
        }
    };
    int e = 0;
    if (kb) {
        unsigned mx = 0;  // fp16 bits of the block's largest finite |q_i|
#pragma unroll 4
        for (int r = warp; r < R; r += kPrepWarps) {
            uint32_t w[EL / 2];
            load(r, w);
#pragma unroll
            for (int i = 0; i < EL / 2; i++) {
                const unsigned x = w[i] & 0x7FFFu, y = (w[i] >> 16) & 0x7FFFu;
                mx = max(mx, max(x < 0x7C00u ? x : 0u, y < 0x7C00u ? y : 0u));
            }
        }
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) red[warp] = mx;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPrepWarps; i++) mx = max(mx, red[i]);
        const unsigned f = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(mx))));
        if (mx) e = static_cast<int>((f >> 23) & 0xFFu) - 126 + (D == 128 ? 4 : 3);
    }
    // x = m_t qk_scale (2^(1-b) sum code q + (2^-b - 1) sum q) = m_t A (U + c), U = 2^(-e - 11) sum code q,
    // c = 2^(-e - 11) (1/2 - 2^(b-1)) sum q
    if (part == 0 && threadIdx.x == 0)
        *reinterpret_cast<float *>(image + C::QIMG) = kb ? p.qk_scale * pow2(12 - kb + e) : p.qk_scale;
    const uint32_t neg = p.sign_bits[EL * lane >> 5] >> (EL * lane & 31);
    // coordinate 32 g + i + 16 u meets the code at place 32 g + 2 i + u, at bit s_i: times 2^(13 - s_i)
    const int u = (EL * lane >> 4) & 1, i0 = EL * lane & 15, g = EL * lane >> 5;
#pragma unroll 1
    for (int r = ROWS * part + warp; r < ROWS * (part + 1); r += kPrepWarps) {
        uint32_t w[EL / 2];
        load(r, w);
        // byte of the row at place k: line k / 64, 16-byte chunk (k % 64) / 8 permuted by the row
        auto place = [&](int k) {
            return image + (k >> 6) * R * 128 + r * 128 + ((((k & 63) >> 3) ^ (r & 7)) << 4) + (k & 7) * 2;
        };
        if (kb == 0) {
#pragma unroll
            for (int i = 0; i < EL / 2; i++) reinterpret_cast<uint32_t *>(place(EL * lane))[i] = w[i];
            continue;
        }
        float x[EL];
#pragma unroll
        for (int i = 0; i < EL / 2; i++) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
        // R q: signs, butterflies in the lane, across lanes, signs, scale
#pragma unroll
        for (int i = 0; i < EL; i++)
            if ((neg >> i) & 1u) x[i] = -x[i];
#pragma unroll
        for (int s = 1; s < EL; s <<= 1)
#pragma unroll
            for (int i = 0; i < EL; i++)
                if (!(i & s)) {
                    const float y = x[i], z = x[i + s];
                    x[i] = y + z, x[i + s] = y - z;
                }
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const float sg = (lane & s) ? -1.f : 1.f;
#pragma unroll
            for (int i = 0; i < EL; i++) x[i] = fmaf(x[i], sg, __shfl_xor_sync(0xffffffffu, x[i], s));
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < EL; i++) {
            x[i] *= ((neg >> i) & 1u) ? -p.inv_sqrt_d : p.inv_sqrt_d;
            sum += x[i];
        }
#pragma unroll
        for (int s = 16; s >= 1; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        // the row's constant, met by 2^-11 twice (hi, lo): 8 rows of 16 bytes per k half
        if (lane == 0) {
            const float y = sum * pow2(-e) * (0.5f - pow2(kb - 1));
            const __half hi = __float2half_rn(y), lo = __float2half_rn(y - __half2float(hi));
            uint8_t *at = image + 2 * C::QPART + (r >> 3) * 256 + (r & 7) * 16;
            *reinterpret_cast<uint4 *>(at) = make_uint4(
                static_cast<uint32_t>(__half_as_ushort(hi)) | static_cast<uint32_t>(__half_as_ushort(lo)) << 16, 0, 0, 0);
            *reinterpret_cast<uint4 *>(at + 128) = make_uint4(0, 0, 0, 0);
        }
        uint32_t hl[EL];  // hi, lo
#pragma unroll
        for (int i = 0; i < EL; i++) {
            const int pos = (kb * (i0 + i)) & 15, o = pos + kb <= 10 ? pos : pos >= 8 ? pos - 8 : pos;
            const float y = x[i] * pow2(13 - e - min(o, 10 - kb));
            const __half hi = __float2half_rn(y), lo = __float2half_rn(y - __half2float(hi));
            hl[i] = static_cast<uint32_t>(__half_as_ushort(hi)) | static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
        }
        // the pair of lanes (u = 0, 1) shares its places: lane u takes the u-th half of the coordinates i
#pragma unroll
        for (int i = 0; i < EL / 2; i++) {
            const uint32_t own = u ? hl[EL / 2 + i] : hl[i];
            const uint32_t other = __shfl_xor_sync(0xffffffffu, u ? hl[i] : hl[EL / 2 + i], 16 / EL);
            uint8_t *at = place(32 * g + 2 * (i0 + u * (EL / 2) + i));
            *reinterpret_cast<uint32_t *>(at) = u ? prmt(other, own, 0x5410u) : prmt(own, other, 0x5410u);
            *reinterpret_cast<uint32_t *>(at + C::QPART) = u ? prmt(other, own, 0x7632u) : prmt(own, other, 0x7632u);
        }
    }
}

// State of a key or value warp's walk through the ring.
struct RingPos {
    int j, st;      // tile, ring stage
    unsigned par;   // parity of the stage's fill
    __device__ __forceinline__ void next(int stages) {
        j++;
        if (++st == stages) st = 0, par ^= 1;
    }
};
// Shared-memory addresses that the key and value warps need.
struct RoleBars {
    unsigned r_full, r_empty, full, empty;  // of buffer / stage 0; the next 8 bytes further
};

// Keys of KB bits from the ring into TMEM, one token a thread, while the tiles have that width.
template <int KB, int D>
__device__ __forceinline__ void keys_loop(RingPos &q, int n_tiles, const RingGeo &ring, unsigned ring_base, const uint8_t *descs,
                                          const RoleBars &bar, unsigned dst, int token, Waiter &wait) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (; q.j < n_tiles; q.next(ring.stages)) {
        const int b = q.j & 1;
        const bool here = bar_test(bar.r_full + 8 * q.st, q.par), free = bar_test(bar.empty + 8 * b, ((q.j >> 1) & 1) ^ 1);
        wait.unless(here, bar.r_full + 8 * q.st, q.par);
        if (wait.gone) return;
        if (((reinterpret_cast<const TileDesc *>(descs)[q.j % kSlots].flags >> 8) & 15) != KB) return;
        uint32_t w[D / 32 * KB];
        load_record<D / 32 * KB>(ring_base + q.st * ring.stage, token, w);
        __syncwarp();
        if (lane == 0) bar_arrive(bar.r_empty + 8 * q.st);
        wait.unless(free, bar.empty + 8 * b, ((q.j >> 1) & 1) ^ 1);
        if (wait.gone) return;
        tc_after();
        // (a loop that shifts the record down: a quarter of the code, which the instruction caches feel)
#pragma unroll 1
        for (int g = 0; g < D / 32; g++) {
            uint32_t out[16];
            key_words<KB>(w, out);
            tmem_st16(dst + b * (D / 2) + 16 * g, out);
#pragma unroll
            for (int i = 0; i + KB < D / 32 * KB; i++) w[i] = w[i + KB];
        }
        tmem_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bar.full + 8 * b);
    }
}

// Values of VB bits from the ring to fp16 rows, one token a thread, while the tiles have
// that width (and law).  Two groups of four warps take alternate tiles, each with its buffer.
template <int VB, int D>
__device__ __forceinline__ void values_loop(RingPos &q, int n_tiles, const RingGeo &ring, unsigned ring_base, const uint8_t *descs,
                                            const RoleBars &bar, const uint8_t *table, uint8_t *dst, int token,
                                            int width, Waiter &wait) {
    const int lane = threadIdx.x & 31;
    table += (token & (level_columns(VB) - 1)) * level_bytes(VB);
    dst += token * 128;
#pragma unroll 1
    for (; q.j < n_tiles; q.next(ring.stages), q.next(ring.stages)) {
        const unsigned par = ((q.j >> 1) & 1) ^ 1;
        const bool here = bar_test(bar.r_full + 8 * q.st, q.par), free = bar_test(bar.empty, par);
        wait.unless(here, bar.r_full + 8 * q.st, q.par);
        if (wait.gone) return;
        const int flags = reinterpret_cast<const TileDesc *>(descs)[q.j % kSlots].flags;
        if (flags >> 16 != width) return;
        uint32_t w[D / 32 * VB];
        load_record<D / 32 * VB>(ring_base + q.st * ring.stage + kTreeTile * (D / 8) * ((flags >> 8) & 15), token, w);
        __syncwarp();
        if (lane == 0) bar_arrive(bar.r_empty + 8 * q.st);
        wait.unless(free, bar.empty, par);
        if (wait.gone) return;
#pragma unroll 1
        for (int g = 0; g < D / 32; g++) {  // 32 dims: four chunks of the line
            uint8_t *line = dst + (g >> 1) * 16384;
            const int c0 = 4 * (g & 1);
            *reinterpret_cast<uint4 *>(line + ((c0 ^ (token & 7)) << 4)) = level_chunk<VB, 0>(w, table);
            *reinterpret_cast<uint4 *>(line + (((c0 + 1) ^ (token & 7)) << 4)) = level_chunk<VB, 1>(w, table);
            *reinterpret_cast<uint4 *>(line + (((c0 + 2) ^ (token & 7)) << 4)) = level_chunk<VB, 2>(w, table);
            *reinterpret_cast<uint4 *>(line + (((c0 + 3) ^ (token & 7)) << 4)) = level_chunk<VB, 3>(w, table);
#pragma unroll
            for (int i = 0; i + VB < D / 32 * VB; i++) w[i] = w[i + VB];
        }
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(bar.full);
    }
}

// Fill the value table of a width (the four warps of a group together).
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
__global__ void __launch_bounds__(Mma<D, R>::kThreads, 1)
    tree_mma_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeLevels lv, const RingGeo ring) {
    using C = Mma<D, R>;
    constexpr int CW = C::CW, kKeyWarp = C::kKeyWarp, kValueWarp = C::kValueWarp, kIssueWarp = C::kIssueWarp,
                  kLoadWarp = C::kLoadWarp;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
    const unsigned sb = su32(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned bars = sb + C::O_B;
    auto k_full = [&](int i) { return bars + 8u * i; };
    auto k_empty = [&](int i) { return bars + 8u * (2 + i); };
    auto v_full = [&](int i) { return bars + 8u * (4 + i); };
    auto v_empty = [&](int i) { return bars + 8u * (6 + i); };
    auto s_full = [&](int i) { return bars + 8u * (8 + i); };
    auto s_empty = [&](int i) { return bars + 8u * (10 + i); };
    const unsigned p_full = bars + 8u * 12, p_empty = bars + 8u * 14;
    // image `ev` of this worker: its buffer, and the parity of the buffer's fill with it
    auto q_buf = [&](int ev) { return ev & ring.q_log; };
    auto q_par = [&](int ev) { return static_cast<unsigned>(ev >> ring.q_log) & 1u; };
    auto q_at = [&](int ev) { return sb + (q_buf(ev) ? C::O_Q2 : C::O_Q); };
    auto q_full = [&](int ev) { return bars + 8u * (16 + q_buf(ev)); };
    auto q_empty = [&](int ev) { return bars + 8u * (18 + q_buf(ev)); };
    const unsigned o_free = bars + 8u * 20;
    auto drain = [&](int i) { return bars + 8u * (21 + i); };
    auto r_full = [&](int i) { return bars + 8u * (23 + i); };
    auto r_empty = [&](int i) { return bars + 8u * (23 + kMaxStages + i); };
    auto t_sync = [&](int i) { return bars + 8u * (23 + 2 * kMaxStages + i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::O_B + C::kBars * 8);

    asm volatile("griddepcontrol.launch_dependents;");  // (the merge waits for this grid's end)
    const unsigned T = total_tiles(p), per = worker_tiles(p, T), worker = blockIdx.x, at0 = worker * per;
    if (at0 >= T) {
        asm volatile("griddepcontrol.wait;" ::: "memory");  // no CTA ends before the grid that it depends on
        return;
    }
    const int n_tiles = static_cast<int>(min(per, T - at0));

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; i++) {
            bar_init(k_full(i), 4);
            bar_init(k_empty(i), 1);
            bar_init(v_full(i), 4);
            bar_init(v_empty(i), 1);
            bar_init(s_full(i), 1);
            bar_init(s_empty(i), 4 * C::NWG);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(q_full(i), 1);
            bar_init(q_empty(i), 1);
        }
        for (int i = 0; i < 2; i++) bar_init(t_sync(i), 4);
        for (int i = 0; i < 4; i++) tmem_slot[1 + i] = 0;  // a softmax group that gave up
        bar_init(p_full, 4 * C::NWG);
        bar_init(p_empty, 1);
        bar_init(o_free, 4 * C::NWG);
        bar_init(drain(0), 1);
        bar_init(drain(1), 1);
        for (int i = 0; i < kMaxStages; i++) {
            bar_init(r_full(i), 65);
            bar_init(r_empty(i), 8);  // four key warps, the four value warps of the tile
        }
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
    constexpr unsigned tbase = 0;
    Waiter wait{p.error, p.wait_polls, false};

    if (warp >= kLoadWarp) {
        // ------------------------------------------------------ records and scales: keys, values
        const int kv = warp - kLoadWarp;
        const uint8_t *src = nullptr;
        const float *scale = nullptr;
        int rec = 0, off = 0, st = 0, kind = 0, ev = -1, issued = -1;
        float inv = 1.f, A = 1.f;
        Walk w = walk_begin(p, at0);
        if (kv == 0) asm volatile("griddepcontrol.wait;" ::: "memory");  // the query images
        for (int j = 0; j < n_tiles; j++) {
            if (w.fresh) {
                const SegView &s = p.seg[w.seg].seg;
                rec = 0;
                kind = kFp16;
                inv = 1.f;
                if (!s.fp16) {
                    const int kb = s.kbits[w.x.h], vb = s.vbits[w.x.h];
                    kind = kb << 8 | vb << 16 | p.seg[w.seg].law << 20;
                    inv = lv.inv[p.seg[w.seg].law][vb];
                    rec = D / 8 * (kv ? vb : kb);
                    off = C::O_RING + (kv ? kTreeTile * (D / 8) * kb : 0);
                    src = (kv ? s.v + w.x.b * s.vblock + s.voff[w.x.h] : s.k + w.x.b * s.kblock + s.koff[w.x.h]) + 16 * lane;
                    scale = (kv ? s.vs : s.ks) + (static_cast<size_t>(w.x.b) * p.H + w.x.h) * s.capacity + 4 * lane;
                }
            }
            if (w.fresh && kv == 0) {
                // the queries for this segment's key width, into the buffer that they are done with first
                ev++;
                const uint8_t *image = p.images + (static_cast<size_t>(group_of(p, w.x)) * p.n_var + p.var[w.seg][w.x.h]) *
                                                      tree_image_stride<D, R>();
                wait(q_empty(ev), q_par(ev) ^ 1);
                if (wait.gone) break;
                if (lane == 0) {
                    issued = ev;
                    bar_expect_tx(q_full(ev), C::QIMG);
                    bulk_load(q_at(ev), image, C::QIMG, q_full(ev));
                }
                A = __ldcg(reinterpret_cast<const float *>(image + C::QIMG));
            }
            TileDesc d;
            d.A = A;
            d.left = w.n - w.t * kTreeTile;
            d.part = w.part;
            d.inv = inv;
            d.b = w.x.b, d.h = w.x.h, d.seg = w.seg, d.t = w.t;
            d.flags = kind | (w.first ? kFirst : 0) | (w.fresh || j == 0 ? kFresh : 0);
            const int n = min(kTreeTile, d.left), chunks = (n * rec + 15) / 16;
            const uint8_t *from = src + static_cast<size_t>(w.t) * (kTreeTile * rec);
            const float *sc = scale + static_cast<size_t>(w.t) * kTreeTile;
            if (j + 1 < n_tiles) {
                walk_next(p, w);
                if (w.fresh) d.flags |= kTurn;
            }
            if (j + 1 == n_tiles || w.first) d.flags |= kLast;
            wait(r_empty(st), ((j / ring.stages) & 1) ^ 1);
            if (wait.gone) break;
            if (kv == 0 && lane == 0) {
                TileDesc *to = reinterpret_cast<TileDesc *>(sm + C::O_D) + j % kSlots;
                to->flags = d.flags, to->left = d.left, to->part = d.part, to->inv = d.inv;
                to->b = d.b, to->h = d.h, to->seg = d.seg, to->t = d.t, to->A = d.A;
                bar_arrive(r_full(st));
            }
            // chunk c = lane + 32 i goes to c ^ ((c >> 3) & m): the same for every i but m = 7's third bit
            const unsigned dst = sb + off + st * ring.stage;
            const int m = chunk_mask(rec);
            const unsigned to = dst + 16 * (lane ^ ((lane >> 3) & m));
            const unsigned to2 = m == 7 ? dst + 16 * (lane ^ (((lane + 32) >> 3) & 7)) : to;
            if (rec && 4 * lane < n) cp16(sb + C::O_S + (j % kSlots) * 1024 + kv * 512 + 16 * lane, sc);
#pragma unroll 4
            for (int i = 0; 32 * i + lane < chunks; i++) cp16(((i & 1) ? to2 : to) + 512 * i, from + 512 * i);
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(r_full(st)) : "memory");
            if (++st == ring.stages) st = 0;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        // the last query images have landed before shared memory goes away
        if (kv == 0 && lane == 0)
            for (int e = max(issued - ring.q_log, 0); e <= issued; e++)
                for (int i = 0; i < kDrainPolls; i++)
                    if (bar_try(q_full(e), q_par(e))) break;
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------------ S^T = K q^T
        constexpr uint32_t id_s = idesc(R, false);
        int ev = -1;
#pragma unroll 1
        for (int j = 0; j < n_tiles; j++) {
            const int b = j & 1;
            const unsigned par = (j >> 1) & 1;
            wait.both(k_full(b), par, s_empty(b), par ^ 1);
            if (wait.gone) break;
            const int flags = reinterpret_cast<const TileDesc *>(sm + C::O_D)[j % kSlots].flags;
            if (flags & kFresh) {
                ev++;
                wait(q_full(ev), q_par(ev));
                if (wait.gone) break;
            }
            tc_after();
            const uint64_t q = desc_k(q_at(ev));
            const unsigned a = C::T_K + b * C::KCOLS, d = C::T_S + b * R;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; k++)
                    mma_ts(d, a + 8 * k, q + (((k >> 2) * R * 128 + 32 * (k & 3)) >> 4), id_s, k != 0);
                if (!(flags & kFp16)) {  // (fp16 queries are exact: no lo part)
#pragma unroll
                    for (int k = 0; k < D / 16; k++)
                        mma_ts(d, a + 8 * k, q + ((C::QPART + (k >> 2) * R * 128 + 32 * (k & 3)) >> 4), id_s, 1);
                    mma_ts(d, C::T_C, desc_k16(q_at(ev) + 2 * C::QPART), id_s, 1);
                }
                mma_commit(k_empty(b));
                mma_commit(s_full(b));
                if (flags & kTurn) mma_commit(q_empty(ev));  // the last product with these queries
            }
            __syncwarp();
        }
        // what was issued has completed before TMEM and shared memory go away
        if (elect_one()) mma_commit(drain(0));
        __syncwarp();
        for (int i = 0; i < kDrainPolls; i++)
            if (bar_try(drain(0), 0)) break;
    } else if (warp == kIssueWarp + 1) {
        // ------------------------------------------------------ O^T += V^T P^T
        constexpr uint32_t id_o = idesc(C::PC, true);
        int parts = 0;
#pragma unroll 1
        for (int j = 0; j < n_tiles; j++) {
            const int b = j & 1;
            wait.both(v_full(b), (j >> 1) & 1, p_full, j & 1);
            if (wait.gone) break;
            const bool first = reinterpret_cast<const TileDesc *>(sm + C::O_D)[j % kSlots].flags & kFirst;
            if (first) {
                if (parts > 0) wait(o_free, (parts - 1) & 1);
                if (wait.gone) break;
                parts++;
            }
            tc_after();
            const uint64_t v = desc_mn(sb + C::O_V + b * C::VBUF, C::HALVES == 2 ? 16384 : 0),
                           pp = desc_mn(sb + C::O_P, C::PLO);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; k++) mma_ss(C::T_O, v + (2048 * k >> 4), pp + (2048 * k >> 4), id_o, k != 0 || !first);
                mma_commit(v_empty(b));
                mma_commit(p_empty);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(drain(1));
        __syncwarp();
        for (int i = 0; i < kDrainPolls; i++)
            if (bar_try(drain(1), 0)) break;
    } else if (warp >= kValueWarp) {
        // ------------------------------------------------------ values into shared memory
        const int vg = (warp - kValueWarp) >> 2, tid = threadIdx.x - (kValueWarp + 4 * vg) * 32;
        const RoleBars bar{r_full(0), r_empty(0), v_full(vg), v_empty(vg)};
        const uint8_t *descs = sm + C::O_D, *table = sm + C::O_T + vg * kTableBytes;
        const unsigned base = sb + C::O_RING;
        uint8_t *dst = sm + C::O_V + vg * C::VBUF;
        RingPos q{0, 0, 0};
        if (vg) q.next(ring.stages);
        unsigned met = 0;  // (bounded, as a group's warps may give up one by one)
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) bar_arrive(t_sync(vg));
            wait(t_sync(vg), met);
            met ^= 1;
        };
        while (q.j < n_tiles) {
            wait(r_full(q.st), q.par);
            if (wait.gone) break;
            const TileDesc &d = reinterpret_cast<const TileDesc *>(descs)[q.j % kSlots];
            const int width = d.flags >> 16, vb = width & 15;
            if (vb) {
                const uint16_t *half = param_table(lv.half[width >> 4] + cb_off(vb));
                meet();  // the other warps have done with the old table
                if (wait.gone) break;
                fill_levels(sm + C::O_T + vg * kTableBytes, half, vb, tid);
                meet();
                if (wait.gone) break;
            }
            switch (vb) {
                case 0: {
                    const SegView &s = p.seg[d.seg].seg;
                    const uint4 *src = reinterpret_cast<const uint4 *>(s.v + d.b * s.vblock + s.voff[d.h]) +
                                       static_cast<size_t>(d.t) * (kTreeTile * D / 8);
                    const int n = d.left;
                    __syncwarp();
                    if (lane == 0) bar_arrive(r_empty(q.st));
                    wait(v_empty(vg), ((q.j >> 1) & 1) ^ 1);
                    if (wait.gone) break;
                    // 16-byte chunks, consecutive threads on consecutive ones; rows behind the tokens are zeros
#pragma unroll 4
                    for (int c = tid; c < kTreeTile * D / 8; c += 128) {
                        const int t = c / (D / 8), e = c % (D / 8);
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (t < n) v = __ldg(src + c);
                        *reinterpret_cast<uint4 *>(dst + (e >> 3) * 16384 + t * 128 + (((e & 7) ^ (t & 7)) << 4)) = v;
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) bar_arrive(v_full(vg));
                    q.next(ring.stages);
                    q.next(ring.stages);
                    break;
                }
                case 1: values_loop<1, D>(q, n_tiles, ring, base, descs, bar, table, dst, tid, width, wait); break;
                case 2: values_loop<2, D>(q, n_tiles, ring, base, descs, bar, table, dst, tid, width, wait); break;
                case 3: values_loop<3, D>(q, n_tiles, ring, base, descs, bar, table, dst, tid, width, wait); break;
                case 4: values_loop<4, D>(q, n_tiles, ring, base, descs, bar, table, dst, tid, width, wait); break;
                case 5: values_loop<5, D>(q, n_tiles, ring, base, descs, bar, table, dst, tid, width, wait); break;
                case 6: values_loop<6, D>(q, n_tiles, ring, base, descs, bar, table, dst, tid, width, wait); break;
                case 7: values_loop<7, D>(q, n_tiles, ring, base, descs, bar, table, dst, tid, width, wait); break;
                default: values_loop<8, D>(q, n_tiles, ring, base, descs, bar, table, dst, tid, width, wait); break;
            }
            if (wait.gone) break;
        }
    } else if (warp >= kKeyWarp) {
        // ------------------------------------------------------ keys into TMEM
        const int kw = warp - kKeyWarp, tid = threadIdx.x - kKeyWarp * 32;
        const unsigned lanes = static_cast<unsigned>(32 * kw) << 16;
        const RoleBars bar{r_full(0), r_empty(0), k_full(0), k_empty(0)};
        const uint8_t *descs = sm + C::O_D;
        const unsigned base = sb + C::O_RING, dst = tbase + lanes + C::T_K;
        {
            const uint32_t c[8] = {0x10001000u, 0, 0, 0, 0, 0, 0, 0};  // 2^-11 twice, zeros
            tmem_st8(tbase + lanes + C::T_C, c);
        }
        RingPos q{0, 0, 0};
        while (q.j < n_tiles) {
            wait(r_full(q.st), q.par);
            if (wait.gone) break;
            const TileDesc &d = reinterpret_cast<const TileDesc *>(descs)[q.j % kSlots];
            switch ((d.flags >> 8) & 15) {
                case 0: {
                    const int b = q.j & 1;
                    const SegView &s = p.seg[d.seg].seg;
                    const uint4 *src = reinterpret_cast<const uint4 *>(s.k + d.b * s.kblock + s.koff[d.h]) +
                                       (static_cast<size_t>(d.t) * kTreeTile + tid) * (D / 8);
                    const bool valid = tid < d.left;
                    __syncwarp();
                    if (lane == 0) bar_arrive(r_empty(q.st));
                    wait(k_empty(b), ((q.j >> 1) & 1) ^ 1);
                    if (wait.gone) break;
                    tc_after();
#pragma unroll
                    for (int i = 0; i < D / 32; i++) {
                        uint32_t out[16];
#pragma unroll
                        for (int c = 0; c < 4; c++) {
                            uint4 v = make_uint4(0, 0, 0, 0);
                            if (valid) v = __ldg(src + 4 * i + c);
                            out[4 * c] = v.x, out[4 * c + 1] = v.y, out[4 * c + 2] = v.z, out[4 * c + 3] = v.w;
                        }
                        tmem_st16(dst + b * C::KCOLS + 16 * i, out);
                    }
                    tmem_wait_st();
                    tc_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(k_full(b));
                    q.next(ring.stages);
                    break;
                }
                case 1: keys_loop<1, D>(q, n_tiles, ring, base, descs, bar, dst, tid, wait); break;
                case 2: keys_loop<2, D>(q, n_tiles, ring, base, descs, bar, dst, tid, wait); break;
                case 3: keys_loop<3, D>(q, n_tiles, ring, base, descs, bar, dst, tid, wait); break;
                case 4: keys_loop<4, D>(q, n_tiles, ring, base, descs, bar, dst, tid, wait); break;
                case 5: keys_loop<5, D>(q, n_tiles, ring, base, descs, bar, dst, tid, wait); break;
                case 6: keys_loop<6, D>(q, n_tiles, ring, base, descs, bar, dst, tid, wait); break;
                case 7: keys_loop<7, D>(q, n_tiles, ring, base, descs, bar, dst, tid, wait); break;
                default: keys_loop<8, D>(q, n_tiles, ring, base, descs, bar, dst, tid, wait); break;
            }
            if (wait.gone) break;
        }
    } else {
        // ------------------------------------------------------ softmax
        const int wg = warp >> 2, qw = warp & 3, tok = 32 * qw + lane;  // TMEM lane = token (or dim of O)
        const unsigned lanes = static_cast<unsigned>(32 * qw) << 16;
        // [CW] m; + R: -m as used (0 while nothing was seen); + 2R: factors
        float *m_row = reinterpret_cast<float *>(sm + C::O_M) + wg * CW;
        float *maxima = reinterpret_cast<float *>(sm + C::O_X) + wg * 4 * CW;
        const unsigned s_addr0 = tbase + lanes + C::T_S + wg * CW, o_addr = tbase + lanes + C::T_O + wg * CW;
        uint8_t *prow = sm + C::O_P + tok * 128;
        float l[CW], A = 1.f;
#pragma unroll
        for (int c = 0; c < CW; c++) l[c] = 0.f;
        if (tok < CW) m_row[R + tok] = 0.f;
        named_sync(1 + wg, 128);
        bool ready = false, lost = false;
        // a group leaves together: a warp that gave up asks for a raise (every warp votes
        // on one per tile, whatever it read), where all four learn of it
        volatile uint32_t *left = tmem_slot + 1 + wg;
#pragma unroll 1
        for (int j = 0; j < n_tiles; j++) {
            const int b = j & 1;
            wait.unless(ready, s_full(b), (j >> 1) & 1);
            tc_after();
            float u[CW];
            tmem_issue<CW>(s_addr0 + b * R, u);
            const TileDesc *desc = reinterpret_cast<const TileDesc *>(sm + C::O_D) + j % kSlots;
            const int4 d = *reinterpret_cast<const int4 *>(desc);  // flags, left, part, inv
            if (d.x & kFresh) A = desc->A;
            // the token's scales (behind the last token: anything)
            const float *sc = reinterpret_cast<const float *>(sm + C::O_S) + (j % kSlots) * 256 + tok;
            const bool valid = tok < d.y;
            float ks = A, sig = 1.f, e = 0.f;  // x = ks U; 2^e <= sig < 2^(e + 1)
            if (!(d.x & kFp16)) {
                ks = sc[0] * A;
                sig = sc[128] * __int_as_float(d.w);
                e = static_cast<float>(max(-64, min(64, static_cast<int>((__float_as_uint(sig) >> 23) & 0xFFu) - 127)));
            }
            if (!valid) ks = sig = 0.f;
            bool raise = (d.x & kFirst) || wait.gone;
            tmem_wait<CW>(u);
#pragma unroll 1
            for (int pass = 0;; pass++) {
                // x - m, and whether some weight outgrew its row's m
                float top = -kInf;
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    const float4 m = *reinterpret_cast<const float4 *>(m_row + R + c);
                    const float2 u0 = ffma2(make_float2(u[c], u[c + 1]), ks, make_float2(m.x, m.y));
                    const float2 u1 = ffma2(make_float2(u[c + 2], u[c + 3]), ks, make_float2(m.z, m.w));
                    u[c] = u0.x, u[c + 1] = u0.y, u[c + 2] = u1.x, u[c + 3] = u1.y;
                    top = fmax3(top, u[c], u[c + 1]);
                    top = fmax3(top, u[c + 2], u[c + 3]);
                }
                raise |= valid && top + e > 8.0f;
                if (pass || !named_or(1 + wg, 128, raise)) break;
                float mine = -kInf;
#pragma unroll
                for (int c = 0; c < CW; c++) {
                    float v = valid ? u[c] + e : -kInf;
                    asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
                    if (lane == c) mine = v;
                }
                if (lane < CW) maxima[qw * CW + lane] = mine;
                if (lane == 0 && wait.gone) *left = 1;
                named_sync(1 + wg, 128);
                lost = *left != 0;
                if (lost) break;
                const bool first = d.x & kFirst;
                if (tok < CW) {
                    const float old = first ? -kInf : m_row[tok];
                    float m = maxima[tok];
#pragma unroll
                    for (int i = 1; i < 4; i++) m = fmaxf(m, maxima[i * CW + tok]);
                    m = fmaxf(old, m - m_row[R + tok]);
                    m_row[tok] = m;
                    m_row[R + tok] = m == -kInf ? 0.f : -m;
                    m_row[2 * R + tok] = old == -kInf ? 0.f : ex2(old - m);
                }
                named_sync(1 + wg, 128);
                if (!first) {
                    // earlier weights to the new max: the sums here, the accumulator in TMEM
                    wait(p_empty, (j - 1) & 1);
                    tc_after();
#pragma unroll
                    for (int c = 0; c < CW; c += 8) {
#pragma unroll
                        for (int x = 0; x < C::PC; x += R) {
                            float o[8];
                            uint32_t r[8];
                            tmem_ld<8>(o_addr + x + c, o);
#pragma unroll
                            for (int i = 0; i < 8; i++) {
                                const float f = m_row[2 * R + c + i];
                                if (x == 0) l[c + i] *= f;
                                r[i] = __float_as_uint(o[i] * f);
                            }
                            tmem_st8(o_addr + x + c, r);
                        }
                    }
                    tmem_wait_st();
                }
                tmem_ld<CW>(s_addr0 + b * R, u);
            }
            if (lost) break;
            tc_before();
            __syncwarp();
            if (lane == 0 && !wait.gone) bar_arrive(s_empty(b));
            const bool p_free = bar_test(p_empty, (j & 1) ^ 1);  // the products with the last P done?
            if (__any_sync(0xffffffffu, !valid)) {  // behind the last token: weight zero, whatever lies there
#pragma unroll
                for (int c = 0; c < CW; c++) u[c] = valid ? u[c] : -kInf;
            }
            uint32_t h[CW / 2], lo[CW / 2];  // hi and 2^11 (w - hi), so that weights down to 2^-36 count
#pragma unroll
            for (int c = 0; c < CW; c += 2) {
                const float2 pr = make_float2(ex2(u[c]), ex2(u[c + 1]));
                const float2 ls = fadd2(make_float2(l[c], l[c + 1]), pr);
                l[c] = ls.x, l[c + 1] = ls.y;
                const float2 w = fmul2(pr, sig);
                const __half2 q = __floats2half2_rn(w.x, w.y);
                h[c / 2] = *reinterpret_cast<const uint32_t *>(&q);
                const float2 left = ffma2(__half22float2(q), -2048.f, fmul2(w, 2048.f));  // (exact)
                const __half2 r = __floats2half2_rn(left.x, left.y);
                lo[c / 2] = *reinterpret_cast<const uint32_t *>(&r);
            }
            wait.unless(p_free, p_empty, (j & 1) ^ 1);
#pragma unroll
            for (int c = 0; c < CW; c += 8)
                *reinterpret_cast<uint4 *>(prow + ((((wg * CW + c) >> 3) ^ (tok & 7)) << 4)) =
                    make_uint4(h[c / 2], h[c / 2 + 1], h[c / 2 + 2], h[c / 2 + 3]);
#pragma unroll
            for (int c = 0; c < CW; c += 8)
                *reinterpret_cast<uint4 *>(prow + C::PLO + (((((C::PLO ? 0 : R) + wg * CW + c) >> 3) ^ (tok & 7)) << 4)) =
                    make_uint4(lo[c / 2], lo[c / 2 + 1], lo[c / 2 + 2], lo[c / 2 + 3]);
            fence_async();
            tc_before();
            __syncwarp();
            if (lane == 0 && !wait.gone) bar_arrive(p_full);
            ready = j + 1 < n_tiles && bar_test(s_full(b ^ 1), ((j + 1) >> 1) & 1);
            if (d.x & kLast) {  // the part's record
                float *rec = p.part + (static_cast<size_t>(worker) + d.z) * R * (D + 4);
                // row sums over the tokens
#pragma unroll
                for (int c = 0; c < CW; c++) {
                    float v = l[c];
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    if (lane == 0) maxima[qw * CW + c] = v;
                    l[c] = 0.f;
                }
                named_sync(1 + wg, 128);
                if (tok < CW) {
                    float *row = rec + (wg * CW + tok) * (D + 4);
                    row[0] = m_row[tok];
                    row[1] = (maxima[tok] + maxima[CW + tok]) + (maxima[2 * CW + tok] + maxima[3 * CW + tok]);
                    m_row[R + tok] = 0.f;
                }
                wait(p_empty, j & 1);
                tc_after();
#pragma unroll
                for (int c = 0; c < CW; c += 8) {
                    float o[8], y[8];
                    tmem_ld<8>(o_addr + c, o);
                    tmem_ld<8>(o_addr + R + c, y);
#pragma unroll
                    for (int i = 0; i < 8; i++)  // (an infinite value: hi's sum tells its sign, lo may be 0 or negative)
                        o[i] = fabsf(o[i]) == kInf ? o[i] : fmaf(y[i], 1.f / 2048.f, o[i]);
                    if (tok < D)
#pragma unroll
                        for (int i = 0; i < 8; i++) rec[(wg * CW + c + i) * (D + 4) + 4 + tok] = o[i];
                }
                tc_before();
                named_sync(1 + wg, 128);  // (also: `maxima` is free again, -m is 0 for all)
                if (lane == 0 && !wait.gone) bar_arrive(o_free);
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
// N(0, 1) weighs their cells, are smallest of 4096 candidates (relative to the levels, all
// alike: 2e-8 at 1 bit, 2e-5 at 3, 9e-5 at 5, 1.7e-4 at 8; s = 1 at 8: 2.3e-4).
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
    double mass[128];
    for (int k = n / 2; k < n; k++) {
        const double a = k == n / 2 ? 0.0 : 0.5 * (static_cast<double>(c[k - 1]) + c[k]);
        const double b = k + 1 == n ? 1e9 : 0.5 * (static_cast<double>(c[k]) + c[k + 1]);
        mass[k - n / 2] = std::erfc(a * 0.70710678118654752) - std::erfc(b * 0.70710678118654752);
    }
    for (int i = 0; i < 4096; i++) {
        const float s = 1.f + static_cast<float>(i) / 4096.f;
        double err = 0.0;
        for (int k = n / 2; k < n; k++) {
            const double d = static_cast<double>(__half2float(__float2half_rn(s * c[k]))) / s - c[k];
            err += mass[k - n / 2] * d * d;
        }
        if (err < best) best = err, s_best = s;
    }
    for (int k = 0; k < n; k++) h.half[k] = __half_as_ushort(__float2half_rn(s_best * c[k]));
    h.inv = 1.f / s_best;
}

template <int D, int R>
cudaError_t tree_mma(const TreeParams &p, const TreeLevels &lv, cudaStream_t s) {
    using C = Mma<D, R>;
    static_assert(C::T_C + 8 <= 512, "TMEM columns");
    int stage = 0;
    for (int i = 0; i < p.n_packed; i++)
        for (int h = 0; h < p.H; h++) stage = std::max(stage, 128 * (D / 8) * (p.seg[i].seg.kbits[h] + p.seg[i].seg.vbits[h]));
    RingGeo ring;
    ring.stage = std::max(stage, 128);
    // A second buffer of queries, so that a segment's first tile does not wait for them, where
    // the ring keeps two stages.  (64 rows of head_dim 128: up to 8 bits of key and value.  One
    // buffer everywhere: 13 drafts over 16 x 9K at head_dim 64 92 us for 85.  Wider records: 32
    // sequences of 512 tokens, 64 rows, K5V4 92 us, in blocks of 64 rows with two buffers
    // and one-fp16 weights 89; K8V8 99, in blocks of 32 rows 116.)
    ring.q_log = (C::kRing - C::QBUF) / ring.stage >= 2 ? 1 : 0;
    ring.stages = std::min(kMaxStages, (C::kRing - ring.q_log * C::QBUF) / ring.stage);
    // Two stages at least: the groups of value warps take alternate tiles, and a wait for a stage's
    // fill is by parity, right for the fill behind the last one that the waiter knows of.
    // (A group that has seen tile j filled knows that tile j - 1 was: fills end in order.  So
    // the fill before its next tile's is known, unless one stage holds both.)
    if (ring.stages < 2) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(tree_mma_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    const int images = p.B * p.H * p.n_rb * p.n_var;
    TreeQueryParams qp;
    qp.H = p.H, qp.g = p.g, qp.n_rb = p.n_rb, qp.n_var = p.n_var, qp.rows = p.N * p.g;
    qp.q = p.q, qp.images = p.images, qp.error = p.error;
    for (int i = 0; i < 3; i++) qp.qs[i] = p.qs[i];
    std::memcpy(qp.var_bits, p.var_bits, sizeof(qp.var_bits));
    std::memcpy(qp.sign_bits, p.sign_bits, sizeof(qp.sign_bits));
    qp.inv_sqrt_d = p.inv_sqrt_d, qp.qk_scale = p.qk_scale;
    tree_queries_kernel<D, R><<<images * std::max(1, R / kPrepRows), 32 * kPrepWarps, 0, s>>>(qp);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.workers);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_mma_kernel<D, R>, p, lv, ring);
}

template <int D>
cudaError_t tree_rows(const TreeParams &p, const TreeLevels &lv, cudaStream_t s) {
    return p.R == 16 ? tree_mma<D, 16>(p, lv, s) : p.R == 32 ? tree_mma<D, 32>(p, lv, s) : tree_mma<D, 64>(p, lv, s);
}

}  // namespace

// The least power of two that holds the rows, up to 64.
int tree_mma_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

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
    return p.d == 128 ? tree_rows<128>(p, lv, s) : tree_rows<64>(p, lv, s);
}

}  // namespace tqk
