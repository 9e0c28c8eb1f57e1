// tq_paged_fp16.cu -- attention of one new token over pages of fp16 rows, head dims 64 and 128: the
// form of tq_paged_mma.cuh without codes.
//
// A stage is 16 tokens: K rows by ldmatrix against the queries as they are (fp16, one part), V rows by
// ldmatrix.trans.  16-byte chunk i of row r lies at i ^ (r & 7), so that the eight rows of an ldmatrix are in
// eight bank groups.  Pages of any size; V rows that are not there are zeros (their weights are).
#include "tq_paged_mma.cuh"

namespace tqk {
namespace pmma {
namespace {

__device__ __forceinline__ void ldmatrix4(uint32_t (&a)[4], unsigned at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&a)[4], unsigned at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(at));
}

constexpr float kInfinity = __builtin_huge_valf();

template <int DIM>
struct Half {
    static constexpr int D = DIM, R = 4, MT = D / 16;
    static constexpr int PT = 16, row = 2 * D, CH = D / 8;       // tokens of a stage; bytes and chunks of a row
    static constexpr int kSlot = 2 * PT * row, kTable = 0;
    static constexpr bool kLinear = false;

    uint32_t bq[2 * MT];
    float scale;

    static __device__ __forceinline__ void fill_table(uint8_t *, const Levels &) {}
    __device__ __forceinline__ Half(const uint8_t *, const Levels &, int) {}
    static constexpr uint32_t kTokenK = row, kTokenV = row;
    // (the V rows: those that do not come stay zeros)
    static __device__ __forceinline__ void clear(uint8_t *slot, int lane) {
        for (int i = lane; i < PT * CH; i += 32) reinterpret_cast<uint4 *>(slot + PT * row)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
    }
    static __device__ __forceinline__ void copy(const uint8_t *k, const uint8_t *v, unsigned slot, int from, int run, uint64_t pol, int lane) {
        const int chunk = lane % CH, first = from + lane / CH;
#pragma unroll
        for (int i = 0; i < PT; i += 32 / CH) {
            const unsigned to = slot + (first + i) * row + 16 * (chunk ^ ((first + i) & 7));
            if (run == PT || lane / CH + i < run) {
                copy16(to, k + i * row, pol);
                copy16(to + PT * row, v + i * row, pol);
            }
        }
    }
    static __device__ __forceinline__ void fill_all(const Source &s, unsigned slot, uint64_t pol, int lane) { copy(s.ka, s.va, slot, 0, PT, pol, lane); }
    static __device__ __forceinline__ bool fill_blocks(const PagedParams &, const Source &, const paged::Walk &, unsigned, uint64_t, int) { return false; }
    static __device__ __forceinline__ void fill(const uint8_t *k, const uint8_t *v, const char *, unsigned slot, int from, int run,
                                                uint64_t pol, int lane) {
        copy(k, v, slot, from, run, pol, lane);
    }
    __device__ __forceinline__ void queries(const PagedParams &p, __half *, int b, int h, int rb, int lane) {
        const int c = lane & 3, head = rb * R + (lane >> 3);
        const uint16_t *q = p.q + b * p.qs[0] + (static_cast<int64_t>(h) * p.g + head) * p.qs[1] + 2 * c;
        const bool some = !((lane >> 2) & 1) && head < p.g;  // (the lo column: nothing)
#pragma unroll
        for (int i = 0; i < 2 * MT; i++)
            bq[i] = some ? static_cast<uint32_t>(q[8 * i]) | (static_cast<uint32_t>(q[8 * i + 1]) << 16) : 0u;
        scale = p.qk_scale;
    }
    template <bool FULL>
    __device__ __forceinline__ void stage(Run<MT> &r, const uint8_t *buf8, int n, const Stage &sg, uint32_t sel, int lane,
                                          std::integral_constant<bool, FULL>) {
        const int g = lane >> 2, c = lane & 3;
        const unsigned buf = smem_u32(buf8);
        // the lane's row address of an ldmatrix
        const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, kch = lane >> 4, vrow = (lane & 7) + (lane >> 4) * 8, vch = (lane >> 3) & 1;
        float e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < MT; kk++) {
            uint32_t a[4];
            ldmatrix4(a, buf + krow * row + 16 * ((2 * kk + kch) ^ (krow & 7)));
            mma16816(e, a[0], a[1], a[2], a[3], bq[2 * kk], bq[2 * kk + 1]);
        }
        float s[2];
        const float v[2] = {1.f, 1.f};
        bool have[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            s[i] = e[2 * i] * scale;
            have[i] = FULL || have_token(sg, g + 8 * i, n);
        }
        uint32_t bp[2];
        softmax<FULL, 1>(r, s, have, v, g, c, sel, bp);
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            uint32_t a[4];
            ldmatrix4_trans(a, buf + PT * row + vrow * row + 16 * ((2 * mt + vch) ^ (vrow & 7)));
            mma16816(r.acc[mt], a[0], a[1], a[2], a[3], bp[0], bp[1]);
        }
        r.tiles++;
    }
    __device__ __forceinline__ void fold(const Run<MT> &r, float *copy, float, float f, int lane) const {
        copy += (lane & 3) * copy_stride(D) + (lane >> 2);
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                float &at = copy[16 * mt + 8 * i];
                // (an infinite value: hi's sum tells its sign, lo may be 0 or negative)
                const float hi = r.acc[mt][2 * i], x = fabsf(hi) == kInfinity ? hi : r.sum(mt, i);
                at = r.some ? fmaf(at, f, x) : x;
            }
    }
    static __device__ __forceinline__ void record(float *rec, const float *copy, float m, float l, int lane) {
#pragma unroll
        for (int i = 0; i < R; i++) {
            float *to = rec + i * (D + 4);
            const float m0 = __shfl_sync(0xffffffffu, m, i), l0 = __shfl_sync(0xffffffffu, l, i);
            if (lane == 0) *reinterpret_cast<float2 *>(to) = make_float2(m0, l0);
            if (4 * lane < D) *reinterpret_cast<float4 *>(to + 4 + 4 * lane) = *reinterpret_cast<const float4 *>(copy + i * copy_stride(D) + 4 * lane);
        }
    }
};

}  // namespace
}  // namespace pmma

cudaError_t launch_paged_fp16(const PagedParams &p, cudaStream_t s) {
    static const pmma::Levels none = {};
    return p.d == 128 ? pmma::launch<pmma::Half<128>>(p, none, s) : pmma::launch<pmma::Half<64>>(p, none, s);
}

}  // namespace tqk
