// tq_pages.cu -- block tables and slot maps of sequences that share a pool of pages,
// from their lengths; pages come off a stack and go back onto it.
//
// With held = ceil(len / P) and need = ceil((len + want) / P) - held of each sequence, the
// pages before sequence b's on the stack are base = the sum of need over the sequences
// before it (a scan), so that every sequence's share, and with it every table entry, is
// known without one waiting for another: entry held + k is stack[n_free - 1 - base - k].
//
// Bound by latency: a decode step of 32 sequences is two dependent loads and a scan (5.9 us alone with cold
// caches, as much for the release; 64 prompts of up to 16384 tokens, slots and release included: 18.5 us).  One
// cluster of eight CTAs does it (every CTA scans all counts, they are few; each writes its
// sequences' entries), and the lengths and the stack's size, which the others read, change
// behind a barrier of the cluster.  Long prompts' slots (n_max > 32: more than one pass of
// the warp that has the sequence) go by a grid of their own behind it.
#include <algorithm>

#include <cooperative_groups.h>

#include "tq_serve.h"

namespace tqk {
namespace {

constexpr int kPageThreads = 512;
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kPageCtas = 8;
constexpr int kFusedRows = 32;

__device__ __forceinline__ int pages_of(int tokens, int page) { return tokens / page + (tokens % page ? 1 : 0); }

// Exclusive scan over the CTA, and the sum (64 bits: counts of many sequences).
__device__ __forceinline__ long long scan(long long x, long long *warp_sum, long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    __syncthreads();  // (warp_sum of an earlier scan has been read)
    if (lane == 31) warp_sum[warp] = y;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int w = 0; w < kPageWarps; w++) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    return before + y - x;
}

struct Place {
    int len, held, got, granted;
    long long base;
};

// A warp's n entries from one place to another, 256 at once: a prompt's entries are as many waits for memory as loads
// that follow one another (16384 tokens in pages of 16 by 32 at once: 32 of them).
template <class Load, class Store>
__device__ __forceinline__ void move_entries(int lane, int n, Load load, Store store) {
    constexpr int U = 8;
    for (int k0 = lane; k0 < n; k0 += 32 * U) {
        int x[U];
#pragma unroll
        for (int u = 0; u < U; u++) x[u] = k0 + 32 * u < n ? load(k0 + 32 * u) : 0;
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 + 32 * u < n) store(k0 + 32 * u, x[u]);
    }
}

// Slot and position of row j of a sequence (held tokens len, granted tokens behind them).
__device__ __forceinline__ void put_row(const PageParams &p, int b, int j, int len, int granted, const int *entries) {
    const bool fits = j < granted;
    const int t = fits ? len + j : 0;
    int slot = -1;
    if (fits) {
        const int page = entries[t / p.page];
        if (page >= 0 && page < p.n_pages) slot = page * p.page + t % p.page;
    }
    if (p.slots) p.slots[static_cast<size_t>(b) * p.n_max + j] = slot;
    if (p.positions) p.positions[static_cast<size_t>(b) * p.n_max + j] = fits ? t : -1;
}

__global__ void __cluster_dims__(kPageCtas, 1, 1) __launch_bounds__(kPageThreads) page_tables_kernel(const __grid_constant__ PageParams p) {
    __shared__ long long warp_sum[kPageWarps];
    __shared__ Place place[kPageThreads];
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x;
    const int most = p.width * p.page;  // tokens that a row of the table can hold (the host checks 32 bits)
    const int free = min(max(*p.n_free, 0), p.n_pages);
    long long taken = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPageThreads) {
        const int b = b0 + threadIdx.x;
        Place x = {0, 0, 0, 0, 0};
        int want = 0, need = 0;
        if (b < p.B) {
            x.len = min(max(p.length[b], 0), most);
            want = min(min(max(p.count[b], 0), p.n_max), most - x.len);
            x.held = pages_of(x.len, p.page);
            need = pages_of(x.len + want, p.page) - x.held;
        }
        long long sum;
        x.base = taken + scan(need, warp_sum, sum);
        taken += sum;
        x.got = static_cast<int>(min(max(free - x.base, 0LL), static_cast<long long>(need)));
        // (the last page held has room for what it has: no product beyond `most`)
        x.granted = min(want, (x.held + x.got) * p.page - x.len);
        place[threadIdx.x] = x;
        __syncthreads();
        const int n = min(kPageThreads, p.B - b0);
        for (int i = warp * kPageCtas + rank; i < n; i += kPageWarps * kPageCtas) {
            const Place y = place[i];
            int *entries = p.table + (b0 + i) * p.table_stride;
            move_entries(lane, y.got, [&](int k) { return p.free_pages[free - 1 - y.base - k]; }, [&](int k, int page) { entries[y.held + k] = page; });
            __syncwarp();
            if (lane == 0) p.granted[b0 + i] = y.granted;
            if (p.n_max <= kFusedRows && lane < p.n_max) put_row(p, b0 + i, lane, y.len, y.granted, entries);
        }
    }
    // every CTA has read the lengths and the stack's size
    cooperative_groups::this_cluster().sync();
    if (rank == 0 && threadIdx.x == 0) *p.n_free = static_cast<int>(max(free - taken, 0LL));
    // (the CTA that granted a sequence its tokens has the count; across chunks it is read back)
    for (int b0 = 0; b0 < p.B; b0 += kPageThreads) {
        const int n = min(kPageThreads, p.B - b0);
        for (int i = warp * kPageCtas + rank; i < n; i += kPageWarps * kPageCtas)
            if (lane == 0) p.length[b0 + i] = min(max(p.length[b0 + i], 0), most) + p.granted[b0 + i];
    }
}

// Slots and positions of long rows: the lengths are those behind the call.
__global__ void __launch_bounds__(256) slot_map_kernel(const __grid_constant__ PageParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int granted = p.granted[b], len = p.length[b] - granted;
        const int *entries = p.table + b * p.table_stride;
        for (long long j = blockIdx.x * 256 + threadIdx.x; j < p.n_max; j += gridDim.x * 256)
            put_row(p, b, static_cast<int>(j), len, granted, entries);
    }
}

__global__ void __cluster_dims__(kPageCtas, 1, 1) __launch_bounds__(kPageThreads) page_release_kernel(const __grid_constant__ PageParams p) {
    __shared__ long long warp_sum[kPageWarps];
    __shared__ Place place[kPageThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x;
    const int most = p.width * p.page;
    const int free = min(max(*p.n_free, 0), p.n_pages);
    auto drop = [&](int b, Place &x) {  // pages to give back
        x.len = min(max(p.length[b], 0), most);
        x.granted = min(max(p.count[b], 0), x.len);
        x.held = pages_of(x.granted, p.page);
        x.got = pages_of(x.len, p.page) - x.held;
        return x.got;
    };
    long long total = 0;
    {
        long long mine = 0;
        Place x;
        for (int b = threadIdx.x; b < p.B; b += kPageThreads) mine += drop(b, x);
        scan(mine, warp_sum, total);
    }
    long long before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPageThreads) {
        const int b = b0 + threadIdx.x;
        Place x = {0, 0, 0, 0, 0};
        if (b < p.B) drop(b, x);
        long long sum;
        x.base = before + scan(x.got, warp_sum, sum);
        before += sum;
        place[threadIdx.x] = x;
        __syncthreads();
        const int n = min(kPageThreads, p.B - b0);
        for (int i = warp * kPageCtas + rank; i < n; i += kPageWarps * kPageCtas) {
            const Place y = place[i];
            const int *entries = p.table + (b0 + i) * p.table_stride;
            // the last given back lies deepest: what was taken last comes back first
            move_entries(lane, y.got, [&](int k) { return entries[y.held + k]; }, [&](int k, int page) {
                const long long at = free + total - 1 - y.base - k;
                if (at < p.n_pages) p.free_pages[at] = page;
            });
        }
    }
    cooperative_groups::this_cluster().sync();
    if (rank == 0 && threadIdx.x == 0) *p.n_free = static_cast<int>(min(free + total, static_cast<long long>(p.n_pages)));
    for (int b = rank * kPageThreads + threadIdx.x; b < p.B; b += kPageCtas * kPageThreads)
        p.length[b] = min(min(max(p.length[b], 0), most), max(p.count[b], 0));
}

}  // namespace

cudaError_t launch_page_tables(const PageParams &p, cudaStream_t s) {
    page_tables_kernel<<<kPageCtas, kPageThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.n_max <= kFusedRows || (!p.slots && !p.positions)) return e;
    cudaLaunchConfig_t cfg = {};
    const int per = std::max(1, 4 * current_sm_count() / p.B);
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(p.n_max / 256 + 1, per)), static_cast<unsigned>(std::min(p.B, 32768)));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, slot_map_kernel, p);
}

cudaError_t launch_page_release(const PageParams &p, cudaStream_t s) {
    page_release_kernel<<<kPageCtas, kPageThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace tqk
