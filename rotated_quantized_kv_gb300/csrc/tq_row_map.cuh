// tq_row_map.cuh -- rows of a ragged write or read.
#pragma once

#include "tq_serve.h"

namespace tqk {
namespace {

// A launch that may run beside the one before it in the stream (beside), which wrote
// nothing that this one touches.
template <class P>
cudaError_t launch_beside(void (*kernel)(P), unsigned grid, int threads, size_t smem, cudaStream_t s, bool beside, const P &p) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(static_cast<unsigned>(threads));
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, p);
}

// Whether the kernels that take 32 threads' rows of `per` vectors each as a block can count
// their blocks, and the rows, in 32 bits (with a grid's warps to spare).
inline bool blocks_fit(int B, int H, int n_max, int per) {
    return n_max <= 1 << 30 && (static_cast<long long>(n_max) + 32 * per - 1) / (32 * per) * H * B <= 1 << 30;
}

// Place of row j of sequence b in the segment: batch element (a page, where rows have
// SLOTS) and position in it; false: nowhere.  (The row kernels are compiled for either: a
// batch element that is one for the whole warp saves a read of 65408 rows 4 of 118 us.)
template <bool SLOTS>
__device__ __forceinline__ bool place_row(const RowMap &m, int b, int j, int capacity, int &block, int &pos) {
    const int n = m.n_rows ? min(m.n_rows[b], m.n_max) : m.n_max;
    if constexpr (SLOTS) {
        if (j >= n) return false;
        const int slot = m.slots[b * m.slot_stride + j];
        block = slot / capacity;
        pos = slot - block * capacity;
        return slot >= 0 && block < m.n_blocks;
    }
    const long long t = static_cast<long long>(m.t_begin[b]) + j;
    block = b;
    pos = static_cast<int>(t);
    return j < n && t >= 0 && t < capacity;
}
__device__ __forceinline__ bool place_row(const RowMap &m, int b, int j, int capacity, int &block, int &pos) {
    return m.slots ? place_row<true>(m, b, j, capacity, block, pos) : place_row<false>(m, b, j, capacity, block, pos);
}

// The same with the source row of a write.
template <bool SLOTS>
__device__ __forceinline__ bool map_row(const RowMap &m, int b, int j, int capacity, int &src, int &block, int &pos) {
    if (!place_row<SLOTS>(m, b, j, capacity, block, pos)) return false;
    src = m.index ? m.index[b * m.index_stride + j] : j;
    return src >= 0 && src < m.n_source;
}
__device__ __forceinline__ bool map_row(const RowMap &m, int b, int j, int capacity, int &src, int &block, int &pos) {
    return m.slots ? map_row<true>(m, b, j, capacity, src, block, pos) : map_row<false>(m, b, j, capacity, src, block, pos);
}

}  // namespace
}  // namespace tqk
