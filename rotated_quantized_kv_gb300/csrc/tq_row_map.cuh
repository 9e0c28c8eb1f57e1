// tq_row_map.cuh -- rows of a ragged write.
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

// Source row and target position of row j of sequence b; false: not written.
__device__ __forceinline__ bool map_row(const RowMap &m, int b, int j, int capacity, int &src, int &pos) {
    const int n = m.n_rows ? min(m.n_rows[b], m.n_max) : m.n_max;
    if (j >= n) return false;
    src = m.index ? m.index[b * m.index_stride + j] : j;
    const long long t = static_cast<long long>(m.t_begin[b]) + j;
    pos = static_cast<int>(t);
    return src >= 0 && src < m.n_source && t >= 0 && t < capacity;
}

}  // namespace
}  // namespace tqk
