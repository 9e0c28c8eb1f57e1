// tq_append_rows_keys.cu -- the keys of a ragged write, one thread per vector.
#include "tq_append_rows.cuh"

namespace tqk {
cudaError_t launch_append_keys(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return append_rows_dispatch<false>(p, bits, beside, s);
}
}  // namespace tqk
