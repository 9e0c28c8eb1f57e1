// tq_append_rows_values.cu -- the values of a ragged write, one thread per vector.
#include "tq_append_rows.cuh"

namespace tqk {
cudaError_t launch_append_values(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return append_rows_dispatch<true>(p, bits, beside, s);
}
}  // namespace tqk
