// tq_read_rows_values_d64.cu -- the values of a read, two vectors of head_dim 64 a thread.
#include "tq_read_rows.cuh"

namespace tqk {
cudaError_t launch_read_values_d64(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return read_rows_dispatch<true, 2>(p, bits, beside, s);
}
}  // namespace tqk
