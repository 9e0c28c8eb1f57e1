// tq_read_rows_values.cu -- the values of a read, one vector of head_dim 128 a thread.
#include "tq_read_rows.cuh"

namespace tqk {
cudaError_t launch_read_values(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return read_rows_dispatch<true, 1>(p, bits, beside, s);
}
}  // namespace tqk
