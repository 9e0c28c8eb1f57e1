// tq_read_rows_values.cu -- the values of a read, one thread per vector.
#include "tq_read_rows.cuh"

namespace tqk {
cudaError_t launch_read_values(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return read_rows_dispatch<true>(p, bits, beside, s);
}
}  // namespace tqk
