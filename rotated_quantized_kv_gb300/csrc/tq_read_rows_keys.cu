// tq_read_rows_keys.cu -- the keys of a read, one vector of head_dim 128 a thread.
#include "tq_read_rows.cuh"

namespace tqk {
cudaError_t launch_read_keys(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return p.rows.slots ? launch_read_keys_slots(p, bits, beside, s) : read_rows_dispatch<false, 1, false>(p, bits, beside, s);
}
}  // namespace tqk
