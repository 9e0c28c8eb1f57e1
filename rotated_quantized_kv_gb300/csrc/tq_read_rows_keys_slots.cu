// tq_read_rows_keys_slots.cu -- the keys of a read, one vector of head_dim 128 a thread, by slot.
#include "tq_read_rows.cuh"

namespace tqk {
cudaError_t launch_read_keys_slots(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return read_rows_dispatch<false, 1, true>(p, bits, beside, s);
}
}  // namespace tqk
