// tq_append_rows_keys_slots.cu -- the keys of a ragged write, one thread per vector, by slot.
#include "tq_append_rows.cuh"

namespace tqk {
cudaError_t launch_append_keys_slots(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return append_rows_dispatch<false, true>(p, bits, beside, s);
}
}  // namespace tqk
