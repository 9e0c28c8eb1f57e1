// tq_append_rows_values.cu -- the values of a ragged write, one thread per vector.
#include "tq_append_rows.cuh"

namespace tqk {
cudaError_t launch_append_values(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s) {
    return p.rows.slots ? launch_append_values_slots(p, bits, beside, s) : append_rows_dispatch<true, false>(p, bits, beside, s);
}
}  // namespace tqk
