// tq_paged_kb8_d128.cu -- attention over packed pages with 8-bit keys, head_dim 128 (every value width).
#include "tq_paged_mma.cuh"

TQ_INSTANTIATE_PAGED(8, 1)
