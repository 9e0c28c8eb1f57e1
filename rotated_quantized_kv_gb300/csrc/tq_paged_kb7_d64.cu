// tq_paged_kb7_d64.cu -- attention over packed pages with 7-bit keys, head_dim 64 (every value width).
#include "tq_paged_mma.cuh"

TQ_INSTANTIATE_PAGED(7, 2)
