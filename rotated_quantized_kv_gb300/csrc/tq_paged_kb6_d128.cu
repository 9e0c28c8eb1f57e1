// tq_paged_kb6_d128.cu -- attention over packed pages with 6-bit keys, head_dim 128 (every value width).
#include "tq_paged_mma.cuh"

TQ_INSTANTIATE_PAGED(6, 1)
