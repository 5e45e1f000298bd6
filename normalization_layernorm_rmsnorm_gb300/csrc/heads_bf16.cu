// heads_bf16.cu -- operators on attention heads for __nv_bfloat16 storage
#include "heads.cuh"
NRM_INSTANTIATE_HEADS(__nv_bfloat16)
