// heads_f16.cu -- operators on attention heads for __half storage
#include "heads.cuh"
NRM_INSTANTIATE_HEADS(__half)
