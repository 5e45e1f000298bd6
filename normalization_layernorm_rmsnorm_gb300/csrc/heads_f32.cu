// heads_f32.cu -- operators on attention heads for float storage
#include "heads.cuh"
NRM_INSTANTIATE_HEADS(float)
