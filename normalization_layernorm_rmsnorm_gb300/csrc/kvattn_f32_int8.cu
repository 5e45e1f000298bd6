// kvattn_f32_int8.cu -- attention over the cache on matrix instructions, float queries, codes in int8
#include "kvattn_mma.cuh"
template nrm_status nrm::attn_mma<float, NRM_CACHE_INT8>(nrm::AttnArgs&, const nrm::DevInfo*, cudaStream_t);
