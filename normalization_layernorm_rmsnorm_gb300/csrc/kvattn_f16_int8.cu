// kvattn_f16_int8.cu -- attention over the cache on matrix instructions, __half queries, codes in int8
#include "kvattn_mma.cuh"
template nrm_status nrm::attn_mma<__half, NRM_CACHE_INT8>(nrm::AttnArgs&, const nrm::DevInfo*, cudaStream_t);
