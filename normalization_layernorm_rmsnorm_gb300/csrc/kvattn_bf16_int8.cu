// kvattn_bf16_int8.cu -- attention over the cache on matrix instructions, __nv_bfloat16 queries, codes in int8
#include "kvattn_mma.cuh"
template nrm_status nrm::attn_mma<__nv_bfloat16, NRM_CACHE_INT8>(nrm::AttnArgs&, const nrm::DevInfo*, cudaStream_t);
