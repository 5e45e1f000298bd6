// kvattn_bf16_int4.cu -- attention over the cache on matrix instructions, __nv_bfloat16 queries, codes in int4
#include "kvattn_mma.cuh"
template nrm_status nrm::attn_mma<__nv_bfloat16, NRM_CACHE_INT4>(nrm::AttnArgs&, const nrm::DevInfo*, cudaStream_t);
