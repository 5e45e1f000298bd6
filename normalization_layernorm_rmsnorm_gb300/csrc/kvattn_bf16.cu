// kvattn_bf16.cu -- attention over the cache for __nv_bfloat16 queries and outputs
#include "kvattn.cuh"
template nrm_status nrm::kv_attention<__nv_bfloat16>(const nrm::AttnArgs&, int, cudaStream_t);
