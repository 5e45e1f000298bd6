// kvattn_f16.cu -- attention over the cache for __half queries and outputs
#include "kvattn.cuh"
template nrm_status nrm::kv_attention<__half>(const nrm::AttnArgs&, int, cudaStream_t);
