// kvattn_f32.cu -- attention over the cache for float queries and outputs
#include "kvattn.cuh"
template nrm_status nrm::kv_attention<float>(const nrm::AttnArgs&, int, cudaStream_t);
