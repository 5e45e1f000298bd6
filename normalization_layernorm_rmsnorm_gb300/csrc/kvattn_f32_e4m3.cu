// kvattn_f32_e4m3.cu -- attention over the cache on matrix instructions, float queries, codes in e4m3
#include "kvattn_mma.cuh"
template nrm_status nrm::attn_mma<float, NRM_CACHE_E4M3>(nrm::AttnArgs&, const nrm::DevInfo*, cudaStream_t);
