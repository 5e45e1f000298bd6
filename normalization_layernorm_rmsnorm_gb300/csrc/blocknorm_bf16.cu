// blocknorm_bf16.cu -- norms around a block for __nv_bfloat16 storage
#include "blocknorm.cuh"
template nrm_status nrm::block_norm_fwd<__nv_bfloat16>(const nrm::BlockArgs&, bool, cudaStream_t);
template nrm_status nrm::block_norm_bwd<__nv_bfloat16>(const nrm::BlockArgs&, bool, bool, cudaStream_t);
