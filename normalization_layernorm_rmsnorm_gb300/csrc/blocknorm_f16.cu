// blocknorm_f16.cu -- norms around a block for __half storage
#include "blocknorm.cuh"
template nrm_status nrm::block_norm_fwd<__half>(const nrm::BlockArgs&, bool, cudaStream_t);
template nrm_status nrm::block_norm_bwd<__half>(const nrm::BlockArgs&, bool, bool, cudaStream_t);
