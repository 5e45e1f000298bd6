// blocknorm_f32.cu -- norms around a block for float storage
#include "blocknorm.cuh"
template nrm_status nrm::block_norm_fwd<float>(const nrm::BlockArgs&, bool, cudaStream_t);
template nrm_status nrm::block_norm_bwd<float>(const nrm::BlockArgs&, bool, bool, cudaStream_t);
