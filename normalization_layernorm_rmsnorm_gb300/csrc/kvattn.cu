// kvattn.cu -- attention over the cache: the kernel for any layout, the joining of
// pieces, the weights, and the choice between the kernels.
#include "kvattn.cuh"

namespace nrm {

template <typename T>
nrm_status kv_attention(const AttnArgs& args, int vec, cudaStream_t s) {
    AttnArgs a = args;
    const DevInfo* dev = dev_info();
    if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    a.err = dev->err;
    void* p[] = {&a};
    nrm_status st;
    if (vec) {
        a.vec = vec;
        st = a.cache.kind == NRM_CACHE_E4M3   ? attn_mma<T, NRM_CACHE_E4M3>(a, dev, s)
             : a.cache.kind == NRM_CACHE_INT8 ? attn_mma<T, NRM_CACHE_INT8>(a, dev, s)
                                              : attn_mma<T, NRM_CACHE_INT4>(a, dev, s);
    } else {
        attn_chunks(a, kAttnScalarHeads);
        a.workers = dev->sms * (kAttnThreads / 32);
        attn_snap(a);
        st = launch_pdl(reinterpret_cast<const void*>(&attn_scalar_kernel<T>), dim3(unsigned(dev->sms)),
                        dim3(kAttnThreads), p, s);
    }
    if (st != NRM_OK) return st;
    // unless no sequence can be cut
    if (attn_most_tiles(a) > a.snap) {
        // a CTA for each head where there are too few pairs to fill the GPU
        const int pairs = a.sequences * a.hk * a.chunks;
        const bool few = pairs < dev->sms;
        st = launch_pdl(a.d <= 128 ? reinterpret_cast<const void*>(&attn_join_kernel<T, 1>)
                                   : reinterpret_cast<const void*>(&attn_join_kernel<T, 2>),
                        dim3(unsigned(pairs), few ? unsigned(a.heads) : 1u), dim3(few ? 32 * kJoinWarps : 128), p, s);
        if (st != NRM_OK) return st;
    }
    if (!a.weights) return NRM_OK;
    return launch_pdl(reinterpret_cast<const void*>(&attn_weights_kernel<T>), dim3(unsigned(4 * dev->sms)),
                      dim3(kAttnThreads), p, s);
}

template nrm_status kv_attention<float>(const AttnArgs&, int, cudaStream_t);
template nrm_status kv_attention<__half>(const AttnArgs&, int, cudaStream_t);
template nrm_status kv_attention<__nv_bfloat16>(const AttnArgs&, int, cudaStream_t);

}  // namespace nrm
