// Paged attention over an fp32 cache: the CUDA-core consumer.
#include "paged_attn_launch.cuh"

namespace sptp {

cudaError_t launch_paged_attn_f32(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return paged::launch_simt<false>(p, num_sms, ctas, s);
}

}  // namespace sptp
