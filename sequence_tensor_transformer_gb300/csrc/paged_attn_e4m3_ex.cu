// Paged attention over an E4M3 cache: the tensor-core consumer, scores with a cap or a bias.
#include "paged_attn_launch.cuh"

namespace sptp {

cudaError_t launch_paged_attn_e4m3_ex(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return paged::launch_tc<true, true>(p, num_sms, ctas, s);
}

}  // namespace sptp
