// Paged attention over a bf16 cache: the tensor-core consumer, scores with a cap or a bias.
#include "paged_attn_launch.cuh"

namespace sptp {

cudaError_t launch_paged_attn_bf16_ex(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return paged::launch_tc<false, true>(p, num_sms, ctas, s);
}

}  // namespace sptp
