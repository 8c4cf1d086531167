// Paged attention over a bf16 cache: the tensor-core consumer.
#include "paged_attn_launch.cuh"

namespace sptp {

cudaError_t launch_paged_attn_bf16(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return paged::launch_tc<false, false>(p, num_sms, ctas, s);
}

}  // namespace sptp
