// Prompts' attention over a bf16 cache, capped scores with a bias: the tensor-core kernel.
#include "prompt_attn_tc.cuh"

namespace sptp {

cudaError_t launch_prompt_bf16_cap_bias(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return prompt::launch_cap<false, true>(p, num_sms, ctas, s);
}

}  // namespace sptp
