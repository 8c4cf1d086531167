// Prompts' attention over a bf16 cache, scores with a cap or a bias: the tensor-core kernel.
#include "prompt_attn_tc.cuh"

namespace sptp {

cudaError_t launch_prompt_bf16_ex(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return prompt::launch_width<false, true>(p, num_sms, ctas, s);
}

}  // namespace sptp
