// Prompts' attention over a bf16 cache: the tensor-core kernel.
#include "prompt_attn_tc.cuh"

namespace sptp {

cudaError_t launch_prompt_bf16(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return prompt::launch_width<false, prompt::kNoCap, false>(p, num_sms, ctas, s);
}

}  // namespace sptp
