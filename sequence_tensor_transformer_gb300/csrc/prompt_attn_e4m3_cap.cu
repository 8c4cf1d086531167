// Prompts' attention over an E4M3 cache, capped scores: the tensor-core kernel.
#include "prompt_attn_tc.cuh"

namespace sptp {

cudaError_t launch_prompt_e4m3_cap(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return prompt::launch_cap<true, false>(p, num_sms, ctas, s);
}

}  // namespace sptp
