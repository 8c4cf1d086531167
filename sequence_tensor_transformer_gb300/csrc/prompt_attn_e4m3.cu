// Prompts' attention over an E4M3 cache: the tensor-core kernel.
#include "prompt_attn_tc.cuh"

namespace sptp {

cudaError_t launch_prompt_e4m3(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    return prompt::launch_width<true, prompt::kNoCap, false>(p, num_sms, ctas, s);
}

}  // namespace sptp
