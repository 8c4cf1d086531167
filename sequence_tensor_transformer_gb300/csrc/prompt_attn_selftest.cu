// Self-test of the way out of prompts' attention: the tensor-core kernel itself, over
// a bf16 or an E4M3 cache, on two CTAs, with a tile of CTA 0 never loaded, so that
// its bounded waits run out without hanging the GPU.
#include "prompt_attn_tc.cuh"

namespace sptp {

cudaError_t launch_prompt_test(PromptParams& p, bool e4m3, int* ctas, cudaStream_t s) {
    using namespace prompt;
    return e4m3 ? launch_tc<Shape<128, true>, kNoCap, false, true>(p, kSelftestCtas, ctas, s)
                : launch_tc<Shape<128, false>, kNoCap, false, true>(p, kSelftestCtas, ctas, s);
}

}  // namespace sptp
