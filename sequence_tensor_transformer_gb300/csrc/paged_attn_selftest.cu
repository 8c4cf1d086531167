// Self-test of the paged attention's way out: the kernel itself, one consumer
// class of each kind (bf16 with one team of consumer warps, E4M3 and fp32 with
// two), with an arrival withheld in CTA 0, so that its bounded waits run out
// without hanging the GPU.
#include "paged_attn_launch.cuh"

namespace sptp {

cudaError_t launch_paged_attn_test(PagedAttnParams& p, bool bf16, bool e4m3, int* ctas, cudaStream_t s) {
    using namespace paged;
    if (p.D > 128) return cudaErrorInvalidValue;
    if (!bf16) return launch<F32Consumer<128, 2>, true>(p, kSelftestCtas, ctas, s);
    return e4m3 ? launch<TcConsumer<128, 2, true, 2>, true>(p, kSelftestCtas, ctas, s)
                : launch<TcConsumer<128, 1, false>, true>(p, kSelftestCtas, ctas, s);
}

}  // namespace sptp
