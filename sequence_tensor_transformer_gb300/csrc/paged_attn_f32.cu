// Paged attention over an fp32 cache: the CUDA-core consumer by row width and
// heads per item.
#include "paged_attn_launch.cuh"

namespace sptp {

cudaError_t launch_paged_attn_f32(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s) {
    using namespace paged;
    const int group = p.Hq / p.Hkv;
    if (group <= 8) {
        if (p.D <= 64) return launch<F32Consumer<64>>(p, num_sms, ctas, s);
        if (p.D <= 128) return launch<F32Consumer<128>>(p, num_sms, ctas, s);
        return launch<F32Consumer<256>>(p, num_sms, ctas, s);
    }
    if (p.D <= 64) return launch<F32Consumer<64, 2>>(p, num_sms, ctas, s);
    if (p.D <= 128) return launch<F32Consumer<128, 2>>(p, num_sms, ctas, s);
    return launch<F32Consumer<256, 2>>(p, num_sms, ctas, s);
}

}  // namespace sptp
