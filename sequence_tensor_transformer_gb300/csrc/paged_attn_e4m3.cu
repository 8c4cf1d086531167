// Paged attention over an E4M3 cache: the tensor-core consumer by row width and
// heads per item.
#include "paged_attn_launch.cuh"

namespace sptp {

cudaError_t launch_paged_attn_e4m3(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s) {
    using namespace paged;
    const int group = p.Hq / p.Hkv;
    if (p.D <= 128) {
        if (group <= 8) return launch<TcConsumer<128, 1, true>>(p, num_sms, ctas, s);
        if (group <= 16) return launch<TcConsumer<128, 2, true>>(p, num_sms, ctas, s);
        return launch<TcConsumer<128, 4, true>>(p, num_sms, ctas, s);
    }
    // a row of more than 128 elements: fewer heads in the registers
    if (group <= 8) return launch<TcConsumer<256, 1, true>>(p, num_sms, ctas, s);
    return launch<TcConsumer<256, 2, true>>(p, num_sms, ctas, s);
}

}  // namespace sptp
