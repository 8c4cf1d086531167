// Paged attention over an E4M3 cache: the tensor-core consumer by row width and
// heads per item.
#include "paged_attn_launch.cuh"

namespace sptp {

cudaError_t launch_paged_attn_e4m3(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s) {
    using namespace paged;
    const int group = p.Hq / p.Hkv;
    if (p.D <= 64) {
        if (group <= 8) return launch<TcConsumer<64, 1, true>>(p, num_sms, ctas, s);
        if (group <= 16) return launch<TcConsumer<64, 2, true>>(p, num_sms, ctas, s);
        return launch<TcConsumer<64, 2, true, 2>>(p, num_sms, ctas, s);
    }
    if (p.D <= 128) {
        if (group <= 8) return launch<TcConsumer<128, 1, true>>(p, num_sms, ctas, s);
        if (group <= 16) return launch<TcConsumer<128, 2, true>>(p, num_sms, ctas, s);
        return launch<TcConsumer<128, 2, true, 2>>(p, num_sms, ctas, s);
    }
    // rows of more than 128 elements: 16 heads are what the registers hold
    if (group <= 8) return launch<TcConsumer<256, 1, true>>(p, num_sms, ctas, s);
    return launch<TcConsumer<256, 2, true>>(p, num_sms, ctas, s);
}

}  // namespace sptp
