// What attention makes of a score before the softmax: a cap, and a bias that
// depends on the distance of the key.  Scores are in units of log 2 (the
// softmax takes powers of two), and so are the cap and the slopes here.
#pragma once

#include <cuda_runtime.h>

namespace sptp {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float pow2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The cap: c tanh(s / c) of a score s (both natural); none if c == 0.
struct ScoreCap {
    float cap;     // c log2(e), 0: none
    float inv;     // 1 / cap
    float twice;   // 2 / c: with x = s log2(e), e^(2 s / c) = 2^(twice x)

    __device__ __forceinline__ explicit ScoreCap(float c) {
        cap = c * kLog2e;
        inv = c == 0.f ? 0.f : 1.f / cap;
        twice = c == 0.f ? 0.f : 2.f / c;
    }
    // tanh u = 1 - 2 / (1 + e^2u) is good to 2^-22 of the cap; below 1/8 of the
    // cap, where that would be much of the score, its series, whose next term
    // is below 2^-29 of the score: u (1 - u^2/3 + 2 u^4/15 - 17 u^6/315).
    __device__ __forceinline__ float operator()(float x) const {
        const float u = x * inv, v = u * u;
        const float near = x * fmaf(v, fmaf(v, fmaf(v, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
        const float far = fmaf(-2.f * cap, __fdividef(1.f, 1.f + pow2_approx(x * twice)), cap);
        return fabsf(u) < 0.125f ? near : far;
    }
};

}  // namespace sptp
