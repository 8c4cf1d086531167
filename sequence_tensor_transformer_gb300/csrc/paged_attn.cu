// Attention of one token per sequence over a paged key-value cache:
//     s_j = scale * q . k_j,  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m).
// One pass over the keys with a running maximum m, sum l and output o; a new
// maximum m' scales l and o by e^(m - m').
//
// One CTA per (shard, sequence, key/value head, up to 8 of its query heads);
// its warps take every fourth key, each with statistics of its own, and are
// joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sptp.h"
#include "sptp_ptx.cuh"

namespace sptp {

namespace {

constexpr int kWarps = 4;
constexpr int kHeads = 8;  // query heads per CTA
constexpr int kMaxD = 256;
constexpr int kPer = kMaxD / 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}


template <typename Q, typename KV>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    __shared__ float qs[kHeads][kMaxD];
    __shared__ float os[kWarps][kHeads][kMaxD];
    __shared__ float ms[kWarps][kHeads], ls[kWarps][kHeads];
    constexpr bool kCodes = sizeof(KV) == 1;
    const int group = p.Hq / p.Hkv, hb = (group + kHeads - 1) / kHeads;
    long long u = blockIdx.x;
    const int h0 = static_cast<int>(u % hb) * kHeads;
    u /= hb;
    const int kvh = static_cast<int>(u % p.Hkv);
    u /= p.Hkv;
    const int shard = static_cast<int>(u % p.P), b = static_cast<int>(u / p.P);
    const int nh = min(kHeads, group - h0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int most = p.max_pages * p.page_size;
    int len = __ldg(p.seq_lens + b);
    if ((len < 0 || len > most) && threadIdx.x == 0) atomicCAS(&p.status->code, 0, SPTP_ERR_SHAPE);
    len = max(0, min(len, most));
    const int start = p.window > 0 ? max(0, len - p.window) : 0;
    const long long qrow = (static_cast<long long>(shard) * p.B + b) * p.Hq + kvh * group + h0;
    for (int i = threadIdx.x; i < nh * p.D; i += kWarps * 32)
        qs[i / p.D][i % p.D] = static_cast<float>(static_cast<const Q*>(p.q)[qrow * p.D + i]) * p.scale;
    __syncthreads();
    float m[kHeads], l[kHeads], o[kHeads][kPer];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[h][i] = 0.f;
    }
    for (int j = start + warp; j < len; j += kWarps) {
        const int page = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + j / p.page_size);
        const bool ok = page >= 0 && page < p.num_pages;
        if (!ok && lane == 0) atomicCAS(&p.status->code, 0, SPTP_ERR_SHAPE);
        const long long row = ((static_cast<long long>(shard) * p.num_pages + (ok ? page : 0)) * p.Hkv + kvh) *
                                  p.page_size + j % p.page_size;
        float ksc = 1.f, vsc = 1.f;
        if (kCodes && ok) {
            ksc = p.k_scale[row];
            vsc = p.v_scale[row];
        }
        float kf[kPer], vf[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int d = lane + 32 * i;
            const bool in = ok && d < p.D;
            kf[i] = in ? static_cast<float>(static_cast<const KV*>(p.k)[row * p.D + d]) : 0.f;
            vf[i] = in ? static_cast<float>(static_cast<const KV*>(p.v)[row * p.D + d]) * vsc : 0.f;
        }
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (h >= nh) break;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < p.D) s = fmaf(qs[h][lane + 32 * i], kf[i], s);
            s = warp_sum(s) * ksc;
            const float top = fmaxf(m[h], s);
            const float old = m[h] == top ? 1.f : expf(m[h] - top);
            const float w = top == -INFINITY ? 0.f : expf(s - top);
            m[h] = top;
            l[h] = l[h] * old + w;
#pragma unroll
            for (int i = 0; i < kPer; ++i) o[h][i] = fmaf(o[h][i], old, w * vf[i]);
        }
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        if (lane == 0) {
            ms[warp][h] = m[h];
            ls[warp][h] = l[h];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) os[warp][h][lane + 32 * i] = o[h][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * p.D; i += kWarps * 32) {
        const int h = i / p.D, d = i % p.D;
        float top = -INFINITY, sum = 0.f, acc = 0.f;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ms[w][h]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = ms[w][h] == -INFINITY ? 0.f : expf(ms[w][h] - top);
            sum = fmaf(ls[w][h], f, sum);
            acc = fmaf(os[w][h][d], f, acc);
        }
        static_cast<Q*>(p.out)[qrow * p.D + i] = static_cast<Q>(sum > 0.f ? acc / sum : 0.f);
        if (p.lse != nullptr && d == 0) p.lse[qrow + h] = sum > 0.f ? top + logf(sum) : -INFINITY;
    }
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnParams& p, bool bf16, bool e4m3, int num_sms, cudaStream_t s) {
    (void)num_sms;
    const int group = p.Hq / p.Hkv;
    const long long grid = static_cast<long long>(p.B) * p.P * p.Hkv * ((group + kHeads - 1) / kHeads);
    if (grid > 0x7fffffffll || (e4m3 && !bf16)) return cudaErrorInvalidValue;
    const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(DeviceStatus), s);
    if (e != cudaSuccess) return e;
    const int g = static_cast<int>(grid);
    if (!bf16)
        paged_attn_kernel<float, float><<<g, kWarps * 32, 0, s>>>(p);
    else if (e4m3)
        paged_attn_kernel<__nv_bfloat16, __nv_fp8_e4m3><<<g, kWarps * 32, 0, s>>>(p);
    else
        paged_attn_kernel<__nv_bfloat16, __nv_bfloat16><<<g, kWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sptp
