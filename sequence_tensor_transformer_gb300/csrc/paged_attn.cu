// The paged attention's dispatch over the cache's element type, and the join of
// the items that were split over several CTAs (paged_attn.cuh has the main
// kernel).
#include <cuda_bf16.h>

#include "sptp.h"
#include "sptp_ptx.cuh"

namespace sptp {

namespace {

constexpr int kJoinThreads = 256;

// Block (h, i): query head h of the item that begins in CTA i's share and goes
// on in later ones, if there is one:  m = max m_k,  out = sum e^(m_k - m) o_k /
// sum e^(m_k - m) l_k over its parts k in ascending order per warp, then over
// the warps.  A warp takes every eighth part, its lanes the elements.  Block
// (0, 0) also sums up the CTAs' status words.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_join(const __grid_constant__ PagedAttnParams p, int ctas) {
    constexpr int kWarps = kJoinThreads / 32, kPer = 8;  // elements per lane: D <= 256
    __shared__ float weight[kPagedMaxCtas];
    __shared__ float o[kWarps][256];
    __shared__ float red[2][kWarps];
    __shared__ int first_bad;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x, i = blockIdx.y;
    if (h == 0 && i == 0) {
        if (tid == 0) first_bad = ctas;
        __syncthreads();
        for (int k = tid; k < ctas; k += kJoinThreads)
            if (p.parts[k].status != 0) atomicMin(&first_bad, k);
        __syncthreads();
        if (tid == 0) {
            DeviceStatus st = {0, 0, 0, 0, 0};
            if (first_bad < ctas) {
                const PagedAttnPart& bad = p.parts[first_bad];
                st.code = bad.status;
                st.where = bad.where;
                st.block = first_bad;
                st.info = bad.info;
            }
            *p.status = st;
        }
    }
    const int n = p.parts[i].join_parts;
    if (n < 2 || i + n > ctas) return;
    const int b = p.parts[i].b, j = p.parts[i].j;
    const int hb = j % p.head_blocks, sk = j / p.head_blocks, group = p.Hq / p.Hkv;
    const int h0 = hb * p.heads_per_item;
    if (h >= min(p.heads_per_item, group - h0)) return;
    // part k lies in slot 0 of CTA i + k; the first one in slot 1
    auto row_of = [&](int k) { return ((i + k) * 2ll + (k == 0 ? 1 : 0)) * p.heads_per_item + h; };
    float top = -INFINITY;
    float2 ml[(kPagedMaxCtas + kJoinThreads - 1) / kJoinThreads];
    int c = 0;
    for (int k = tid; k < n; k += kJoinThreads, ++c) {
        ml[c] = p.part_ml[row_of(k)];
        top = fmaxf(top, ml[c].x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) red[0][warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red[0][w]);
    float sum = 0.f;
    c = 0;
    for (int k = tid; k < n; k += kJoinThreads, ++c) {
        const float f = ml[c].x == -INFINITY ? 0.f : exp2f(ml[c].x - top);
        weight[k] = f;
        sum = fmaf(f, ml[c].y, sum);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += red[1][w];
    float acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int k = warp; k < n; k += kWarps) {
        const float f = weight[k];
        const float* row = p.part_o + row_of(k) * p.D;
#pragma unroll
        for (int e = 0; e < kPer / 4; ++e) {
            const int d = e * 128 + lane * 4;
            if (d < p.D) {
                const float4 v = *reinterpret_cast<const float4*>(row + d);
                acc[4 * e] = fmaf(f, v.x, acc[4 * e]);
                acc[4 * e + 1] = fmaf(f, v.y, acc[4 * e + 1]);
                acc[4 * e + 2] = fmaf(f, v.z, acc[4 * e + 2]);
                acc[4 * e + 3] = fmaf(f, v.w, acc[4 * e + 3]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[warp][(e >> 2) * 128 + lane * 4 + (e & 3)] = acc[e];
    __syncthreads();
    const int shard = sk / p.Hkv, kvh = sk - shard * p.Hkv;
    const long long qrow = (static_cast<long long>(shard) * p.B + b) * p.Hq + kvh * group + h0 + h;
    if (tid < p.D) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += o[w][tid];
        v = sum == 0.f ? 0.f : v / sum;
        static_cast<T*>(p.out)[qrow * p.D + tid] = static_cast<T>(v);
    }
    if (p.lse != nullptr && tid == 0) p.lse[qrow] = sum == 0.f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
}

}  // namespace

cudaError_t launch_paged_attn(PagedAttnParams& p, bool bf16, bool e4m3, int num_sms, cudaStream_t s) {
    if (e4m3 && !bf16) return cudaErrorInvalidValue;
    int ctas = 0;
    cudaError_t e = !bf16  ? launch_paged_attn_f32(p, num_sms, &ctas, s)
                    : e4m3 ? launch_paged_attn_e4m3(p, num_sms, &ctas, s)
                           : launch_paged_attn_bf16(p, num_sms, &ctas, s);
    if (e != cudaSuccess) return e;
    // The join is launched beside the main kernel's end (a programmatic
    // dependency): it waits for the parts on the device.
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(p.heads_per_item, ctas);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, paged_attn_join<__nv_bfloat16>, p, ctas)
                : cudaLaunchKernelEx(&cfg, paged_attn_join<float>, p, ctas);
}

}  // namespace sptp
