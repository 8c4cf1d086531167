// sptp_paged_attn_prompt: the split into items, the dispatch over the element
// type, and the join of the items whose parts lie in several CTAs' shares
// (prompt_plan.cuh has the split, prompt_attn_{tc,f32} the main kernels).
#include <cuda_bf16.h>

#include "attn_scores.cuh"
#include "prompt_attn.h"
#include "sptp.h"

namespace sptp {

namespace {

// m = max m_k,  out = sum e^(m_k - m) o_k / sum e^(m_k - m) l_k  over the parts
// k of a row, in their order.
//
// Blocks kJoinBlocks c .. are CTA c's counterparts; an item of n parts is joined
// by those of its n CTAs, which take its rows in turn, so that one long item
// (many parts) and many short ones spread over the SMs.  A warp joins a row, or,
// since the loads of what other SMs have just written take about a microsecond
// each, the eight warps of a block share one of more than kAlone parts, their
// sums added in order.  The last block sums up the CTAs' status words.
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocks = 8;
constexpr int kAlone = 16;
constexpr int kBatch = 4;  // parts whose loads a lane has in flight

__device__ __forceinline__ void add_scaled(float4& a, float f, const float4& v) {
    a.x = fmaf(f, v.x, a.x);
    a.y = fmaf(f, v.y, a.y);
    a.z = fmaf(f, v.z, a.z);
    a.w = fmaf(f, v.w, a.w);
}

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) prompt_join(const __grid_constant__ PromptParams p, int ctas) {
    __shared__ float4 sums[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    admit_next();
    await_previous();
    if (blockIdx.x == ctas * kJoinBlocks) {
        // the first CTA that failed; if none did, the first that met an index outside its range
        __shared__ int first_bad, first_failed;
        if (threadIdx.x == 0) first_bad = first_failed = ctas;
        __syncthreads();
        for (int c = threadIdx.x; c < ctas; c += kJoinWarps * 32) {
            const int status = p.parts[c].status;
            if (status != 0) atomicMin(&first_bad, c);
            if (status != 0 && status != SPTP_ERR_SHAPE) atomicMin(&first_failed, c);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            DeviceStatus st = {0, 0, 0, 0, 0};
            const int at = first_failed < ctas ? first_failed : first_bad;
            if (at < ctas) {
                st.code = p.parts[at].status;
                st.where = p.parts[at].where;
                st.block = at;
                st.info = p.parts[at].info;
            }
            *p.status = st;
        }
        return;
    }
    const int c = blockIdx.x / kJoinBlocks;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const PromptItem it = p.parts[c].items[which];
        const int n = it.parts;
        if (n < 2 || it.first < 0 || it.first + n > ctas) continue;
        const int rows = it.tokens * it.heads;
        const bool shared = n > kAlone;
        const int sub = shared ? warp : 0, ways = shared ? kJoinWarps : 1;
        const int first = (c - it.first) * kJoinBlocks + blockIdx.x % kJoinBlocks, step = n * kJoinBlocks;
#pragma unroll 1
        for (int r0 = first; r0 < rows; r0 += shared ? step : step * kJoinWarps) {
            const int row = shared ? r0 : r0 + warp * step;
            const bool mine = row < rows;
            // part k: slot 0 of share first + k; the first: slot 1
            const long long base = 2ll * it.first * p.part_rows + row;
            auto slot = [&](int k) { return base + max(2 * k, 1) * static_cast<long long>(p.part_rows); };
            float top = -INFINITY, sum = 0.f;
            if (mine) {
                for (int k = lane; k < n; k += 32) top = fmaxf(top, p.part_ml[slot(k)].x);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                if (top == -INFINITY) top = 0.f;
                for (int k = lane; k < n; k += 32) {
                    const float2 r = p.part_ml[slot(k)];
                    sum = fmaf(pow2_approx(r.x - top), r.y, sum);
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const long long orow = (it.token0 + row / it.heads) * p.Hq + it.head0 + row % it.heads;
            if (p.lse != nullptr && mine && lane == 0 && sub == 0)
                p.lse[orow] = sum == 0.f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
#pragma unroll 1
            for (int d0 = 0; d0 < p.D; d0 += 128) {
                const int d = d0 + lane * 4;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                if (mine && d < p.D) {
#pragma unroll 1
                    for (int k0 = sub; k0 < n; k0 += kBatch * ways) {
                        float4 v[kBatch];
                        float m[kBatch];
#pragma unroll
                        for (int u = 0; u < kBatch; ++u) {
                            const int k = k0 + u * ways;
                            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                            m[u] = -INFINITY;
                            if (k < n) {
                                m[u] = p.part_ml[slot(k)].x;
                                v[u] = *reinterpret_cast<const float4*>(p.part_o + slot(k) * p.D + d);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < kBatch; ++u) {
                            // in two factors: a part far below the top may have values that are as much larger
                            const float f = pow2_approx(0.5f * (m[u] - top));
                            add_scaled(acc, f, make_float4(f * v[u].x, f * v[u].y, f * v[u].z, f * v[u].w));
                        }
                    }
                }
                if (shared) {
                    sums[warp][lane] = acc;
                    __syncthreads();
                    if (warp == 0)
                        for (int w = 1; w < kJoinWarps; ++w) add_scaled(acc, 1.f, sums[w][lane]);
                    __syncthreads();
                }
                if (!mine || sub != 0 || d >= p.D) continue;
                T* out = static_cast<T*>(p.out) + orow * p.D + d;
                if constexpr (sizeof(T) == 2) {
                    reinterpret_cast<__nv_bfloat162*>(out)[0] = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
                    reinterpret_cast<__nv_bfloat162*>(out)[1] = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                } else {
                    *reinterpret_cast<float4*>(out) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                }
            }
        }
    }
}

}  // namespace

void plan_prompt(PromptParams& p, int rows, int tile_rows) {
    const int group = p.Hq / p.Hkv;
    p.head_blocks = (group + tile_rows - 1) / tile_rows;
    p.heads = (group + p.head_blocks - 1) / p.head_blocks;
    p.head_blocks = (group + p.heads - 1) / p.heads;
    p.tokens = tile_rows / p.heads * (rows / tile_rows);
    p.items_per_block = p.P * p.Hkv * p.head_blocks;
    // division by the page size: with 2^(l-1) < d <= 2^l and mul = floor(2^(31+l) / d) + 1, the error
    // mul - 2^(31+l) / d <= 1 adds less than key / 2^(31+l) < 1 / d to the quotient
    int l = 0;
    while ((1ll << l) < p.page_size) ++l;
    p.page_mul = static_cast<uint32_t>((1ull << (31 + l)) / static_cast<uint32_t>(p.page_size) + 1);
    p.page_shift = l - 1;
}

int prompt_grid(const PromptParams& p, int most, int tk) {
    const long long span = static_cast<long long>(p.max_pages) * p.page_size;
    const long long blocks = p.M / p.tokens + static_cast<long long>(p.B < p.M ? p.B : p.M);
    const long long tiles = (span + tk - 1) / tk;
    const long long all = blocks >= most ? most : tiles * blocks * p.items_per_block;
    const long long n = all < most ? all : most;
    return static_cast<int>(n < kPromptMaxCtas ? n : kPromptMaxCtas);
}

cudaError_t launch_prompt_attn(PromptParams& p, bool bf16, bool e4m3, int num_sms, cudaStream_t s) {
    int ctas = 0;
    // (the plain kernels find a row's maximum among unscaled scores; those with a bias
    // take slopes of 0 where there are none)
    static PromptLaunch* const kernels[2][2][2] = {
        {{launch_prompt_bf16, launch_prompt_bf16_bias}, {launch_prompt_bf16_cap, launch_prompt_bf16_cap_bias}},
        {{launch_prompt_e4m3, launch_prompt_e4m3_bias}, {launch_prompt_e4m3_cap, launch_prompt_e4m3_cap_bias}}};
    const bool cap = p.cap != 0.f, bias = p.slopes != nullptr || (!cap && !(p.scale > 0.f));
    cudaError_t e = p.withhold_full >= 0 ? launch_prompt_test(p, e4m3, &ctas, s)
                                         : (bf16 ? kernels[e4m3][cap][bias] : launch_prompt_f32)(p, num_sms, &ctas, s);
    if (e != cudaSuccess) return e;
    const int grid = ctas * kJoinBlocks + 1;
    return bf16 ? launch_after(prompt_join<__nv_bfloat16>, grid, kJoinWarps * 32, 0, s, p, ctas)
                : launch_after(prompt_join<float>, grid, kJoinWarps * 32, 0, s, p, ctas);
}

}  // namespace sptp
