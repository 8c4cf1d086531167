// sptp_paged_attn_prompt: the split into items, the dispatch over the element
// type, and the join of the items whose parts lie in several CTAs' shares
// (prompt_plan.cuh has the split, prompt_attn_{tc,f32} the main kernels).
#include <cuda_bf16.h>

#include <type_traits>

#include "attn_scores.cuh"
#include "prompt_attn.h"
#include "sptp.h"

namespace sptp {

namespace {

// m = max m_k,  out = sum e^(m_k - m) o_k / sum e^(m_k - m) l_k  over the parts
// k of a row, in their order.
//
// Every part has an entry (its CTA and the slot there) and an entry kJoinBlocks
// blocks, which all join the entry's item and take its rows in turn, so that one long
// item (many parts) and many short ones spread over the SMs.  The loads of what other
// SMs have just written take about a microsecond each: a warp has the parts of four
// rows of two parts under way at once, or of two of up to kFew; a row of more is a warp's, or, of more
// than kAlone, the eight warps' of a block, their sums added in order.  The last block
// looks through the sequences' rows and lengths and sums up the CTAs' status words.
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocks = 4;
constexpr int kFew = 4;
constexpr int kAlone = 16;
constexpr int kBatch = 4;  // parts whose loads a lane has in flight

__device__ __forceinline__ void add_scaled(float4& a, float f, const float4& v) {
    a.x = fmaf(f, v.x, a.x);
    a.y = fmaf(f, v.y, a.y);
    a.z = fmaf(f, v.z, a.z);
    a.w = fmaf(f, v.w, a.w);
}

template <typename T>
__device__ __forceinline__ void store4(T* out, const float4& v) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(out) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
        *reinterpret_cast<float4*>(out) = v;
    }
}

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) prompt_join(const __grid_constant__ PromptParams p, int ctas) {
    __shared__ float4 sums[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    admit_next();
    await_previous();
    if (blockIdx.x == ctas * 2 * kJoinBlocks) {
        // the first CTA that failed; if none did, the first sequence whose rows or length are outside
        // their range (every one is looked at: the main kernel's numbers of blocks pass over
        // some where row starts descend), or the first CTA that met a page outside
        __shared__ int first_bad, first_failed, first_sequence;
        if (threadIdx.x == 0) {
            first_bad = first_failed = ctas;
            first_sequence = p.B;
        }
        __syncthreads();
        const int most = p.max_pages * p.page_size;
        for (int b = threadIdx.x; b < p.B; b += kJoinWarps * 32) {
            const int s = __ldg(p.row_starts + b), e = __ldg(p.row_starts + b + 1), len = __ldg(p.seq_lens + b);
            if (s < 0 || e > p.M || e < s || len < 0 || len > most || e - s > len) atomicMin(&first_sequence, b);
        }
        for (int c = threadIdx.x; c < ctas; c += kJoinWarps * 32) {
            const int status = p.parts[c].status;
            if (status != 0) atomicMin(&first_bad, c);
            if (status != 0 && status != SPTP_ERR_SHAPE) atomicMin(&first_failed, c);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            DeviceStatus st = {0, 0, 0, 0, 0};
            const int at = first_failed < ctas ? first_failed : first_bad;
            if (first_failed == ctas && first_sequence < p.B) {
                st.code = SPTP_ERR_SHAPE;
                st.where = kWhereKvPage;
                st.info = first_sequence;
            } else if (at < ctas) {
                st.code = p.parts[at].status;
                st.where = p.parts[at].where;
                st.block = at;
                st.info = p.parts[at].info;
            }
            *p.status = st;
        }
        return;
    }
    const int entry = blockIdx.x / kJoinBlocks, c = entry / 2;
    const PromptItem it = p.parts[c].items[entry % 2];
    const int n = it.parts;
    if (n < 2 || it.first < 0 || it.first + n > ctas) return;
    const int rows = it.tokens * it.heads;
    const int first = (c - it.first) * kJoinBlocks + blockIdx.x % kJoinBlocks, step = n * kJoinBlocks;
    // part k of a row: slot 0 of share first + k; the first: slot 1
    auto slot = [&](int row, int k) {
        return (2ll * it.first + max(2 * k, 1)) * p.part_rows + row;
    };
    auto out_row = [&](int row) { return (it.token0 + row / it.heads) * p.Hq + it.head0 + row % it.heads; };
    auto lse = [&](float top, float sum) { return sum == 0.f ? -INFINITY : top * 0.6931471805599453f + logf(sum); };
    // in two factors: a part far below the top may have values that are as much larger
    auto add_part = [](float4& acc, float m, float top, const float4& v) {
        const float f = pow2_approx(0.5f * (m - top));
        add_scaled(acc, f, make_float4(f * v.x, f * v.y, f * v.z, f * v.w));
    };
    // ROWS rows of up to PARTS parts, all their loads first
    auto few = [&](auto parts, auto at_once) {
        constexpr int PARTS = decltype(parts)::value, ROWS = decltype(at_once)::value;
#pragma unroll 1
        for (int r0 = first + warp * step; r0 < rows; r0 += ROWS * step * kJoinWarps) {
#pragma unroll 1
            for (int d = lane * 4; d < p.D; d += 128) {
                float2 ml[ROWS][PARTS];
                float4 v[ROWS][PARTS];
#pragma unroll
                for (int e = 0; e < ROWS; ++e) {
                    const int row = r0 + e * step * kJoinWarps;
                    const long long at = 2ll * it.first * p.part_rows + row;
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
                        const bool is = row < rows && k < n;
                        const long long s = at + max(2 * k, 1) * static_cast<long long>(p.part_rows);
                        ml[e][k] = is ? p.part_ml[s] : make_float2(-INFINITY, 0.f);
                        v[e][k] = is ? *reinterpret_cast<const float4*>(p.part_o + s * p.D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
#pragma unroll
                for (int e = 0; e < ROWS; ++e) {
                    const int row = r0 + e * step * kJoinWarps;
                    if (row >= rows) break;
                    float top = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) top = fmaxf(top, ml[e][k].x);
                    if (top == -INFINITY) top = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
                        sum = fmaf(pow2_approx(ml[e][k].x - top), ml[e][k].y, sum);
                        add_part(acc, ml[e][k].x, top, v[e][k]);
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    const long long orow = out_row(row);
                    store4(static_cast<T*>(p.out) + orow * p.D + d,
                           make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
                    if (p.lse != nullptr && d == 0) p.lse[orow] = lse(top, sum);
                }
            }
        }
    };
    if (n <= 2) {
        few(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
        return;
    }
    if (n <= kFew) {
        few(std::integral_constant<int, kFew>(), std::integral_constant<int, 2>());
        return;
    }
    const bool shared = n > kAlone;
    const int sub = shared ? warp : 0, ways = shared ? kJoinWarps : 1;
#pragma unroll 1
    for (int r0 = first; r0 < rows; r0 += shared ? step : step * kJoinWarps) {
        const int row = shared ? r0 : r0 + warp * step;
        const bool mine = row < rows;
        float top = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int d0 = 0; d0 < p.D; d0 += 128) {
            const int d = d0 + lane * 4;
            const bool in = mine && d < p.D;
            float4 v[kBatch];
            float m[kBatch];
            auto load = [&](int k0) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int k = k0 + u * ways;
                    const bool is = in && k < n;
                    m[u] = is ? p.part_ml[slot(row, k)].x : -INFINITY;
                    v[u] = is ? *reinterpret_cast<const float4*>(p.part_o + slot(row, k) * p.D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            };
            load(sub);  // on its way while the maximum is found
            if (mine && d0 == 0) {
                for (int k = lane; k < n; k += 32) top = fmaxf(top, p.part_ml[slot(row, k)].x);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                if (top == -INFINITY) top = 0.f;
                for (int k = lane; k < n; k += 32) {
                    const float2 r = p.part_ml[slot(row, k)];
                    sum = fmaf(pow2_approx(r.x - top), r.y, sum);
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (p.lse != nullptr && lane == 0 && sub == 0) p.lse[out_row(row)] = lse(top, sum);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int k0 = sub; k0 < n; k0 += kBatch * ways) {
                if (k0 != sub) load(k0);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) add_part(acc, m[u], top, v[u]);
            }
            if (shared) {
                sums[warp][lane] = acc;
                __syncthreads();
                if (warp == 0)
                    for (int w = 1; w < kJoinWarps; ++w) add_scaled(acc, 1.f, sums[w][lane]);
                __syncthreads();
            }
            if (!in || sub != 0) continue;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            store4(static_cast<T*>(p.out) + out_row(row) * p.D + d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
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
    const int grid = ctas * 2 * kJoinBlocks + 1;
    return bf16 ? launch_after(prompt_join<__nv_bfloat16>, grid, kJoinWarps * 32, 0, s, p, ctas)
                : launch_after(prompt_join<float>, grid, kJoinWarps * 32, 0, s, p, ctas);
}

}  // namespace sptp
