// The attention of sptp_paged_attn_prompt in fp32 on the CUDA cores:
//     s_j = cap tanh(scale q.k_j / cap) - slope |pos - j|,
//     out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
// for 64 query rows and 64 keys at a time, one pass over the keys with a running
// maximum and sum per row.  A thread holds 4 rows x 4 keys of the scores and 4
// rows x DP / 16 elements of the outputs; queries, keys, values and weights lie
// in shared memory, the next tile's keys and values on their way there while this
// one's are used (rows of more than 128 elements: no room for two tiles).
#include <atomic>

#include "attn_scores.cuh"
#include "prompt_plan.cuh"
#include "sptp.h"

namespace sptp {
namespace prompt {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;
constexpr int kItemCost = kTileCost;

template <int DP>
struct F32Smem {
    static constexpr int QS = DP + 4, KS = DP + 4, VS = DP, WS = kKeys + 4;  // row strides, floats
    static constexpr int BUFFERS = DP <= 128 ? 2 : 1, BUFFER = kKeys * (KS + VS);
    static constexpr int Q = 0, W = Q + kRows * QS, K = W + kRows * WS;
    static constexpr int BYTES = (K + BUFFERS * BUFFER) * 4;
    static constexpr int CTAS = BYTES <= 113 * 1024 ? 2 : 1;
};

template <int DP>
__global__ void __launch_bounds__(kThreads, F32Smem<DP>::CTAS) prompt_f32_kernel(const __grid_constant__ PromptParams p) {
    using L = F32Smem<DP>;
    constexpr int NV = DP / 64;  // float4 of a row's outputs per thread
    extern __shared__ __align__(16) float smem[];
    float *sq = smem + L::Q, *sw = smem + L::W;
    __shared__ long long warp_cost[kThreads / 32];
    __shared__ Cursor<kKeys, kItemCost> share_at;
    __shared__ int bad_at, bad_any;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    admit_next();
    if (tid == 0) bad_at = bad_any = 0;
    await_previous();
    bool bad = false;
    const Share share = find_share<kThreads>(p, warp_cost, &share_at, &bad);
    if (bad) bad_any = 1;
    PromptPart* part = p.parts + blockIdx.x;
    if (tid == 0) part->items[0].parts = part->items[1].parts = 0;
    const long long numbers = block_numbers(p);
    const ScoreCap cap(p.cap);
    const float to_log2 = p.scale * kLog2e;
    Cursor<kKeys, kItemCost> c = share_at;
    bool more = c.k.tiles != 0;
    while (more && c.tile_at() < share.end) {
        const Piece r = piece_of(p, c, share);
        const int rows = c.k.n * r.heads;
        const int q_stride = p.Hq * p.D;
        // queries: row = token * heads + head
        for (int i = tid; i < kRows * (DP / 4); i += kThreads) {
            const int row = i / (DP / 4), d = i % (DP / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < rows && d < p.D)
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + (r.token0 + row / r.heads) * q_stride +
                                                     (r.head0 + row % r.heads) * p.D + d);
            *reinterpret_cast<float4*>(sq + row * L::QS + d) = v;
        }
        int lo[4], hi[4], pos[4];
        float slope[4], m[4], l[4];
        float4 o[4][NV];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = ty * 4 + i, h = row % r.heads;
            pos[i] = c.k.pos0 + row / r.heads;
            const bool in = row < rows;
            lo[i] = in ? first_key(p, pos[i]) : 0;
            hi[i] = in ? min(c.k.len, end_key(pos[i], c.k.prefix)) : 0;
            slope[i] = p.slopes != nullptr && in ? __ldg(p.slopes + r.shard * p.Hq + r.head0 + h) * kLog2e : 0.f;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n) o[i][n] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // keys and values of tile t, zeros where no row sees one
        auto load = [&](int t) {
            const int key0 = c.key0() + t * kKeys;
            const int from = max(0, c.k.lo - key0), to = min(kKeys, c.k.hi - key0);
            float *sk = smem + L::K + t % L::BUFFERS * L::BUFFER, *sv = sk + kKeys * L::KS;
            constexpr int PER = kThreads / kKeys;  // threads of a key
            const int key = tid / PER;
            long long row = -1;
            if (key >= from && key < to) {
                row = pool_row(p, c.k.b, r.shard, r.kvh, key0 + key);
                if (row < 0) {
                    bad_any = 1;
                    bad_at = c.k.b;
                }
            }
            const float* k = static_cast<const float*>(p.k) + max(row, 0ll) * p.D;
            const float* v = static_cast<const float*>(p.v) + max(row, 0ll) * p.D;
#pragma unroll 4
            for (int d = tid % PER * 4; d < DP; d += PER * 4) {
                const bool has = row >= 0 && d < p.D;
                copy16_or_zero(sk + key * L::KS + d, has ? k + d : k, has);
                copy16_or_zero(sv + key * L::VS + d, has ? v + d : v, has);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if (r.here > 0) load(0);
        for (int t = 0; t < r.here; ++t) {
            const int key0 = c.key0() + t * kKeys;
            const int from = max(0, c.k.lo - key0), to = min(kKeys, c.k.hi - key0);  // keys that some row sees
            const float *sk = smem + L::K + t % L::BUFFERS * L::BUFFER, *sv = sk + kKeys * L::KS;
            if (L::BUFFERS == 2 && t + 1 < r.here) {
                load(t + 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
            float s[4][4] = {};
#pragma unroll 4
            for (int d = 0; d < DP; d += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (ty * 4 + i) * L::QS + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * L::KS + d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] += a[i].x * b[j].x + a[i].y * b[j].y + a[i].z * b[j].z + a[i].w * b[j].w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + tx + 16 * j;
                    float x = s[i][j] * to_log2;
                    if (p.cap != 0.f) x = cap.cap * tanhf(x * cap.inv);
                    if (p.slopes != nullptr) x -= slope[i] * static_cast<float>(abs(pos[i] - key));
                    s[i][j] = key >= lo[i] && key < hi[i] ? x : -INFINITY;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float base = top == -INFINITY ? 0.f : top;
                const float old = pow2_approx(m[i] - base);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w = pow2_approx(s[i][j] - base);
                    sum += w;
                    sw[(ty * 4 + i) * L::WS + tx + 16 * j] = w;
                }
                l[i] = l[i] * old + sum;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    o[i][n].x *= old;
                    o[i][n].y *= old;
                    o[i][n].z *= old;
                    o[i][n].w *= old;
                }
            }
            __syncwarp();  // the weights of a warp's 8 rows are its own
            for (int k = from & ~3; k < to; k += 4) {
                float4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(sw + (ty * 4 + i) * L::WS + k);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        const float4 v = *reinterpret_cast<const float4*>(sv + (k + kk) * L::VS + n * 64 + tx * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float f = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
                            o[i][n].x = fmaf(f, v.x, o[i][n].x);
                            o[i][n].y = fmaf(f, v.y, o[i][n].y);
                            o[i][n].z = fmaf(f, v.z, o[i][n].z);
                            o[i][n].w = fmaf(f, v.w, o[i][n].w);
                        }
                    }
            }
            __syncthreads();
            if (L::BUFFERS == 1 && t + 1 < r.here) load(t + 1);
        }
        const bool whole = r.begins && r.ends;
        if (tid == 0 && !whole) part->items[r.begins ? 1 : 0] = split_item(c, r, share);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = ty * 4 + i;
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
            if (row >= rows) continue;
            float* to;
            float f = 1.f;
            if (whole) {
                const long long orow = (r.token0 + row / r.heads) * p.Hq + r.head0 + row % r.heads;
                f = l[i] == 0.f ? 0.f : 1.f / l[i];
                to = static_cast<float*>(p.out) + orow * p.D;
                if (p.lse != nullptr && tx == 0)
                    p.lse[orow] = l[i] == 0.f ? -INFINITY : m[i] * 0.6931471805599453f + logf(l[i]);
            } else {
                // slot 1 if the item begins in this share, slot 0 if in an earlier one
                const long long at = (blockIdx.x * 2ll + (r.begins ? 1 : 0)) * p.part_rows + row;
                if (tx == 0) p.part_ml[at] = make_float2(m[i], l[i]);
                to = p.part_o + at * p.D;
            }
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int d = n * 64 + tx * 4;
                if (d < p.D)
                    *reinterpret_cast<float4*>(to + d) = make_float4(o[i][n].x * f, o[i][n].y * f, o[i][n].z * f, o[i][n].w * f);
            }
        }
        __syncthreads();
        more = c.next_item(p, numbers);
    }
    __syncthreads();
    if (tid == 0) {
        part->status = bad_any ? SPTP_ERR_SHAPE : 0;
        part->where = bad_any ? kWhereKvPage : 0;
        part->info = bad_at;
    }
}

template <int DP>
cudaError_t launch_one(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(prompt_f32_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, F32Smem<DP>::BYTES);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    *ctas = prompt_grid(p, num_sms * F32Smem<DP>::CTAS, kKeys);
    return launch_after(prompt_f32_kernel<DP>, *ctas, kThreads, F32Smem<DP>::BYTES, s, p);
}

}  // namespace
}  // namespace prompt

cudaError_t launch_prompt_f32(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    using namespace prompt;
    plan_prompt(p, kRows, kRows);
    if (p.D <= 64) return launch_one<64>(p, num_sms, ctas, s);
    if (p.D <= 128) return launch_one<128>(p, num_sms, ctas, s);
    return launch_one<256>(p, num_sms, ctas, s);
}

}  // namespace sptp
