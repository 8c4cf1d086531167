// The attention of sptp_paged_attn_prompt in fp32 on the CUDA cores:
//     s_j = cap tanh(scale q.k_j / cap) - slope |pos - j|,
//     out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
// for 64 query rows and 64 keys at a time, one pass over the keys with a running
// maximum and sum per row.  A thread holds 4 rows x 4 keys of the scores and 4
// rows x DP / 16 elements of the outputs; queries, keys, values and weights lie
// in shared memory, the next tile's keys and values on their way there while this
// one's are used (rows of more than 128 elements: no room for two tiles).
//
// What bounds it are the loads from shared memory: 16 bytes for each lane of a warp
// take 4 clocks, so the 8 loads for a thread's 4 x 4 products of 4 elements take 32
// clocks of the SM and the products 16.  8 x 4 (48 for 32) leaves 8 warps an SM, which
// wait for one another: 319 us instead of 305 for 2500 causal capped rows of 2 shards,
// 8 heads of 64 on 2, and 4.29 ms instead of 4.33 behind 20000 cached keys (36 TFLOP/s).
#include <atomic>
#include <type_traits>

#include "attn_scores.cuh"
#include "prompt_plan.cuh"
#include "sptp.h"

namespace sptp {
namespace prompt {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;
constexpr int R = 4, STEP = kRows / R;  // rows of a thread: ty + STEP i
constexpr int kItemCost = kTileCost;

template <int DP>
struct F32Smem {
    static constexpr int QS = DP + 4, KS = DP + 4, VS = DP, WS = kKeys + 4;  // row strides, floats
    static constexpr int BUFFERS = DP <= 128 ? 2 : 1, BUFFER = kKeys * (KS + VS);
    static constexpr int Q = 0, W = Q + kRows * QS, K = W + kRows * WS;
    static constexpr int BYTES = (K + BUFFERS * BUFFER) * 4;
    static constexpr int CTAS = BYTES <= 113 * 1024 ? 2 : 1;
};

struct __align__(16) RowMask {
    int lo, hi, pos;  // first and last key + 1 that the row sees, and its position
    float slope;      // in units of log 2
};

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float low(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a)); }
__device__ __forceinline__ float high(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a >> 32)); }

template <int DP>
__global__ void __launch_bounds__(kThreads, F32Smem<DP>::CTAS) prompt_f32_kernel(const __grid_constant__ PromptParams p) {
    using L = F32Smem<DP>;
    constexpr int NV = DP / 64;  // float4 of a row's outputs per thread
    extern __shared__ __align__(16) float smem[];
    float *sq = smem + L::Q, *sw = smem + L::W;
    __shared__ long long warp_cost[kThreads / 32];
    __shared__ Cursor<kKeys, kItemCost> share_at;
    __shared__ int bad_at, bad_any;
    __shared__ RowMask masks[kRows];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    admit_next();
    if (tid == 0) bad_at = bad_any = 0;
    await_previous();
    const Share share = find_share<kThreads>(p, warp_cost, &share_at);
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
        if (tid < kRows) {
            const int h = tid % r.heads, pos = c.k.pos0 + tid / r.heads;
            const bool in = tid < rows;
            RowMask k;
            k.pos = pos;
            k.lo = in ? first_key(p, pos) : 0;
            k.hi = in ? min(c.k.len, end_key(pos, c.k.prefix)) : 0;
            k.slope = p.slopes != nullptr && in ? __ldg(p.slopes + r.shard * p.Hq + r.head0 + h) * kLog2e : 0.f;
            masks[tid] = k;
        }
        float m[R], l[R];
        uint64_t o[R][NV][2];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n) o[i][n][0] = o[i][n][1] = 0;
        }
        const int all_lo = first_key(p, c.k.pos0 + c.k.n - 1), all_hi = end_key(c.k.pos0, c.k.prefix);  // every row sees
        // keys and values of tile t, zeros where no row sees one
        auto load = [&](int t) {
            const int key0 = c.key0() + t * kKeys;
            const int from = max(0, c.k.lo - key0), to = min(kKeys, c.k.hi - key0);
            float *sk = smem + L::K + t % L::BUFFERS * L::BUFFER, *sv = sk + kKeys * L::KS;
            // a warp's keys: their rows looked up by a lane each, copied by the row
            constexpr int KEYS = kKeys / (kThreads / 32), LANES = DP / 4 < 32 ? DP / 4 : 32;
            const int lane = tid & 31, first = tid / 32 * KEYS;
            long long mine = -1;
            if (lane < KEYS && first + lane >= from && first + lane < to) {
                mine = pool_row(p, c.k.b, r.shard, r.kvh, key0 + first + lane);
                if (mine < 0) {
                    bad_any = 1;
                    bad_at = c.k.b;
                }
            }
#pragma unroll
            for (int i = 0; i < KEYS; i += 32 / LANES) {
                const int j = i + lane / LANES, key = first + j;
                const long long row = __shfl_sync(0xffffffffu, mine, j);
                const float* k = static_cast<const float*>(p.k) + max(row, 0ll) * p.D;
                const float* v = static_cast<const float*>(p.v) + max(row, 0ll) * p.D;
#pragma unroll
                for (int d = lane % LANES * 4; d < DP; d += LANES * 4) {
                    const bool has = row >= 0 && d < p.D;
                    copy16_or_zero(sk + key * L::KS + d, has ? k + d : k, has);
                    copy16_or_zero(sv + key * L::VS + d, has ? v + d : v, has);
                }
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
            // elements d, d + 2 .. and d + 1, d + 3 .. of the products apart: packed arithmetic
            uint64_t s[R][4] = {};
#pragma unroll 4
            for (int d = 0; d < DP; d += 4) {
                ulonglong2 b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 16 * j) * L::KS + d);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(sq + (ty + STEP * i) * L::QS + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = fma2(a.y, b[j].y, fma2(a.x, b[j].x, s[i][j]));
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const RowMask k = masks[ty + STEP * i];
                float x[4], top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + tx + 16 * j;
                    x[j] = (low(s[i][j]) + high(s[i][j])) * to_log2;
                    if (p.cap != 0.f) x[j] = cap.cap * tanhf(x[j] * cap.inv);
                    if (p.slopes != nullptr) x[j] -= k.slope * static_cast<float>(abs(k.pos - key));
                    x[j] = key >= k.lo && key < k.hi ? x[j] : -INFINITY;
                    top = fmaxf(top, x[j]);
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float base = top == -INFINITY ? 0.f : top;
                const float old = pow2_approx(m[i] - base);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w = pow2_approx(x[j] - base);
                    sum += w;
                    sw[(ty + STEP * i) * L::WS + tx + 16 * j] = w;
                }
                l[i] = l[i] * old + sum;
                const uint64_t f = pack2(old, old);
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    o[i][n][0] = mul2(o[i][n][0], f);
                    o[i][n][1] = mul2(o[i][n][1], f);
                }
            }
            __syncwarp();  // the weights of a warp's rows are its own
            auto add_values = [&](auto masked) {
                constexpr bool MASKED = decltype(masked)::value;
                for (int k = from & ~3; k < to; k += 4) {
                    ulonglong2 v[4][NV];
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int n = 0; n < NV; ++n)
                            v[kk][n] = *reinterpret_cast<const ulonglong2*>(sv + (k + kk) * L::VS + n * 64 + tx * 4);
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float4 w = *reinterpret_cast<const float4*>(sw + (ty + STEP * i) * L::WS + k);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const float f = kk == 0 ? w.x : kk == 1 ? w.y : kk == 2 ? w.z : w.w;
                            const uint64_t ff = pack2(f, f);
#pragma unroll
                            for (int n = 0; n < NV; ++n) {
                                // (0 times what a row does not see need not be 0)
                                if (MASKED && f == 0.f) continue;
                                o[i][n][0] = fma2(ff, v[kk][n].x, o[i][n][0]);
                                o[i][n][1] = fma2(ff, v[kk][n].y, o[i][n][1]);
                            }
                        }
                    }
                }
            };
            if (key0 < all_lo || key0 + kKeys > all_hi)
                add_values(std::true_type());
            else
                add_values(std::false_type());
            __syncthreads();
            if (L::BUFFERS == 1 && t + 1 < r.here) load(t + 1);
        }
        const bool whole = r.begins && r.ends;
        if (tid == 0 && !whole) part->items[r.begins ? 1 : 0] = split_item(c, r, share);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = ty + STEP * i;
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
                    *reinterpret_cast<float4*>(to + d) = make_float4(low(o[i][n][0]) * f, high(o[i][n][0]) * f,
                                                                           low(o[i][n][1]) * f, high(o[i][n][1]) * f);
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
