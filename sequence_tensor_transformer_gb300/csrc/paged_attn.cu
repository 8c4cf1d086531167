// The paged attention's dispatch over the cache's element type, and the join of
// the items that were split over several CTAs (paged_attn.cuh has the main
// kernel).
#include <cuda_bf16.h>

#include "attn.h"
#include "sptp.h"
#include "sptp_ptx.cuh"

namespace sptp {

namespace {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The join of the items whose parts lie in several shares:  m = max m_k,  out =
// sum e^(m_k - m) o_k / sum e^(m_k - m) l_k  over the parts k.
//
// Block c is CTA c's counterpart, one half of it for each of the (at most) two
// such items that the share has a part of.  An item of n parts is joined by
// the n halves of its shares, which take its slices (64 elements of one head)
// in turn, so that one long row (few items, many parts) and many short ones
// (many items, two parts) both spread over the SMs.
//
// Bound by latency: a load of what another SM has just written takes about a
// microsecond.  So a warp reads its parts of a slice in one batch, beside the
// maxima, and `ways` warps share a slice of more than kBatch parts; their sums
// are added in order.  The last block sums up the CTAs' status words.
constexpr int kHalf = 8;   // warps
constexpr int kJoinThreads = 2 * kHalf * 32;
constexpr int kBatch = 8;  // parts whose loads a warp has in flight

template <typename T>
__global__ void __launch_bounds__(kJoinThreads, 2) paged_attn_join(const __grid_constant__ PagedAttnParams p, int ctas,
                                                               int head_shift) {
    __shared__ float2 sums[2][kHalf][32];
    __shared__ int first_bad, first_failed;
    const int tid = threadIdx.x, lane = tid & 31, c = blockIdx.x;
    admit_next();
    await_previous();
    if (c == ctas) {
        // the first CTA that failed; if none did, the first that met an
        // index outside its range
        if (tid == 0) first_bad = first_failed = ctas;
        __syncthreads();
        const int mine = tid < ctas ? p.parts[tid].status : 0;
        if (mine != 0) atomicMin(&first_bad, tid);
        if (mine != 0 && mine != SPTP_ERR_SHAPE) atomicMin(&first_failed, tid);
        __syncthreads();
        if (tid == 0) {
            DeviceStatus st = {0, 0, 0, 0, 0};
            const int at = first_failed < ctas ? first_failed : first_bad;
            if (at < ctas) {
                const PagedAttnPart& bad = p.parts[at];
                st.code = bad.status;
                st.where = bad.where;
                st.block = at;
                st.info = bad.info;
            }
            *p.status = st;
        }
        return;
    }
    const int which = tid / (kHalf * 32), warp = tid / 32 % kHalf;
    const PagedAttnItem it = p.parts[c].items[which];
    const int n = it.parts;
    if (n < 2 || it.first < 0 || it.first + n > ctas) return;
    const int way_shift = n <= kBatch ? 0 : n <= 4 * kBatch ? 2 : 3, ways = 1 << way_shift;
    const int side_by_side = kHalf >> way_shift;  // slices that the half works on at a time
    const int sub = warp & (ways - 1);
    const int slices = it.heads << head_shift;
#pragma unroll 1
    for (int s0 = c - it.first; s0 < slices; s0 += n * side_by_side) {
        const int s = s0 + n * (warp >> way_shift);
        const int h = s >> head_shift, d = ((s & ((1 << head_shift) - 1)) * 64) + lane * 2;
        const bool mine = s < slices;
        float top = -INFINITY, sum = 0.f;
        float2 acc = make_float2(0.f, 0.f);
        if (mine) {
            // part k: slot 0 of share first + k; the first part: slot 1
            const float2* ml = p.part_ml + 2ll * it.first * p.heads_per_item + h;
            const float* o = p.part_o + (2ll * it.first * p.heads_per_item + h) * p.D + d;
#pragma unroll 1
            for (int b = sub; b < n; b += kBatch * ways) {
                float2 v[kBatch];
                float m[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int k = b + u * ways;
                    const int row = max(2 * k, 1) * p.heads_per_item;
                    v[u] = make_float2(0.f, 0.f);
                    m[u] = -INFINITY;
                    if (k < n) {
                        m[u] = ml[row].x;
                        if (d < p.D) v[u] = *reinterpret_cast<const float2*>(o + static_cast<long long>(row) * p.D);
                    }
                }
                if (b == sub) {  // the statistics, while these loads are under way
                    constexpr int kTurns = 3;
                    float2 q[kTurns];
#pragma unroll
                    for (int t = 0; t < kTurns; ++t) {
                        const int k = t * 32 + lane;
                        q[t] = make_float2(-INFINITY, 0.f);
                        if (k < n) q[t] = ml[max(2 * k, 1) * p.heads_per_item];
                    }
#pragma unroll
                    for (int t = 0; t < kTurns; ++t) top = fmaxf(top, q[t].x);
#pragma unroll 1
                    for (int k = kTurns * 32 + lane; k < n; k += 32) top = fmaxf(top, ml[2 * k * p.heads_per_item].x);
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    if (top == -INFINITY) top = 0.f;
#pragma unroll
                    for (int t = 0; t < kTurns; ++t) sum = fmaf(ex2(q[t].x - top), q[t].y, sum);
#pragma unroll 1
                    for (int k = kTurns * 32 + lane; k < n; k += 32) {
                        const float2 r = ml[2 * k * p.heads_per_item];
                        sum = fmaf(ex2(r.x - top), r.y, sum);
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    // in two factors: a part far below the top may have
                    // values that are as much larger, and 2^-126 is the least factor
                    const float f = ex2(0.5f * (m[u] - top));
                    acc.x = fmaf(f, f * v[u].x, acc.x);
                    acc.y = fmaf(f, f * v[u].y, acc.y);
                }
            }
        }
        if (ways > 1) {
            auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + which), "n"(kHalf * 32) : "memory"); };
            sums[which][warp][lane] = acc;
            sync();
            if (sub == 0)
                for (int w = 1; w < ways; ++w) {
                    acc.x += sums[which][warp + w][lane].x;
                    acc.y += sums[which][warp + w][lane].y;
                }
            sync();
        }
        if (!mine || sub != 0 || d >= p.D) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        T* out = static_cast<T*>(p.out) + (it.qrow + h) * p.D + d;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        else
            *reinterpret_cast<float2*>(out) = make_float2(acc.x * inv, acc.y * inv);
        if (p.lse != nullptr && d == 0)
            p.lse[it.qrow + h] = sum == 0.f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
    }
}
static_assert(kJoinThreads >= kPagedMaxCtas, "one thread per status word");

}  // namespace

cudaError_t launch_paged_attn(PagedAttnParams& p, bool bf16, bool e4m3, int num_sms, cudaStream_t s) {
    if (e4m3 && !bf16) return cudaErrorInvalidValue;
    int ctas = 0;
    const bool test = p.withhold_full >= 0 || p.withhold_empty >= 0;
    cudaError_t e = test    ? launch_paged_attn_test(p, bf16, e4m3, &ctas, s)
                    : !bf16 ? launch_paged_attn_f32(p, num_sms, &ctas, s)
                    : e4m3  ? launch_paged_attn_e4m3(p, num_sms, &ctas, s)
                            : launch_paged_attn_bf16(p, num_sms, &ctas, s);
    if (e != cudaSuccess) return e;
    const int head_shift = p.D <= 64 ? 0 : p.D <= 128 ? 1 : 2;  // slices of a head: 1, 2 or 4
    return bf16 ? launch_after(paged_attn_join<__nv_bfloat16>, ctas + 1, kJoinThreads, 0, s, p, ctas, head_shift)
                : launch_after(paged_attn_join<float>, ctas + 1, kJoinThreads, 0, s, p, ctas, head_shift);
}

}  // namespace sptp
