// Attention of one token per sequence over a paged key-value cache:
//     s_j = scale q . k_j,  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),
// one pass over the keys with a running maximum m, sum l and output o; a new
// maximum m' scales l and o by e^(m - m').  (In the kernels: powers of two,
// scores in units of log 2.)
//
// Bound by HBM: every key and value is read once, 2 D bytes of a bf16 key for
// 4 D flops per query head.  What the layout is for is to keep the reads going
// on every SM whatever the lengths are:
//  - An item is one (sequence, shard, key/value head) with the query heads that
//    read it (more than kMaxHeads of them: several items).  Its keys are cut
//    into tiles of TK; the tiles of all items, in order, are dealt out to the
//    CTAs of one resident wave in equal contiguous shares.  Every CTA works
//    out its own share from the lengths, so nothing depends on the host
//    knowing them.  An item that crosses a share's end leaves its parts'
//    (m, l, o) in the workspace; a second launch (paged_attn_join) joins them in
//    a fixed order.
//  - One producer warp walks over the share and keeps a ring of tiles filled by
//    TMA (one box per page and 128 bytes of row), running ahead across item
//    borders, so that the reads never wait for the arithmetic of an item's end.
//  - Four consumer warps take a quarter of each tile's keys, each with
//    statistics of its own, and meet only where an item ends.
#pragma once

#include <cuda_bf16.h>

#include "sptp.h"
#include "sptp_ptx.cuh"

namespace sptp {
namespace paged {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kMaxStages = 8;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// c += A (16 x 16) B (16 x 8), bf16 operands, fp32 sums
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------- consumers
// A consumer class holds one warp's query fragments and statistics and has
//   TK, STAGES, CTAS, HEADS, DP        tile and launch shape
//   ROW_BYTES, BOXES, K_BYTES          a key's bytes, boxes per row, a stage's keys
//   begin(p, q row, heads)             a new item
//   tile(stage, lo, hi)                keys [lo, hi) of the stage's tile
//   stats(ms, ls), add(obuf)           at an item's end

// Tensor-core consumer for a bf16 or E4M3 cache, DP >= D elements per row, up
// to 8 NT query heads.
//
// Both products have the keys or the value's elements as the 16 rows of
// m16n8k16 and the query heads as its 8 columns, so that a group of up to 8
// heads wastes nothing:  S^T = K q^T  and  O^T = V^T W^T.  A thread then holds
// the scores, statistics and outputs of the same two heads throughout, and
// the weights go from one product to the other through a transpose within the
// warp (movmatrix), not through shared memory.
//
// E4M3: a code's 7 magnitude bits, moved into a bf16's exponent and mantissa,
// are the value times 2^-120, subnormal codes among them, so that a pair of
// codes becomes a pair of bf16 by two shifts and masks.  q carries 2^100 over
// its own exponent and the weights carry 2^100 over the largest v scale so
// far, so that no product comes near the ends of fp32's range; both powers of
// two leave with the score and at the item's end.  (Converting to fp16 instead
// would lose rows of v whose scales differ by more than fp16's range.)
template <int DP_, int NT_, bool CODES_>
struct TcConsumer {
    static constexpr int DP = DP_, NT = NT_;
    static constexpr bool CODES = CODES_;
    static constexpr bool F32 = false;
    static constexpr int HEADS = 8 * NT;
    static constexpr int ROW_BYTES = DP * (CODES ? 1 : 2);
    static constexpr int BOXES = ROW_BYTES / 128;
    // 32 KB a stage, or 64 keys where a row is wider
    static constexpr int TK = ROW_BYTES == 128 ? 128 : 64;
    static constexpr int K_BYTES = TK * ROW_BYTES;
    static constexpr int SCALE_BYTES = CODES ? TK * 4 : 0;
    static constexpr int STAGE_BYTES = 2 * K_BYTES;
    // two CTAs per SM where shared memory and registers allow
    static constexpr int CTAS =
        NT < 4 && STAGE_BYTES <= 32768 &&
                98304 + 6 * SCALE_BYTES + HEADS * (DP + 4) * 4 + 10 * HEADS * 4 + 2048 <= 113 * 1024
            ? 2
            : 1;
    static constexpr int STAGES = (CTAS == 2 ? 98304 : 196608) / STAGE_BYTES;
    static constexpr int SLICES = TK / (16 * kConsumers);
    static constexpr int KSTEPS = DP / 16;  // of 16 elements of q and k
    static constexpr int MTILES = DP / 16;  // of 16 elements of v
    static_assert(ROW_BYTES % 128 == 0 && STAGES >= 3 && STAGES <= kMaxStages, "layout");

    uint32_t qf[KSTEPS][NT][2];
    float m[NT][2], l[NT][2], qs[NT][2];
    float o[MTILES][NT][4];
    int vexp;  // E4M3: the exponent field that the weights are relative to

    static __device__ __forceinline__ uint32_t even_pair(uint32_t c) {
        const uint32_t t = c << 8;
        return (t & 0x80008000u) | ((c << 4) & 0x07f007f0u);
    }
    static __device__ __forceinline__ uint32_t odd_pair(uint32_t c) {
        return (c & 0x80008000u) | ((c >> 4) & 0x07f007f0u);
    }

    __device__ __forceinline__ void begin(const PagedAttnParams& p, long long qrow, int heads) {
        const int lane = threadIdx.x & 31, g = lane >> 2, i = lane & 3;
        const float to_log2 = p.scale * 1.4426950408889634f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + g;
            const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(p.q) + (qrow + h) * p.D;
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) {
                if constexpr (!CODES) {
                    const int d = k * 16 + i * 2;
                    qf[k][nt][0] = h < heads && d < p.D ? __ldg(reinterpret_cast<const uint32_t*>(row + d)) : 0u;
                    qf[k][nt][1] = h < heads && d + 8 < p.D ? __ldg(reinterpret_cast<const uint32_t*>(row + d + 8)) : 0u;
                } else {
                    // elements 4i .. 4i+3 of the step, even ones and odd ones
                    const int d = k * 16 + i * 4;
                    uint2 u = make_uint2(0, 0);
                    if (h < heads && d < p.D) u = __ldg(reinterpret_cast<const uint2*>(row + d));
                    qf[k][nt][0] = __byte_perm(u.x, u.y, 0x5410);
                    qf[k][nt][1] = __byte_perm(u.x, u.y, 0x7632);
                }
            }
            if constexpr (CODES) {
                // |q| of the row below 2^(e+1); q * 2^(100 - e) is exact but for
                // elements 2^-226 of the largest
                __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&qf[k][nt][r])));
                float amax = fmaxf(__low2float(top), __high2float(top));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const int e = max(static_cast<int>(__float_as_uint(amax) >> 23), 1) - 127;
                // 2^(100 - e) in two factors, each within bf16's range
                const float up = __uint_as_float(static_cast<uint32_t>(127 + 100 - max(e, -26)) << 23);
                const float up2 = e < -26 ? __uint_as_float(static_cast<uint32_t>(127 - 26 - e) << 23) : 1.f;
#pragma unroll
                for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[k][nt][r]));
                        qf[k][nt][r] = pack_bf16(f.x * up2 * up, f.y * up2 * up);
                    }
                // the score's factor of this row: scale 2^(e - 100 + 120)
                const float back = __uint_as_float(static_cast<uint32_t>(min(127 + e + 20, 254)) << 23);
                const float f = to_log2 * back;
                qs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * i);
                qs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * i + 4);
            } else {
                qs[nt][0] = qs[nt][1] = to_log2;
            }
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < MTILES; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
        vexp = 100;
    }

    __device__ __forceinline__ void tile(uint32_t stage, const float* scales, int lo, int hi) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, i = lane & 3;
        const int key0 = warp * 16 * SLICES;  // this warp's keys of the tile
        if (key0 >= hi || key0 + 16 * SLICES <= lo) return;
        const bool partial = lo > key0 || hi < key0 + 16 * SLICES;
        float s[SLICES][NT][4];
        // S^T = K q^T
        {
            const uint32_t rowa = stage + (key0 + (lane & 15)) * 128;
            const uint32_t x = static_cast<uint32_t>((lane >> 4) ^ (lane & 7)) << 4;
#pragma unroll
            for (int sl = 0; sl < SLICES; ++sl) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[sl][nt][e] = 0.f;
#pragma unroll
                for (int c = 0; c < ROW_BYTES / 32; ++c) {  // two 16-byte chunks at a time
                    uint32_t a[4];
                    ldmatrix_x4(rowa + sl * 16 * 128 + (c >> 2) * TK * 128 + (x ^ ((c & 3) << 5)), a);
                    if constexpr (!CODES) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_bf16(s[sl][nt], a, qf[c][nt][0], qf[c][nt][1]);
                    } else {
                        const uint32_t a0[4] = {even_pair(a[0]), even_pair(a[1]), odd_pair(a[0]), odd_pair(a[1])};
                        const uint32_t a1[4] = {even_pair(a[2]), even_pair(a[3]), odd_pair(a[2]), odd_pair(a[3])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_bf16(s[sl][nt], a0, qf[2 * c][nt][0], qf[2 * c][nt][1]);
                            mma_bf16(s[sl][nt], a1, qf[2 * c + 1][nt][0], qf[2 * c + 1][nt][1]);
                        }
                    }
                }
            }
        }
        // scores in units of log 2, and the keys outside [lo, hi) away
        float vs[SLICES][2], vtop = 0.f;
#pragma unroll
        for (int sl = 0; sl < SLICES; ++sl) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int key = key0 + sl * 16 + g + 8 * r;
                const bool in = !partial || (key >= lo && key < hi);
                float ks = 1.f;
                if constexpr (CODES) {
                    ks = scales[key];
                    vs[sl][r] = in ? scales[TK + key] : 0.f;
                    vtop = fmaxf(vtop, vs[sl][r]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& v = s[sl][nt][2 * r + e];
                        v = in ? (CODES ? v * ks * qs[nt][e] : v * qs[nt][e]) : -INFINITY;
                    }
            }
        }
        float vf = 1.f, vold = 1.f;  // E4M3: factors of the new weights and the old outputs
        if constexpr (CODES) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, off));
            const int e = static_cast<int>(__float_as_uint(vtop) >> 23);
            if (e > vexp) {  // the same in every lane
                vold = __uint_as_float(static_cast<uint32_t>(max(127 - (e - vexp), 0)) << 23);
                vexp = e;
            }
            vf = __uint_as_float(static_cast<uint32_t>(min(127 + 227 - vexp, 254)) << 23);
        }
        uint32_t w[SLICES][NT][2];
        float old[NT][2];
        bool moved = vold != 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = m[nt][e];
#pragma unroll
                for (int sl = 0; sl < SLICES; ++sl) top = fmaxf(top, fmaxf(s[sl][nt][e], s[sl][nt][2 + e]));
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float base = top == -INFINITY ? 0.f : top;
                old[nt][e] = ex2(m[nt][e] - base);
                moved |= top != m[nt][e];
                m[nt][e] = top;
                float sum = 0.f;
#pragma unroll
                for (int sl = 0; sl < SLICES; ++sl)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float& v = s[sl][nt][2 * r + e];
                        v = ex2(v - base);
                        sum += v;
                        if constexpr (CODES) v *= vs[sl][r] * vf;
                    }
                l[nt][e] = fmaf(l[nt][e], old[nt][e], sum);
                old[nt][e] *= vold;
            }
#pragma unroll
            for (int sl = 0; sl < SLICES; ++sl) {
                // the weights, rounded to bf16 for the product with v
                w[sl][nt][0] = movmatrix_trans(pack_bf16(s[sl][nt][0], s[sl][nt][1]));
                w[sl][nt][1] = movmatrix_trans(pack_bf16(s[sl][nt][2], s[sl][nt][3]));
            }
        }
        if (__any_sync(0xffffffffu, moved)) {  // a maximum moved
#pragma unroll
            for (int t = 0; t < MTILES; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][nt][e] *= old[nt][e & 1];
        }
        // O^T += V^T W^T
#pragma unroll
        for (int sl = 0; sl < SLICES; ++sl) {
            // what lies in a masked row may be anything (NaN for one), and 0
            // times that is not 0: such values are cleared (E4M3 codes are
            // finite however they are read)
            uint32_t keep0 = ~0u, keep1 = ~0u;
            if (!CODES && partial) {
                auto pair = [&](int key) {
                    return (key >= lo && key < hi ? 0xffffu : 0u) | (key + 1 >= lo && key + 1 < hi ? 0xffff0000u : 0u);
                };
                keep0 = pair(key0 + sl * 16 + 2 * i);
                keep1 = pair(key0 + sl * 16 + 8 + 2 * i);
            }
            if constexpr (!CODES) {
                const uint32_t rowa = stage + K_BYTES + (key0 + sl * 16 + (lane & 7) + ((lane >> 4) << 3)) * 128;
                const uint32_t x = static_cast<uint32_t>(((lane >> 3) & 1) ^ (lane & 7)) << 4;
#pragma unroll
                for (int t = 0; t < MTILES; ++t) {
                    uint32_t a[4];
                    ldmatrix_x4_trans(rowa + (t >> 2) * TK * 128 + (x ^ ((t & 3) << 5)), a);
                    if (partial) {
                        a[0] &= keep0;
                        a[1] &= keep0;
                        a[2] &= keep1;
                        a[3] &= keep1;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_bf16(o[t][nt], a, w[sl][nt][0], w[sl][nt][1]);
                }
            } else {
                const uint32_t rowa = stage + K_BYTES + (key0 + sl * 16 + (lane & 15)) * 128;
                const uint32_t x = static_cast<uint32_t>((lane >> 4) ^ (lane & 7)) << 4;
#pragma unroll
                for (int c = 0; c < MTILES / 2; ++c) {
                    uint32_t a[4];
                    ldmatrix_x4_trans(rowa + (c >> 2) * TK * 128 + (x ^ ((c & 3) << 5)), a);
                    const uint32_t a0[4] = {even_pair(a[0]), odd_pair(a[0]), even_pair(a[1]), odd_pair(a[1])};
                    const uint32_t a1[4] = {even_pair(a[2]), odd_pair(a[2]), even_pair(a[3]), odd_pair(a[3])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_bf16(o[2 * c][nt], a0, w[sl][nt][0], w[sl][nt][1]);
                        mma_bf16(o[2 * c + 1][nt], a1, w[sl][nt][0], w[sl][nt][1]);
                    }
                }
            }
        }
    }

    // This warp's statistics of its heads, for the lanes that hold them.
    __device__ __forceinline__ void stats(float* ms, float* ls) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (lane < 4) {
                    ms[nt * 8 + 2 * lane + e] = m[nt][e];
                    ls[nt * 8 + 2 * lane + e] = sum;
                }
            }
    }

    // Adds (or, the first, stores) this warp's outputs, relative to the maxima
    // `top`, to obuf [HEADS][DP + 4].
    __device__ __forceinline__ void add(float* obuf, const float* top, bool first) {
        const int lane = threadIdx.x & 31, g = lane >> 2, i = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = nt * 8 + 2 * i + e;
                float f = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - top[h]);
                // E4M3: 2^(vexp - 127 - 100 + 120), the second part below
                if constexpr (CODES) f *= __uint_as_float(static_cast<uint32_t>(vexp) << 23);
                float* row = obuf + h * (DP + 4);
#pragma unroll
                for (int t = 0; t < MTILES; ++t)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int d = CODES ? t * 16 + 2 * g + r : t * 16 + g + 8 * r;
                        float v = o[t][nt][2 * r + e] * f;
                        if constexpr (CODES) v *= 0x1p20f;
                        row[d] = first ? v : row[d] + v;
                    }
            }
    }
};

// fp32 consumer: CUDA cores, fp32 throughout.  Lane i holds elements [V i, V i +
// V) of q, of o and of each row it reads (conflict-free); a row's product with
// 8 heads leaves 32 lanes' partial sums of 8 scores.  Four keys at a time give
// 32 such sums, which 31 exchanges turn into one finished score per lane
// (lane = key * 8 + head).
template <int DP_>
struct F32Consumer {
    static constexpr int DP = DP_;
    static constexpr bool CODES = false;
    static constexpr bool F32 = true;
    static constexpr int HEADS = 8;
    static constexpr int ROW_BYTES = DP * 4;
    static constexpr int BOXES = 1;
    static constexpr int TK = 16384 / ROW_BYTES;
    static constexpr int K_BYTES = TK * ROW_BYTES;
    static constexpr int SCALE_BYTES = 0;
    static constexpr int STAGE_BYTES = 2 * K_BYTES;
    static constexpr int CTAS = 2;
    static constexpr int STAGES = 3;
    static constexpr int V = DP / 32;
    static constexpr int KEYS = TK / kConsumers;  // of a warp, a multiple of 4

    float q[HEADS][V], o[HEADS][V];
    float m, l;  // of head lane & 7: m of all keys, l of keys lane >> 3 (mod 4)

    static __device__ __forceinline__ void load_row(uint32_t addr, float (&f)[V]) {
        if constexpr (V == 2) {
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f[0]), "=f"(f[1]) : "r"(addr) : "memory");
        } else {
#pragma unroll
            for (int v = 0; v < V; v += 4)
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f[v]), "=f"(f[v + 1]), "=f"(f[v + 2]), "=f"(f[v + 3])
                             : "r"(addr + v * 128)
                             : "memory");
        }
    }
    // element of lane i's vector slot v: V = 8 rows are read as two halves of
    // 128 elements, so that every access is conflict-free
    static __device__ __forceinline__ int elem(int lane, int v) {
        return V == 8 ? (v >> 2) * 128 + lane * 4 + (v & 3) : lane * V + v;
    }

    __device__ __forceinline__ void begin(const PagedAttnParams& p, long long qrow, int heads) {
        const int lane = threadIdx.x & 31;
        const float to_log2 = p.scale * 1.4426950408889634f;
#pragma unroll
        for (int h = 0; h < HEADS; ++h)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int d = elem(lane, v);
                q[h][v] = h < heads && d < p.D ? __ldg(static_cast<const float*>(p.q) + (qrow + h) * p.D + d) * to_log2 : 0.f;
                o[h][v] = 0.f;
            }
        m = -INFINITY;
        l = 0.f;
    }

    __device__ __forceinline__ void tile(uint32_t stage, const float*, int lo, int hi) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const uint32_t at = stage + lane * (V == 2 ? 8 : 16);
#pragma unroll 1
        for (int k0 = warp * KEYS; k0 < (warp + 1) * KEYS; k0 += 4) {
            if (k0 >= hi || k0 + 4 <= lo) continue;
            float s[32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float f[V];
                load_row(at + (k0 + k) * ROW_BYTES, f);
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    float a = q[h][0] * f[0];
#pragma unroll
                    for (int v = 1; v < V; ++v) a = fmaf(q[h][v], f[v], a);
                    s[k * 8 + h] = a;
                }
            }
            // halves exchanged, each lane keeping the sums of its side
#pragma unroll
            for (int n = 16; n > 0; n >>= 1) {
                const bool up = (lane & n) != 0;
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const float give = up ? s[j] : s[j + n], keep = up ? s[j + n] : s[j];
                    s[j] = keep + __shfl_xor_sync(0xffffffffu, give, n);
                }
            }
            const int key = k0 + (lane >> 3);
            const bool in = key >= lo && key < hi;
            float x = in ? s[0] : -INFINITY;
            float top = fmaxf(m, x);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float base = top == -INFINITY ? 0.f : top;
            const float old = ex2(m - base), w = ex2(x - base);
            const bool moved = top != m;
            m = top;
            l = fmaf(l, old, w);
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    const float f = __shfl_sync(0xffffffffu, old, h);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[h][v] *= f;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float f[V];
                load_row(at + K_BYTES + (k0 + k) * ROW_BYTES, f);
                if (k0 + k < lo || k0 + k >= hi) {  // whatever a masked row holds
#pragma unroll
                    for (int v = 0; v < V; ++v) f[v] = 0.f;
                }
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    const float wk = __shfl_sync(0xffffffffu, w, k * 8 + h);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[h][v] = fmaf(wk, f[v], o[h][v]);
                }
            }
        }
    }

    __device__ __forceinline__ void stats(float* ms, float* ls) {
        const int lane = threadIdx.x & 31;
        float sum = l + __shfl_xor_sync(0xffffffffu, l, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (lane < 8) {
            ms[lane] = m;
            ls[lane] = sum;
        }
    }

    __device__ __forceinline__ void add(float* obuf, const float* top, bool first) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const float mine = __shfl_sync(0xffffffffu, m, h);
            const float f = mine == -INFINITY ? 0.f : ex2(mine - top[h]);
            float* row = obuf + h * (DP + 4);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int d = elem(lane, v);
                row[d] = first ? o[h][v] * f : row[d] + o[h][v] * f;
            }
        }
    }
};

// ---------------------------------------------------------------- the frame

struct Meta {       // of a ring stage, written by the producer
    int b, j;       // sequence, item of the sequence
    int lo, hi;     // keys of the tile that count
    int flags;
};
enum : int { kFirst = 1, kLast = 2, kItemBegins = 4, kItemEnds = 8 };

// Length and first key of a sequence; both within the table.
struct Span {
    int start, len;
};

__device__ __forceinline__ Span span_of(const PagedAttnParams& p, int b, bool* bad) {
    const int most = p.max_pages * p.page_size;
    const int n = __ldg(p.seq_lens + b);
    if (n < 0 || n > most) *bad = true;
    Span s;
    s.len = max(0, min(n, most));
    s.start = p.window > 0 ? max(0, s.len - p.window) : 0;
    return s;
}

// Tiles of an item: those that hold keys [start, len); one for an empty row,
// so that every item belongs to some CTA.
template <int TK>
__device__ __forceinline__ int tiles_of(const Span& s) {
    return s.len > 0 ? (s.len + TK - 1) / TK - s.start / TK : 1;
}

// Position in the list of tiles: tile t of `tiles` of item j of sequence b.
template <int TK>
struct Cursor {
    int b, j, t, tiles;
    Span s;

    __device__ __forceinline__ void load(const PagedAttnParams& p) {
        bool bad = false;
        s = span_of(p, b, &bad);
        tiles = tiles_of<TK>(s);
    }
    __device__ __forceinline__ void next(const PagedAttnParams& p) {
        if (++t < tiles) return;
        t = 0;
        if (++j < p.items_per_seq) return;
        j = 0;
        if (++b < p.B) load(p);
    }
};

template <class C>
struct Smem {
    static constexpr int RING = C::STAGES * C::STAGE_BYTES;
    static constexpr int SCALES = RING;  // [STAGES][2][TK] floats
    static constexpr int OBUF = SCALES + C::STAGES * 2 * C::SCALE_BYTES;
    static constexpr int STATS = OBUF + C::HEADS * (C::DP + 4) * 4;  // m, l [warps][HEADS]; top, sum [HEADS]
    static constexpr int BYTES = STATS + (2 * kConsumers + 2) * C::HEADS * 4 + 1024;  // 1024: alignment of the ring
};

template <class C>
__global__ void __launch_bounds__(kThreads, C::CTAS) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    constexpr int TK = C::TK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ Meta meta[kMaxStages];
    __shared__ DeviceStatus status;  // this CTA's, copied to the workspace at the end
    __shared__ int abort_flag;
    __shared__ long long warp_tiles[kThreads / 32];
    __shared__ long long share_first;
    __shared__ int share_count;
    __shared__ Cursor<TK> share_at;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // the join may be scheduled as soon as every CTA of this launch runs
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (tid == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kConsumers);
        }
        fence_mbar_init();
        abort_flag = 0;
        status.code = status.where = status.info = 0;
        share_count = 0;
        tma_prefetch_map(&p.map_k);
        tma_prefetch_map(&p.map_v);
    }

    // This CTA's share: every thread counts the tiles of a run of sequences, a
    // scan over the threads gives the total and the thread in whose run the
    // share begins.
    const int run = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * run), b1 = min(p.B, b0 + run);
    long long mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) mine += tiles_of<TK>(span_of(p, b, &bad));
    mine *= p.items_per_seq;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) warp_tiles[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_tiles[w];
        total += warp_tiles[w];
    }
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    const long long first = share * blockIdx.x;
    if (bad) {
        status.code = SPTP_ERR_SHAPE;
        status.where = kWhereKvPage;
    }
    if (first >= before && first < before + mine) {
        long long rest = first - before;
        Cursor<TK> c;
        c.b = b0;
        for (;; ++c.b) {
            c.load(p);
            const long long n = static_cast<long long>(c.tiles) * p.items_per_seq;
            if (rest < n) break;
            rest -= n;
        }
        c.j = static_cast<int>(rest / c.tiles);
        c.t = static_cast<int>(rest - static_cast<long long>(c.j) * c.tiles);
        share_at = c;
        share_first = first;
        share_count = static_cast<int>(min(share, total - first));
    }
    __syncthreads();
    const int count = share_count;
    WaitCtx wc{&status, &abort_flag, kWaitLimitNs};
    PagedAttnPart* part = p.parts + blockIdx.x;

    if (warp == kConsumers) {
        // -------------------------------------------------- producer
        int join_parts = 0, join_b = 0, join_j = 0;
        const int R = p.box_rows, nb = TK / R;
        Cursor<TK> c, n;
        if (count > 0) {
            c = share_at;
            n = c;
        }
        // page of this lane's box of a tile (-1: bad, -2: no key of it counts)
        auto page_of = [&](const Cursor<TK>& at) {
            const int key = (at.s.start / TK + at.t) * TK + lane * R;
            if (lane >= nb || key >= at.s.len || key + R <= at.s.start) return -2;
            const int page = __ldg(p.page_table + static_cast<long long>(at.b) * p.max_pages + key / p.page_size);
            return page >= 0 && page < p.num_pages ? page : -1;
        };
        int page = count > 0 ? page_of(c) : -2;
        int issued = 0;
        for (int i = 0, s = 0; i < count; ++i) {
            // the next tile's pages are read while this one waits for its stage
            int page_next = -2;
            if (i + 1 < count) {
                n.next(p);
                page_next = page_of(n);
            }
            const uint32_t phase = (i / C::STAGES) & 1;
            if (!mbar_wait(&empty[s], phase ^ 1, wc, kWhereKvEmpty, i)) break;
            const int tile0 = (c.s.start / TK + c.t) * TK;
            const int key = tile0 + lane * R;
            const int shard = c.j / (p.Hkv * p.head_blocks), kvh = c.j / p.head_blocks % p.Hkv;
            const int bad_row = p.P * p.num_pages * p.Hkv * p.page_size;  // outside the map: zeros
            int row = bad_row;
            if (page >= 0)
                row = ((shard * p.num_pages + page) * p.Hkv + kvh) * p.page_size + key % p.page_size;
            float* sc = reinterpret_cast<float*>(smem + Smem<C>::SCALES + s * 2 * C::SCALE_BYTES);
            if (page == -1) {
                status.code = SPTP_ERR_SHAPE;
                status.where = kWhereKvPage;
                status.info = c.b;
                if constexpr (C::CODES) {
                    for (int r = 0; r < R; ++r) sc[lane * R + r] = sc[TK + lane * R + r] = 0.f;
                    fence_proxy_async_smem();
                }
            }
            const uint32_t loads = __ballot_sync(0xffffffffu, page != -2);
            const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
            if (lane == 0) {
                Meta md;
                md.b = c.b;
                md.j = c.j;
                md.lo = max(0, c.s.start - tile0);
                md.hi = max(0, min(TK, c.s.len - tile0));
                md.flags = (c.t == 0 ? kItemBegins : 0) | (c.t == c.tiles - 1 ? kItemEnds : 0) |
                           (i == 0 || c.t == 0 ? kFirst : 0) | (i == count - 1 || c.t == c.tiles - 1 ? kLast : 0);
                meta[s] = md;
                // an item that begins here and goes on in the next CTA
                if (i == count - 1 && c.t != c.tiles - 1) {
                    const long long item0 = share_first + i - c.t;
                    if (item0 >= share_first) {
                        join_parts = static_cast<int>((item0 + c.tiles - 1) / share - blockIdx.x) + 1;
                        join_b = c.b;
                        join_j = c.j;
                    }
                }
                mbar_arrive_expect_tx(&full[s], __popc(loads) * 2 * R * C::ROW_BYTES +
                                                    (C::CODES ? __popc(good) * 2 * R * 4 : 0));
            }
            __syncwarp();
            issued = i + 1;
            uint8_t* st = smem + s * C::STAGE_BYTES;
            for (int base = 0; base < nb * C::BOXES * 2; base += 32) {
                const int box = base + lane;
                const int r = box % nb, which = box / nb;
                const int brow = __shfl_sync(0xffffffffu, row, r);
                // a checked build: a page's rows, or the row of zeros
                if (box < nb * C::BOXES * 2 && (loads >> r & 1) != 0 &&
                    checked(brow >= 0 && (brow == bad_row || brow + R <= bad_row), &status, &abort_flag, kWhereBoundsTma,
                            brow)) {
                    const int cb = which >> 1;
                    const bool is_v = which & 1;
                    uint8_t* dst = st + (is_v ? C::K_BYTES : 0) +
                                   (C::F32 ? r * R * C::ROW_BYTES : cb * TK * 128 + r * R * 128);
                    const int x = C::F32 ? 0 : cb * (C::CODES ? 128 : 64);
                    // boxes past a narrow row's end lie outside the map: zeros
                    tma_load_2d(dst, is_v ? &p.map_v : &p.map_k, &full[s], x, brow);
                }
            }
            if constexpr (C::CODES) {
                if (page >= 0) {
                    bulk_load(sc + lane * R, p.k_scale + row, R * 4, &full[s]);
                    bulk_load(sc + TK + lane * R, p.v_scale + row, R * 4, &full[s]);
                }
            }
            c = n;
            page = page_next;
            if (++s == C::STAGES) s = 0;
        }
        if (lane == 0) {
            part->join_parts = join_parts;
            part->b = join_b;
            part->j = join_j;
        }
        if (abort_flag) {
            // left early: wait (bounded) for the copies still in flight
            int local_abort = 0;
            WaitCtx drain{&status, &local_abort, kWaitLimitNs};
            for (int i = max(0, issued - C::STAGES); i < issued; ++i)
                mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, drain, kWhereDrain, i);
        }
    } else {
        // -------------------------------------------------- consumers
        float* obuf = reinterpret_cast<float*>(smem + Smem<C>::OBUF);
        float* ms = reinterpret_cast<float*>(smem + Smem<C>::STATS);
        float* ls = ms + kConsumers * C::HEADS;
        float* top = ls + kConsumers * C::HEADS;
        float* sum = top + C::HEADS;
        const int group = p.Hq / p.Hkv;
        bool begun = false;
        C c;
        for (int i = 0, s = 0; i < count; ++i) {
            if (!mbar_wait(&full[s], (i / C::STAGES) & 1, wc, kWhereKvFull, i)) break;
            const Meta md = meta[s];
            const int hb = md.j % p.head_blocks, sk = md.j / p.head_blocks;
            const int shard = sk / p.Hkv, kvh = sk - shard * p.Hkv;
            const int h0 = hb * p.heads_per_item, heads = min(p.heads_per_item, group - h0);
            const long long qrow = (static_cast<long long>(shard) * p.B + md.b) * p.Hq + kvh * group + h0;
            if (md.flags & kFirst) {
                c.begin(p, qrow, heads);
                begun = (md.flags & kItemBegins) != 0;
            }
            c.tile(smem_u32(smem) + s * C::STAGE_BYTES,
                   reinterpret_cast<const float*>(smem + Smem<C>::SCALES + s * 2 * C::SCALE_BYTES), md.lo, md.hi);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == C::STAGES) s = 0;
            if (!(md.flags & kLast)) continue;

            // ---- the item's end, or this share's: the four warps' parts
            c.stats(ms + warp * C::HEADS, ls + warp * C::HEADS);
            consumers_sync();
            if (tid < C::HEADS) {
                float t = -INFINITY, n = 0.f;
#pragma unroll
                for (int w = 0; w < kConsumers; ++w) t = fmaxf(t, ms[w * C::HEADS + tid]);
#pragma unroll
                for (int w = 0; w < kConsumers; ++w) {
                    const float mw = ms[w * C::HEADS + tid];
                    n += mw == -INFINITY ? 0.f : ls[w * C::HEADS + tid] * ex2(mw - t);
                }
                top[tid] = t;
                sum[tid] = n;
            }
            consumers_sync();
            for (int w = 0; w < kConsumers; ++w) {  // in turn: a fixed order of the sums
                if (warp == w) c.add(obuf, top, w == 0);
                consumers_sync();
            }
            if (begun && (md.flags & kItemEnds)) {
                // the whole item: o / l, rounded once
                for (int e = tid * 2; e < heads * p.D; e += kConsumers * 64) {
                    const int h = e / p.D, d = e - h * p.D;
                    const float n = sum[h], inv = n == 0.f ? 0.f : 1.f / n;
                    const float x = obuf[h * (C::DP + 4) + d] * inv, y = obuf[h * (C::DP + 4) + d + 1] * inv;
                    if constexpr (C::F32)
                        *reinterpret_cast<float2*>(static_cast<float*>(p.out) + qrow * p.D + e) = make_float2(x, y);
                    else
                        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + qrow * p.D + e) =
                            __floats2bfloat162_rn(x, y);
                }
                if (p.lse != nullptr && tid < heads)
                    p.lse[qrow + tid] = sum[tid] == 0.f ? -INFINITY : top[tid] * 0.6931471805599453f + logf(sum[tid]);
            } else {
                // a part: slot 1 if the item begins in this share (it goes on
                // in the next), slot 0 if it began in an earlier one
                const long long at = (blockIdx.x * 2ll + (begun ? 1 : 0)) * p.heads_per_item;
                for (int e = tid * 2; e < heads * p.D; e += kConsumers * 64) {
                    const int h = e / p.D, d = e - h * p.D;
                    *reinterpret_cast<float2*>(p.part_o + at * p.D + e) =
                        make_float2(obuf[h * (C::DP + 4) + d], obuf[h * (C::DP + 4) + d + 1]);
                }
                if (tid < heads) p.part_ml[at + tid] = make_float2(top[tid], sum[tid]);
            }
            consumers_sync();  // obuf and the statistics are free again
        }
    }
    __syncthreads();
    if (tid == 0) {
        part->status = status.code;
        part->where = status.where;
        part->info = status.info;
    }
}

}  // namespace paged
}  // namespace sptp
