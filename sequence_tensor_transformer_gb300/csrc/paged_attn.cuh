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
//    read it (more than HEADS of them: several items).  Its keys are cut into
//    tiles of TK; the tiles of all items, in order, are dealt out to the CTAs
//    of one resident wave in contiguous shares of equal cost: kTileCost a tile
//    and kItemCost an item (its first loads, its end).  Every CTA works out its
//    own share from the lengths, so nothing depends on the host knowing them.
//    An item that crosses a share's end leaves its parts' (m, l, o) in the
//    workspace; a second launch (paged_attn_join) joins them in a fixed order.
//  - One producer warp walks over the share and keeps a ring of tiles filled by
//    TMA (one box per page and 128 bytes of row, an item's queries with its
//    first tile), running ahead across item borders, so that the reads never
//    wait for the arithmetic.
//  - Four consumer warps score a quarter of each tile's keys, agree on the new
//    maxima, leave the weights in shared memory, and then each sums up all the
//    tile's weighted values for a quarter of the row's elements.  Two barriers
//    a tile; in return no warp has outputs of another's elements, and an item's
//    end costs next to nothing, which is what batches of short rows are made of.
//
// Measured (back to back on the device; of the copy bandwidth): 4 rows of 131071
// bf16 keys of 128 (268 MB) 48.6 us, 0.83; 64 sequences of 64 .. 16384 keys, 4
// heads each (403 MB) 67.7 us, 0.89; 64 of 4096 (540 MB) 0.91; E4M3, 96 sequences
// of 16 .. 8000 keys, 8 heads each (271 MB) 51.0 us, 0.79; 4 rows of 333 keys 7.9
// us.  About 8 us of every call are latency: two launches, the lengths, the page
// table, a first and a last tile, the join.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "attn.h"
#include "sptp.h"
#include "sptp_ptx.cuh"

namespace sptp {
namespace paged {

constexpr int kMaxStages = 8;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 x; 0 gives -infinity
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Consumer warps work in teams of four; a team takes up to HEADS of an item's
// query heads.
constexpr int kTeam = 4;

__device__ __forceinline__ int team_warp() { return (threadIdx.x >> 5) & (kTeam - 1); }
__device__ __forceinline__ int team_index() { return threadIdx.x / (32 * kTeam); }


// Barrier of this thread's team (a constant where there is one team).
template <int TEAMS>
__device__ __forceinline__ void team_sync() {
    if constexpr (TEAMS == 1)
        asm volatile("bar.sync 1, %0;" ::"n"(kTeam * 32) : "memory");
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team_index()), "n"(kTeam * 32) : "memory");
}
// The same, and whether `ok` holds in every thread.  A warp whose bounded wait
// for a tile gave up still comes to the barrier, and all leave together: none
// is left waiting there.
template <int TEAMS>
__device__ __forceinline__ bool team_agrees(bool ok) {
    uint32_t all;
    if constexpr (TEAMS == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.u32 p, %1, 0;\n\t"
            "bar.red.and.pred q, 1, %2, p;\n\t"
            "selp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(all)
            : "r"(static_cast<uint32_t>(ok)), "n"(kTeam * 32)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.u32 p, %1, 0;\n\t"
            "bar.red.and.pred q, %2, %3, p;\n\t"
            "selp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(all)
            : "r"(static_cast<uint32_t>(ok)), "r"(1 + team_index()), "n"(kTeam * 32)
            : "memory");
    return all != 0;
}

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

// the same on fp16 operands
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Four E4M3 codes as fp16 (exact): bytes 0, 1 and bytes 2, 3
__device__ __forceinline__ void unpack_e4m3(uint32_t c, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
}

// The same for a register of the transposed v, which holds two elements of two
// keys each: the keys together, elements 2g to `lo` and 2g + 1 to `hi`
__device__ __forceinline__ void unpack_values(uint32_t c, uint32_t& lo, uint32_t& hi) {
    unpack_e4m3(__byte_perm(c, 0, 0x3120), lo, hi);
}

// Two fp32 in a register pair, and a * b + c on both at once
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 split2(uint64_t p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ float pow2_bits(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// ---------------------------------------------------------------- consumers
// A consumer class is one warp's part of the arithmetic of its team:
//   HEADS, TEAMS, DP       query heads of a team, teams, elements of a row, at most
//   TK                     keys of a tile
//   ROW_BYTES, BOXES       a key's bytes, TMA boxes per row
//   begin(q, keep, heads)  a new item; q its rows in shared memory, keep room for
//                          them (KEEP_BYTES); no barrier of the warps
//   tile(...)              keys [lo, hi) of a tile; false if a warp's `ok` is
//   finish(...)            an item's end, or its part's

// Tensor-core consumer for a bf16 or E4M3 cache, DP >= D elements per row, up
// to 8 NT query heads.
//
// Both products have the keys or the value's elements as the 16 rows of
// m16n8k16 and the query heads as its 8 columns, so that a group of up to 8
// heads wastes nothing:  S^T = K q^T  and  O^T = V^T W^T.  A thread holds the
// scores, statistics and outputs of the same two heads (of every eight)
// throughout.
//
// E4M3: codes become fp16 (exact), and both products run on fp16.  q comes as
// 2^(kRoomQ - e) q, its largest element in [1, 2) times 2^kRoomQ, so fp16 holds
// a bf16 q exactly down to 2^-31 of that, and to 2^-39 of it below (an element
// far larger than the others may meet zeros of k); 2^(e - kRoomQ) and k's scale
// join the score in fp32.  v's scale goes into the
// weight: with t_j its logarithm and M2 the largest s_j + t_j so far (not the
// largest score, which may belong to a row of zeros) the product takes the
// weight 2^(s_j + t_j - M2 + kRoom), an exponential of its own beside the one
// that goes into the sum l, which keeps its own maximum m.  Neither is made
// from the other: a score far below m may be the one that counts, where its
// scale is as much larger (they go from 2^-126, a row of zeros, to 2^119), and
// would be flushed to 0 or meet an infinite factor.  Weights are 2^kRoom at
// most, which fp16 holds, and are flushed below 2^-(25 + kRoom) of the largest,
// so that a long row's tail adds up.  (The sum's exponential times a factor
// loses all of that and is hardly faster: 96 sequences 50.5 and 50.7 us; 64 of
// 2500 keys with 16 heads per key head, D = 64, 128 and 256, 51.9 / 72.4 /
// 144.3 and 53.2 / 73.2 / 149.0.)
template <int DP_, int NT_, bool CODES_, int TEAMS_ = 1>
struct TcConsumer {
    static constexpr int DP = DP_, NT = NT_, TEAMS = TEAMS_;
    static constexpr bool CODES = CODES_;
    static constexpr bool F32 = false;
    static constexpr int HEADS = 8 * NT;
    static constexpr int ROW_BYTES = DP * (CODES ? 1 : 2);
    static constexpr int ELEM = CODES ? 1 : 2;  // bytes
    static constexpr int SPAN = ROW_BYTES < 128 ? 64 : 128;  // bytes of a swizzled row in shared memory
    static constexpr int BOXES = ROW_BYTES / SPAN;
    // 32 KB a tile, or 64 keys where rows are wider
    static constexpr int TK = ROW_BYTES > 256 ? 64 : 16384 / ROW_BYTES;
    static constexpr int Q_STRIDE = DP * 2 + 16;                        // bytes; 8 rows in distinct banks
    static constexpr int W_STRIDE = TK * 2 + 16;
    static constexpr int W_BYTES = HEADS * W_STRIDE;
    static constexpr int KEEP_BYTES = 0;
    static constexpr int CTAS = TEAMS == 1 && ROW_BYTES <= 256 ? 2 : 1;
    static constexpr int K_BYTES = TK * ROW_BYTES;
    static constexpr int SLICES = TK / (16 * kTeam);  // of 16 keys, a warp's
    static constexpr int KSTEPS = DP / 16;                 // of 16 elements of q and k
    static constexpr int MTILES = DP / 16 / kTeam;    // of 16 elements of v, a warp's
    static_assert(ROW_BYTES % SPAN == 0 && (!CODES || MTILES == 1 || MTILES % 2 == 0), "layout");

    // Byte of 16-byte chunk `chunk` of key `row` within a tile's keys: columns of
    // SPAN bytes, swizzled as TMA leaves them.
    static __device__ __forceinline__ uint32_t at(int row, int chunk) {
        constexpr int PER = SPAN / 16;
        const int swizzle = SPAN == 128 ? row & 7 : (row >> 1) & 3;
        return chunk / PER * (TK * SPAN) + row * SPAN + (((chunk % PER) ^ swizzle) << 4);
    }

    uint32_t qf[KSTEPS][NT][2];
    float m[NT][2], l[NT][2], qs[NT][2];
    float m2[NT][2];  // E4M3: M2
    static constexpr int kRoom = 13, kRoomQ = 14;
    float o[MTILES][NT][4];

    // element of the head's row in o[t][..][2 r + ..]
    static __device__ __forceinline__ int elem(int t, int r) {
        const int lane = threadIdx.x & 31, warp = team_warp(), g = lane >> 2;
        return warp * (DP / kTeam) + t * 16 + (CODES ? 2 * g + r : g + 8 * r);
    }

    __device__ __forceinline__ void begin(const PagedAttnParams& p, const uint8_t* q, uint8_t*, int heads) {
        const int lane = threadIdx.x & 31, g = lane >> 2, i = lane & 3;
        const float to_log2 = p.scale * 1.4426950408889634f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + g;
            const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(q + h * Q_STRIDE);
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) {
                if constexpr (!CODES) {
                    const int d = k * 16 + i * 2;
                    qf[k][nt][0] = h < heads && d < p.D ? *reinterpret_cast<const uint32_t*>(row + d) : 0u;
                    qf[k][nt][1] = h < heads && d + 8 < p.D ? *reinterpret_cast<const uint32_t*>(row + d + 8) : 0u;
                } else {
                    const int d = k * 16 + i * 4;  // elements 4i .. 4i+3 of the step
                    uint2 u = make_uint2(0, 0);
                    if (h < heads && d < p.D) u = *reinterpret_cast<const uint2*>(row + d);
                    qf[k][nt][0] = u.x;
                    qf[k][nt][1] = u.y;
                }
            }
            qs[nt][0] = qs[nt][1] = to_log2;
            if constexpr (CODES) {
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
                // 2^(kRoomQ - e) in two factors, each a normal number
                const int x = kRoomQ - e;
                const float f1 = pow2_bits(x >> 1), f2 = pow2_bits(x - (x >> 1));
#pragma unroll
                for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[k][nt][r]));
                        qf[k][nt][r] = pack_f16(f.x * f1 * f2, f.y * f1 * f2);
                    }
                const float f = to_log2 * pow2_bits(e);
                qs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * i);
                qs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * i + 4);
            }
            m[nt][0] = m[nt][1] = m2[nt][0] = m2[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < MTILES; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
    }

    // stage: the tile in shared memory (K, then V); scales: E4M3, of its keys;
    // maxima [1 or 2][kTeam][HEADS] and weights (W_BYTES): this tile's, of
    // all the warps
    // (Whole tiles have code of their own, without a branch that would keep the
    // loads and products of one step apart from the next one's.)
    __device__ __forceinline__ bool tile(bool ok, uint32_t stage, const float* scales, float* maxima, uint8_t* weights,
                                         int lo, int hi) {
        return lo == 0 && hi == TK ? tile_of<false>(ok, stage, scales, maxima, weights, lo, hi)
                                   : tile_of<true>(ok, stage, scales, maxima, weights, lo, hi);
    }

    template <bool partial>
    __device__ __forceinline__ bool tile_of(bool ok, uint32_t stage, const float* scales, float* maxima,
                                            uint8_t* weights, int lo, int hi) {
        const int lane = threadIdx.x & 31, warp = team_warp(), g = lane >> 2, i = lane & 3;
        const int key0 = warp * 16 * SLICES;  // this warp's keys of the tile
        const bool some = !partial || (key0 < hi && key0 + 16 * SLICES > lo);
        float s[SLICES][NT][4];
        float vlog[SLICES][2];  // E4M3: logarithm of v's scale
        float top[NT][2], top2[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = top2[nt][0] = top2[nt][1] = -INFINITY;
        if (some) {
            // S^T = K q^T
#pragma unroll
            for (int sl = 0; sl < SLICES; ++sl) {
                float s2[NT][4];  // a second chain of sums
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[sl][nt][e] = s2[nt][e] = 0.f;
#pragma unroll
                for (int c = 0; c < ROW_BYTES / 32; ++c) {  // two 16-byte chunks at a time
                    uint32_t a[4];
                    ldmatrix_x4(stage + at(key0 + sl * 16 + (lane & 15), 2 * c + (lane >> 4)), a);
                    if constexpr (!CODES) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_bf16(c & 1 ? s2[nt] : s[sl][nt], a, qf[c][nt][0], qf[c][nt][1]);
                    } else {
                        uint32_t a0[4], a1[4];
                        unpack_e4m3(a[0], a0[0], a0[2]);
                        unpack_e4m3(a[1], a0[1], a0[3]);
                        unpack_e4m3(a[2], a1[0], a1[2]);
                        unpack_e4m3(a[3], a1[1], a1[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(s[sl][nt], a0, qf[2 * c][nt][0], qf[2 * c][nt][1]);
                            mma_f16(s2[nt], a1, qf[2 * c + 1][nt][0], qf[2 * c + 1][nt][1]);
                        }
                    }
                }
                // scores in units of log 2, and the keys outside [lo, hi) away
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int key = key0 + sl * 16 + g + 8 * r;
                    const bool in = !partial || (key >= lo && key < hi);
                    float ks = 1.f;
                    if constexpr (CODES) {
                        ks = scales[key] * (1.f / (1 << kRoomQ));
                        vlog[sl][r] = lg2(in ? scales[TK + key] : 0.f);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& v = s[sl][nt][2 * r + e];
                            v += s2[nt][2 * r + e];
                            v = in ? (CODES ? v * ks * qs[nt][e] : v * qs[nt][e]) : -INFINITY;
                            top[nt][e] = fmaxf(top[nt][e], v);
                            if constexpr (CODES) top2[nt][e] = fmaxf(top2[nt][e], v + vlog[sl][r]);
                        }
                }
            }
        }
        // the tile's maxima, of all the warps
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(0xffffffffu, top[nt][e], off));
                    if constexpr (CODES) top2[nt][e] = fmaxf(top2[nt][e], __shfl_xor_sync(0xffffffffu, top2[nt][e], off));
                }
        }
        if (lane < 4) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float* at = maxima + warp * HEADS + nt * 8 + 2 * lane;
                *reinterpret_cast<float2*>(at) = make_float2(top[nt][0], top[nt][1]);
                if constexpr (CODES)
                    *reinterpret_cast<float2*>(at + kTeam * HEADS) = make_float2(top2[nt][0], top2[nt][1]);
            }
        }
        if (!team_agrees<TEAMS>(ok)) return false;
        float old[NT][2];
        bool moved = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float2 t2 = make_float2(m[nt][0], m[nt][1]), u2 = make_float2(m2[nt][0], m2[nt][1]);
#pragma unroll
            for (int w = 0; w < kTeam; ++w) {
                const float* at = maxima + w * HEADS + nt * 8 + 2 * i;
                const float2 o2 = *reinterpret_cast<const float2*>(at);
                t2.x = fmaxf(t2.x, o2.x);
                t2.y = fmaxf(t2.y, o2.y);
                if constexpr (CODES) {
                    const float2 p2 = *reinterpret_cast<const float2*>(at + kTeam * HEADS);
                    u2.x = fmaxf(u2.x, p2.x);
                    u2.y = fmaxf(u2.y, p2.y);
                }
            }
            top[nt][0] = t2.x;
            top[nt][1] = t2.y;
            top2[nt][0] = u2.x;
            top2[nt][1] = u2.y;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float base = top[nt][e] == -INFINITY ? 0.f : top[nt][e];
                old[nt][e] = ex2(m[nt][e] - base);
                l[nt][e] *= old[nt][e];
                float base2 = 0.f;  // E4M3
                if constexpr (CODES) {
                    if (top2[nt][e] != -INFINITY) base2 = top2[nt][e];
                    old[nt][e] = ex2(m2[nt][e] - base2);
                    base2 -= kRoom;
                    moved |= top2[nt][e] != m2[nt][e];
                    m2[nt][e] = top2[nt][e];
                } else {
                    moved |= top[nt][e] != m[nt][e];
                }
                m[nt][e] = top[nt][e];
                if (some) {
                    float sum = 0.f;
#pragma unroll
                    for (int sl = 0; sl < SLICES; ++sl)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float& v = s[sl][nt][2 * r + e];
                            const float w = ex2(v - base);
                            sum += w;
                            if constexpr (CODES)
                                v = ex2(v - base2 + vlog[sl][r]);
                            else
                                v = w;
                        }
                    l[nt][e] += sum;
                }
            }
            if (some) {
                // the weights, rounded to bf16 (E4M3: fp16) for the product with
                // v; turned so that a thread stores two keys of one head
                uint8_t* row = weights + (nt * 8 + g) * W_STRIDE + (key0 + 2 * i) * 2;
#pragma unroll
                for (int sl = 0; sl < SLICES; ++sl)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        *reinterpret_cast<uint32_t*>(row + (sl * 16 + 8 * r) * 2) =
                            movmatrix_trans(CODES ? pack_f16(s[sl][nt][2 * r], s[sl][nt][2 * r + 1])
                                                  : pack_bf16(s[sl][nt][2 * r], s[sl][nt][2 * r + 1]));
            }
        }
        team_sync<TEAMS>();
        if (__any_sync(0xffffffffu, moved)) {  // a maximum moved
#pragma unroll
            for (int t = 0; t < MTILES; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][nt][e] *= old[nt][e & 1];
        }
        // O^T += V^T W^T: all keys, this warp's elements
        const uint32_t wrow = smem_u32(weights) + (lane & 7) * W_STRIDE + (lane >> 3) * 16;
#pragma unroll
        for (int k2 = 0; k2 < TK / 32; ++k2) {  // two steps of 16 keys
            if (partial && (k2 * 32 >= hi || k2 * 32 + 32 <= lo)) continue;
            uint32_t w[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) ldmatrix_x4(wrow + nt * 8 * W_STRIDE + k2 * 64, w[nt]);
            // what lies in a masked row may be anything (NaN for one), and 0
            // times that is not 0: such values are cleared
            auto keep = [&](int key) {
                return (key >= lo && key < hi ? 0xffffu : 0u) | (key + 1 >= lo && key + 1 < hi ? 0xffff0000u : 0u);
            };
            const int chunk0 = warp * (ROW_BYTES / 16 / kTeam);  // this warp's part of the row
            if constexpr (!CODES) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const int k0 = k2 * 32 + kk * 16;
                    if (partial && (k0 >= hi || k0 + 16 <= lo)) continue;
#pragma unroll
                    for (int t = 0; t < MTILES; ++t) {
                        uint32_t a[4];
                        ldmatrix_x4_trans(stage + K_BYTES + at(k0 + (lane & 7) + ((lane >> 4) << 3),
                                                               chunk0 + 2 * t + ((lane >> 3) & 1)),
                                          a);
                        if (partial) {
                            const uint32_t keep0 = keep(k0 + 2 * i), keep1 = keep(k0 + 8 + 2 * i);
                            a[0] &= keep0;
                            a[1] &= keep0;
                            a[2] &= keep1;
                            a[3] &= keep1;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_bf16(o[t][nt], a, w[nt][2 * kk], w[nt][2 * kk + 1]);
                    }
                }
            } else if constexpr (MTILES == 1) {
                uint32_t a[4];  // 16 elements of 32 keys
                ldmatrix_x4_trans(stage + K_BYTES + at(k2 * 32 + lane, chunk0), a);
                if (partial) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) a[n] &= keep(k2 * 32 + 8 * n + 2 * i);
                }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    if (partial && (k2 * 32 + kk * 16 >= hi || k2 * 32 + kk * 16 + 16 <= lo)) continue;
                    uint32_t f[4];
                    unpack_values(a[2 * kk], f[0], f[1]);
                    unpack_values(a[2 * kk + 1], f[2], f[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(o[0][nt], f, w[nt][2 * kk], w[nt][2 * kk + 1]);
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const int k0 = k2 * 32 + kk * 16;
                    if (partial && (k0 >= hi || k0 + 16 <= lo)) continue;
#pragma unroll
                    for (int t = 0; t < MTILES; t += 2) {
                        uint32_t a[4];
                        ldmatrix_x4_trans(stage + K_BYTES + at(k0 + (lane & 15), chunk0 + t + (lane >> 4)), a);
                        if (partial) {
                            const uint32_t keep0 = keep(k0 + 2 * i), keep1 = keep(k0 + 8 + 2 * i);
                            a[0] &= keep0;
                            a[1] &= keep1;
                            a[2] &= keep0;
                            a[3] &= keep1;
                        }
                        uint32_t a0[4], a1[4];
                        unpack_values(a[0], a0[0], a0[1]);
                        unpack_values(a[1], a0[2], a0[3]);
                        unpack_values(a[2], a1[0], a1[1]);
                        unpack_values(a[3], a1[2], a1[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(o[t][nt], a0, w[nt][2 * kk], w[nt][2 * kk + 1]);
                            mma_f16(o[t + 1][nt], a1, w[nt][2 * kk], w[nt][2 * kk + 1]);
                        }
                    }
                }
            }
        }
        return true;
    }

    // The item's end, or its part's: sums [kTeam][HEADS] in shared memory, this
    // thread's outputs to the rows that row_of(head, m, l, holds element 0) gives.
    template <typename RowOf>
    __device__ __forceinline__ void finish(float* sums, RowOf row_of) {
        const int lane = threadIdx.x & 31, warp = team_warp(), i = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (lane < 4) sums[warp * HEADS + nt * 8 + 2 * lane + e] = sum;
            }
        team_sync<TEAMS>();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = nt * 8 + 2 * i + e;
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < kTeam; ++w) sum += sums[w * HEADS + h];
                const auto row = row_of(h, m[nt][e], sum, elem(0, 0) == 0);
                // E4M3: o is relative to M2 - kRoom, the sum to m (in two
                // factors: 2^(M2 - m) may be the least normal number)
                const float f = CODES && sum != 0.f ? row.f * ex2(m2[nt][e] - m[nt][e]) : row.f;
                constexpr float kUnit = CODES ? 1.f / (1 << kRoom) : 1.f;
                if (row.at == nullptr) continue;
#pragma unroll
                for (int t = 0; t < MTILES; ++t) {
                    const float v0 = o[t][nt][e] * kUnit * f, v1 = o[t][nt][2 + e] * kUnit * f;
                    if constexpr (CODES) {
                        row.put(elem(t, 0), v0, v1);
                    } else {
                        row.put(elem(t, 0), v0);
                        row.put(elem(t, 1), v1);
                    }
                }
            }
    }
};

// fp32 consumer: CUDA cores, fp32 throughout, up to 8 query heads a team.
//
// What bounds it beside HBM is shared memory: a query or a weight that all
// lanes read from one place costs as much as a row of 32 values.  So a lane
// scores two keys (half a row of each, the halves' sums exchanged at the end)
// for the HPW heads of its warp, and sums up four elements of the values of one
// key in KEYS_A_STEP: each query read serves two products, each weight four.
// The swizzle that TMA leaves the rows in keeps the lanes' reads apart.
template <int DP_, int TEAMS_ = 1>
struct F32Consumer {
    static constexpr int DP = DP_, TEAMS = TEAMS_;
    static constexpr bool CODES = false;
    static constexpr bool F32 = true;
    static constexpr int HEADS = 8;
    static constexpr int ELEM = 4;  // bytes
    static constexpr int ROW_BYTES = DP * 4;
    static constexpr int SPAN = 128;
    static constexpr int BOXES = ROW_BYTES / 128;
    static constexpr int TK = 16384 / ROW_BYTES;
    static constexpr int K_BYTES = TK * ROW_BYTES;
    static constexpr int Q_STRIDE = ROW_BYTES;
    static constexpr int W_STRIDE = HEADS + 4;  // floats of a key's weights
    static constexpr int W_BYTES = TK * W_STRIDE * 4;
    static constexpr int CTAS = TEAMS == 1 ? 2 : 1;
    // scores
    static constexpr int KEY_GROUPS = TK > 32 ? TK / 32 : 1;   // of the warps
    static constexpr int HPW = HEADS * KEY_GROUPS / kTeam;     // heads of a warp
    static constexpr int KPL = TK < 32 ? 1 : 2;                // keys of a lane, 16 apart
    static constexpr int LANES = TK < 32 ? TK : 32;            // that hold a key each in the end
    static constexpr int CHUNKS = DP / 8;                      // 16-byte chunks of half a row
    static constexpr int KEEP_BYTES = kTeam * HPW * ROW_BYTES;
    // outputs
    static constexpr int OWN = DP / kTeam;                     // elements of a warp
    static constexpr int QUADS = OWN / 4;                      // of four, a lane each
    static constexpr int KEYS_A_STEP = 32 / QUADS;
    static_assert((HPW == 2 || HPW == 4) && TK % KEYS_A_STEP == 0, "layout");

    const uint8_t* q;          // this warp's heads of the item's queries
    uint64_t o[HEADS / 2][4];  // of two heads each
    float m;                   // of head lane & 7
    float l[HPW];              // of this lane's keys
    float to_log2;
    int heads;

    __device__ __forceinline__ void begin(const PagedAttnParams& p, const uint8_t* rows, uint8_t* keep, int n) {
        // the stage that the queries came with is given back: this warp's heads
        // are copied, cleared where the item has no head or the row no element
        const int lane = threadIdx.x & 31, warp = team_warp(), h0 = warp / KEY_GROUPS * HPW;
        uint8_t* mine = keep + warp * HPW * ROW_BYTES;
        __syncwarp();  // the last item's queries are no longer read
        for (int i = lane; i < HPW * DP / 4; i += 32) {
            const int h = i / (DP / 4), d = i % (DP / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (h0 + h < n && d < p.D) v = *reinterpret_cast<const float4*>(rows + (h0 + h) * Q_STRIDE + d * 4);
            *reinterpret_cast<float4*>(mine + h * ROW_BYTES + d * 4) = v;
        }
        __syncwarp();
        q = mine;
        heads = n;
        to_log2 = p.scale * 1.4426950408889634f;
#pragma unroll
        for (int h = 0; h < HEADS / 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[h][e] = 0;
        m = -INFINITY;
#pragma unroll
        for (int h = 0; h < HPW; ++h) l[h] = 0.f;
    }

    __device__ __forceinline__ bool tile(bool ok, uint32_t stage, const float*, float* maxima, uint8_t* weights, int lo,
                                         int hi) {
        const int lane = threadIdx.x & 31, warp = team_warp();
        const int key0 = KEY_GROUPS > 1 ? warp % KEY_GROUPS * 32 : 0;
        const int key = key0 + lane % LANES;     // whose scores this lane holds in the end
        const int h0 = warp / KEY_GROUPS * HPW;  // this warp's heads
        const bool in = key >= lo && key < hi;
        float* w = reinterpret_cast<float*>(weights);  // [TK][W_STRIDE]
        float x[HPW];
#pragma unroll
        for (int h = 0; h < HPW; ++h) x[h] = 0.f;
        if (h0 < heads) {
            const int side = lane >> 4;  // of the row
            const int first = key0 + (lane & 15);
            const uint32_t row = stage + first * 128;
            const ulonglong2* qv = reinterpret_cast<const ulonglong2*>(q);
            uint64_t x2[KPL][HPW][2];  // sums of elements 0 and 1, 2 and 3 of the chunks
#pragma unroll
            for (int j = 0; j < KPL; ++j)
#pragma unroll
                for (int h = 0; h < HPW; ++h) x2[j][h][0] = x2[j][h][1] = 0;
#pragma unroll 8
            for (int c0 = 0; c0 < CHUNKS; ++c0) {
                const int c = side * CHUNKS + (c0 ^ side);  // the sides in different banks
                const uint32_t at = row + (c >> 3) * (TK * 128) + (((c & 7) ^ (first & 7)) << 4);
                uint64_t k[KPL][2];
#pragma unroll
                for (int j = 0; j < KPL; ++j)
                    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                                 : "=l"(k[j][0]), "=l"(k[j][1])
                                 : "r"(at + j * 16 * 128)
                                 : "memory");
#pragma unroll
                for (int h = 0; h < HPW; ++h) {
                    const ulonglong2 a = qv[h * (DP / 4) + c];
#pragma unroll
                    for (int j = 0; j < KPL; ++j) {
                        x2[j][h][0] = fma2(a.x, k[j][0], x2[j][h][0]);
                        x2[j][h][1] = fma2(a.y, k[j][1], x2[j][h][1]);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < HPW; ++h) {
                float y[KPL];
#pragma unroll
                for (int j = 0; j < KPL; ++j) {
                    const float2 u = split2(x2[j][h][0]), v = split2(x2[j][h][1]);
                    y[j] = (u.x + u.y) + (v.x + v.y);
                }
                // the other side's sum of the key that this lane keeps
                const float mine = KPL == 2 && side ? y[KPL - 1] : y[0], give = KPL == 2 && !side ? y[KPL - 1] : y[0];
                x[h] = mine + __shfl_xor_sync(0xffffffffu, give, 16);
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < HPW; ++h) {
            x[h] = in ? x[h] * to_log2 : -INFINITY;
            float t = x[h];
#pragma unroll
            for (int off = 1; off < LANES; off <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
            if ((lane & 7) == h0 + h) top = t;
        }
        if (lane < 8) maxima[warp * HEADS + lane] = top;
        if (!team_agrees<TEAMS>(ok)) return false;
        top = m;
#pragma unroll
        for (int n = 0; n < kTeam; ++n) top = fmaxf(top, maxima[n * HEADS + (lane & 7)]);
        const float base = top == -INFINITY ? 0.f : top;
        const float old = ex2(m - base);
        const bool moved = top != m;
        m = top;
#pragma unroll
        for (int h = 0; h < HPW; ++h) {
            x[h] = ex2(x[h] - __shfl_sync(0xffffffffu, base, h0 + h));
            l[h] = fmaf(l[h], __shfl_sync(0xffffffffu, old, h0 + h), x[h]);
        }
        if (lane < LANES) {
            float* at = w + key * W_STRIDE + h0;
            if constexpr (HPW == 4)
                *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[2], x[3]);
            else
                *reinterpret_cast<float2*>(at) = make_float2(x[0], x[1]);
        }
        team_sync<TEAMS>();
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int h = 0; h < HEADS / 2; ++h) {
                const uint64_t f = pair2(__shfl_sync(0xffffffffu, old, 2 * h), __shfl_sync(0xffffffffu, old, 2 * h + 1));
#pragma unroll
                for (int e = 0; e < 4; ++e) o[h][e] = fma2(o[h][e], f, 0);
            }
        }
        const int quad = warp * QUADS + lane % QUADS;  // chunk of the row
        // (rows of 64: of the two keys that eight lanes read, one is 4 further,
        // in the other half of the banks)
        const int sub = lane / QUADS, k1 = QUADS == 4 ? (sub & 1) << 2 | sub >> 1 : sub;
        const uint32_t vat = stage + K_BYTES + (quad >> 3) * (TK * 128);
        const bool many = heads > 4;
        auto add_key = [&](int k) {
            const ulonglong2* w4 = reinterpret_cast<const ulonglong2*>(w + k * W_STRIDE);
            float f[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                         : "r"(vat + k * 128 + (((quad & 7) ^ (k & 7)) << 4))
                         : "memory");
            const ulonglong2 wa = w4[0];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t ff = pair2(f[e], f[e]);
                o[0][e] = fma2(wa.x, ff, o[0][e]);
                o[1][e] = fma2(wa.y, ff, o[1][e]);
            }
            if (many) {
                const ulonglong2 wb = w4[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t ff = pair2(f[e], f[e]);
                    o[2][e] = fma2(wb.x, ff, o[2][e]);
                    o[3][e] = fma2(wb.y, ff, o[3][e]);
                }
            }
        };
        if (lo == 0 && hi == TK) {
#pragma unroll 4
            for (int k = 0; k < TK; k += KEYS_A_STEP) add_key(k + k1);
        } else {
            // keys [lo, hi) alone: a masked row may hold anything
            for (int k = lo + k1; k < hi; k += KEYS_A_STEP) add_key(k);
        }
        return true;
    }

    template <typename RowOf>
    __device__ __forceinline__ void finish(float* sums, RowOf row_of) {
        const int lane = threadIdx.x & 31, warp = team_warp(), h0 = warp / KEY_GROUPS * HPW;
        float mine = 0.f;
#pragma unroll
        for (int h = 0; h < HPW; ++h) {
            float n = l[h];
#pragma unroll
            for (int off = 1; off < LANES; off <<= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
            if (lane == h0 + h) mine = n;
        }
        if (lane < 8) sums[warp * HEADS + lane] = mine;
        team_sync<TEAMS>();
        // sums over the KEYS_A_STEP lanes that share elements, each lane keeping
        // the heads of its side at every exchange: QUADS / 4 of them at the end
        float v[HEADS * 4];
#pragma unroll
        for (int h = 0; h < HEADS / 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 both = split2(o[h][e]);
                v[2 * h * 4 + e] = both.x;
                v[(2 * h + 1) * 4 + e] = both.y;
            }
        int head = 0;
#pragma unroll
        for (int off = 16; off >= QUADS; off >>= 1) {  // off values are kept
            const bool up = (lane & off) != 0;
            head += up ? off / 4 : 0;
#pragma unroll
            for (int i = 0; i < off; ++i) {
                const float give = up ? v[i] : v[i + off], kept = up ? v[i + off] : v[i];
                v[i] = kept + __shfl_xor_sync(0xffffffffu, give, off);
            }
        }
#pragma unroll
        for (int j = 0; j < QUADS / 4; ++j) {
            const int h = head + j;
            const float mh = __shfl_sync(0xffffffffu, m, h);
            float n = 0.f;
#pragma unroll
            for (int k = 0; k < kTeam; ++k) n += sums[k * HEADS + h];
            const int d = warp * OWN + lane % QUADS * 4;
            const auto row = row_of(h, mh, n, d == 0);
            if (row.at != nullptr)
                row.put(d, v[4 * j] * row.f, v[4 * j + 1] * row.f, v[4 * j + 2] * row.f, v[4 * j + 3] * row.f);
        }
    }
};

// ---------------------------------------------------------------- the frame

// Where one head's D outputs go, and what they are multiplied by; at == nullptr:
// nowhere.  Element numbers are multiples of how many are put at once, as D is.
template <typename T>
struct OutRow {
    T* at;
    float f;
    int D;

    __device__ __forceinline__ void put(int d, float v) const {
        if (d >= D) return;
        if constexpr (sizeof(T) == 2)
            at[d] = __float2bfloat16_rn(v);
        else
            at[d] = v;
    }
    __device__ __forceinline__ void put(int d, float v0, float v1) const {
        if (d >= D) return;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<__nv_bfloat162*>(at + d) = __floats2bfloat162_rn(v0, v1);
        else
            *reinterpret_cast<float2*>(at + d) = make_float2(v0, v1);
    }
    __device__ __forceinline__ void put(int d, float v0, float v1, float v2, float v3) const {
        static_assert(sizeof(T) == 4, "fp32 outputs");
        if (d < D) *reinterpret_cast<float4*>(at + d) = make_float4(v0, v1, v2, v3);
    }
};

struct Meta {       // of a ring stage, written by the producer
    long long qrow;  // row of q and out of the item's first head
    int heads;       // of the item
    int lo, hi;      // keys of the tile that count
    int flags;
};
enum : int {
    kFirst = 1,       // the first tile of an item or of this share
    kLast = 2,        // the last one
    kItemBegins = 4,  // the item's own first tile
    kItemEnds = 8,
    kEnd = 16,        // the share's last tile, or (lo = hi, no other flag) no tile at all
};

// Cost of a tile and of an item, for the shares.  An item (its first loads, the
// pipeline of its arithmetic, its end) costs about as much as one tile more: a
// batch of 96 E4M3 rows took 63.7, 58.5, 54.3, 51.8 and 52.4 us with item costs
// of 0, 1, 2, 4 and 8.
constexpr int kTileCost = 4;
constexpr int kItemCost = 4;

// Length and first key of a sequence; both within the table.
struct Span {
    int start, len;
};

__device__ __forceinline__ Span clip(const PagedAttnParams& p, int n) {
    Span s;
    s.len = max(0, min(n, p.max_pages * p.page_size));
    s.start = p.window > 0 ? max(0, s.len - p.window) : 0;
    return s;
}

__device__ __forceinline__ Span span_of(const PagedAttnParams& p, int b, bool* bad) {
    const int n = __ldg(p.seq_lens + b);
    if (n < 0 || n > p.max_pages * p.page_size) *bad = true;
    return clip(p, n);
}

// Tiles of an item: those that hold keys [start, len); one for an empty row,
// so that every item belongs to some CTA.
template <int TK>
__device__ __forceinline__ int tiles_of(const Span& s) {
    return s.len > 0 ? (s.len + TK - 1) / TK - s.start / TK : 1;
}

// Position in the list of tiles: tile t of `tiles` of item j of sequence b; the
// item's cost begins at `at`.
template <int TK>
struct Cursor {
    long long at;
    int b, j, t, tiles;
    Span s;

    __device__ __forceinline__ void load(const PagedAttnParams& p) {
        bool bad = false;
        s = span_of(p, b, &bad);
        tiles = tiles_of<TK>(s);
    }
    __device__ __forceinline__ int item_cost() const { return tiles * kTileCost + kItemCost; }
    __device__ __forceinline__ long long tile_at() const { return at + static_cast<long long>(t) * kTileCost; }
    __device__ __forceinline__ int key0() const { return (s.start / TK + t) * TK; }
    __device__ __forceinline__ void next_item(const PagedAttnParams& p) {
        at += item_cost();
        t = 0;
        if (++j < p.items_per_seq) return;
        j = 0;
        if (++b < p.B) load(p);
    }
};

// Sixteen bytes to shared memory behind the thread's back, or zeros.
__device__ __forceinline__ void copy16_or_zero(void* dst, const void* src, bool has) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(has ? 16 : 0)
                 : "memory");
}

// One of the arrivals that `bar` expects, once the thread's copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// mbar_wait by a whole warp: true if every lane's wait was.  A lane gives up by
// itself (its own clock, or the abort flag seen); what follows a wait has the
// warp's lanes work together, so they go on or leave as one.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w, int where, int info) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, w, where, info));
}

template <class C>
struct Smem {
    static constexpr int SCALE_BYTES = C::CODES ? C::TK * 4 : 0;
    static constexpr int HEADS = C::HEADS * C::TEAMS;  // of an item
    static constexpr int Q_BYTES = HEADS * C::Q_STRIDE;
    static constexpr int STAGE_BYTES = 2 * C::K_BYTES;
    // of a team: maxima (two sets, for two tiles), sums [kTeam][HEADS], weights [2]
    static constexpr int MAXIMA = (C::CODES ? 2 : 1) * kTeam * C::HEADS;
    static constexpr int STATS_BYTES = (2 * MAXIMA + kTeam * C::HEADS) * 4;
    static constexpr int TEAM_BYTES = STATS_BYTES + 2 * C::W_BYTES + C::KEEP_BYTES;
    static constexpr int FIXED = C::TEAMS * TEAM_BYTES + 1024;  // 1024: alignment of the ring
    // what a CTA may have: 227 KB, or half of an SM's 228 KB less 1 KB each;
    // less the kernel's static shared memory
    static constexpr int ROOM = (C::CTAS == 2 ? 113 * 1024 : 227 * 1024) - 512;
    static constexpr int FIT = (ROOM - FIXED) / (STAGE_BYTES + 2 * SCALE_BYTES + Q_BYTES);
    static constexpr int STAGES = FIT < kMaxStages ? FIT : kMaxStages;
    static constexpr int SCALES = STAGES * STAGE_BYTES;  // [STAGES][2][TK] floats
    static constexpr int QROWS = SCALES + STAGES * 2 * SCALE_BYTES;
    static constexpr int TEAM = QROWS + STAGES * Q_BYTES;
    static constexpr int BYTES = TEAM + C::TEAMS * TEAM_BYTES + 1024;
    static_assert(STAGES >= 2 && STATS_BYTES % 16 == 0 && Q_BYTES % 16 == 0 && C::W_BYTES % 16 == 0, "layout");
};

// TEST: a self-test of the way out (paged_attn_selftest.cu), in which CTA 0 lets
// a wait run out: its producer does not fill tile withhold_full of its share, or
// its consumers do not give back the stage of tile withhold_empty.
template <class C, bool TEST = false>
__global__ void __launch_bounds__(32 * (kTeam * C::TEAMS + 1), C::CTAS)
    paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    using L = Smem<C>;
    constexpr int kThreads = 32 * (kTeam * C::TEAMS + 1);
    constexpr int TK = C::TK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ Meta meta[kMaxStages];
    // This CTA's findings, copied to the workspace at the end: waits that ran out
    // and failed checks; and apart from them, since the outputs stay defined, a
    // length or page outside its range (and its sequence)
    __shared__ DeviceStatus status;
    __shared__ int out_of_range, out_of_range_at;
    __shared__ int abort_flag;
    __shared__ long long warp_cost[kThreads / 32];
    __shared__ Cursor<TK> share_at;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    admit_next();
    if (tid == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(&full[s], C::CODES ? 1 + 32 : 1);  // E4M3: and each lane's scales
            mbar_init(&empty[s], kTeam * C::TEAMS);
        }
        fence_mbar_init();
        abort_flag = 0;
        status.code = status.where = status.info = 0;
        out_of_range = out_of_range_at = 0;
        share_at.b = -1;
        tma_prefetch_map(&p.map_k);
        tma_prefetch_map(&p.map_v);
    }
    await_previous();

    // This CTA's share: every thread adds up the cost of a run of sequences, a
    // scan over the threads gives the total and the thread in whose run the
    // share begins.
    const int run = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * run), b1 = min(p.B, b0 + run);
    long long mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) mine += tiles_of<TK>(span_of(p, b, &bad)) * kTileCost + kItemCost;
    mine *= p.items_per_seq;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) warp_cost[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_cost[w];
        total += warp_cost[w];
    }
    // A tile belongs to the share in which its cost begins; a share is at least
    // one tile's cost, so that an item's parts lie in successive shares.
    const long long share = max(static_cast<long long>(kTileCost), (total + gridDim.x - 1) / gridDim.x);
    const long long begin = share * blockIdx.x, end = begin + share;
    if (bad) out_of_range = 1;
    if (begin >= before && begin < before + mine) {
        Cursor<TK> c;
        c.at = before;
        for (c.b = b0;; ++c.b) {
            c.load(p);
            const long long n = static_cast<long long>(c.item_cost()) * p.items_per_seq;
            if (begin < c.at + n) break;
            c.at += n;
        }
        c.j = static_cast<int>((begin - c.at) / c.item_cost());
        c.at += static_cast<long long>(c.j) * c.item_cost();
        c.t = static_cast<int>((begin - c.at + kTileCost - 1) / kTileCost);
        if (c.t >= c.tiles) c.next_item(p);
        if (c.b < p.B && c.tile_at() < end) share_at = c;
    }
    __syncthreads();
    WaitCtx wc{&status, &abort_flag, p.wait_limit_ns};
    PagedAttnPart* part = p.parts + blockIdx.x;

    if (warp == kTeam * C::TEAMS) {
        // -------------------------------------------------- producer
        PagedAttnItem early = {0, 0, 0, 0, 0, 0}, late = early;
        const int R = p.box_rows, r_shift = __ffs(R) - 1;  // powers of two
        const int nb_shift = __ffs(TK / R) - 1, nb = 1 << nb_shift;
        const int per = 32 >> nb_shift;  // tiles whose rows the lanes look up at once
        const int group = p.Hq / p.Hkv;
        const int pages_rows = p.Hkv * p.page_size;               // of a shard's page
        // outside the maps, all of a box's rows: zeros (before them, since a box
        // behind a pool of almost 2^31 rows would pass the coordinates' 32 bits)
        constexpr int bad_row = -TK;
        const int q_bytes = p.D * (C::F32 ? 4 : 2);
        // this lane's box of a tile: nb x BOXES x 2 of them, at most 32
        static_assert(TK / 16 * C::BOXES * 2 <= 32, "one box per lane");
        const int box_r = lane & (nb - 1), box_cb = lane >> nb_shift >> 1;
        const bool box_v = lane >> nb_shift & 1, box_in = lane < nb * C::BOXES * 2;
        const uint32_t box_at = (box_v ? C::K_BYTES : 0) + (box_cb * TK + box_r * R) * C::SPAN;
        const int box_x = box_cb * (C::SPAN / C::ELEM);
        const CUtensorMap* box_map = box_v ? &p.map_v : &p.map_k;

        Cursor<TK> c = share_at;
        bool more = c.b >= 0, fresh = true;  // fresh: the first item of this share
        if (!more) {
            if (lane == 0) meta[0] = Meta{0, 0, 0, 0, kEnd};
            __syncwarp();
            if (C::CODES || lane == 0) mbar_arrive(&full[0]);
            if (C::CODES && lane == 0) mbar_arrive(&full[0]);
        }
        // page of rows [key, key + R) (-1: bad, -2: no key of them counts)
        auto page_of = [&](int b, const Span& sp, int key) {
            if (key >= sp.len || key + R <= sp.start) return -2;
            const int index = static_cast<int>(__umulhi(static_cast<uint32_t>(key), p.page_mul) >> p.page_shift);
            const int page = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + index);
            return page >= 0 && page < p.num_pages ? page : -1;
        };
        int page = more ? page_of(c.b, c.s, c.key0() + lane * R) : -2;
        int raw_next = more && c.b + 1 < p.B ? __ldg(p.seq_lens + c.b + 1) : 0;
        int issued = 0, s = 0;
        uint32_t phase = 1;
        while (more) {
            // one item: its tiles that lie in this share
            const long long room = (end - c.tile_at() + kTileCost - 1) / kTileCost;
            const int here = static_cast<int>(min(static_cast<long long>(c.tiles - c.t), room));
            const bool begins = c.t == 0, ends = c.t + here == c.tiles;
            const int hb = c.j % p.head_blocks, sk = c.j / p.head_blocks;
            const int shard = sk / p.Hkv, kvh = sk - shard * p.Hkv;
            const int h0 = hb * p.heads_per_item, heads = min(p.heads_per_item, group - h0);
            const long long qrow = (static_cast<long long>(shard) * p.B + c.b) * p.Hq + kvh * group + h0;
            const int pool_row = (shard * p.num_pages * p.Hkv + kvh) * p.page_size;
            const int key_begin = c.key0();
            if ((fresh && !begins) || !ends) {
                // it began in an earlier share, or goes on in the next
                PagedAttnItem it;
                it.first = static_cast<int>(c.at / share);
                it.parts =
                    static_cast<int>((c.at + static_cast<long long>(c.tiles - 1) * kTileCost) / share) - it.first + 1;
                it.heads = heads;
                it.qrow = qrow;
                it.pad = 0;
                it.pad2 = 0;
                (begins ? late : early) = it;
            }
            // the item after it
            Cursor<TK> n = c;
            n.t = 0;
            n.at += c.item_cost();
            if (++n.j == p.items_per_seq) {
                n.j = 0;
                ++n.b;
                n.s = clip(p, raw_next);
                n.tiles = tiles_of<TK>(n.s);
            }
            more = n.b < p.B && n.at < end;
            for (int u0 = 0; u0 < here; u0 += per) {
                const int key = key_begin + u0 * TK + lane * R;  // of this lane's rows
                int row = bad_row;
                if (page >= 0) {
                    const int index = static_cast<int>(__umulhi(static_cast<uint32_t>(key), p.page_mul) >> p.page_shift);
                    row = pool_row + page * pages_rows + key - index * p.page_size;
                }
                const uint32_t loads = __ballot_sync(0xffffffffu, page != -2);
                const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
                // rows of tiles that this share does not have are not reported
                if (page == -1 && (lane >> nb_shift) < here - u0) {
                    out_of_range = 1;
                    out_of_range_at = c.b;
                }
                // the next tiles' pages, while these are waited for
                if (u0 + per < here)
                    page = page_of(c.b, c.s, key + per * TK);
                else if (more)
                    page = page_of(n.b, n.s, n.key0() + lane * R);
                const int tiles = min(per, here - u0);
                for (int u = 0; u < tiles; ++u) {
                    if (!warp_wait(&empty[s], phase, wc, kWhereKvEmpty, issued)) {
                        more = false;
                        u0 = here;
                        break;
                    }
                    const uint32_t mask = (1u << nb) - 1u;
                    const uint32_t tile_loads = loads >> (u << nb_shift) & mask, tile_good = good >> (u << nb_shift) & mask;
                    const bool first = u0 + u == 0, last = u0 + u + 1 == here;
                    const int src = (u << nb_shift) + box_r;
                    const int brow = __shfl_sync(0xffffffffu, row, src);
                    if (TEST && blockIdx.x == 0 && issued == p.withhold_full) {
                        ++issued;
                        if (++s == L::STAGES) {
                            s = 0;
                            phase ^= 1;
                        }
                        continue;
                    }
                    if (lane == 0) {
                        const int tile0 = key_begin + (u0 + u) * TK;
                        Meta md;
                        md.qrow = qrow;
                        md.heads = heads;
                        md.lo = max(0, c.s.start - tile0);
                        md.hi = max(0, min(TK, c.s.len - tile0));
                        md.flags = (first ? kFirst | (begins ? kItemBegins : 0) : 0) |
                                   (last ? kLast | (ends ? kItemEnds : 0) | (more ? 0 : kEnd) : 0);
                        meta[s] = md;
                        mbar_arrive_expect_tx(&full[s], __popc(tile_loads) * 2 * R * C::ROW_BYTES +
                                                            (first ? heads * q_bytes : 0));
                    }
                    __syncwarp();
                    ++issued;
                    if (first && lane < heads)
                        bulk_load(smem + L::QROWS + s * L::Q_BYTES + lane * C::Q_STRIDE,
                                  static_cast<const uint8_t*>(p.q) + (qrow + lane) * q_bytes, q_bytes, &full[s]);
                    // a checked build: a page's rows, or the row of zeros
                    if (box_in && (tile_loads >> box_r & 1) &&
                        checked(brow == bad_row || (brow >= 0 && brow <= p.P * p.num_pages * pages_rows - R), &status,
                                &abort_flag, kWhereBoundsTma, brow))
                        // boxes past a narrow row's end lie outside the map: zeros
                        tma_load_2d(smem + s * L::STAGE_BYTES + box_at, box_map, &full[s], box_x, brow);
                    if constexpr (C::CODES) {
                        // Four keys' scales a lane at a time (0 where there is no
                        // page), by copies of the lanes: a bulk copy for each page's
                        // 64 bytes kept the copy engine busy for longer than its boxes
                        // (pages of 16: rows of 128 61.1 and 53.0 us, of 64 57.7 and 42.9).
                        float* sc = reinterpret_cast<float*>(smem + L::SCALES + s * 2 * L::SCALE_BYTES);
#pragma unroll
                        for (int k0 = 0; k0 < TK; k0 += 128) {
                            // (every lane shuffles, also where a tile has fewer than 128 keys)
                            const int k = k0 + 4 * lane, r = min(k, TK - 1) >> r_shift;  // key, box
                            const int at = __shfl_sync(0xffffffffu, row, (u << nb_shift) + r) + (k & (R - 1));
                            const bool has = tile_good >> r & 1;
                            if (k >= TK) continue;
                            copy16_or_zero(sc + k, p.k_scale + (has ? at : 0), has);
                            copy16_or_zero(sc + TK + k, p.v_scale + (has ? at : 0), has);
                        }
                        arrive_after_copies(&full[s]);
                    }
                    if (++s == L::STAGES) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (n.b != c.b) raw_next = n.b + 1 < p.B ? __ldg(p.seq_lens + n.b + 1) : 0;
            c = n;
            fresh = false;
        }
        if (lane == 0) {
            part->items[0] = early;
            part->items[1] = late;
        }
        if (abort_flag) {
            // left early: wait (bounded) for the copies still in flight
            int local_abort = 0;
            WaitCtx drain{&status, &local_abort, p.wait_limit_ns};
            for (int i = max(0, issued - L::STAGES); i < issued; ++i)
                mbar_wait(&full[i % L::STAGES], (i / L::STAGES) & 1, drain, kWhereDrain, i);
        }
    } else {
        // -------------------------------------------------- consumers
        uint8_t* mine = smem + L::TEAM + team_index() * L::TEAM_BYTES;  // this team's
        float* stats = reinterpret_cast<float*>(mine);
        uint8_t* weights = mine + L::STATS_BYTES;
        uint8_t* keep = weights + 2 * C::W_BYTES;
        bool begun = false;
        C c;
        uint32_t phase = 0;
        for (int i = 0, s = 0;; ++i) {
            const bool ok = warp_wait(&full[s], phase, wc, kWhereKvFull, i);
            const Meta md = ok ? meta[s] : Meta{0, 0, 0, 0, 0};
            // this team's heads: an equal part of the item's
            const int part_heads = (md.heads + C::TEAMS - 1) / C::TEAMS, h0 = team_index() * part_heads;
            const int heads = max(0, min(part_heads, md.heads - h0));
            if (md.flags & kFirst || i == 0) {
                c.begin(p, smem + L::QROWS + s * L::Q_BYTES + h0 * C::Q_STRIDE, keep, heads);
                begun = (md.flags & kItemBegins) != 0;
            }
            if (!c.tile(ok, smem_u32(smem) + s * L::STAGE_BYTES,
                        reinterpret_cast<const float*>(smem + L::SCALES + s * 2 * L::SCALE_BYTES),
                        stats + (i & 1) * L::MAXIMA, weights + (i & 1) * C::W_BYTES, md.lo, md.hi))
                break;
            __syncwarp();
            if (lane == 0 && !(TEST && blockIdx.x == 0 && i == p.withhold_empty)) mbar_arrive(&empty[s]);
            if (++s == L::STAGES) {
                s = 0;
                phase ^= 1;
            }
            if (md.flags & kLast) {
                float* sums = stats + 2 * L::MAXIMA;
                if (begun && (md.flags & kItemEnds)) {
                    // the whole item: o times 1 / l
                    const long long qrow = md.qrow + h0;
                    using T = std::conditional_t<C::F32, float, __nv_bfloat16>;
                    c.finish(sums, [&](int h, float m, float n, bool first) {
                        if (h >= heads) return OutRow<T>{nullptr, 0.f, 0};
                        if (first && p.lse != nullptr)
                            p.lse[qrow + h] = n == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(n);
                        return OutRow<T>{static_cast<T*>(p.out) + (qrow + h) * p.D, n == 0.f ? 0.f : __frcp_rn(n), p.D};
                    });
                } else {
                    // a part: slot 1 if the item begins in this share (it goes
                    // on in the next), slot 0 if it began in an earlier one
                    const long long at = (blockIdx.x * 2ll + (begun ? 1 : 0)) * p.heads_per_item + h0;
                    c.finish(sums, [&](int h, float m, float n, bool first) {
                        if (h >= heads) return OutRow<float>{nullptr, 0.f, 0};
                        if (first) p.part_ml[at + h] = make_float2(m, n);
                        return OutRow<float>{p.part_o + (at + h) * p.D, 1.f, p.D};
                    });
                }
            }
            if (md.flags & kEnd) break;
        }
    }
    __syncthreads();
    if (tid == 0) {
        const bool failed = status.code != 0;
        part->status = failed ? status.code : out_of_range ? SPTP_ERR_SHAPE : 0;
        part->where = failed ? status.where : out_of_range ? kWhereKvPage : 0;
        part->info = failed ? status.info : out_of_range_at;
    }
}

}  // namespace paged
}  // namespace sptp
