// The attention of sptp_paged_attn_prompt on the tensor cores:
//     s_j = cap tanh(scale q.k_j / cap) - slope |pos - j|,
//     out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
// one pass over the keys with a base m that follows the row's maximum, and a sum (in
// the kernel: powers of two, scores in units of log 2).
//
// Bound by the tensor cores for many rows: 4 D flops per row and key.  A CTA has
// two tiles of 128 query rows (rows of 128 < D <= 256: one), token by token with
// the query heads of one key/value head side by side, so that few tokens of a
// large group fill a tile too; both read the same tiles of TK keys.  Scores S =
// Q K^T (both operands from shared memory) and outputs O += P V (weights P from
// tensor memory, where they take the place of their scores) are tcgen05 products
// with fp32 sums in tensor memory.
//  - One warp walks over the CTA's share (prompt_plan.cuh) and keeps a ring of K
//    and V tiles filled by TMA, a box per page; it leaves a description of each
//    item for the others.
//  - One warp issues the products, the two tiles of rows in turn: S of a tile's next
//    keys right behind O of its last ones.  While a tile is in its softmax, the
//    other one's products run.  (With a warp each, their products interleaved, and
//    both tiles were in their softmax at once, the tensor cores idle.)
//  - Two warps look through the tiles of V that some row does not see whole and take out
//    what is infinite or NaN (a weight of 0 would spread it to the rows that do not see
//    it); it is added to the outputs of those that do.
//  - E4M3: four warps turn the tiles of codes that TMA brings into bf16 tiles,
//    code times the row's power of two, which is exact; the rest is the same.
//  - Four warps per tile of rows do its softmax, a thread a row, scores in
//    registers: no exchange between threads.  The base m that the weights refer to
//    lies above the largest score so far and moves only when one is 2^16 above it, so
//    that the outputs in tensor memory are rarely rescaled.
//
// Measured, causal, heads of 128: 4 shards of 16384 rows and 7 heads on one, 1.45 ms
// (1330 TFLOP/s), 1.62 with a bias, 2.36 with a cap (there the softmax is what lasts:
// 8 multiply-adds a score for the cap beside an exponential and its sum), 2.53 with both.
#pragma once

#include <atomic>
#include <cuda_bf16.h>

#include "attn_scores.cuh"
#include "prompt_plan.cuh"
#include "sptp.h"

namespace sptp {
namespace prompt {

constexpr int kTileRows = 128;
// A row's base, in units of log 2, is kHead above the score that it was taken for and
// moves, which rescales the row's outputs in tensor memory and makes its warp's other
// rows wait, when a score is kSlack above it.  Weights are thus within 2^16 of the
// largest score's, which costs no bits (both their types have eight bits of exponent):
// scores 2^-110 of the largest vanish, and values whose sum over a row's keys is below 2^111 stay
// finite.  16384 capped rows of scores of deviation 6: 2.35 ms, with 16 and 8 2.40, with
// 16 and 0 2.57, with 8 and 0 2.77.
constexpr float kSlack = 16.f, kHead = 16.f;
constexpr int kItems = 4;      // descriptions under way
// An item costs as much as two and a half tiles (16384 causal rows, heads of 128: 1.48,
// 1.435 and 1.437 ms with costs of 2, 2.5 and 3; pieces of nine prompts 400, 402 and 406 us).
constexpr int kItemCost = 5 * kTileCost / 2;
constexpr float kPlainCap = 128.f;  // up to here 2^-22 of the cap is no more than a score is off by itself
// No cap; one up to kPlainCap; one above it, or so far from the scale that scale / cap is no normal number
enum CapForm : int { kNoCap, kCap, kWideCap };

enum : int { kBegins = 1, kEnds = 2, kStop = 4 };

// An item's part that the CTA works on, from the producer to the others.
struct Work {
    long long token0;      // shard * M + first row
    int flags;
    int here, key0;        // tiles of keys, first key
    int a[2], b[2];        // tiles [a, b) of them that each tile of rows sees
    int n, heads;          // rows are token * heads + head
    int head0, slope0;     // of the shard; index in slopes
    int pos0, len, prefix;
    int lo, hi;            // keys that any row sees
    int all_lo, all_hi;    // keys that every row sees
    int seq, shard, kvh;   // the sequence, the cache's shard and head
    int unfinite;          // a value that some rows see and others do not is infinite or NaN

    // whether some row does not see a key of the TK from `key` on
    __device__ __forceinline__ bool masked(int key, int TK) const { return key < all_lo || key + TK > all_hi; }
};

template <int DP_, bool CODES_>
struct Shape {
    static constexpr int DP = DP_;                      // elements of a row, at most
    static constexpr bool CODES = CODES_;               // an E4M3 cache
    static constexpr int NQ = DP <= 128 ? 2 : 1;        // tiles of rows
    static constexpr int TK = DP <= 128 ? 128 : 64;     // keys of a tile
    static constexpr int CB = DP / 64;                  // 128-byte columns of a row
    static constexpr int Q_BYTES = kTileRows * DP * 2;  // a tile of rows
    static constexpr int SLOT = TK * DP * 2;            // a tile of K or V
    static constexpr int SLOTS = DP == 64 ? 8 : CODES ? 4 : 5;
    // E4M3: two tiles of codes in columns of SPAN bytes, and their scales
    static constexpr int SPAN = DP == 64 ? 64 : 128, CODE_BOXES = DP / SPAN;
    static constexpr int STAGES = 2, STAGE = TK * DP;
    static constexpr int CODES_AT = NQ * Q_BYTES + SLOTS * SLOT, SCALES_AT = CODES_AT + (CODES ? STAGES * STAGE : 0);
    static constexpr int BYTES = SCALES_AT + (CODES ? STAGES * TK * 4 : 0) + 1024;
    // warps: softmax, four for the others, four that convert codes
    static constexpr int PRODUCER = 4 * NQ, ISSUER = 4 * NQ + 1, CONVERTER = 4 * NQ + 4;
    static constexpr int SIFTER = 4 * NQ + 2, SIFTERS = 2;  // bf16
    static constexpr int WARPS = CONVERTER + (CODES ? 4 : 0);
    // tensor memory columns
    static constexpr int S = 128;                       // between the tiles' scores
    static constexpr int O = 256;                       // first of the outputs; DP between the tiles'
};

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// The products and their commits are issued by one elected lane (the same one
// every time) of a warp that runs through them as a whole, so that their operands
// are uniform registers from the start.
// D (+)= A B^T, both operands bf16 in shared memory.
__device__ __forceinline__ void issue_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|l, 0xffffffff;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D (+)= A B with A (128 x 16 bf16, two elements a column) in tensor memory.
__device__ __forceinline__ void issue_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|l, 0xffffffff;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void issue_commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred l;\n\t"
        "elect.sync _|l, 0xffffffff;\n\t"
        "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// A value that all lanes have, in a uniform register.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Two fp32 in a register pair, and arithmetic on both at once
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float reciprocal_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of a V tile as the second operand: TK rows (the inner dimension) of
// 128 bytes, 128-byte swizzle, elements along the rows: 8 rows are 1024 bytes
// apart, columns of 64 elements `column` bytes.
__device__ __forceinline__ uint64_t smem_desc_rows(uint32_t smem_addr, uint32_t column) {
    uint64_t desc = 0;
    desc |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    desc |= static_cast<uint64_t>(column >> 4) << 16;
    desc |= static_cast<uint64_t>(1024u >> 4) << 32;
    desc |= static_cast<uint64_t>(1u) << 46;
    desc |= static_cast<uint64_t>(2u) << 61;
    return desc;
}
constexpr uint32_t kSecondByRows = 1u << 16;  // instruction descriptor: the second operand lies along its other dimension

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two E4M3 codes (bytes 0 and 1, or 2 and 3 of c) as bf16, times `scale` twice.  A
// code's exponent and mantissa at the end of bf16's exponent are its value times
// 2^-120, subnormals included: times 2^120, and then the row's scale.  Both are
// powers of two, so nothing is rounded.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t c, bool upper, __nv_bfloat162 scale) {
    const uint32_t t = __byte_perm(c, 0, upper ? 0x3424 : 0x1404);
    const uint32_t bits = (t & 0x80008000u) | ((t >> 4) & 0x07f007f0u);
    const __nv_bfloat162 unit = __floats2bfloat162_rn(1.329227995784916e36f, 1.329227995784916e36f);  // 2^120
    const __nv_bfloat162 v = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&bits), unit), scale);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <class C>
struct Bars {
    uint64_t c_full[C::STAGES], c_empty[C::STAGES];  // E4M3: tiles of codes
    uint64_t full[C::SLOTS], empty[C::SLOTS];  // K and V tiles
    uint64_t masked[C::SLOTS];                 // bf16: a masked tile of V is on its way there
    uint64_t checked[C::SLOTS];                // and has been looked through
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2];                        // scores in tensor memory (and all products before them done)
    uint64_t p_ready[2];                       // weights there, outputs rescaled (a warp each)
    uint64_t o_full[2];                        // outputs of an item done
    uint64_t w_full[kItems], w_empty[kItems];  // descriptions
    uint64_t drain;
    Work work[kItems];
    uint32_t tmem;
    int abort_flag;
    DeviceStatus status;
    int out_of_range, out_of_range_at;
};

// ---------------------------------------------------------------- softmax of one tile of rows
// tanh u = u P(u^2) for |u| <= 1/2, off by 1.4e-8 of itself: the polynomial of degree
// 4 in u^2 with the least largest relative error (a Remez fit).
__host__ __device__ constexpr float tanh_term(int i) {
    return i == 0 ? 0.999999986872f : i == 1 ? -0.333330693943f : i == 2 ? 0.133247793204f : i == 3 ? -0.0529860754004f : 0.0171350067528f;
}

template <class C, CapForm CAP, bool BIAS>
struct Softmax {
    static constexpr int TK = C::TK;

    float m, l;  // the base in use, in units of log 2; the sum
    float to_log2, slope;
    int lo, hi, pos;  // keys that this row sees; its position
    bool in;          // a token has it
    int simple;       // BIAS: keys before it lie behind all of the warp's rows; 0 if one has a slope above 1

    static constexpr int N = 32;      // scores at a time
    static constexpr int P = TK / 2;  // column of the weights, in the place of scores that are read before

    static __device__ __forceinline__ uint64_t both(float x) { return pair2(x, x); }
    static __device__ __forceinline__ uint64_t at(const float (&s)[N], int j) { return pair2(s[j], s[j + 1]); }
    static __device__ __forceinline__ void put(float (&s)[N], int j, uint64_t v) {
        const float2 f = split2(v);
        s[j] = f.x;
        s[j + 1] = f.y;
    }

    // The cap, cap tanh(s / cap), of 32 scores that also still lie at s_at.
    // kCap: where no |score| of the warp's rows passes half the cap, three of four by a
    // series on the fused multiply-adds (7 of them each), the rest on the function unit (an
    // exponential and a reciprocal), so that both units have their share; else all of them
    // there.  The function unit's are off by 2^-22 of the cap.
    // kWideCap: up to half the cap the series for all of them, as a factor of the score, so
    // that they are off by 2^-22 of the score however large the cap is.  (In one kernel
    // with the other, 16384 rows with a cap of 50 took 2.46 ms instead of 2.34: more
    // instructions to fetch.)
    __device__ __forceinline__ void apply_cap(const PromptParams& p, const ScoreCap& cap, float (&s)[N], uint32_t s_at) {
        const float to_u = to_log2 * cap.inv;  // (kWideCap: may be 0 or infinite)
        // cap - 2 cap / (1 + e^(2 s / cap)): off by 2^-22 of the cap
        auto by_units = [&](int j) {
            const float2 x = split2(mul2(at(s, j), both(to_log2 * cap.twice)));
            const float2 d = split2(add2(pair2(pow2_approx(x.x), pow2_approx(x.y)), both(1.f)));
            put(s, j, fma2(pair2(reciprocal_approx(d.x), reciprocal_approx(d.y)), both(-2.f * cap.cap), both(cap.cap)));
        };
        auto by_series = [&](int j) {
            // kCap: u = s / cap times the series times the cap; kWideCap: s times the series
            const uint64_t x = mul2(at(s, j), both(CAP == kWideCap ? to_log2 : to_u));
            const uint64_t u = CAP == kWideCap ? mul2(x, both(cap.inv)) : x, v = mul2(u, u);
            const float unit = CAP == kWideCap ? 1.f : cap.cap;
            uint64_t y = both(tanh_term(4) * unit);
#pragma unroll
            for (int i = 3; i >= 0; --i) y = fma2(y, v, both(tanh_term(i) * unit));
            put(s, j, mul2(x, y));
        };
        float most[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) most[i] = max3(fabsf(s[i]), fabsf(s[4 + i]), fabsf(s[8 + i]));
#pragma unroll
        for (int i = 0; i < 4; ++i) most[i] = max3(most[i], fabsf(s[12 + i]), fabsf(s[16 + i]));
#pragma unroll
        for (int i = 0; i < 4; ++i) most[i] = max3(most[i], fabsf(s[20 + i]), fabsf(s[24 + i]));
#pragma unroll
        for (int i = 0; i < 4; ++i) most[i] = fmaxf(most[i], fabsf(s[28 + i]));
        const float all = max3(most[0], most[1], fmaxf(most[2], most[3]));
        // (of rows that a token has: what the others hold must not choose the arithmetic)
        const bool far = __any_sync(0xffffffffu, in && !(all * fabsf(to_u) <= 0.5f));
        if (!far) {
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                if (CAP == kCap && j % 8 == 2)
                    by_units(j);
                else
                    by_series(j);
            }
        } else if constexpr (CAP == kCap) {
#pragma unroll
            for (int j = 0; j < N; j += 2) by_units(j);
        } else {
            // scores next to a cap in the hundreds: rare, and little code
#pragma unroll 1
            for (int c = 0; c < N; c += 16) {
                uint32_t x[16];
                tmem_ld_16cols(s_at + c, x);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(cap(__uint_as_float(x[i]) * to_log2));
                tmem_st_16cols(s_at + c, x);
            }
            tmem_st_wait();
            uint32_t raw[N];
            tmem_ld_32cols(s_at, raw);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < N; ++j) s[j] = __uint_as_float(raw[j]);
        }
    }

    // A new base for the score `now`: the sum, the outputs (unless this is an item's
    // first tile) and the weights of this tile so far (from the 32 c0-th score on) relative to it.
    __device__ __forceinline__ void move(float now, bool moves, uint32_t s_at, uint32_t o_at, int o_cols, bool first, int c0,
                                      uint64_t (&sum)[4]) {
        now += kHead;
        const float f = moves ? pow2_approx(m - now) : 1.f;
        if (moves) m = now;
        l *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = mul2(sum[i], both(f));
        tmem_st_wait();
#pragma unroll 1
        for (int c = c0 * 16; c < TK / 2; c += 16) {
            uint32_t w[16];
            tmem_ld_16cols(s_at + P + c, w);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
                w[i] = pack_bf16(v.x * f, v.y * f);
            }
            tmem_st_16cols(s_at + P + c, w);
        }
        if (first) return;
#pragma unroll 1
        for (int c = 0; c < o_cols; c += 16) {
            uint32_t o[16];
            tmem_ld_16cols(o_at + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st_16cols(o_at + c, o);
        }
    }

    // A tile of keys from key0 on: weights to P, 32 at a time, the last keys first (a
    // bias by distance is least there), in a loop whose code stays in the instruction cache (with the 128 scores
    // of a tile unrolled, fetching instructions took longer than running them).
    __device__ __forceinline__ void tile(const PromptParams& p, const ScoreCap& cap, uint32_t s_at, uint32_t o_at, int o_cols,
                                         int key0, bool first) {
        uint64_t sum[4] = {0, 0, 0, 0};
        const bool masked = __any_sync(0xffffffffu, lo > key0 || hi < key0 + TK);
#pragma unroll 1
        for (int c = TK / N - 1; c >= 0; --c) {
            float s[N];
            {
                uint32_t raw[N];
                tmem_ld_32cols(s_at + c * N, raw);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < N; ++j) s[j] = __uint_as_float(raw[j]);
            }
            // scores in units of log 2 are unit s + bias
            float unit = to_log2, bias = 0.f;
            const int key = key0 + c * N;
            // bit j: key j of the 32 is seen
            const int from = max(lo - key, 0), to = min(max(hi - key, 0), N);
            const uint32_t seen = from >= to ? 0u : (0xffffffffu >> (32 - (to - from))) << from;
            if constexpr (CAP != kNoCap) {
                if (masked) {  // (nor must what lies where no key is)
#pragma unroll
                    for (int j = 0; j < N; ++j) s[j] = seen >> j & 1u ? s[j] : 0.f;
                }
                apply_cap(p, cap, s, s_at + c * N);
                unit = 1.f;
            }
            if constexpr (BIAS) {
                const float far = static_cast<float>(pos - key);
                if (key + N <= simple) {
                    // slope (j - pos), of which the part without j can wait: off by the roundings
                    // of 31 slope and of the whole bias, 2^-17 for slopes up to 1.  (Each
                    // key's distance times the slope: 16384 rows 1.84 ms instead of 1.60.)
#pragma unroll
                    for (int j = 0; j < N; j += 2) put(s, j, fma2(at(s, j), both(unit), pair2(slope * j, slope * (j + 1))));
                    bias = -slope * far;
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) s[j] = fmaf(s[j], unit, -slope * fabsf(far - j));
                }
                unit = 1.f;
            }
            if (masked) {
#pragma unroll
                for (int j = 0; j < N; ++j) s[j] = seen >> j & 1u ? s[j] : -INFINITY;
            }
            float top[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = max3(s[i], s[4 + i], s[8 + i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = max3(top[i], s[12 + i], s[16 + i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = max3(top[i], s[20 + i], s[24 + i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], s[28 + i]);
            const float now = fmaf(max3(top[0], top[1], fmaxf(top[2], top[3])), unit, bias);
            const bool moves = now > m + kSlack;  // (from -infinity to any other, too)
            if (__any_sync(0xffffffffu, moves)) move(now, moves, s_at, o_at, o_cols, first, c + 1, sum);
            const uint64_t unit2 = both(unit), base = both(bias - (m == -INFINITY ? 0.f : m));
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 y = split2(fma2(at(s, 2 * i), unit2, base));
                const float a = pow2_approx(y.x), b = pow2_approx(y.y);
                sum[i & 3] = add2(sum[i & 3], pair2(a, b));
                w[i] = pack_bf16(a, b);
            }
            tmem_st_16cols(s_at + P + c * 16, w);
        }
        const float2 all = split2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
        l += all.x + all.y;
        tmem_st_wait();
    }
};

// Adds, to a row of out (whole) or of the parts' outputs that this thread has written,
// what is infinite or NaN among the values of keys [lo, hi) in masked tiles (E4M3: by
// their scale), which is missing from its products.  Rare, so from global memory, key by key.
template <int TK, bool CODES>
__device__ __noinline__ void add_unfinite(const PromptParams& p, const Work& d, int lo, int hi, bool whole, long long row) {
    const int end = min(hi, d.key0 + d.here * TK);
    for (int key = max(lo, d.key0); key < end; ++key) {
        const int tile = key / TK * TK;
        if (!d.masked(tile, TK)) {
            key = tile + TK - 1;
            continue;
        }
        const long long from = pool_row(p, d.seq, d.shard, d.kvh, key);
        if (from < 0) continue;
        const float scale = CODES ? p.v_scale[from] : 1.f;
        if (CODES && fabsf(scale) <= 3.4e38f) continue;
        for (int c = 0; c < p.D; ++c) {
            float x;
            if (CODES) {
                const int code = static_cast<const uint8_t*>(p.v)[from * p.D + c];
                x = (code & 0x7f) == 0 ? 0.f : code & 0x80 ? -1.f : 1.f;
                x *= scale;
            } else {
                x = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v)[from * p.D + c]);
            }
            if (fabsf(x) <= 3.4e38f) continue;
            if (whole) {
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + row * p.D + c;
                *to = __float2bfloat16(__bfloat162float(*to) + x);
            } else {
                p.part_o[row * p.D + c] += x;
            }
        }
    }
}

template <class C, CapForm CAP, bool BIAS, bool TEST = false>
__global__ void __launch_bounds__(32 * C::WARPS, 1) prompt_tc_kernel(const __grid_constant__ PromptParams p) {
    constexpr int TK = C::TK, NQ = C::NQ, kThreads = 32 * C::WARPS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* slots = smem + NQ * C::Q_BYTES;
    uint8_t* codes = smem + C::CODES_AT;                              // E4M3
    float* scales = reinterpret_cast<float*>(smem + C::SCALES_AT);  // E4M3: [STAGES][TK]
    __shared__ Bars<C> bars;
    __shared__ long long warp_cost[C::WARPS];
    __shared__ Cursor<TK, kItemCost> share_at;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int s = 0; s < C::SLOTS; ++s) {
            mbar_init(&bars.full[s], C::CODES ? 4 : 1);
            mbar_init(&bars.empty[s], 1);
            mbar_init(&bars.masked[s], 1);
            mbar_init(&bars.checked[s], C::SIFTERS);
        }
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&bars.c_full[s], 1 + 32);
            mbar_init(&bars.c_empty[s], 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars.q_full[t], 1);
            mbar_init(&bars.q_empty[t], 1);
            mbar_init(&bars.s_full[t], 1);
            mbar_init(&bars.p_ready[t], 4);
            mbar_init(&bars.o_full[t], 1);
        }
        mbar_init(&bars.drain, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&bars.w_full[i], 1);
            mbar_init(&bars.w_empty[i], 4 * NQ + 1 + (C::CODES ? 4 : C::SIFTERS));
        }
        fence_mbar_init();
        bars.abort_flag = 0;
        bars.status.code = bars.status.where = bars.status.info = 0;
        bars.out_of_range = bars.out_of_range_at = 0;
        tma_prefetch_map(&p.map_q);
        tma_prefetch_map(&p.map_k);
        tma_prefetch_map(&p.map_v);
    }
    if (warp == C::ISSUER) {
        tmem_alloc(&bars.tmem, 512);
        tmem_relinquish();
    }
    // rows of a tile of queries that no box has
    {
        const int used = kTileRows / p.heads * p.heads;
        for (int i = tid; i < NQ * C::CB * (kTileRows - used) * 8; i += kThreads) {
            const int row = used + i / 8 % (kTileRows - used), column = i / 8 / (kTileRows - used);
            *reinterpret_cast<uint4*>(smem + column * kTileRows * 128 + row * 128 + i % 8 * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    await_previous();
    tc_fence_before();
    __syncthreads();
    // Not before the tensor memory is this CTA's: a CTA of the next call's launch that came
    // earlier could hold it while it waits for this launch to end.
    admit_next();
    const Share share = find_share<kThreads>(p, warp_cost, &share_at);
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    WaitCtx wc{&bars.status, &bars.abort_flag, p.wait_limit_ns};
    PromptPart* part = p.parts + blockIdx.x;

    if (warp < C::PRODUCER) {
        // -------------------------------------------------- softmax, a thread a row
        const int t = warp / 4, r = tid % kTileRows;
        const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lane_at + t * C::S, o_at = tmem + lane_at + C::O + t * C::DP;
        const int o_cols = (p.D + 15) / 16 * 16;
        const ScoreCap cap(p.cap);
        Softmax<C, CAP, BIAS> sm;
        sm.to_log2 = p.scale * kLog2e;
        int w = 0;
        uint32_t w_phase = 0, s_phase = 0, o_phase = 0;
        while (true) {
            if (!warp_sleep(&bars.w_full[w], w_phase, wc, kWherePromptItem, -1)) break;
            const Work& d = bars.work[w];
            if (d.flags & kStop) break;
            const int heads = d.heads, tile_tokens = kTileRows / p.heads;
            const int local = r / heads, head = r - local * heads, token = t * tile_tokens + local;
            const bool in = local < tile_tokens && token < d.n;
            const bool some = __any_sync(0xffffffffu, in);  // (a warp without any row leaves what is there)
            sm.in = in;
            sm.m = -INFINITY;
            sm.l = 0.f;
            sm.pos = d.pos0 + token;
            // (a row of the tile that no token has is not masked: it would cost its warp
            // as much as one that is)
            sm.lo = in ? first_key(p, sm.pos) : 0;
            sm.hi = in ? min(d.len, end_key(sm.pos, d.prefix)) : 0x7fffffff;
            sm.slope = BIAS && p.slopes != nullptr && in ? __ldg(p.slopes + d.slope0 + head) * kLog2e : 0.f;
            if constexpr (BIAS)
                sm.simple = __reduce_min_sync(0xffffffffu, fabsf(sm.slope) > kLog2e               ? 0
                                                           : in && p.prefix_lens != nullptr ? max(0, sm.pos + 1)
                                                                                             : 0x7fffffff);
            const int a = d.a[t], b = d.b[t], key0 = d.key0;
            bool ok = true;
            for (int j = b - 1; j >= a; --j) {
                if (!(ok = warp_sleep(&bars.s_full[t], s_phase, wc, kWherePromptScores, j))) break;
                s_phase ^= 1;
                tc_fence_after();
                if (some) sm.tile(p, cap, s_at, o_at, o_cols, key0 + j * TK, j == b - 1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_ready[t]);
            }
            if (!ok) break;
            if (a < b) {
                if (!warp_sleep(&bars.o_full[t], o_phase, wc, kWherePromptOutputs, b)) break;
                o_phase ^= 1;
                tc_fence_after();
            }
            if (some) {
                const bool whole = (d.flags & (kBegins | kEnds)) == (kBegins | kEnds);
                const long long orow = (d.token0 + token) * p.Hq + d.head0 + head;
                // slot 1 if the item begins in this share, slot 0 if in an earlier one
                const int row = token * heads + head;
                const long long at = (blockIdx.x * 2ll + (d.flags & kBegins ? 1 : 0)) * p.part_rows + row;
                const float f = !whole ? 1.f : sm.l == 0.f ? 0.f : 1.f / sm.l;
                if (in) {
                    if (!whole)
                        p.part_ml[at] = make_float2(sm.m, sm.l);
                    else if (p.lse != nullptr)
                        p.lse[orow] = sm.l == 0.f ? -INFINITY : sm.m * 0.6931471805599453f + logf(sm.l);
                }
#pragma unroll 1
                for (int c0 = 0; c0 < o_cols; c0 += 32) {
                    const int halves = c0 + 16 < o_cols ? 2 : 1;  // of 16 columns
                    uint32_t o[2][16] = {};
                    if (a < b) {
                        tmem_ld_16cols(o_at + c0, o[0]);
                        if (halves == 2) tmem_ld_16cols(o_at + c0 + 16, o[1]);
                        tmem_ld_wait();
                    }
                    if (!in) continue;
#pragma unroll
                    for (int h = 0; h < 32; h += 8) {
                        if (c0 + h >= p.D) break;
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(o[h / 16][h % 16 + i]) * f;
                        if (whole) {
                            uint4 u = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                 pack_bf16(v[6], v[7]));
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * p.D + c0 + h) = u;
                        } else {
                            float4* to = reinterpret_cast<float4*>(p.part_o + at * p.D + c0 + h);
                            to[0] = make_float4(v[0], v[1], v[2], v[3]);
                            to[1] = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
                if (in && *const_cast<const volatile int*>(&d.unfinite))
                    add_unfinite<TK, C::CODES>(p, d, sm.lo, sm.hi, whole, whole ? orow : at);
                // the outputs are read before the next item's products (issued behind
                // this warp's next arrival) write there
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.w_empty[w]);
            if (++w == kItems) {
                w = 0;
                w_phase ^= 1;
            }
        }
    } else if (C::CODES && warp >= C::CONVERTER) {
        // -------------------------------------------------- E4M3 tiles to bf16
        // A thread has a row (or half of one), 16 codes at a time: eight lanes' reads and
        // writes are in different banks, swizzled as they are.  Elements behind the
        // row's end are not read by any product.
        constexpr int PARTS = 128 / TK, PER = C::SPAN / 16;
        const int row = (tid - 32 * C::CONVERTER) % TK, first = (tid - 32 * C::CONVERTER) / TK;
        const int swizzle = C::SPAN == 128 ? row & 7 : (row >> 1) & 3;
        const int chunks = (p.D + 15) / 16;
        int stage = 0, slot = 0, w = 0;
        uint32_t c_phase = 0, phase = 1, w_phase = 0;
        bool ok = true;
        while (ok) {
            if (!warp_sleep(&bars.w_full[w], w_phase, wc, kWherePromptItem, -2)) break;
            Work& d = bars.work[w];
            if (d.flags & kStop) break;
            const int tiles = 2 * d.here;
            for (int i = 0; i < tiles; ++i) {
                const int key0 = d.key0 + (d.here - 1 - i / 2) * TK;
                // V: rows that no row of the batch sees become zeros
                const int from = i & 1 ? d.lo - key0 : 0, to = i & 1 ? d.hi - key0 : TK;
                if (!(ok = warp_sleep(&bars.c_full[stage], c_phase, wc, kWhereKvFull, i))) break;
                if (!(ok = warp_sleep(&bars.empty[slot], phase, wc, kWhereKvEmpty, i))) break;
                const uint8_t* in = codes + stage * C::STAGE + row * C::SPAN;
                uint8_t* out = slots + slot * C::SLOT + row * 128;
                const float f = scales[stage * TK + row];
                const __nv_bfloat162 f2 = __floats2bfloat162_rn(f, f);
                bool seen = row >= from && row < to;
                if ((i & 1) && seen && !(fabsf(f) <= 3.4e38f) && d.masked(key0, TK)) {
                    d.unfinite = 1;  // (see the warps that look through bf16 tiles)
                    seen = false;
                }
#pragma unroll 4
                for (int c = first; c < chunks; c += PARTS) {
                    const uint4 u = *reinterpret_cast<const uint4*>(in + c / PER * (TK * C::SPAN) + (((c % PER) ^ swizzle) << 4));
                    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                    if (seen) {
                        lo = make_uint4(codes_to_bf16(u.x, false, f2), codes_to_bf16(u.x, true, f2),
                                        codes_to_bf16(u.y, false, f2), codes_to_bf16(u.y, true, f2));
                        hi = make_uint4(codes_to_bf16(u.z, false, f2), codes_to_bf16(u.z, true, f2),
                                        codes_to_bf16(u.w, false, f2), codes_to_bf16(u.w, true, f2));
                    }
                    uint8_t* at = out + c / 4 * (TK * 128);
                    *reinterpret_cast<uint4*>(at + (((c % 4 * 2) ^ (row & 7)) << 4)) = lo;
                    *reinterpret_cast<uint4*>(at + (((c % 4 * 2 + 1) ^ (row & 7)) << 4)) = hi;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars.full[slot]);
                    mbar_arrive(&bars.c_empty[stage]);
                }
                if (++stage == C::STAGES) {
                    stage = 0;
                    c_phase ^= 1;
                }
                if (++slot == C::SLOTS) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.w_empty[w]);
            if (++w == kItems) {
                w = 0;
                w_phase ^= 1;
            }
        }
    } else {
        if (warp == C::PRODUCER) {
            // -------------------------------------------------- producer
            const int R = p.box_rows, nb = TK / R;
            const long long numbers = block_numbers(p);
            const int tile_tokens = kTileRows / p.heads;
            constexpr int kBadRow = -TK;  // outside the maps, all of a box's rows: zeros
            if (lane == 0) part->items[0].parts = part->items[1].parts = 0;
            Cursor<TK, kItemCost> c = share_at;
            bool more = c.k.tiles != 0, ok = true;
            int slot = 0, issued = 0, w = 0, q_used[2] = {0, 0};
            uint32_t phase = 1, w_phase = 1, q_phase[2] = {1, 1};
            while (ok) {
                if (!(ok = warp_sleep(&bars.w_empty[w], w_phase, wc, kWherePromptItem, issued))) break;
                more = more && c.tile_at() < share.end;
                Work d = {};
                Piece r = {};
                if (!more) {
                    d.flags = kStop;
                } else {
                    r = piece_of(p, c, share);
                    d.token0 = r.token0;
                    d.flags = (r.begins ? kBegins : 0) | (r.ends ? kEnds : 0);
                    d.key0 = c.key0();
                    d.n = c.k.n;
                    d.heads = r.heads;
                    d.head0 = r.head0;
                    d.slope0 = r.shard * p.Hq + r.head0;
                    d.pos0 = c.k.pos0;
                    d.len = c.k.len;
                    d.prefix = c.k.prefix;
                    d.lo = c.k.lo;
                    d.hi = c.k.hi;
                    d.all_lo = first_key(p, d.pos0 + d.n - 1);
                    d.all_hi = end_key(d.pos0, d.prefix);
                    d.seq = c.k.b;
                    d.shard = r.shard;
                    d.kvh = r.kvh;
                    d.here = d.hi > d.lo ? r.here : 0;
                    for (int t = 0; t < NQ; ++t) {
                        const int t0 = t * tile_tokens, n = min(tile_tokens, d.n - t0);  // its rows' tokens
                        if (n <= 0) continue;
                        const int lo = first_key(p, d.pos0 + t0), hi = end_key(d.pos0 + t0 + n - 1, d.prefix);
                        if (hi <= lo) continue;
                        const int from = max(lo, d.key0) - d.key0, to = min(hi, d.key0 + d.here * TK) - d.key0;
                        if (to <= from) continue;
                        d.a[t] = from / TK;
                        d.b[t] = (to + TK - 1) / TK;
                    }
                    if (lane == 0 && !(r.begins && r.ends)) part->items[r.begins ? 1 : 0] = split_item(c, r, share);
                }
                if (lane == 0) {
                    bars.work[w] = d;
                    mbar_arrive(&bars.w_full[w]);
                }
                __syncwarp();
                if (++w == kItems) {
                    w = 0;
                    w_phase ^= 1;
                }
                if (!more) break;
                // the tiles: K of the first, the queries, then V and the next K in turn
                const int pages_rows = p.Hkv * p.page_size;
                const int pool = (r.shard * p.num_pages * p.Hkv + r.kvh) * p.page_size;
                // row of this lane's box (lanes below nb) of tile j: -1: bad page, -2: no key of it is seen
                auto row_of = [&](int j) {
                    const int key = d.key0 + j * TK + lane * R;
                    if (lane >= nb || j < 0 || key >= d.hi || key + R <= d.lo) return -2;
                    const int index = static_cast<int>(__umulhi(static_cast<uint32_t>(key), p.page_mul) >> p.page_shift);
                    const int page = __ldg(p.page_table + static_cast<long long>(c.k.b) * p.max_pages + index);
                    if (page < 0 || page >= p.num_pages) {
                        bars.out_of_range = 1;
                        bars.out_of_range_at = c.k.b;
                        return -1;
                    }
                    return pool + page * pages_rows + key - index * p.page_size;
                };
                // a tile's boxes, and an E4M3 tile's scales; sift: a masked tile of V
                auto load = [&](const CUtensorMap* map, const float* scale, int row, bool sift) {
                    constexpr int kSlots = C::CODES ? C::STAGES : C::SLOTS;
                    uint64_t* full = C::CODES ? &bars.c_full[slot] : &bars.full[slot];
                    if (!warp_sleep(C::CODES ? &bars.c_empty[slot] : &bars.empty[slot], phase, wc, kWhereKvEmpty, issued)) return false;
                    const uint32_t loads = __ballot_sync(0xffffffffu, row != -2);
                    const bool skip = TEST && blockIdx.x == 0 && issued == p.withhold_full;
                    constexpr int kBoxes = C::CODES ? C::CODE_BOXES : C::CB, kSpan = C::CODES ? C::SPAN : 128;
                    if (lane == 0 && !skip) mbar_arrive_expect_tx(full, __popc(loads) * R * kSpan * kBoxes);
                    if (!C::CODES && lane == 0 && sift) mbar_arrive(&bars.masked[slot]);
                    __syncwarp();
                    // lane: box lane % nb of column lane / nb
                    const int box = lane % nb, cb = lane / nb;
                    const int at = __shfl_sync(0xffffffffu, row, box);
                    uint8_t* to = C::CODES ? codes + slot * C::STAGE : slots + slot * C::SLOT;
                    if (cb < kBoxes && at != -2 && !skip &&
                        checked(at == -1 || (at >= 0 && at <= p.P * p.num_pages * pages_rows - R), &bars.status,
                                &bars.abort_flag, kWhereBoundsTma, at))
                        tma_load_2d(to + (cb * TK + box * R) * kSpan, map, full, cb * (C::CODES ? C::SPAN : 64),
                                    at == -1 ? kBadRow : at);
                    if constexpr (C::CODES) {
                        // four keys' scales a lane (0 where there is no page)
                        const int k = min(lane * 4, TK - 4);
                        const int first = __shfl_sync(0xffffffffu, row, k / R);
                        if (lane * 4 < TK)
                            copy16_or_zero(scales + slot * TK + k, scale + (first >= 0 ? first + k % R : 0), first >= 0);
                        arrive_after_copies(full);
                    }
                    ++issued;
                    if (++slot == kSlots) {
                        slot = 0;
                        phase ^= 1;
                    }
                    return true;
                };
                int row = row_of(d.here - 1), next;
                for (int j = d.here - 1; j >= 0; --j) {
                    next = row_of(j - 1);
                    if (!(ok = load(&p.map_k, p.k_scale, row, false))) break;
                    if (j == d.here - 1) {
                        for (int t = 0; t < NQ && ok; ++t) {
                            if (d.a[t] == d.b[t]) continue;
                            if (!(ok = warp_sleep(&bars.q_empty[t], q_phase[t], wc, kWherePromptQuery, t))) break;
                            q_phase[t] ^= 1;
                            ++q_used[t];
                            if (lane == 0) {
                                mbar_arrive_expect_tx(&bars.q_full[t], tile_tokens * p.heads * 128 * C::CB);
                                const int token = static_cast<int>(d.token0 - static_cast<long long>(r.shard) * p.M) + t * tile_tokens;
                                for (int cb = 0; cb < C::CB; ++cb)
                                    tma_load_4d(smem + t * C::Q_BYTES + cb * kTileRows * 128, &p.map_q, &bars.q_full[t], cb * 64,
                                                d.head0, token, r.shard);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
                    if (!(ok = load(&p.map_v, p.v_scale, row, d.masked(d.key0 + j * TK, TK)))) break;
                    row = next;
                }
                if (ok) more = c.next_item(p, numbers);
            }
            if (bars.abort_flag) {
                // left early: wait (bounded) for the copies still in flight
                if (C::CODES) asm volatile("cp.async.wait_all;" ::: "memory");
                int local_abort = 0;
                WaitCtx drain{&bars.status, &local_abort, p.wait_limit_ns};
                constexpr int kSlots = C::CODES ? C::STAGES : C::SLOTS;
                for (int i = max(0, issued - kSlots); i < issued; ++i)
                    if (!(TEST && blockIdx.x == 0 && i == p.withhold_full))
                        mbar_wait(C::CODES ? &bars.c_full[i % kSlots] : &bars.full[i % kSlots], (i / kSlots) & 1, drain,
                                  kWhereDrain, i);
                for (int t = 0; t < NQ; ++t)
                    if (q_used[t] > 0) mbar_wait(&bars.q_full[t], (q_used[t] - 1) & 1, drain, kWhereDrain, t);
            }
        } else if (warp == C::ISSUER) {
            // -------------------------------------------------- products
            const int ksteps = (p.D + 15) / 16;
            const uint32_t s_idesc = idesc_bf16_f32(kTileRows, TK);
            const uint32_t o_idesc = idesc_bf16_f32(kTileRows, ksteps * 16) | kSecondByRows;
            // (descriptors count in 16 bytes, and no tile's addresses carry out of that field)
            const uint64_t q_desc = smem_desc_kmajor_sw128(smem_u32(smem)), k_desc = smem_desc_kmajor_sw128(smem_u32(slots));
            const uint64_t v_desc = smem_desc_rows(smem_u32(slots), TK * 128);
            int slot = 0, w = 0;
            uint32_t phase = 0, w_phase = 0, checked = 0, q_phase[NQ] = {}, p_phase[NQ] = {};
            bool ok = true;
            auto next_slot = [&] {
                if (++slot == C::SLOTS) {
                    slot = 0;
                    phase ^= 1;
                }
            };
            while (true) {
                if (!(ok = warp_sleep(&bars.w_full[w], w_phase, wc, kWherePromptItem, 0))) break;
                const Work& d = bars.work[w];
                if (uniform(d.flags) & kStop) break;
                const int here = uniform(d.here);
                const int key0 = uniform(d.key0), all_lo = uniform(d.all_lo), all_hi = uniform(d.all_hi);
                int a[NQ], b[NQ];
#pragma unroll
                for (int t = 0; t < NQ; ++t) {
                    a[t] = uniform(d.a[t]);
                    b[t] = uniform(d.b[t]);
                }
                // the last keys first; V of tile j and K of tile j - 1: a tile of rows' next
                // scores are issued right behind its outputs, so that the two tiles take
                // turns on the tensor cores, each in its softmax while the other has them
                for (int j = here; j >= 0 && here > 0; --j) {
                    int v_slot = 0;
                    if (j < here) {
                        if (!(ok = warp_sleep(&bars.full[slot], phase, wc, kWhereKvFull, j))) break;
                        if (!C::CODES && (key0 + j * TK < all_lo || key0 + (j + 1) * TK > all_hi)) {
                            if (!(ok = warp_sleep(&bars.checked[slot], checked >> slot & 1u, wc, kWherePromptChecked, j))) break;
                            checked ^= 1u << slot;
                        }
                        v_slot = slot;
                        next_slot();
                    }
                    bool have_k = false;
#pragma unroll
                    for (int t = 0; t < NQ; ++t) {
                        if (j < here && j >= a[t] && j < b[t]) {
                            if (!(ok = warp_sleep(&bars.p_ready[t], p_phase[t], wc, kWherePromptWeights, j))) break;
                            p_phase[t] ^= 1;
                            tc_fence_after();
                            const uint64_t vd = v_desc + v_slot * (C::SLOT >> 4);
                            const uint32_t adds = j != b[t] - 1;
#pragma unroll
                            for (int k = 0; k < TK / 16; ++k)
                                issue_ts(tmem + C::O + t * C::DP, tmem + t * C::S + TK / 2 + k * 8, vd + k * (2048 >> 4),
                                         o_idesc, k != 0 ? 1u : adds);
                            if (j == a[t]) issue_commit(&bars.o_full[t]);
                        }
                        if (j > 0 && !have_k) {
                            if (!(ok = warp_sleep(&bars.full[slot], phase, wc, kWhereKvFull, j))) break;
                            have_k = true;
                        }
                        if (j - 1 >= a[t] && j - 1 < b[t]) {
                            if (j == b[t]) {
                                if (!(ok = warp_sleep(&bars.q_full[t], q_phase[t], wc, kWherePromptQuery, j))) break;
                                q_phase[t] ^= 1;
                            }
                            tc_fence_after();
                            const uint64_t qd = q_desc + t * (C::Q_BYTES >> 4), kd = k_desc + slot * (C::SLOT >> 4);
#pragma unroll
                            for (int k = 0; k < C::DP / 16; ++k)
                                if (k < ksteps)
                                    issue_ss(tmem + t * C::S, qd + ((k >> 2) * (kTileRows * 8) + (k & 3) * 2),
                                             kd + ((k >> 2) * (TK * 8) + (k & 3) * 2), s_idesc, k != 0);
                            issue_commit(&bars.s_full[t]);
                            if (j - 1 == a[t]) issue_commit(&bars.q_empty[t]);
                        }
                    }
                    if (!ok) break;
                    if (j < here) issue_commit(&bars.empty[v_slot]);
                    if (j > 0) {
                        issue_commit(&bars.empty[slot]);
                        next_slot();
                    }
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.w_empty[w]);
                if (++w == kItems) {
                    w = 0;
                    w_phase ^= 1;
                }
            }
            // the products still under way write to tensor memory, which is given back below
            int local_abort = 0;
            WaitCtx drain{&bars.status, &local_abort, p.wait_limit_ns};
            issue_commit(&bars.drain);
            warp_sleep(&bars.drain, 0, drain, kWhereDrain, -1);
        } else if (!C::CODES && warp >= C::SIFTER) {
            // -------------------------------------------------- masked tiles of V
            // A weight is 0 where a row does not see a key, and 0 times what lies there may
            // not be: values that no row of the item sees become zeros, and so does what is
            // infinite or NaN among those that some rows see; the softmax warps then give it
            // to those rows.  (E4M3: the converters do the same by a row's scale.)  All of a
            // batch's loads go before their use: with a load and a branch
            // at a time, by one warp, 16384 plain rows took 1.68 ms instead of 1.43.
            // These warps pass over the tiles that every row sees, up to a whole item of them,
            // and a wait tells a phase of a barrier from the next one only.  So the wait for
            // a tile comes behind one for the producer's word that it is on its way, which it
            // gives once the slot's last tile is used up; a slot has no other such word until this
            // tile is checked.
            int slot = 0, w = 0;
            uint32_t phase = 0, w_phase = 0, sifted = 0;  // sifted: bit s, phase of masked[s]
            bool ok = true;
            auto next_slot = [&] {
                if (++slot == C::SLOTS) {
                    slot = 0;
                    phase ^= 1;
                }
            };
            while (true) {
                if (!warp_sleep(&bars.w_full[w], w_phase, wc, kWherePromptItem, -3)) break;
                Work& d = bars.work[w];
                if (d.flags & kStop) break;
                bool unfinite = false;
                for (int j = d.here - 1; j >= 0; --j) {
                    next_slot();  // K
                    const int key = d.key0 + j * TK;
                    if (d.masked(key, TK)) {
                        if (!(ok = warp_sleep(&bars.masked[slot], sifted >> slot & 1u, wc, kWherePromptMasked, j))) break;
                        sifted ^= 1u << slot;
                        if (!(ok = warp_sleep(&bars.full[slot], phase, wc, kWhereKvFull, j))) break;
                        const int from = d.lo - key, to = d.hi - key;
                        // the sign bit of each half whose exponent is all ones
                        auto ones = [](uint32_t v) { return ((v & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                        auto odd = [&](const uint4& u) { return ones(u.x) | ones(u.y) | ones(u.z) | ones(u.w); };
                        constexpr int BATCH = 8, STRIDE = 32 * C::SIFTERS;
                        static_assert(TK * C::CB * 8 % (BATCH * STRIDE) == 0, "whole batches");
                        uint4* tile = reinterpret_cast<uint4*>(slots + slot * C::SLOT);
#pragma unroll 1
                        for (int i = (warp - C::SIFTER) * 32 + lane; i < TK * C::CB * 8; i += BATCH * STRIDE) {
                            uint4 u[BATCH];
#pragma unroll
                            for (int e = 0; e < BATCH; ++e) u[e] = tile[i + e * STRIDE];
                            uint32_t any = 0;
#pragma unroll
                            for (int e = 0; e < BATCH; ++e) {
                                const int row = (i + e * STRIDE) / 8 % TK;
                                if (row < from || row >= to)
                                    tile[i + e * STRIDE] = make_uint4(0, 0, 0, 0);
                                else
                                    any |= odd(u[e]);
                            }
                            if (any == 0) continue;
                            unfinite = true;
                            auto finite = [&](uint32_t v) { return v & ~((ones(v) >> 15) * 0xffffu); };
#pragma unroll 1
                            for (int e = 0; e < BATCH; ++e) {
                                const uint4 v = tile[i + e * STRIDE];
                                tile[i + e * STRIDE] = make_uint4(finite(v.x), finite(v.y), finite(v.z), finite(v.w));
                            }
                        }
                        fence_proxy_async_smem();
                        unfinite = __any_sync(0xffffffffu, unfinite);
                        if (lane == 0) {
                            if (unfinite) d.unfinite = 1;
                            mbar_arrive(&bars.checked[slot]);
                        }
                        __syncwarp();
                    }
                    next_slot();
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.w_empty[w]);
                if (++w == kItems) {
                    w = 0;
                    w_phase ^= 1;
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == C::ISSUER) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0) {
        const bool failed = bars.status.code != 0;
        part->status = failed ? bars.status.code : bars.out_of_range ? SPTP_ERR_SHAPE : 0;
        part->where = failed ? bars.status.where : bars.out_of_range ? kWhereKvPage : 0;
        part->info = failed ? bars.status.info : bars.out_of_range_at;
    }
}

namespace {  // internal: a process may load the library and its checked build, each with `done` of its own

template <class C, CapForm CAP, bool BIAS, bool TEST = false>
cudaError_t launch_tc(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    plan_prompt(p, C::NQ * kTileRows, kTileRows);
    // the largest boxes that never cross a page
    p.box_rows = 16;
    while (p.box_rows < C::TK && p.page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
    const uint64_t rows = static_cast<uint64_t>(p.P) * p.num_pages * p.Hkv * p.page_size;
    const int es = C::CODES ? 1 : 2, span = C::CODES ? C::SPAN : 64;
    if (!encode_map_rows(&p.map_k, p.k, es, p.D, rows, span, p.box_rows) ||
        !encode_map_rows(&p.map_v, p.v, es, p.D, rows, span, p.box_rows) ||
        !encode_map_queries(&p.map_q, p.q, p.D, p.Hq, p.M, p.P, p.heads, kTileRows / p.heads))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(prompt_tc_kernel<C, CAP, BIAS, TEST>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    *ctas = prompt_grid(p, num_sms < kPromptWideCtas ? num_sms : kPromptWideCtas, C::TK);
    if (TEST && *ctas > kSelftestCtas) *ctas = kSelftestCtas;
    return launch_after(prompt_tc_kernel<C, CAP, BIAS, TEST>, *ctas, 32 * C::WARPS, C::BYTES, s, p);
}

// By row width, and the form of the cap.
template <bool CODES, CapForm CAP, bool BIAS>
cudaError_t launch_width(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    if (p.D <= 64) return launch_tc<Shape<64, CODES>, CAP, BIAS>(p, num_sms, ctas, s);
    if (p.D <= 128) return launch_tc<Shape<128, CODES>, CAP, BIAS>(p, num_sms, ctas, s);
    return launch_tc<Shape<256, CODES>, CAP, BIAS>(p, num_sms, ctas, s);
}

template <bool CODES, bool BIAS>
cudaError_t launch_cap(PromptParams& p, int num_sms, int* ctas, cudaStream_t s) {
    const float to_u = fabsf(p.scale / p.cap);
    return p.cap <= kPlainCap && to_u > 1e-30f && to_u < 1e30f ? launch_width<CODES, kCap, BIAS>(p, num_sms, ctas, s)
                                                                : launch_width<CODES, kWideCap, BIAS>(p, num_sms, ctas, s);
}

}  // namespace

}  // namespace prompt
}  // namespace sptp
