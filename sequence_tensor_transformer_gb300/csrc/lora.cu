// Low-rank adapters of many requests at once beside a shared projection:
//     out[p][m] = base[p][m] + gain_a B_a (A_a x_m),   a = ids[m]
// in two launches: t = A_a x_m (fp32, in the workspace), then the rest.
//
// Bound by HBM: x, base and out move once, and each adapter that a row names.
// Rows may name adapters in any order; what is done with a tile of rows is done
// for each of its distinct adapters in turn, on the tensor cores for all its
// rows (16 of them cost as much as one), and kept for the rows that named it.
// So a tile of one prompt's rows reads one adapter, and a tile of 16 new tokens
// of 16 requests reads 16, each once.
//
// bf16: m16n8k16 products with fp32 sums.  The order in which a product's inner
// elements are taken is free as long as both operands agree, and so is that of
// its columns: a lane's fragments are 16 (x, A, out) or 8 (B) contiguous bytes,
// loaded from global memory without a detour.  t goes into its product as the
// sum of two bf16, so that it keeps 16 bits and the result is rounded once.
#include <cuda_bf16.h>

#include <atomic>

#include "lora.h"
#include "sptp.h"
#include "sptp_ptx.cuh"

namespace sptp {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
// The bf16 next below x in magnitude (0: 0): of x's sign and finite unless x is NaN.
__device__ __forceinline__ uint32_t below(float x) {
    const uint32_t u = __float_as_uint(x);
    return u << 1 == 0 ? 0u : (u - 1) & 0xffff0000u;
}
// v = hi + lo up to 2^-16 of it, both of its sign and neither 0 unless it is: so an infinite
// v (lo is infinite, hi is not) and a finite one times an infinity give the infinity that v
// itself does, where hi rounded to the nearest would leave infinity - infinity or 0 times infinity.
__device__ __forceinline__ void split2bf(float x, float y, uint32_t& hi, uint32_t& lo) {
    const uint32_t hx = below(x), hy = below(y);
    hi = hx >> 16 | hy;
    lo = pack2(x - __uint_as_float(hx), y - __uint_as_float(hy));
}

// The adapters of 16 rows: lane r < 16 has row r's (-1: none or no row), and `first`
// the lanes whose row is the first with its adapter.
struct Ids {
    int id;
    uint32_t first;

    __device__ __forceinline__ Ids(const LoraParams& p, int m0, int rows) {
        const int lane = threadIdx.x & 31;
        id = lane < rows && m0 + lane < p.M ? __ldg(p.ids + m0 + lane) : -1;
        if (id >= p.adapters || id < 0) id = -1;
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        first = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
    }
    __device__ __forceinline__ int of(int row) const { return __shfl_sync(0xffffffffu, id, row); }
};

// The status words: the first row whose adapter is outside its range (beside another
// call's: only if there is one, and the other call recorded nothing).  By the last block
// of the second launch.
__device__ __forceinline__ void report_rows(const LoraParams& p) {
    __shared__ int first;
    if (threadIdx.x == 0) first = p.M;
    __syncthreads();
    int mine = p.M;
    for (int m = threadIdx.x; m < p.M; m += kThreads)
        if (__ldg(p.ids + m) >= p.adapters) mine = min(mine, m);
    if (mine < p.M) atomicMin(&first, mine);
    __syncthreads();
    if (threadIdx.x == 0) {
        DeviceStatus st = {0, 0, 0, 0, 0};
        if (first < p.M) {
            st.code = SPTP_ERR_SHAPE;
            st.where = kWhereAdapter;
            st.info = first;
        }
        if (!p.beside || (st.code != 0 && p.status->code == 0)) *p.status = st;
    }
}

// 16 bytes into shared memory, zeros where there are none.
__device__ __forceinline__ void copy_row(void* to, const void* base, long long elem, bool in) {
    copy16_or_zero(to, static_cast<const __nv_bfloat16*>(base) + (in ? elem : 0), in);
}

// ---------------------------------------------------------------- t = A x, bf16
// A block has 16 rows and one split of K.  Its warps share out the rows' adapters,
// and the split's elements where there are fewer adapters than warps (their sums
// are then added in a fixed order).  A thread's loads go through a ring of its own in
// shared memory, so that as many are under way as HBM's latency takes whatever the
// registers are: 16384 rows of 3584 elements, rank 16, 32 us and 39 with unrolled
// loads; 3001 rows of 2 x 2048, rank 64, 17 and 24.
template <int NT>
struct DownRing {
    static constexpr int ITEMS = 2 + NT, STAGES = NT <= 4 ? 3 : 2;
    static constexpr int BYTES = STAGES * ITEMS * kThreads * 16;
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 2) lora_down_bf16(const __grid_constant__ LoraParams p) {
    constexpr int STAGES = DownRing<NT>::STAGES, ITEMS = DownRing<NT>::ITEMS;
    extern __shared__ __align__(16) uint4 down_ring[];  // [STAGES][ITEMS][threads]: a thread's loads under way
    __shared__ __align__(16) float sums[kWarps / 2][16 * NT * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, i = lane & 3;
    await_previous();
    const int tiles = (p.M + 15) / 16;
    const int m0 = blockIdx.x % tiles * 16;
    const int rest = blockIdx.x / tiles, split = rest % p.splits, shard = rest / p.splits;
    const Ids ids(p, m0, 16);
    const int count = __popc(ids.first);
    if (count == 0) return;
    int groups = 1;
    while (groups < count && groups < kWarps) groups *= 2;
    const int ways = kWarps / groups, group = warp / ways, sub = warp % ways;
    const int k0 = split * p.split_k, k1 = min(p.f, k0 + p.split_k);
    const long long xrow = (static_cast<long long>(shard) * p.M + m0 + g) * p.f;
    const bool in0 = m0 + g < p.M, in1 = m0 + g + 8 < p.M;
    float* t = p.t + ((static_cast<long long>(split) * (p.rowwise ? p.P : 1) + shard) * p.M + m0) * p.R;
    uint32_t left = ids.first;
    for (int n = 0; n < group; ++n) left &= left - 1;
    for (int n0 = 0; n0 < count; n0 += groups) {
        const bool mine = left != 0;
        const int a = mine ? ids.of(__ffs(left) - 1) : -2;
        const bool me0 = ids.of(g) == a, me1 = ids.of(g + 8) == a;
        for (int n = 0; n < groups; ++n) left &= left - 1;
        for (int r0 = 0; r0 < p.R; r0 += NT * 8) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
            if (mine) {
                const long long arow = (static_cast<long long>(a) * p.R + r0 + g) * p.K + (p.rowwise ? shard * p.f : 0);
                const int steps = (k1 - k0 - sub * 32 + ways * 32 - 1) / (ways * 32);
                auto load = [&](int step, int slot) {
                    const int k = k0 + (step * ways + sub) * 32 + i * 8;
                    const bool in = k < k1;
                    uint4* to = down_ring + slot * ITEMS * kThreads + threadIdx.x;
                    if (step < steps) {
                        copy_row(to, p.x, xrow + k, in && in0);
                        copy_row(to + kThreads, p.x, xrow + 8ll * p.f + k, in && in1);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            copy_row(to + (2 + nt) * kThreads, p.A, arow + static_cast<long long>(nt) * 8 * p.K + k,
                                     in && r0 + nt * 8 < p.R);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                int slot = 0;
#pragma unroll
                for (int st = 0; st < STAGES - 1; ++st) load(st, st);
                for (int step = 0; step < steps; ++step) {
                    // into the slot that the last step has used up
                    load(step + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
                    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
                    const uint4* from = down_ring + slot * ITEMS * kThreads + threadIdx.x;
                    const uint4 u = from[0], v = from[kThreads];
                    const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 w = from[(2 + nt) * kThreads];
                        mma_bf16(acc[nt], a0, w.x, w.y);
                        mma_bf16(acc[nt], a1, w.z, w.w);
                    }
                    if (++slot == STAGES) slot = 0;
                }
            }
            // (the second launch's blocks only wait until this one is over, in room that its
            // blocks could have: 3001 rows of rank 64 66 us when admitted first, and 63)
            admit_next();
            for (int half = ways / 2; half > 0; half /= 2) {  // warps [half, 2 half) of a group to [0, half)
                float* at = &sums[group * half + (sub < half ? sub : sub - half)][0] + lane * 2;
                if (sub >= half && sub < 2 * half)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float2*>(at + (nt * 2 + e) * 64) = make_float2(acc[nt][2 * e], acc[nt][2 * e + 1]);
                __syncthreads();
                if (sub < half)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 o = *reinterpret_cast<const float2*>(at + (nt * 2 + e) * 64);
                            acc[nt][2 * e] += o.x;
                            acc[nt][2 * e + 1] += o.y;
                        }
                __syncthreads();
            }
            if (sub != 0) continue;
            // this adapter's rows: elements (g, 2i), (g, 2i + 1), (g + 8, ..) of each 16 x 8
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (r0 + nt * 8 >= p.R) break;
                float* at = t + static_cast<long long>(g) * p.R + r0 + nt * 8 + 2 * i;
                if (me0) *reinterpret_cast<float2*>(at) = make_float2(acc[nt][0], acc[nt][1]);
                if (me1) *reinterpret_cast<float2*>(at + 8ll * p.R) = make_float2(acc[nt][2], acc[nt][3]);
            }
        }
    }
}

// A lane's elements of B's row for products kt .. kt + WIDE - 1.
template <int WIDE, int KT, int J>
__device__ __forceinline__ void load_b(const __nv_bfloat16* row, bool in, uint2 (&b)[KT][J], int kt, int j) {
    if constexpr (WIDE == 2) {
        const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(row)) : make_uint4(0, 0, 0, 0);
        b[kt][j] = make_uint2(v.x, v.y);
        b[kt + 1][j] = make_uint2(v.z, v.w);
    } else {
        b[kt][j] = in ? __ldg(reinterpret_cast<const uint2*>(row)) : make_uint2(0, 0);
    }
}

// ---------------------------------------------------------------- out = base + B t, bf16
// A block has 16 rows; its warps take chunks of 32 NC columns in turn, side by side:
// 1 KB of a row at a time with NC = 2.  (With rows of its own for each warp, so that
// they share B, the GPU worked its way through the columns of all rows at once, 128
// bytes of a row here and there: 16384 rows of 4608 columns 95 us instead of 70.)
template <int KT, int NC>
__global__ void __launch_bounds__(kThreads, KT <= 4 ? 2 : 1)
    lora_up_bf16(const __grid_constant__ LoraParams p, int col_blocks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, i = lane & 3;
    admit_next();
    await_previous();
    if (blockIdx.x == gridDim.x - 1) {
        report_rows(p);
        return;
    }
    const int m0 = blockIdx.x / col_blocks * 16;
    if (m0 >= p.M) return;
    const Ids ids(p, m0, 16);
    const bool in_place = p.out == p.base;
    if (ids.first == 0 && in_place) return;
    const int id0 = ids.of(g), id1 = ids.of(g + 8);
    const bool row0 = m0 + g < p.M && (!in_place || id0 >= 0), row1 = m0 + g + 8 < p.M && (!in_place || id1 >= 0);
    // the chunks of all shards, this warp's from `first` on
    const int chunks = (p.n + 32 * NC - 1) / (32 * NC);  // of a shard
    const int first = blockIdx.x % col_blocks * kWarps + warp, step = col_blocks * kWarps;
    struct Place {
        int shard, chunk;
    };
    auto advance = [&](Place& q) {
        for (q.chunk += step; q.chunk >= chunks; q.chunk -= chunks) ++q.shard;
    };
    // lane i has columns 8 i .. 8 i + 7 of each 32: 2 j and 2 j + 1 of them in product j
    auto first_of = [&](const Place& q) {  // element of row g
        return (static_cast<long long>(q.shard) * p.M + m0 + g) * p.n + q.chunk * (32 * NC) + 8 * i;
    };
    auto load_base = [&](const Place& q, uint4 (&v)[NC][2]) {
        const bool in = q.shard < p.P;
        const uint4* b = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.base) + (in ? first_of(q) : 0));
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const bool cin = in && q.chunk * (32 * NC) + c * 32 + 8 * i < p.n;
            v[c][0] = cin && row0 ? b[c * 4] : make_uint4(0, 0, 0, 0);
            v[c][1] = cin && row1 ? b[c * 4 + p.n] : make_uint4(0, 0, 0, 0);  // 8 rows on: 8 n elements, n times 16 bytes
        }
    };
    Place q = {first / chunks, first % chunks}, coming = q;
    uint4 ahead[NC][2];  // the next chunk's base
    load_base(coming, ahead);
    advance(coming);
    // a lane's first element of product kt: 4 i of each 16, or with an even number of
    // products 8 i and 8 i + 4 of each 32, so that 16 bytes of B do for two (3001 rows of
    // rank 64, 2 x 4096 columns: 65 us with the first launch, and 70)
    constexpr int WIDE = KT % 2 == 0 ? 2 : 1;
    auto inner = [&](int kt) { return kt / WIDE * (16 * WIDE) + 4 * WIDE * i + kt % WIDE * 4; };
    // this lane's part of t, times the gain: rows g and g + 8
    uint32_t hi[KT][4], lo[KT][4];
    auto load_t = [&](int shard) {
        const int shards = p.rowwise ? p.P : 1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int a = e ? id1 : id0;
            const float gain = a < 0 ? 0.f : p.gains != nullptr ? __ldg(p.gains + a) : 1.f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (a >= 0 && inner(kt) < p.R) {
                    const float* at = p.t + (static_cast<long long>(shard) * p.M + m0 + g + 8 * e) * p.R + inner(kt);
                    const long long stride = static_cast<long long>(shards) * p.M * p.R;
#pragma unroll 8
                    for (int s = 0; s < p.splits; ++s) {
                        const float4 u = *reinterpret_cast<const float4*>(at + s * stride);
                        v.x += u.x;
                        v.y += u.y;
                        v.z += u.z;
                        v.w += u.w;
                    }
                }
                split2bf(v.x * gain, v.y * gain, hi[kt][e], lo[kt][e]);
                split2bf(v.z * gain, v.w * gain, hi[kt][2 + e], lo[kt][2 + e]);
            }
        }
    };
    // base + the products with the columns whose B is in b, both rows of 32 columns
    auto add = [&](const uint4 (&was)[2], const uint2 (&b)[KT][NC * 4], int c, uint4 (&now)[2]) {
        uint32_t *w0 = reinterpret_cast<uint32_t*>(&now[0]), *w1 = reinterpret_cast<uint32_t*>(&now[1]);
        const uint32_t *o0 = reinterpret_cast<const uint32_t*>(&was[0]), *o1 = reinterpret_cast<const uint32_t*>(&was[1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f0 = unpack2(o0[j]), f1 = unpack2(o1[j]);
            float sum[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                mma_bf16(sum, lo[kt], b[kt][c * 4 + j].x, b[kt][c * 4 + j].y);
                mma_bf16(sum, hi[kt], b[kt][c * 4 + j].x, b[kt][c * 4 + j].y);
            }
            w0[j] = pack2(sum[0], sum[1]);
            w1[j] = pack2(sum[2], sum[3]);
        }
    };
    // one adapter for all 16 rows, and the ranks all there: no row or element is left out
    const bool plain = __all_sync(0xffffffffu, id0 >= 0 && id0 == id1) && __popc(ids.first) == 1 && p.R == KT * 16;
    const int a0 = ids.first != 0 ? ids.of(__ffs(ids.first) - 1) : 0;
    int have = -1;  // shard whose t is there
    for (; q.shard < p.P; advance(q)) {
        uint4 was[NC][2];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) was[c][e] = ahead[c][e];
        load_base(coming, ahead);
        advance(coming);
        if (have < 0 || (p.rowwise && have != q.shard)) load_t(p.rowwise ? q.shard : 0);
        have = q.shard;
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + first_of(q));
        const int col0 = q.chunk * (32 * NC);
        const long long b0 = (p.rowwise ? 0 : static_cast<long long>(q.shard) * p.n) + col0 + 8 * (g >> 1) + (g & 1);
        if (plain && col0 + 32 * NC <= p.n) {
            const __nv_bfloat16* rows = static_cast<const __nv_bfloat16*>(p.B) + (static_cast<long long>(a0) * p.N + b0) * p.R + inner(0);
            uint2 b[KT][NC * 4];
#pragma unroll
            for (int j = 0; j < NC * 4; ++j)
#pragma unroll
                for (int kt = 0; kt < KT; kt += WIDE)
                    load_b<WIDE>(rows + (j / 4 * 32 + 2 * (j % 4)) * (KT * 16) + kt * 16, true, b, kt, j);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                uint4 now[2];
                add(was[c], b, c, now);
                out[c * 4] = now[0];
                out[c * 4 + p.n] = now[1];
            }
            continue;
        }
        bool cin[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            cin[c] = col0 + c * 32 + 8 * i < p.n;
            // rows without an adapter
            if (cin[c] && row0 && id0 < 0) out[c * 4] = was[c][0];
            if (cin[c] && row1 && id1 < 0) out[c * 4 + p.n] = was[c][1];
        }
        for (uint32_t left = ids.first; left != 0; left &= left - 1) {
            const int a = ids.of(__ffs(left) - 1);
            const __nv_bfloat16* rows = static_cast<const __nv_bfloat16*>(p.B) + (static_cast<long long>(a) * p.N + b0) * p.R + inner(0);
            uint2 b[KT][NC * 4];
#pragma unroll
            for (int j = 0; j < NC * 4; ++j) {
                const int n = j / 4 * 32 + 2 * (j % 4);  // from this lane's first row of B
                const bool in = col0 + n + 8 * (g >> 1) + (g & 1) < p.n;
#pragma unroll
                for (int kt = 0; kt < KT; kt += WIDE)
                    load_b<WIDE>(rows + n * p.R + kt * 16, in && inner(kt) < p.R, b, kt, j);
            }
            // all 16 rows' products with each adapter, kept by the rows that named it
            // (so another adapter's infinities do not reach a row)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                uint4 now[2];
                add(was[c], b, c, now);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (cin[c] && (e ? id1 : id0) == a) out[c * 4 + (e ? p.n : 0)] = now[e];
            }
        }
    }
}

// Few rows, most with an adapter of their own: a block has one row and 512 columns, a
// lane two of them, on the CUDA cores (16 rows' products for each of 16 adapters took
// ten times the instructions: 64 rows of 61 requests 23 us with them, 15 this way; the
// two cross at some 200 rows).
__global__ void __launch_bounds__(kThreads) lora_up_row_bf16(const __grid_constant__ LoraParams p, int col_blocks) {
    __shared__ float part[kThreads];
    __shared__ __align__(16) float st[kLoraMaxRank];
    const int tid = threadIdx.x;
    admit_next();
    await_previous();
    if (blockIdx.x == gridDim.x - 1) {
        report_rows(p);
        return;
    }
    const int m = blockIdx.x / col_blocks, block = blockIdx.x % col_blocks;
    int a = __ldg(p.ids + m);
    if (a >= p.adapters) a = -1;
    const bool in_place = p.out == p.base;
    if (a < 0 && in_place) return;
    // a shard's columns come in whole blocks of 512
    const int shard_blocks = (p.n + 2 * kThreads - 1) / (2 * kThreads);
    const int shard = block / shard_blocks, col = (block % shard_blocks) * 2 * kThreads + 2 * tid;
    const bool in = col < p.n;
    const long long at = (static_cast<long long>(shard) * p.M + m) * p.n + col;
    const uint32_t was = in ? *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.base) + at) : 0u;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at);
    if (a < 0) {
        if (in) *out = was;
        return;
    }
    const uint4* rows = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(p.B) +
        (static_cast<long long>(a) * p.N + (p.rowwise ? 0 : static_cast<long long>(shard) * p.n) + (in ? col : 0)) * p.R);
    const int eights = p.R / 8;
    uint4 b0[2], b1[2];  // of both columns; the first 16 elements, while t is read
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        b0[e] = e < eights ? __ldg(rows + e) : make_uint4(0, 0, 0, 0);
        b1[e] = e < eights ? __ldg(rows + eights + e) : make_uint4(0, 0, 0, 0);
    }
    // t: R elements, kThreads / R threads each
    {
        const int shards = p.rowwise ? p.P : 1, ways = kThreads / p.R, r = tid % p.R, way = tid / p.R;
        const float* from = p.t + (static_cast<long long>(p.rowwise ? shard : 0) * p.M + m) * p.R + r;
        float v = 0.f;
        if (way < ways)
#pragma unroll 4
            for (int s = way; s < p.splits; s += ways) v += from[static_cast<long long>(s) * shards * p.M * p.R];
        part[tid] = v;
        __syncthreads();
        if (tid < p.R) {
            for (int w = 1; w < ways; ++w) v += part[w * p.R + tid];
            st[tid] = p.gains != nullptr ? v * __ldg(p.gains + a) : v;
        }
        __syncthreads();
    }
    float2 sum = unpack2(was);
    auto add8 = [&](const uint4& u, const uint4& v, int r) {
        const uint32_t *x = reinterpret_cast<const uint32_t*>(&u), *y = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t2 = *reinterpret_cast<const float2*>(st + r + 2 * j), f = unpack2(x[j]), h = unpack2(y[j]);
            sum.x = fmaf(t2.x, f.x, fmaf(t2.y, f.y, sum.x));
            sum.y = fmaf(t2.x, h.x, fmaf(t2.y, h.y, sum.y));
        }
    };
    add8(b0[0], b1[0], 0);
    if (eights > 1) add8(b0[1], b1[1], 8);
#pragma unroll 4
    for (int e = 2; e < eights; ++e) add8(__ldg(rows + e), __ldg(rows + eights + e), 8 * e);
    if (in) *out = pack2(sum.x, sum.y);
}

// ---------------------------------------------------------------- fp32, CUDA cores
constexpr int kRowsF = 8;

// A warp has 8 rows, one split and 8 elements of t: lanes along K, four elements
// each, and sums over the lanes at the end.
constexpr int kDownWarps = 2;  // of a block: few rows spread over the SMs
__global__ void __launch_bounds__(32 * kDownWarps) lora_down_f32(const __grid_constant__ LoraParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    await_previous();
    const int tiles = (p.M + kRowsF - 1) / kRowsF, parts = p.R / 8;
    long long unit = static_cast<long long>(blockIdx.x) * kDownWarps + warp;
    const int r0 = static_cast<int>(unit % parts) * 8;
    unit /= parts;
    const int m0 = static_cast<int>(unit % tiles) * kRowsF;
    unit /= tiles;
    const int split = static_cast<int>(unit % p.splits), shard = static_cast<int>(unit / p.splits);
    if (shard >= (p.rowwise ? p.P : 1)) return;
    const Ids ids(p, m0, kRowsF);
    admit_next();
    const int k0 = split * p.split_k, k1 = min(p.f, k0 + p.split_k);
    const float* x = static_cast<const float*>(p.x) + (static_cast<long long>(shard) * p.M + m0) * p.f;
    float* t = p.t + ((static_cast<long long>(split) * (p.rowwise ? p.P : 1) + shard) * p.M + m0) * p.R + r0;
    for (uint32_t left = ids.first; left != 0; left &= left - 1) {
        const int a = ids.of(__ffs(left) - 1);
        const uint32_t mine = __ballot_sync(0xffffffffu, ids.id == a);  // rows
        const float* A = static_cast<const float*>(p.A) + (static_cast<long long>(a) * p.R + r0) * p.K + (p.rowwise ? shard * p.f : 0);
        float acc[kRowsF][8] = {};
        for (int k = k0 + lane * 4; k < k1; k += 128) {
            float4 w[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) w[r] = __ldg(reinterpret_cast<const float4*>(A + static_cast<long long>(r) * p.K + k));
#pragma unroll
            for (int m = 0; m < kRowsF; ++m) {
                if (!(mine >> m & 1)) continue;
                const float4 v = __ldg(reinterpret_cast<const float4*>(x + static_cast<long long>(m) * p.f + k));
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    acc[m][r] = fmaf(v.x, w[r].x, fmaf(v.y, w[r].y, fmaf(v.z, w[r].z, fmaf(v.w, w[r].w, acc[m][r]))));
            }
        }
#pragma unroll
        for (int m = 0; m < kRowsF; ++m) {
            if (!(mine >> m & 1)) continue;
            float keep = 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float v = acc[m][r];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
                if (lane == r) keep = v;
            }
            if (lane < 8) t[static_cast<long long>(m) * p.R + lane] = keep;
        }
    }
}

// A block has 8 rows and an adapter's rows of B at a time; a thread has two columns
// for every read of t.  Above rank 16, LANES = 4 lanes share a column's 16-byte pieces
// of B, so that a load touches 8 of B's rows and not 32 (4911 rows of rank 64, two
// launches: 173 us, and 223 with a lane a column); up to it, where the sums over the
// lanes would cost more than that, a column is one lane's (3000 rows of rank 16: 84 us,
// and 117 with four).
constexpr int kColsF = 2;
template <int LANES>
__global__ void __launch_bounds__(kThreads) lora_up_f32(const __grid_constant__ LoraParams p, int col_blocks) {
    constexpr int WIDTH = kThreads / LANES * kColsF;  // columns of a round
    __shared__ __align__(16) float st[kRowsF][kLoraMaxRank];
    admit_next();
    const int m0 = blockIdx.x / col_blocks * kRowsF;
    await_previous();
    if (blockIdx.x == gridDim.x - 1) {
        report_rows(p);
        return;
    }
    const Ids ids(p, m0, kRowsF);
    const bool in_place = p.out == p.base;
    if (ids.first == 0 && in_place) return;
    const uint32_t some = __ballot_sync(0xffffffffu, ids.id >= 0);  // rows with an adapter
    const int shards = p.rowwise ? p.P : 1;
    for (int shard = 0; shard < shards; ++shard) {
        __syncthreads();
        for (int u = threadIdx.x; u < kRowsF * p.R; u += kThreads) {
            const int m = u / p.R, r = u % p.R;
            const int a = m0 + m < p.M ? __ldg(p.ids + m0 + m) : -1;
            float v = 0.f;
            if (a >= 0 && a < p.adapters) {
                const float* at = p.t + (static_cast<long long>(shard) * p.M + m0 + m) * p.R + r;
#pragma unroll 4
                for (int s = 0; s < p.splits; ++s) v += at[static_cast<long long>(s) * shards * p.M * p.R];
                if (p.gains != nullptr) v *= __ldg(p.gains + a);
            }
            st[m][r] = v;
        }
        __syncthreads();
        const int part = threadIdx.x % LANES;
        const int rounds = (p.N + WIDTH * col_blocks - 1) / (WIDTH * col_blocks);
        for (int round = 0; round < rounds; ++round) {  // (whole warps: sums are exchanged between lanes)
            const int col0 = (round * col_blocks + blockIdx.x % col_blocks) * WIDTH + threadIdx.x / LANES;
            long long at0[kColsF];
            bool in[kColsF];
            float was[kColsF][kRowsF / LANES], acc[kColsF][kRowsF] = {};
#pragma unroll
            for (int c = 0; c < kColsF; ++c) {
                const int col = col0 + c * (kThreads / LANES);
                in[c] = col < p.N;
                const int sh = p.rowwise || !in[c] ? shard : col / p.n;
                at0[c] = (static_cast<long long>(sh) * p.M + m0) * p.n + (p.rowwise ? col : col - sh * p.n);
                // this lane's rows: part, part + LANES ..
#pragma unroll
                for (int e = 0; e < kRowsF / LANES; ++e) {
                    const int m = e * LANES + part;
                    was[c][e] = in[c] && m0 + m < p.M ? static_cast<const float*>(p.base)[at0[c] + static_cast<long long>(m) * p.n] : 0.f;
                }
            }
            for (uint32_t left = ids.first; left != 0; left &= left - 1) {
                const int a = ids.of(__ffs(left) - 1);
                const uint32_t mine = __ballot_sync(0xffffffffu, ids.id == a);
                const float4* row = reinterpret_cast<const float4*>(static_cast<const float*>(p.B) +
                                                                    (static_cast<long long>(a) * p.N + col0) * p.R);
                const int next = kThreads / LANES * (p.R / 4);  // from a column's row of B to the other's
#pragma unroll 2
                for (int r = part; r < p.R / 4; r += LANES) {
                    float4 w[kColsF];
#pragma unroll
                    for (int c = 0; c < kColsF; ++c) w[c] = in[c] ? __ldg(row + c * next + r) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int m = 0; m < kRowsF; ++m) {
                        if (!(mine >> m & 1)) continue;
                        const float4 v = *reinterpret_cast<const float4*>(&st[m][r * 4]);
#pragma unroll
                        for (int c = 0; c < kColsF; ++c)
                            acc[c][m] = fmaf(v.x, w[c].x, fmaf(v.y, w[c].y, fmaf(v.z, w[c].z, fmaf(v.w, w[c].w, acc[c][m]))));
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < kColsF; ++c)
#pragma unroll
                for (int m = 0; m < kRowsF; ++m) {
                    float v = acc[c][m];
#pragma unroll
                    for (int off = 1; off < LANES; off *= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
                    if (m % LANES == part && in[c] && m0 + m < p.M && (!in_place || (some >> m & 1)))
                        static_cast<float*>(p.out)[at0[c] + static_cast<long long>(m) * p.n] = was[c][m / LANES] + v;
                }
        }
    }
}

// A kernel's dynamic shared memory, asked for once on each device.
template <class K>
struct RoomFor {
    K kernel;
    int bytes;
    std::atomic<unsigned long long> done{0};

    RoomFor(K k, int b) : kernel(k), bytes(b) {}
    cudaError_t made() {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        const unsigned long long bit = 1ull << (dev & 63);
        if (e != cudaSuccess || (done.load(std::memory_order_relaxed) & bit)) return e;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

template <int NT>
cudaError_t down(const LoraParams& p, cudaStream_t s) {
    static RoomFor room{lora_down_bf16<NT>, DownRing<NT>::BYTES};
    const cudaError_t e = room.made();
    if (e != cudaSuccess) return e;
    return launch_after(lora_down_bf16<NT>, (p.M + 15) / 16 * p.splits * (p.rowwise ? p.P : 1), kThreads, DownRing<NT>::BYTES, s, p);
}

template <int KT, int NC>
cudaError_t up(const LoraParams& p, int num_sms, cudaStream_t s) {
    // Blocks of columns: fewer than fill the SMs twice (each reads t and the adapters'
    // numbers), one where the rows alone do.
    const int tiles = (p.M + 15) / 16, chunks = (p.n + 32 * NC - 1) / (32 * NC) * p.P;
    int col_blocks = 4 * num_sms / tiles;
    const int most = (chunks + kWarps - 1) / kWarps;
    col_blocks = col_blocks < 1 ? 1 : col_blocks > most ? most : col_blocks;
    return launch_after(lora_up_bf16<KT, NC>, tiles * col_blocks + 1, kThreads, 0, s, p, col_blocks);
}

template <int LANES>
cudaError_t up_f32(const LoraParams& p, int row_tiles, int num_sms, cudaStream_t s) {
    constexpr int WIDTH = kThreads / LANES * kColsF;
    int col_blocks = (4 * num_sms + row_tiles - 1) / row_tiles;
    const int most_cols = (p.N + WIDTH - 1) / WIDTH;
    if (col_blocks > most_cols) col_blocks = most_cols;
    return launch_after(lora_up_f32<LANES>, row_tiles * col_blocks + 1, kThreads, 0, s, p, col_blocks);
}

}  // namespace

cudaError_t launch_lora(LoraParams& p, bool bf16, int num_sms, cudaStream_t s) {
    cudaError_t e;
    if (!bf16) {
        const int row_tiles = (p.M + kRowsF - 1) / kRowsF;
        const long long units = static_cast<long long>(row_tiles) * (p.R / 8) * p.splits * (p.rowwise ? p.P : 1);
        e = launch_after(lora_down_f32, static_cast<int>((units + kDownWarps - 1) / kDownWarps), 32 * kDownWarps, 0, s, p);
        if (e != cudaSuccess) return e;
        return p.R <= 16 ? up_f32<1>(p, row_tiles, num_sms, s) : up_f32<4>(p, row_tiles, num_sms, s);
    }
    e = p.R <= 16 ? down<2>(p, s) : p.R <= 32 ? down<4>(p, s) : down<8>(p, s);
    if (e != cudaSuccess) return e;
    if (p.M < kLoraFew) {
        const int col_blocks = (p.n + 2 * kThreads - 1) / (2 * kThreads) * p.P;
        return launch_after(lora_up_row_bf16, p.M * col_blocks + 1, kThreads, 0, s, p, col_blocks);
    }
    if (p.R <= 16) return up<1, 2>(p, num_sms, s);
    if (p.R <= 32) return up<2, 1>(p, num_sms, s);
    if (p.R <= 64) return up<4, 1>(p, num_sms, s);
    return up<8, 1>(p, num_sms, s);
}

}  // namespace sptp
