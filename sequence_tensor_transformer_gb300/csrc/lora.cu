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
// v = hi + lo up to 2^-16 of it
__device__ __forceinline__ void split2bf(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack2(x, y);
    const float2 h = unpack2(hi);
    lo = pack2(x - h.x, y - h.y);
}

// The adapters of a tile of ROWS rows, each distinct one once, in the order in
// which they first come.
template <int ROWS>
struct Tile {
    int id[ROWS];       // -1: none
    int distinct[ROWS];
    int count;
};

template <int ROWS>
__device__ __forceinline__ void load_tile(Tile<ROWS>& t, const LoraParams& p, int m0) {
    const int tid = threadIdx.x;
    if (tid < ROWS) {
        const int a = m0 + tid < p.M ? __ldg(p.ids + m0 + tid) : -1;
        t.id[tid] = a < 0 || a >= p.adapters ? -1 : a;
    }
    __syncthreads();
    if (tid < 32) {
        int n = 0;
#pragma unroll
        for (int r0 = 0; r0 < ROWS; r0 += 32) {
            const int r = r0 + tid;
            const int a = r < ROWS ? t.id[r] : -1;
            bool first = a >= 0;
            for (int i = 0; first && i < r; ++i) first = t.id[i] != a;
            const uint32_t mask = __ballot_sync(0xffffffffu, first);
            if (first) t.distinct[n + __popc(mask & ((1u << tid) - 1u))] = a;
            n += __popc(mask);
        }
        if (tid == 0) t.count = n;
    }
    __syncthreads();
}

__device__ __forceinline__ uint4 load16(const void* base, long long elem, bool in) {
    return in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + elem)) : make_uint4(0, 0, 0, 0);
}

// The status words: the first row whose adapter is outside its range.  By the
// last block of the second launch.
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
        *p.status = st;
    }
}

// ---------------------------------------------------------------- t = A x, bf16
// A block has 16 MT rows and one split of K.  Its warps share out the tile's
// adapters, and the split's elements where there are fewer adapters than warps
// (their sums are then added in order).
template <int MT, int NT>
__global__ void __launch_bounds__(kThreads) lora_down_bf16(const __grid_constant__ LoraParams p) {
    constexpr int ROWS = 16 * MT;
    __shared__ Tile<ROWS> tile;
    __shared__ __align__(16) float sums[kWarps / 2][ROWS * NT * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, i = lane & 3;
    admit_next();
    await_previous();
    const int tiles = (p.M + ROWS - 1) / ROWS;
    const int m0 = blockIdx.x % tiles * ROWS;
    const int rest = blockIdx.x / tiles, split = rest % p.splits, shard = rest / p.splits;
    load_tile(tile, p, m0);
    const int count = tile.count;
    if (count == 0) return;
    int groups = 1;
    while (groups < count && groups < kWarps) groups *= 2;
    const int ways = kWarps / groups, group = warp / ways, sub = warp % ways;
    const int k0 = split * p.split_k, k1 = min(p.f, k0 + p.split_k);
    const long long xrow = static_cast<long long>(shard) * p.M + m0;
    float* t = p.t + (static_cast<long long>(rest % p.splits) * (p.rowwise ? p.P : 1) + shard) * p.M * p.R;
    for (int r0 = 0; r0 < p.R; r0 += NT * 8) {
        for (int first = 0; first < count; first += groups) {
            const bool mine = first + group < count;
            const int a = mine ? tile.distinct[first + group] : -1;
            float acc[MT][NT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
            if (mine) {
                bool has[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    has[mt] = __any_sync(0xffffffffu, tile.id[mt * 16 + (lane & 15)] == a);
                const long long arow = (static_cast<long long>(a) * p.R + r0 + g) * p.K + (p.rowwise ? shard * p.f : 0);
#pragma unroll 4
                for (int k = k0 + sub * 32; k < k1; k += ways * 32) {
                    const int kk = k + i * 8;
                    const bool in = kk < k1;
                    uint4 w[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        w[nt] = load16(p.A, arow + static_cast<long long>(nt) * 8 * p.K + kk, in && r0 + nt * 8 < p.R);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if (!has[mt]) continue;
                        const uint4 u = load16(p.x, (xrow + mt * 16 + g) * p.f + kk, in && m0 + mt * 16 + g < p.M);
                        const uint4 v = load16(p.x, (xrow + mt * 16 + g + 8) * p.f + kk, in && m0 + mt * 16 + g + 8 < p.M);
                        const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_bf16(acc[mt][nt], a0, w[nt].x, w[nt].y);
                            mma_bf16(acc[mt][nt], a1, w[nt].z, w[nt].w);
                        }
                    }
                }
            }
            // rows of this adapter: lane's elements (g, 2i), (g, 2i + 1), (g + 8, ..) of each 16 x 8
            auto each = [&](auto f) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) f(acc[mt][nt][2 * e], acc[mt][nt][2 * e + 1], mt * 16 + g + 8 * e, nt * 8 + 2 * i);
            };
            for (int half = ways / 2; half > 0; half /= 2) {  // warps [half, 2 half) of a group to [0, half)
                if (sub >= half && sub < 2 * half)
                    each([&](float x, float y, int row, int r) {
                        *reinterpret_cast<float2*>(&sums[group * half + sub - half][row * NT * 8 + r]) = make_float2(x, y);
                    });
                __syncthreads();
                if (sub < half)
                    each([&](float& x, float& y, int row, int r) {
                        const float2 o = *reinterpret_cast<const float2*>(&sums[group * half + sub][row * NT * 8 + r]);
                        x += o.x;
                        y += o.y;
                    });
                __syncthreads();
            }
            if (mine && sub == 0)
                each([&](float x, float y, int row, int r) {
                    if (tile.id[row] == a && r0 + r < p.R)
                        *reinterpret_cast<float2*>(t + static_cast<long long>(m0 + row) * p.R + r0 + r) = make_float2(x, y);
                });
        }
    }
}

// ---------------------------------------------------------------- out = base + B t, bf16
// A block has 16 MT rows; its warps take chunks of 32 columns in turn.
template <int MT, int KT>
__global__ void __launch_bounds__(kThreads) lora_up_bf16(const __grid_constant__ LoraParams p, int col_blocks) {
    constexpr int ROWS = 16 * MT;
    __shared__ Tile<ROWS> tile;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, i = lane & 3;
    admit_next();
    const int m0 = blockIdx.x / col_blocks * ROWS;
    await_previous();
    if (blockIdx.x == gridDim.x - 1) {
        report_rows(p);
        return;
    }
    load_tile(tile, p, m0);
    const int count = tile.count;
    const bool in_place = p.out == p.base;
    if (count == 0 && in_place) return;
    const int shards = p.rowwise ? p.P : 1;
    const int chunks = (p.N + 31) / 32;  // of a shard's columns (rowwise) or of all shards'
    for (int shard = 0; shard < shards; ++shard) {
        // this lane's part of t, times the gain: rows g and g + 8 of each 16, elements 4 i .. 4 i + 3 of each 16
        uint32_t hi[MT][KT][4], lo[MT][KT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = mt * 16 + g + 8 * e, a = tile.id[row];
                const float gain = a < 0 ? 0.f : p.gains != nullptr ? __ldg(p.gains + a) : 1.f;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (a >= 0 && kt * 16 + 4 * i < p.R) {
                        const float* at = p.t + (static_cast<long long>(shard) * p.M + m0 + row) * p.R + kt * 16 + 4 * i;
                        const long long stride = static_cast<long long>(shards) * p.M * p.R;
#pragma unroll 4
                        for (int s = 0; s < p.splits; ++s) {
                            const float4 u = *reinterpret_cast<const float4*>(at + s * stride);
                            v.x += u.x;
                            v.y += u.y;
                            v.z += u.z;
                            v.w += u.w;
                        }
                    }
                    split2bf(v.x * gain, v.y * gain, hi[mt][kt][e], lo[mt][kt][e]);
                    split2bf(v.z * gain, v.w * gain, hi[mt][kt][2 + e], lo[mt][kt][2 + e]);
                }
            }
        for (int chunk = blockIdx.x % col_blocks * kWarps + warp; chunk < chunks; chunk += col_blocks * kWarps) {
            // lane i has columns 8 i .. 8 i + 7 of the chunk: 2 j and 2 j + 1 of them in product j
            const int col = chunk * 32 + 8 * i;
            const bool cin = col < p.N;
            const int sh = p.rowwise ? shard : col / p.n;
            const long long at0 = (static_cast<long long>(sh) * p.M + m0) * p.n + (p.rowwise ? col : col - sh * p.n);
            uint4 was[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = mt * 16 + g + 8 * e;
                    const bool need = cin && m0 + row < p.M && (!in_place || tile.id[row] >= 0);
                    was[mt][e] = make_uint4(0, 0, 0, 0);
                    if (need)
                        was[mt][e] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.base) + at0 +
                                                                     static_cast<long long>(row) * p.n);
                }
            float acc[MT][4][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[mt][j][e] = 0.f;
#pragma unroll 2
            for (int d = 0; d < count; ++d) {
                const int a = tile.distinct[d];
                uint2 b[KT][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = chunk * 32 + 8 * (g >> 1) + 2 * j + (g & 1);
                    const __nv_bfloat16* row =
                        static_cast<const __nv_bfloat16*>(p.B) + (static_cast<long long>(a) * p.N + n) * p.R + 4 * i;
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
                        b[kt][j] = n < p.N && kt * 16 + 4 * i < p.R ? __ldg(reinterpret_cast<const uint2*>(row + kt * 16))
                                                                    : make_uint2(0, 0);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const bool me0 = tile.id[mt * 16 + g] == a, me1 = tile.id[mt * 16 + g + 8] == a;
                    if (!__any_sync(0xffffffffu, me0 || me1)) continue;
                    // (sums of their own, kept by this adapter's rows: another's
                    // infinities do not reach a row)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt) {
                            mma_bf16(c, hi[mt][kt], b[kt][j].x, b[kt][j].y);
                            mma_bf16(c, lo[mt][kt], b[kt][j].x, b[kt][j].y);
                        }
                        if (me0) {
                            acc[mt][j][0] = c[0];
                            acc[mt][j][1] = c[1];
                        }
                        if (me1) {
                            acc[mt][j][2] = c[2];
                            acc[mt][j][3] = c[3];
                        }
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = mt * 16 + g + 8 * e;
                    if (!cin || m0 + row >= p.M || (in_place && tile.id[row] < 0)) continue;
                    uint4 now = was[mt][e];
                    if (tile.id[row] >= 0) {
                        uint32_t* w = reinterpret_cast<uint32_t*>(&now);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = unpack2(w[j]);
                            w[j] = pack2(f.x + acc[mt][j][2 * e], f.y + acc[mt][j][2 * e + 1]);
                        }
                    }
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at0 + static_cast<long long>(row) * p.n) = now;
                }
        }
    }
}

// ---------------------------------------------------------------- fp32, CUDA cores
constexpr int kRowsF = 8;

// A block has 8 rows and one split; a warp 8 elements of t at a time: lanes along
// K, four elements each, and sums over the lanes at the end.
__global__ void __launch_bounds__(kThreads) lora_down_f32(const __grid_constant__ LoraParams p) {
    __shared__ Tile<kRowsF> tile;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    admit_next();
    await_previous();
    const int tiles = (p.M + kRowsF - 1) / kRowsF;
    const int m0 = blockIdx.x % tiles * kRowsF;
    const int rest = blockIdx.x / tiles, split = rest % p.splits, shard = rest / p.splits;
    load_tile(tile, p, m0);
    const int k0 = split * p.split_k, k1 = min(p.f, k0 + p.split_k);
    const float* x = static_cast<const float*>(p.x) + (static_cast<long long>(shard) * p.M + m0) * p.f;
    float* t = p.t + (static_cast<long long>(split) * (p.rowwise ? p.P : 1) + shard) * p.M * p.R;
    const int units = tile.count * (p.R / 8);
    for (int u = warp; u < units; u += kWarps) {
        const int a = tile.distinct[u / (p.R / 8)], r0 = u % (p.R / 8) * 8;
        const float* A = static_cast<const float*>(p.A) + (static_cast<long long>(a) * p.R + r0) * p.K + (p.rowwise ? shard * p.f : 0);
        float acc[kRowsF][8] = {};
        for (int k = k0 + lane * 4; k < k1; k += 128) {
            float4 w[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) w[r] = __ldg(reinterpret_cast<const float4*>(A + static_cast<long long>(r) * p.K + k));
#pragma unroll
            for (int m = 0; m < kRowsF; ++m) {
                if (tile.id[m] != a) continue;
                const float4 v = __ldg(reinterpret_cast<const float4*>(x + static_cast<long long>(m) * p.f + k));
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    acc[m][r] = fmaf(v.x, w[r].x, fmaf(v.y, w[r].y, fmaf(v.z, w[r].z, fmaf(v.w, w[r].w, acc[m][r]))));
            }
        }
#pragma unroll
        for (int m = 0; m < kRowsF; ++m) {
            if (tile.id[m] != a) continue;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float v = acc[m][r];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
                if (lane == r) t[static_cast<long long>(m0 + m) * p.R + r0 + r] = v;
            }
        }
    }
}

// A block has 8 rows; a thread a column of all of them, an adapter's rows at a time.
__global__ void __launch_bounds__(kThreads) lora_up_f32(const __grid_constant__ LoraParams p, int col_blocks) {
    __shared__ Tile<kRowsF> tile;
    __shared__ __align__(16) float st[kRowsF][kLoraMaxRank];
    admit_next();
    const int m0 = blockIdx.x / col_blocks * kRowsF;
    await_previous();
    if (blockIdx.x == gridDim.x - 1) {
        report_rows(p);
        return;
    }
    load_tile(tile, p, m0);
    const bool in_place = p.out == p.base;
    if (tile.count == 0 && in_place) return;
    const int shards = p.rowwise ? p.P : 1;
    for (int shard = 0; shard < shards; ++shard) {
        __syncthreads();
        for (int u = threadIdx.x; u < kRowsF * p.R; u += kThreads) {
            const int m = u / p.R, r = u % p.R, a = tile.id[m];
            float v = 0.f;
            if (a >= 0) {
                const float* at = p.t + (static_cast<long long>(shard) * p.M + m0 + m) * p.R + r;
                for (int s = 0; s < p.splits; ++s) v += at[static_cast<long long>(s) * shards * p.M * p.R];
                if (p.gains != nullptr) v *= __ldg(p.gains + a);
            }
            st[m][r] = v;
        }
        __syncthreads();
        for (int col = blockIdx.x % col_blocks * kThreads + threadIdx.x; col < p.N; col += col_blocks * kThreads) {
            const int sh = p.rowwise ? shard : col / p.n;
            const long long at0 = (static_cast<long long>(sh) * p.M + m0) * p.n + (p.rowwise ? col : col - sh * p.n);
            float acc[kRowsF] = {};
            for (int d = 0; d < tile.count; ++d) {
                const int a = tile.distinct[d];
                const float4* row = reinterpret_cast<const float4*>(static_cast<const float*>(p.B) +
                                                                    (static_cast<long long>(a) * p.N + col) * p.R);
#pragma unroll 4
                for (int r = 0; r < p.R / 4; ++r) {
                    const float4 w = __ldg(row + r);
#pragma unroll
                    for (int m = 0; m < kRowsF; ++m) {
                        if (tile.id[m] != a) continue;
                        const float4 v = *reinterpret_cast<const float4*>(&st[m][r * 4]);
                        acc[m] = fmaf(v.x, w.x, fmaf(v.y, w.y, fmaf(v.z, w.z, fmaf(v.w, w.w, acc[m]))));
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < kRowsF; ++m) {
                if (m0 + m >= p.M || (in_place && tile.id[m] < 0)) continue;
                const long long at = at0 + static_cast<long long>(m) * p.n;
                static_cast<float*>(p.out)[at] = static_cast<const float*>(p.base)[at] + acc[m];
            }
        }
    }
}

template <int MT, int NT>
cudaError_t down(const LoraParams& p, cudaStream_t s) {
    const int grid = (p.M + 16 * MT - 1) / (16 * MT) * p.splits * (p.rowwise ? p.P : 1);
    return launch_after(lora_down_bf16<MT, NT>, grid, kThreads, 0, s, p);
}

template <int MT, int KT>
cudaError_t up(const LoraParams& p, int num_sms, cudaStream_t s) {
    // blocks of columns: a few chunks a warp, fewer where the rows alone do not fill the SMs
    const int tiles = (p.M + 16 * MT - 1) / (16 * MT), chunks = (p.N + 31) / 32;
    int col_blocks = (2 * num_sms + tiles - 1) / tiles;
    const int most = (chunks + kWarps - 1) / kWarps;
    if (col_blocks > most) col_blocks = most;
    return launch_after(lora_up_bf16<MT, KT>, tiles * col_blocks + 1, kThreads, 0, s, p, col_blocks);
}

}  // namespace

cudaError_t launch_lora(LoraParams& p, bool bf16, int num_sms, cudaStream_t s) {
    cudaError_t e;
    const bool many = p.M >= kLoraMany;
    if (!bf16) {
        const int row_tiles = (p.M + kRowsF - 1) / kRowsF;
        e = launch_after(lora_down_f32, row_tiles * p.splits * (p.rowwise ? p.P : 1), kThreads, 0, s, p);
        if (e != cudaSuccess) return e;
        int col_blocks = (4 * num_sms + row_tiles - 1) / row_tiles;
        const int most_cols = (p.N + kThreads - 1) / kThreads;
        if (col_blocks > most_cols) col_blocks = most_cols;
        return launch_after(lora_up_f32, row_tiles * col_blocks + 1, kThreads, 0, s, p, col_blocks);
    }
    if (p.R <= 16)
        e = many ? down<4, 2>(p, s) : down<1, 2>(p, s);
    else if (p.R <= 32)
        e = many ? down<4, 4>(p, s) : down<1, 4>(p, s);
    else
        e = many ? down<2, 8>(p, s) : down<1, 8>(p, s);
    if (e != cudaSuccess) return e;
    if (p.R <= 16) return many ? up<4, 1>(p, num_sms, s) : up<1, 1>(p, num_sms, s);
    if (p.R <= 32) return many ? up<4, 2>(p, num_sms, s) : up<1, 2>(p, num_sms, s);
    if (p.R <= 64) return many ? up<2, 4>(p, num_sms, s) : up<1, 4>(p, num_sms, s);
    return up<1, 8>(p, num_sms, s);
}

}  // namespace sptp
