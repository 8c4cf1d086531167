// Rotary positions, alone (sptp_rope) and on the way into a paged key-value
// cache (sptp_rope_append_kv).  Pair i of a head at position m turns by
// m * f_i: (a, b) -> gain (a cos t - b sin t, a sin t + b cos t); the gradient
// is the same with -t.
//
// Angles.  f_i is kept in turns per position as a 64-bit binary fraction u_i,
// so m * u_i mod 2^64 (one integer product) is the angle's fraction of a turn
// without rounding: its top bits, as a signed number, are converted to fp32
// (2^-25 of a turn) and go to sincospif.  No 64-bit floating point, no table
// over the positions, and a far position is as exact as a near one.
//
// Both are bound by HBM: every element is read once and written once with
// 16-byte accesses, and nothing else is large.  A block takes one to four
// tokens: its first loads are under way while its threads work out the tokens'
// cosines and sines, each once, into shared memory.  A lane owns one slot of a
// head, two 16-byte vectors (half layout: the vectors at c and c + rot/2 hold
// each other's partners; interleaved: any two; elements that do not turn: any
// two), L lanes cover a head, and a warp walks over its rows (heads of a token,
// all shards') with the slot's cosines and sines in registers.
//
// Measured, 16384 rows of 36 heads of 128 over 4 shards in bf16 (302 MB): 46.3 us
// (6.5 TB/s, 0.97 of the copy bandwidth) rotated alone, 48.6 us (0.93) with k and
// v into pages; with each lane working out its own angles 49.9 and 62.7 us.  One
// row: 2.0 us, a launch.
#include <cuda_bf16.h>

#include "attn.h"
#include "e4m3.cuh"
#include "sptp.h"
#include "sptp_ptx.cuh"

namespace sptp {

namespace {

enum class Op { kRope, kAppend, kAppendE4M3 };

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;

// How the rows of the tokens are dealt out (host).
struct Split {
    int L;           // lanes of a head
    int hpw;         // heads that a warp has side by side, 32 / L
    int tokens;      // of a block: 1, 2 or 4; a token has kWarps / tokens of its warps
    int parts;       // blocks that share a token's rows (tokens == 1)
    int per;         // rows of a warp
    int checker;     // append: the first block writes the status words
    uint32_t mul;    // row / H = (2 row * mul) >> (32 + shift) for rows below 2^24
    int shift;
};

template <typename T>
struct Elems {
    static constexpr int E = 16 / sizeof(T);
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4 u, float (&f)[Elems<T>::E]) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __bfloat1622float2(h[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    } else {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[Elems<T>::E]) {
    if constexpr (sizeof(T) == 2) {
        uint4 u;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        return u;
    } else {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
}

// Turns the pairs of one slot in place.
template <typename T, bool INTER>
__device__ __forceinline__ void turn(uint4& ua, uint4& ub, const float (&c)[Elems<T>::E], const float (&s)[Elems<T>::E]) {
    constexpr int E = Elems<T>::E;
    float a[E], b[E], y[E], z[E];
    unpack<T>(ua, a);
    unpack<T>(ub, b);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if constexpr (INTER) {
            // pairs 0 .. E/2-1 lie in a, the others in b
            const float* src = e < E / 2 ? a : b;
            float* dst = e < E / 2 ? y : z;
            const int i = 2 * (e % (E / 2));
            dst[i] = src[i] * c[e] - src[i + 1] * s[e];
            dst[i + 1] = src[i] * s[e] + src[i + 1] * c[e];
        } else {
            y[e] = a[e] * c[e] - b[e] * s[e];
            z[e] = a[e] * s[e] + b[e] * c[e];
        }
    }
    ua = pack<T>(y);
    ub = pack<T>(z);
}

// The page that a token's key and value go to; -1 if an index is out of range.
__device__ __forceinline__ int kv_page(const RopeParams& p, int seq, int pos) {
    if (seq < 0 || seq >= p.B || pos < 0 || pos / p.page_size >= p.max_pages) return -1;
    const int page = __ldg(p.page_table + static_cast<long long>(seq) * p.max_pages + pos / p.page_size);
    return page >= 0 && page < p.num_pages ? page : -1;
}

// The status words of an append, written once by a block of its own: it looks at
// all rows' indexes, beside the blocks that move the data (which skip the bad
// ones silently), so that no launch has to clear the words first.  That takes
// it about 1 us per 1024 rows, hidden behind the data where a row is large; a
// launch that clears the words, and blocks that report what they meet, cost 3.5
// us (16384 rows of 18 KB: 53.0 and 49.5 us).  So one block checks where there
// are few rows, or rows of kCheckBytes, which take as long to move.
constexpr int kCheckRows = 2048;
constexpr int kCheckBytes = 8192;

__device__ __forceinline__ void check_rows(const RopeParams& p) {
    constexpr int N = 8;
    __shared__ int first_bad;
    if (threadIdx.x == 0) first_bad = 0x7fffffff;
    __syncthreads();
    int seq[N], pos[N];
    auto load = [&](int m0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int m = m0 + i * kThreads + static_cast<int>(threadIdx.x);
            seq[i] = m < p.M ? __ldg(p.seq_ids + m) : -1;
            pos[i] = m < p.M ? __ldg(p.positions + m) : 0;
        }
    };
    load(0);
    for (int m0 = 0; m0 < p.M; m0 += N * kThreads) {
        int page[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // (entry 0 where there is none to look up)
            const bool in = seq[i] >= 0 && seq[i] < p.B && pos[i] >= 0 && pos[i] / p.page_size < p.max_pages;
            const int at = __ldg(p.page_table + (in ? static_cast<long long>(seq[i]) * p.max_pages + pos[i] / p.page_size : 0));
            page[i] = seq[i] < 0 ? 0 : in ? at : -1;
        }
        load(m0 + N * kThreads < p.M ? m0 + N * kThreads : p.M);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (page[i] < 0 || page[i] >= p.num_pages) atomicMin(&first_bad, m0 + i * kThreads + static_cast<int>(threadIdx.x));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool bad = first_bad != 0x7fffffff;
        // a checked build clears the words before the launch: another block
        // may have written them, and a failed check stays there
        if (kBoundsChecked) {
            if (bad && atomicCAS(&p.status->code, 0, SPTP_ERR_SHAPE) == 0) {
                p.status->where = kWhereKvSlot;
                p.status->info = first_bad;
            }
            return;
        }
        DeviceStatus st;
        st.code = bad ? SPTP_ERR_SHAPE : SPTP_OK;
        st.where = bad ? kWhereKvSlot : 0;
        st.block = 0;
        st.info = bad ? first_bad : 0;
        st.flag = 0;
        *p.status = st;
    }
}

// One slot of N rows.
template <int N>
struct Batch {
    uint4 va[N], vb[N];
    int pp[N], hh[N];  // shard, head (-1: none)
};

// Rows whose loads a lane has in flight: four at a time alone; for an append,
// which waits for a page before its first store and has more to do per row,
// three and the next three, at one block less per SM (device us, one batch at a
// time / one ahead: 16384 bf16 rows of 18 KB 49.1 / 48.6, 3001 of them 12.1 /
// 11.3, 16384 E4M3 rows of 48 heads 67.4 / 65.8, 3001 of them 15.8 / 14.1; alone
// 46.3 / 48.1 to 50.5).
template <typename T, bool INTER, Op OP>
__global__ void __launch_bounds__(kThreads, OP == Op::kRope ? 6 : 5) rope_kernel(const __grid_constant__ RopeParams p,
                                                                              const __grid_constant__ Split sp) {
    constexpr int E = Elems<T>::E;
    constexpr int kUnroll = OP == Op::kRope ? 4 : 3;
    constexpr bool kAhead = OP != Op::kRope;
    __shared__ __align__(16) float cosines[4][kMaxPairs], sines[4][kMaxPairs];
    admit_next();
    await_previous();
    // the first block, so that it starts with the others and not after them
    if (OP != Op::kRope && sp.checker && blockIdx.x == 0) {
        check_rows(p);
        return;
    }
    const uint32_t block = blockIdx.x - (OP != Op::kRope ? sp.checker : 0);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hg = lane / sp.L, slot = lane - hg * sp.L;
    const int half = p.rot / 2;
    const int turning = half / E;  // slots that turn
    // the slot's two vectors (element offsets); a tail slot may lack the second
    const bool turns = slot < turning;
    const int still = ((p.D - p.rot) / E + 1) / 2;  // slots that do not
    const int ea = turns ? slot * E : p.rot + (slot - turning) * E;
    const int eb = ea + (turns ? half : still * E);
    const bool lives = hg < sp.hpw && slot < turning + still;
    const bool has_b = lives && eb < p.D;
    // this warp's token and rows
    const int wpt = kWarps / sp.tokens;
    const int m0 = block / sp.parts * sp.tokens, mi = warp / wpt, m = m0 + mi;
    const int r0 = (block % sp.parts * wpt + warp % wpt) * sp.per;
    const int r1 = m < p.M ? min(p.P * p.H, r0 + sp.per) : 0;

    Batch<kUnroll> now, next;
    auto load = [&](Batch<kUnroll>& to, int base) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int r = base + i * sp.hpw + hg;
            to.pp[i] = static_cast<int>(__umulhi(2u * static_cast<uint32_t>(r), sp.mul) >> sp.shift);
            to.hh[i] = lives && r < r1 ? r - to.pp[i] * p.H : -1;
            // in place, what does not turn stays where it is
            if (OP == Op::kRope && p.out == p.x && (to.hh[i] >= p.Hr || !turns)) to.hh[i] = -1;
            to.va[i] = to.vb[i] = make_uint4(0, 0, 0, 0);
            if (to.hh[i] >= 0) {
                const T* src =
                    static_cast<const T*>(p.x) + ((static_cast<long long>(to.pp[i]) * p.M + m) * p.H + to.hh[i]) * p.D;
                to.va[i] = __ldcs(reinterpret_cast<const uint4*>(src + ea));
                if (has_b) to.vb[i] = __ldcs(reinterpret_cast<const uint4*>(src + eb));
            }
        }
    };
    load(now, r0);

    // the angles of the block's tokens, while the first rows are under way
    for (int j = tid; j < sp.tokens * half; j += kThreads) {
        const int t = sp.tokens == 1 ? 0 : j / half, i = j - t * half;
        if (m0 + t < p.M) {
            const unsigned long long f = static_cast<unsigned long long>(static_cast<long long>(__ldg(p.positions + m0 + t))) *
                                         __ldg(p.turns + i);
            // signed: [-1/2, 1/2) turn = [-1, 1) half turns
            float s, c;
            sincospif(__ll2float_rn(static_cast<long long>(f)) * 0x1p-63f, &s, &c);
            cosines[t][i] = c * p.gain;
            sines[t][i] = s * (p.transpose ? -p.gain : p.gain);
        }
    }
    int page = -1, off = 0;
    if constexpr (OP != Op::kRope) {
        if (m < p.M) {
            const int seq = __ldg(p.seq_ids + m), pos = __ldg(p.positions + m);
            page = seq < 0 ? -2 : kv_page(p, seq, pos);  // -2: a padding row
            off = pos % p.page_size;
            if (page == -1 && !sp.checker && r0 == 0 && lane == 0 &&
                atomicCAS(&p.status->code, 0, SPTP_ERR_SHAPE) == 0) {
                p.status->where = kWhereKvSlot;
                p.status->info = m;
            }
        }
    }
    __syncthreads();
    if (OP != Op::kRope && page == -2) return;
    float c[E], s[E];
    if (turns && lives) {
        // half: pairs slot E + e; interleaved: the vectors' own E/2 pairs each
        const int ia = INTER ? slot * (E / 2) : slot * E;
        const int ib = INTER ? half / 2 + slot * (E / 2) : slot * E + E / 2;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            c[e] = cosines[mi][ia + e];
            c[E / 2 + e] = cosines[mi][ib + e];
            s[e] = sines[mi][ia + e];
            s[E / 2 + e] = sines[mi][ib + e];
        }
    }
    for (int base = r0; base < r1; base += sp.hpw * kUnroll) {
        const int after = base + sp.hpw * kUnroll;
        if (!kAhead && base != r0) load(now, base);
        if (kAhead && after < r1) load(next, after);
        auto& va = now.va;
        auto& vb = now.vb;
        const auto& pp = now.pp;
        const auto& hh = now.hh;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (turns && hh[i] >= 0 && hh[i] < p.Hr) turn<T, INTER>(va[i], vb[i], c, s);
            if constexpr (OP == Op::kRope) {
                if (hh[i] < 0) continue;
                T* dst = static_cast<T*>(p.out) + ((static_cast<long long>(pp[i]) * p.M + m) * p.H + hh[i]) * p.D;
                __stcs(reinterpret_cast<uint4*>(dst + ea), va[i]);
                if (has_b) __stcs(reinterpret_cast<uint4*>(dst + eb), vb[i]);
            } else {
                const bool is_q = hh[i] < p.Hq, is_v = hh[i] >= p.Hq + p.Hkv;
                const int kvh = hh[i] - p.Hq - (is_v ? p.Hkv : 0);
                // row of the cache, or of q_out
                const long long row = is_q ? (static_cast<long long>(pp[i]) * p.M + m) * p.Hq + hh[i]
                                           : ((pp[i] * p.num_pages + page) * p.Hkv + kvh) * p.page_size + off;
                const bool stores =
                    hh[i] >= 0 &&
                    (is_q || (page >= 0 && checked_index(row, static_cast<long long>(p.P) * p.num_pages * p.Hkv * p.page_size,
                                                         p.status, nullptr, kWhereBoundsStore)));
                if (stores && (is_q || OP == Op::kAppend)) {
                    T* dst = static_cast<T*>(is_q ? p.out : is_v ? p.v_cache : p.k_cache) + row * p.D;
                    __stcs(reinterpret_cast<uint4*>(dst + ea), va[i]);
                    if (has_b) __stcs(reinterpret_cast<uint4*>(dst + eb), vb[i]);
                }
                if constexpr (OP == Op::kAppendE4M3) {
                    // the head's row maximum over its L lanes (a power of two
                    // here); every lane of the warp takes part
                    float amax = fmaxf(absmax_bf16x8(va[i]), absmax_bf16x8(vb[i]));
                    for (int o = sp.L / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    if (stores && !is_q) {
                        const int ex = e4m3_row_exponent(amax);
                        const float inv = pow2f(-ex);
                        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + row * p.D;
                        *reinterpret_cast<uint2*>(dst + ea) = e4m3_quant8(va[i], inv);
                        if (has_b) *reinterpret_cast<uint2*>(dst + eb) = e4m3_quant8(vb[i], inv);
                        if (slot == 0) (is_v ? p.v_scale : p.k_scale)[row] = pow2f(ex);
                    }
                }
            }
        }
        if (kAhead) now = next;
    }
}

template <typename T, Op OP>
cudaError_t launch_typed(const RopeParams& p, int num_sms, cudaStream_t s) {
    constexpr int E = Elems<T>::E;
    Split sp;
    sp.L = p.rot / (2 * E) + ((p.D - p.rot) / E + 1) / 2;  // slots of a head
    if (OP == Op::kAppendE4M3) {  // a power of two, for the row maximum's exchanges
        int pow = 1;
        while (pow < sp.L) pow *= 2;
        sp.L = pow;
    }
    sp.hpw = 32 / sp.L;
    // Warps per token: enough for 40 per SM (24 are resident), or 10 for an
    // append, whose blocks each wait for their tokens' pages; at most one for
    // each group of heads.  (4097 rows of 40 heads: 11.6, 11.2 and 13.7 us for
    // 20, 40 and 80; 3001 appended E4M3 rows of 48: 19.9, 22.7 and 34 us for 10, 20 and 80.)
    const int rows = p.P * p.H;
    const int most = (rows + sp.hpw - 1) / sp.hpw;
    long long warps = (static_cast<long long>(num_sms) * (OP == Op::kRope ? 40 : 10) + p.M - 1) / p.M;
    if (warps > most) warps = most;
    const int wpt = warps <= 1 ? 1 : warps <= 2 ? 2 : 4;
    sp.tokens = kWarps / wpt;
    sp.parts = static_cast<int>((warps + wpt - 1) / wpt);
    if (sp.tokens > 1) sp.parts = 1;
    // whole groups of heads side by side
    sp.per = ((rows + wpt * sp.parts - 1) / (wpt * sp.parts) + sp.hpw - 1) / sp.hpw * sp.hpw;
    // with H <= 2^l and mul = floor(2^(31+l) / H) + 1, the error mul - 2^(31+l) / H <= 1 adds less than
    // row / 2^(31+l) < 1 / H to the quotient
    int l = 0;
    while ((1 << l) < p.H) ++l;
    sp.mul = static_cast<uint32_t>((1ull << (31 + l)) / static_cast<uint32_t>(p.H) + 1);
    sp.shift = l;
    long long grid = (static_cast<long long>(p.M) + sp.tokens - 1) / sp.tokens * sp.parts;
    const long long row_bytes = static_cast<long long>(rows) * p.D * sizeof(T) * 2;
    sp.checker = OP != Op::kRope && p.B > 0 && (p.M <= kCheckRows || row_bytes >= kCheckBytes) ? 1 : 0;
    if (sp.checker) ++grid;
    if (OP != Op::kRope && (!sp.checker || kBoundsChecked)) {
        const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(DeviceStatus), s);
        if (e != cudaSuccess) return e;
    }
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    return p.interleaved ? launch_after(rope_kernel<T, true, OP>, static_cast<int>(grid), kThreads, 0, s, p, sp)
                         : launch_after(rope_kernel<T, false, OP>, static_cast<int>(grid), kThreads, 0, s, p, sp);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool bf16, int num_sms, cudaStream_t s) {
    return bf16 ? launch_typed<__nv_bfloat16, Op::kRope>(p, num_sms, s) : launch_typed<float, Op::kRope>(p, num_sms, s);
}

cudaError_t launch_rope_append(const RopeParams& p, bool bf16, bool e4m3, int num_sms, cudaStream_t s) {
    if (e4m3) return bf16 ? launch_typed<__nv_bfloat16, Op::kAppendE4M3>(p, num_sms, s) : cudaErrorInvalidValue;
    return bf16 ? launch_typed<__nv_bfloat16, Op::kAppend>(p, num_sms, s)
                : launch_typed<float, Op::kAppend>(p, num_sms, s);
}

}  // namespace sptp
