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
// 16-byte accesses, and nothing else is large.  A lane owns one slot of a
// head, two 16-byte vectors that hold each other's partners (half layout: the
// vectors at c and c + rot/2; interleaved: two adjacent ones; elements that do
// not turn: two adjacent ones), and walks over the heads of its row with the
// slot's cosines and sines in registers, so an angle is computed once per
// token and slot, not once per head.  L lanes (a power of two) cover a head.
#include <cuda_bf16.h>

#include "e4m3.cuh"
#include "sptp.h"
#include "sptp_ptx.cuh"

namespace sptp {

namespace {

enum class Op { kRope, kAppend, kAppendE4M3 };

constexpr int kThreads = 128;  // four warps: four work units of the same kind
constexpr int kUnroll = 4;     // heads whose loads a lane has in flight

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

// Where a token's keys and values go: its row of the cache without the shard
// and head, or -1 (padding or an index out of its range).
__device__ __forceinline__ int kv_page(const RopeParams& p, int seq, int pos) {
    if (seq < 0 || seq >= p.B || pos < 0 || pos / p.page_size >= p.max_pages) return -1;
    const int page = __ldg(p.page_table + static_cast<long long>(seq) * p.max_pages + pos / p.page_size);
    return page >= 0 && page < p.num_pages ? page : -1;
}

// The status words of an append of up to kCheckRows rows, written once: a block
// of its own looks at all rows' indexes, in one round of loads, beside the
// blocks that move the data (which skip the bad ones silently), so that no
// launch has to clear the words first.  More rows are checked by the blocks
// that move them, after a launch that clears the words: 1.5 us that a batch of
// new tokens would feel and a prompt does not (for 16384 rows one block took 3
// times as long as moving the data).
constexpr int kCheckRows = 8 * kThreads;

__device__ __noinline__ void check_rows(const RopeParams& p) {
    __shared__ int first_bad;
    if (threadIdx.x == 0) first_bad = 0x7fffffff;
    __syncthreads();
    int seq[8], pos[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = i * kThreads + threadIdx.x;
        seq[i] = m < p.M ? __ldg(p.seq_ids + m) : -1;
        pos[i] = m < p.M ? __ldg(p.positions + m) : 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (seq[i] >= 0 && kv_page(p, seq[i], pos[i]) < 0) atomicMin(&first_bad, i * kThreads + static_cast<int>(threadIdx.x));
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool bad = first_bad != 0x7fffffff;
        // a checked build clears the words before the launch: another block
        // may have written them
        if (kBoundsChecked && !bad) return;
        DeviceStatus st;
        st.code = bad ? SPTP_ERR_SHAPE : SPTP_OK;
        st.where = bad ? kWhereKvSlot : 0;
        st.block = 0;
        st.info = bad ? first_bad : 0;
        st.flag = 0;
        *p.status = st;
    }
}

// Unit u = token u / parts, and of its P * H heads the `per` of part u % parts;
// one warp each.
template <typename T, bool INTER, Op OP>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p, int L, int parts,
                                                        int per) {
    constexpr int E = Elems<T>::E;
    const bool one_block_checks = OP != Op::kRope && p.M <= kCheckRows;
    if (one_block_checks && blockIdx.x == gridDim.x - 1) {
        check_rows(p);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int slot = lane & (L - 1), hg = lane / L, hpw = 32 / L;
    const int half = p.rot / 2;
    const int turning = half / E;  // slots that turn
    // the slot's two vectors (element offsets); a tail slot may lack the second
    const bool turns = slot < turning;
    const int ea = turns ? (INTER ? 2 * slot * E : slot * E) : p.rot + 2 * (slot - turning) * E;
    const int eb = turns && !INTER ? ea + half : ea + E;
    const bool has_a = ea < p.D, has_b = eb < p.D;
    const int rows = p.P * p.H;
    const long long units = static_cast<long long>(p.M) * parts;
    const long long blocks = one_block_checks ? gridDim.x - 1 : gridDim.x;
    for (long long u = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; u < units;
         u += blocks * (kThreads / 32)) {
        const int m = static_cast<int>(u / parts);
        const int r0 = static_cast<int>(u - static_cast<long long>(m) * parts) * per;
        const int r1 = min(rows, r0 + per);
        const int pos = __ldg(p.positions + m);
        int seq = 0, page = -1, off = 0;
        if constexpr (OP != Op::kRope) {
            seq = __ldg(p.seq_ids + m);
            if (seq < 0) continue;  // a padding row
            page = kv_page(p, seq, pos);
            off = pos % p.page_size;
            if (page < 0 && !one_block_checks && r0 == 0 && lane == 0 &&
                atomicCAS(&p.status->code, 0, SPTP_ERR_SHAPE) == 0) {
                p.status->where = kWhereKvSlot;
                p.status->info = m;
            }
        }
        float c[E], s[E];
        bool have = false;
        for (int base = r0; base < r1; base += hpw * kUnroll) {
            uint4 va[kUnroll], vb[kUnroll];
            int pp[kUnroll], hh[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int r = base + i * hpw + hg;
                pp[i] = r / p.H;
                hh[i] = r < r1 ? r - pp[i] * p.H : -1;
                va[i] = vb[i] = make_uint4(0, 0, 0, 0);
                if (hh[i] >= 0) {
                    // in place, what does not turn stays where it is
                    if (OP == Op::kRope && p.out == p.x && (hh[i] >= p.Hr || !turns)) {
                        hh[i] = -1;
                        continue;
                    }
                    const T* src = static_cast<const T*>(p.x) +
                                   ((static_cast<long long>(pp[i]) * p.M + m) * p.H + hh[i]) * p.D;
                    if (has_a) va[i] = __ldcs(reinterpret_cast<const uint4*>(src + ea));
                    if (has_b) vb[i] = __ldcs(reinterpret_cast<const uint4*>(src + eb));
                }
            }
            if (!have) {  // the loads of the first heads are under way
                have = true;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    c[e] = p.gain;
                    s[e] = 0.f;
                    if (turns) {
                        const unsigned long long f = static_cast<unsigned long long>(static_cast<long long>(pos)) *
                                                     __ldg(p.turns + slot * E + e);
                        // signed: [-1/2, 1/2) turn = [-1, 1) half turns
                        const float t = __ll2float_rn(static_cast<long long>(f)) * 0x1p-63f;
                        sincospif(t, &s[e], &c[e]);
                        c[e] *= p.gain;
                        s[e] *= p.transpose ? -p.gain : p.gain;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (turns && hh[i] >= 0 && hh[i] < p.Hr) turn<T, INTER>(va[i], vb[i], c, s);
                if constexpr (OP == Op::kRope) {
                    if (hh[i] < 0) continue;
                    T* dst = static_cast<T*>(p.out) + ((static_cast<long long>(pp[i]) * p.M + m) * p.H + hh[i]) * p.D;
                    if (has_a) __stcs(reinterpret_cast<uint4*>(dst + ea), va[i]);
                    if (has_b) __stcs(reinterpret_cast<uint4*>(dst + eb), vb[i]);
                } else {
                    const bool is_q = hh[i] >= 0 && hh[i] < p.Hq;
                    if (is_q) {
                        T* dst = static_cast<T*>(p.out) +
                                 ((static_cast<long long>(pp[i]) * p.M + m) * p.Hq + hh[i]) * p.D;
                        if (has_a) *reinterpret_cast<uint4*>(dst + ea) = va[i];
                        if (has_b) *reinterpret_cast<uint4*>(dst + eb) = vb[i];
                    }
                    const bool is_v = hh[i] >= p.Hq + p.Hkv;
                    const int kvh = hh[i] - p.Hq - (is_v ? p.Hkv : 0);
                    const long long row =
                        ((static_cast<long long>(pp[i]) * p.num_pages + page) * p.Hkv + kvh) * p.page_size + off;
                    const bool is_kv = hh[i] >= p.Hq && page >= 0 &&
                                       checked_index(row, static_cast<long long>(p.P) * p.num_pages * p.Hkv * p.page_size,
                                                     p.status, nullptr, kWhereBoundsStore);
                    if constexpr (OP == Op::kAppend) {
                        if (is_kv) {
                            T* dst = static_cast<T*>(is_v ? p.v_cache : p.k_cache) + row * p.D;
                            if (has_a) *reinterpret_cast<uint4*>(dst + ea) = va[i];
                            if (has_b) *reinterpret_cast<uint4*>(dst + eb) = vb[i];
                        }
                    } else {
                        // the head's row maximum over its L lanes; every lane
                        // of the warp takes part
                        float amax = fmaxf(absmax_bf16x8(va[i]), absmax_bf16x8(vb[i]));
                        for (int o = L / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                        if (is_kv) {
                            const int ex = e4m3_row_exponent(amax);
                            const float inv = pow2f(-ex);
                            uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + row * p.D;
                            if (has_a) *reinterpret_cast<uint2*>(dst + ea) = e4m3_quant8(va[i], inv);
                            if (has_b) *reinterpret_cast<uint2*>(dst + eb) = e4m3_quant8(vb[i], inv);
                            if (slot == 0) (is_v ? p.v_scale : p.k_scale)[row] = pow2f(ex);
                        }
                    }
                }
            }
        }
    }
}

template <typename T, Op OP>
cudaError_t launch_typed(const RopeParams& p, int num_sms, cudaStream_t s) {
    constexpr int E = Elems<T>::E;
    const int slots = p.rot / (2 * E) + (p.D - p.rot + 2 * E - 1) / (2 * E);
    int L = 1;
    while (L < slots) L *= 2;
    const int hpw = 32 / L;
    // A warp takes a whole token where there are tokens enough for 16 warps
    // per SM; below that a token's heads are cut into parts, down to one
    // head per lane group.
    const int rows = p.P * p.H;
    const long long want = static_cast<long long>(num_sms) * 16;
    long long parts = (want + p.M - 1) / p.M;
    const int most = (rows + hpw - 1) / hpw;
    if (parts > most) parts = most;
    // whole lane groups per part
    const int per = ((rows + static_cast<int>(parts) - 1) / static_cast<int>(parts) + hpw - 1) / hpw * hpw;
    parts = (rows + per - 1) / per;
    const long long units = p.M * parts;
    long long grid = (units + kThreads / 32 - 1) / (kThreads / 32);
    const long long cap = static_cast<long long>(num_sms) * 16;
    if (grid > cap) grid = cap;
    if (OP != Op::kRope) {
        if (p.M <= kCheckRows) ++grid;  // the block that checks the indexes
        if (p.M > kCheckRows || kBoundsChecked) {
            const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(DeviceStatus), s);
            if (e != cudaSuccess) return e;
        }
    }
    const int g = static_cast<int>(grid), n = static_cast<int>(parts);
    if (p.interleaved)
        rope_kernel<T, true, OP><<<g, kThreads, 0, s>>>(p, L, n, per);
    else
        rope_kernel<T, false, OP><<<g, kThreads, 0, s>>>(p, L, n, per);
    return cudaGetLastError();
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
