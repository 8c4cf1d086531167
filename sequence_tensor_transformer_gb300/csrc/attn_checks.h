// Argument checks of the calls on attention rows and a paged key-value cache.
#pragma once

#include <cmath>

#include "checks.h"
#include "sptp.h"

namespace sptp {

inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// One buffer of a call: its bytes, and the alignment its pointer needs.
struct Buf {
    const void* p;
    size_t bytes;
    size_t align;
};

inline int check_aligned(const Buf* b, int n) {
    for (int i = 0; i < n; ++i)
        if (b[i].p != nullptr && !aligned_to(b[i].p, b[i].align)) return SPTP_ERR_SHAPE;
    return SPTP_OK;
}

// No output on top of an input or of another output.
inline int check_alias(const Buf* outs, int n_out, const Buf* ins, int n_in) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (overlaps(outs[o].p, outs[o].bytes, ins[i].p, ins[i].bytes)) return SPTP_ERR_ALIAS;
        for (int j = o + 1; j < n_out; ++j)
            if (overlaps(outs[o].p, outs[o].bytes, outs[j].p, outs[j].bytes)) return SPTP_ERR_ALIAS;
    }
    return SPTP_OK;
}

inline int check_heads(int P, int Hq, int Hkv, int D) {
    if (P < 1 || P > kMaxGroups || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return SPTP_ERR_SHAPE;
    if (D < 8 || D > 256 || D % 8 != 0) return SPTP_ERR_SHAPE;
    if (static_cast<long long>(P) * (Hq + 2ll * Hkv) >= (1ll << 24)) return SPTP_ERR_SHAPE;
    return SPTP_OK;
}

inline int check_cache(int P, int Hkv, int D, int B, int max_pages, int num_pages, int page_size, int dtype, int kv_type) {
    if (!dtype_ok(dtype) || (kv_type != SPTP_KV_SAME && kv_type != SPTP_KV_E4M3)) return SPTP_ERR_DTYPE;
    if (kv_type == SPTP_KV_E4M3 && dtype != SPTP_BF16) return SPTP_ERR_DTYPE;
    if (kv_type == SPTP_KV_E4M3 && D % 16 != 0) return SPTP_ERR_SHAPE;
    if (B < 0 || max_pages < 1 || num_pages < 1 || page_size < 16 || page_size % 16 != 0) return SPTP_ERR_SHAPE;
    if (static_cast<long long>(max_pages) * page_size >= (1ll << 30)) return SPTP_ERR_SHAPE;
    // rows of the pool (a TMA coordinate), each product below 2^31 before the next
    long long rows = static_cast<long long>(num_pages) * page_size;
    if (rows >= (1ll << 31)) return SPTP_ERR_SHAPE;
    rows *= P;
    if (rows >= (1ll << 31)) return SPTP_ERR_SHAPE;
    rows *= Hkv;
    return rows < (1ll << 31) ? SPTP_OK : SPTP_ERR_SHAPE;
}

// Elements of an activation tensor, M rows; -1 if it is beyond any GPU (and the
// kernels' 32-bit row numbers).
inline long long elems(long long P, long long M, long long heads, long long D) {
    const long long row = P * heads * D;  // < 2^32
    return M < (1ll << 30) && M <= (1ll << 42) / row ? M * row : -1;
}

// A cap on the scores: none (0), or one that has room for its reciprocal.
inline bool score_cap_ok(float cap) { return cap == 0.f || (cap >= 1e-30f && cap <= 1e30f); }

}  // namespace sptp
