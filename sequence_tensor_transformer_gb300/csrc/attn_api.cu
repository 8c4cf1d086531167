// C ABI of the attention sub-layer between the QKV projection and the output
// projection: the frequency table of the rotary positions (host), the
// rotation, its append to a paged key-value cache and the attention of one
// token per sequence over that cache.  Argument checks and launches; the
// kernels are in rope.cu and paged_attn.cu.
#include <cmath>
#include <cstring>

#include "attn.h"
#include "checks.h"
#include "sptp.h"
#include "sptp_internal.h"

using namespace sptp;

namespace {

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// One buffer of a call: its bytes, and the alignment its pointer needs.
struct Buf {
    const void* p;
    size_t bytes;
    size_t align;
};

int check_aligned(const Buf* b, int n) {
    for (int i = 0; i < n; ++i)
        if (b[i].p != nullptr && !aligned_to(b[i].p, b[i].align)) return SPTP_ERR_SHAPE;
    return SPTP_OK;
}

// No output on top of an input or of another output.
int check_alias(const Buf* outs, int n_out, const Buf* ins, int n_in) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (overlaps(outs[o].p, outs[o].bytes, ins[i].p, ins[i].bytes)) return SPTP_ERR_ALIAS;
        for (int j = o + 1; j < n_out; ++j)
            if (overlaps(outs[o].p, outs[o].bytes, outs[j].p, outs[j].bytes)) return SPTP_ERR_ALIAS;
    }
    return SPTP_OK;
}

int check_heads(int P, int Hq, int Hkv, int D) {
    if (P < 1 || P > kMaxGroups || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return SPTP_ERR_SHAPE;
    if (D < 8 || D > 256 || D % 8 != 0) return SPTP_ERR_SHAPE;
    if (static_cast<long long>(P) * (Hq + 2ll * Hkv) >= (1ll << 24)) return SPTP_ERR_SHAPE;
    return SPTP_OK;
}

int check_cache(int P, int Hkv, int D, int B, int max_pages, int num_pages, int page_size, int dtype, int kv_type) {
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

// Query heads whose parts one CTA of the attention may leave, at most.
int part_heads(int group) { return group < 32 ? group : 32; }

struct PagedLayout {
    size_t parts, ml, o, total;
};

PagedLayout paged_layout(int group, int D) {
    PagedLayout L;
    const size_t rows = static_cast<size_t>(kPagedMaxCtas) * 2 * part_heads(group);
    L.parts = SPTP_WS_HEADER_BYTES;
    L.ml = L.parts + align_up(sizeof(PagedAttnPart) * kPagedMaxCtas);
    L.o = L.ml + align_up(rows * sizeof(float2));
    L.total = L.o + align_up(rows * D * sizeof(float));
    return L;
}

// Elements of an activation tensor, M rows; -1 if it is beyond any GPU (and the
// kernels' 32-bit row numbers).
long long elems(long long P, long long M, long long heads, long long D) {
    const long long row = P * heads * D;  // < 2^32
    return M < (1ll << 30) && M <= (1ll << 42) / row ? M * row : -1;
}

// sptp_paged_attn_decode, and its self-test.
int attend(const sptp_paged_attn_decode_args& a, unsigned long long limit_ns, int withhold_full, int withhold_empty) {
    const bool e4m3 = a.kv_type == SPTP_KV_E4M3;
    if (!a.k_cache || !a.v_cache || !a.workspace || (e4m3 && (!a.k_scale || !a.v_scale)) ||
        (a.B != 0 && (!a.q || !a.page_table || !a.seq_lens || !a.out)))
        return SPTP_ERR_NULL;
    int rc = check_cache(a.P, a.Hkv, a.D, a.B, a.max_pages, a.num_pages, a.page_size, a.dtype, a.kv_type);
    if (rc == SPTP_ERR_DTYPE) return rc;
    int rc2 = check_heads(a.P, a.Hq, a.Hkv, a.D);
    if (rc2 != SPTP_OK || rc != SPTP_OK) return SPTP_ERR_SHAPE;
    if (a.window < 0 || !std::isfinite(a.scale)) return SPTP_ERR_SHAPE;
    const long long n = elems(a.P, a.B, a.Hq, a.D);
    if (n < 0) return SPTP_ERR_SHAPE;
    const sptp_dtype dtype = static_cast<sptp_dtype>(a.dtype);
    const size_t es = esize(dtype), rows = static_cast<size_t>(a.P) * a.num_pages * a.Hkv * a.page_size;
    const size_t cb = rows * a.D * (e4m3 ? 1 : es), sb = e4m3 ? rows * 4 : 0, qb = static_cast<size_t>(n) * es;
    const size_t need = sptp_paged_attn_workspace_size(a.P, a.B, a.Hq, a.Hkv, a.D);
    const Buf ins[] = {{a.q, qb, 16}, {a.k_cache, cb, 16}, {a.v_cache, cb, 16},
                       {e4m3 ? a.k_scale : nullptr, sb, 16}, {e4m3 ? a.v_scale : nullptr, sb, 16},
                       {a.page_table, static_cast<size_t>(a.B) * a.max_pages * 4, 4},
                       {a.seq_lens, static_cast<size_t>(a.B) * 4, 4}};
    const Buf outs[] = {{a.out, qb, 16}, {a.lse, static_cast<size_t>(a.P) * a.B * a.Hq * 4, 16}, {a.workspace, need, kAlign}};
    if ((rc = check_aligned(ins, 7)) != SPTP_OK || (rc = check_aligned(outs, 3)) != SPTP_OK) return rc;
    if (a.ws_bytes < need) return SPTP_ERR_WORKSPACE;
    if ((rc = check_alias(outs, 3, ins, 7)) != SPTP_OK) return rc;
    if (a.B == 0) return SPTP_OK;
    DevInfo di;
    if ((rc = device_info(&di)) != SPTP_OK) return rc;
    PagedAttnParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = a.q;
    p.k = a.k_cache;
    p.v = a.v_cache;
    p.k_scale = static_cast<const float*>(a.k_scale);
    p.v_scale = static_cast<const float*>(a.v_scale);
    p.page_table = static_cast<const int*>(a.page_table);
    p.seq_lens = static_cast<const int*>(a.seq_lens);
    p.P = a.P;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.D = a.D;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.window = a.window;
    p.scale = a.scale;
    p.out = a.out;
    p.lse = static_cast<float*>(a.lse);
    p.wait_limit_ns = limit_ns;
    p.withhold_full = withhold_full;
    p.withhold_empty = withhold_empty;
    p.status = ws_status(a.workspace);
    const PagedLayout lay = paged_layout(a.Hq / a.Hkv, a.D);
    p.parts = reinterpret_cast<PagedAttnPart*>(mptr(a.workspace, lay.parts));
    p.part_ml = reinterpret_cast<float2*>(mptr(a.workspace, lay.ml));
    p.part_o = reinterpret_cast<float*>(mptr(a.workspace, lay.o));
    return cuda_status(launch_paged_attn(p, dtype == SPTP_BF16, e4m3, di.sms, static_cast<cudaStream_t>(a.cuda_stream)));
}

}  // namespace

extern "C" {

int sptp_rope_turns(int rot, double theta, sptp_rope_scaling scaling, double factor, double orig_len, double alpha,
                    double beta, unsigned long long* turns) {
    if (!turns) return SPTP_ERR_NULL;
    if (scaling < SPTP_ROPE_NONE || scaling > SPTP_ROPE_PARTS) return SPTP_ERR_UNIMPLEMENTED;
    if (rot < 16 || rot > 256 || rot % 16 != 0 || !(theta > 1.0) || !std::isfinite(theta)) return SPTP_ERR_SHAPE;
    if (scaling == SPTP_ROPE_NONE) factor = 1.0;
    if (!(factor >= 1.0) || !std::isfinite(factor)) return SPTP_ERR_SHAPE;
    if (scaling == SPTP_ROPE_PARTS && (!(orig_len > 0.0) || !std::isfinite(orig_len) || !std::isfinite(alpha) ||
                                       !std::isfinite(beta) || !(beta > alpha)))
        return SPTP_ERR_SHAPE;
    if (scaling == SPTP_ROPE_NTK) theta *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
    if (!std::isfinite(theta)) return SPTP_ERR_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot);
        if (scaling == SPTP_ROPE_LINEAR) f /= factor;
        if (scaling == SPTP_ROPE_PARTS) {
            const double c = std::fmin(1.0, std::fmax(0.0, (orig_len * f / two_pi - alpha) / (beta - alpha)));
            f = c * f + (1.0 - c) * (f / factor);
        }
        // f <= 1, so f / 2 pi is below 1/6 of a turn
        turns[i] = static_cast<unsigned long long>(std::nearbyint(std::ldexp(f / two_pi, 64)));
    }
    return SPTP_OK;
}

int sptp_rope(const void* x, const int* positions, const unsigned long long* turns, int P, int M, int H, int Hr,
              int D, int rot, int interleaved, int transpose, float gain, sptp_dtype dtype, void* out,
              void* cuda_stream) {
    if (!turns || (M != 0 && (!x || !positions || !out))) return SPTP_ERR_NULL;
    if (!dtype_ok(dtype)) return SPTP_ERR_DTYPE;
    if (P < 1 || P > kMaxGroups || M < 0 || H < 1 || Hr < 1 || Hr > H || D < 8 || D > 256 || D % 8 != 0)
        return SPTP_ERR_SHAPE;
    if (static_cast<long long>(P) * H >= (1ll << 24) || rot < 16 || rot > D || rot % 16 != 0 || !std::isfinite(gain))
        return SPTP_ERR_SHAPE;
    const long long n = elems(P, M, H, D);
    if (n < 0) return SPTP_ERR_SHAPE;
    const size_t xb = static_cast<size_t>(n) * esize(dtype);
    const Buf ins[] = {{x, xb, 16}, {positions, static_cast<size_t>(M) * 4, 4}, {turns, static_cast<size_t>(rot) * 4, 8}};
    const Buf outs[] = {{out, xb, 16}};
    int rc = check_aligned(ins, 3);
    if (rc == SPTP_OK) rc = check_aligned(outs, 1);
    if (rc != SPTP_OK) return rc;
    const int skip = out == x ? 1 : 0;
    if ((rc = check_alias(outs, 1, ins + skip, 3 - skip)) != SPTP_OK) return rc;
    if (M == 0) return SPTP_OK;
    DevInfo di;
    if ((rc = device_info(&di)) != SPTP_OK) return rc;
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = x;
    p.positions = positions;
    p.turns = turns;
    p.P = P;
    p.M = M;
    p.H = H;
    p.Hr = Hr;
    p.D = D;
    p.rot = rot;
    p.interleaved = interleaved;
    p.transpose = transpose;
    p.gain = gain;
    p.out = out;
    return cuda_status(launch_rope(p, dtype == SPTP_BF16, di.sms, static_cast<cudaStream_t>(cuda_stream)));
}

int sptp_rope_append_kv(const void* qkv, const int* positions, const int* seq_ids, const int* page_table,
                        const unsigned long long* turns, int P, int M, int Hq, int Hkv, int D, int rot,
                        int interleaved, float gain, int B, int max_pages, int num_pages, int page_size,
                        sptp_dtype dtype, sptp_kv_type kv_type, void* q_out, void* k_cache, void* v_cache,
                        float* k_scale, float* v_scale, void* workspace, size_t ws_bytes, void* cuda_stream) {
    const bool e4m3 = kv_type == SPTP_KV_E4M3;
    if (!k_cache || !v_cache || !workspace || (rot != 0 && !turns) || (e4m3 && (!k_scale || !v_scale)) ||
        (M != 0 && (!qkv || !positions || !seq_ids || (B != 0 && !page_table) || !q_out)))
        return SPTP_ERR_NULL;
    int rc = check_cache(P, Hkv, D, B, max_pages, num_pages, page_size, dtype, kv_type);
    if (rc == SPTP_ERR_DTYPE) return rc;
    int rc2 = check_heads(P, Hq, Hkv, D);
    if (rc2 != SPTP_OK || rc != SPTP_OK) return SPTP_ERR_SHAPE;
    if (M < 0 || rot < 0 || rot > D || rot % 16 != 0 || !std::isfinite(gain)) return SPTP_ERR_SHAPE;
    const int H = Hq + 2 * Hkv;
    const long long n = elems(P, M, H, D);
    if (n < 0) return SPTP_ERR_SHAPE;
    const size_t es = esize(dtype), rows = static_cast<size_t>(P) * num_pages * Hkv * page_size;
    const size_t cb = rows * D * (e4m3 ? 1 : es), sb = e4m3 ? rows * 4 : 0;
    const Buf ins[] = {{qkv, static_cast<size_t>(n) * es, 16},
                       {positions, static_cast<size_t>(M) * 4, 4},
                       {seq_ids, static_cast<size_t>(M) * 4, 4},
                       {page_table, static_cast<size_t>(B) * max_pages * 4, 4},
                       {rot != 0 ? turns : nullptr, static_cast<size_t>(rot) * 4, 8}};
    const Buf outs[] = {{q_out, static_cast<size_t>(P) * M * Hq * D * es, 16}, {k_cache, cb, 16}, {v_cache, cb, 16},
                        {workspace, SPTP_WS_HEADER_BYTES, kAlign},
                        {e4m3 ? k_scale : nullptr, sb, 16}, {e4m3 ? v_scale : nullptr, sb, 16}};
    if ((rc = check_aligned(ins, 5)) != SPTP_OK || (rc = check_aligned(outs, 6)) != SPTP_OK) return rc;
    if (ws_bytes < SPTP_WS_HEADER_BYTES) return SPTP_ERR_WORKSPACE;
    if ((rc = check_alias(outs, 6, ins, 5)) != SPTP_OK) return rc;
    if (M == 0) return SPTP_OK;
    DevInfo di;
    if ((rc = device_info(&di)) != SPTP_OK) return rc;
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = qkv;
    p.positions = positions;
    p.turns = turns;
    p.P = P;
    p.M = M;
    p.H = H;
    p.Hr = rot != 0 ? Hq + Hkv : 0;
    p.D = D;
    p.rot = rot;
    p.interleaved = interleaved;
    p.gain = gain;
    p.out = q_out;
    p.seq_ids = seq_ids;
    p.page_table = page_table;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.B = B;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.status = ws_status(workspace);
    return cuda_status(
        launch_rope_append(p, dtype == SPTP_BF16, e4m3, di.sms, static_cast<cudaStream_t>(cuda_stream)));
}

size_t sptp_paged_attn_workspace_size(int P, int B, int Hq, int Hkv, int D) {
    if (check_heads(P, Hq, Hkv, D) != SPTP_OK || B < 0) return 0;
    return paged_layout(Hq / Hkv, D).total;
}

int sptp_paged_attn_decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int* page_table, const int* seq_lens, int P, int B, int Hq,
                           int Hkv, int D, int max_pages, int num_pages, int page_size, int window, float scale,
                           sptp_dtype dtype, sptp_kv_type kv_type, void* out, float* lse, void* workspace,
                           size_t ws_bytes, void* cuda_stream) {
    sptp_paged_attn_decode_args a;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    a.cuda_stream = cuda_stream;
    a.ws_bytes = ws_bytes;
    a.P = P;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.window = window;
    a.dtype = dtype;
    a.kv_type = kv_type;
    a.scale = scale;
    return attend(a, kWaitLimitNs, -1, -1);
}

int sptp_rope_packed(const sptp_rope_args* a) {
    if (!a) return SPTP_ERR_NULL;
    return sptp_rope(a->x, static_cast<const int*>(a->positions), static_cast<const unsigned long long*>(a->turns), a->P,
                     a->M, a->H, a->Hr, a->D, a->rot, a->interleaved, a->transpose, a->gain,
                     static_cast<sptp_dtype>(a->dtype), a->out, a->cuda_stream);
}

int sptp_rope_append_kv_packed(const sptp_rope_append_kv_args* a) {
    if (!a) return SPTP_ERR_NULL;
    return sptp_rope_append_kv(
        a->qkv, static_cast<const int*>(a->positions), static_cast<const int*>(a->seq_ids),
        static_cast<const int*>(a->page_table), static_cast<const unsigned long long*>(a->turns), a->P, a->M, a->Hq,
        a->Hkv, a->D, a->rot, a->interleaved, a->gain, a->B, a->max_pages, a->num_pages, a->page_size,
        static_cast<sptp_dtype>(a->dtype), static_cast<sptp_kv_type>(a->kv_type), a->q_out, a->k_cache, a->v_cache,
        static_cast<float*>(a->k_scale), static_cast<float*>(a->v_scale), a->workspace, a->ws_bytes, a->cuda_stream);
}

int sptp_paged_attn_decode_packed(const sptp_paged_attn_decode_args* a) {
    return a ? attend(*a, kWaitLimitNs, -1, -1) : SPTP_ERR_NULL;
}

int sptp_paged_attn_wait_selftest(const sptp_paged_attn_decode_args* a, int withhold_full, int withhold_empty,
                                  unsigned long long limit_ns) {
    if (!a) return SPTP_ERR_NULL;
    if (limit_ns == 0 || limit_ns > 10000000000ull || a->D > 128) return SPTP_ERR_SHAPE;
    if ((withhold_full < 0) == (withhold_empty < 0)) return SPTP_ERR_SHAPE;
    return attend(*a, limit_ns, withhold_full, withhold_empty);
}

}  // extern "C"
