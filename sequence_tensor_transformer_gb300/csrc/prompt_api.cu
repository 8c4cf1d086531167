// C ABI of the attention of many rows per sequence over a paged key-value cache:
// argument checks and the launch; the kernels are in prompt_attn_*.cu.
#include <cmath>
#include <cstring>

#include "attn_checks.h"
#include "prompt_attn.h"
#include "sptp.h"

using namespace sptp;

namespace {

struct PromptLayout {
    size_t parts, ml, o, total;
    int rows;
};

// Room for the parts of either element type's kernel: items of up to 256 rows
// with one CTA an SM, or of 64 rows with two.
PromptLayout prompt_layout(int M, int group, int D, bool bf16) {
    PromptLayout L;
    const long long most = static_cast<long long>(M) * group;
    auto part_rows = [&](bool b) { return static_cast<int>(most < prompt_item_rows(D, b) ? most : prompt_item_rows(D, b)); };
    const size_t wide = static_cast<size_t>(kPromptWideCtas) * 2 * part_rows(true);
    const size_t narrow = static_cast<size_t>(kPromptMaxCtas) * 2 * part_rows(false);
    const size_t rows = wide > narrow ? wide : narrow;
    L.rows = part_rows(bf16);
    L.parts = SPTP_WS_HEADER_BYTES;
    L.ml = L.parts + align_up(sizeof(PromptPart) * kPromptMaxCtas);
    L.o = L.ml + align_up(rows * sizeof(float2));
    L.total = L.o + align_up(rows * D * sizeof(float));
    return L;
}

int attend_rows(const sptp_paged_attn_prompt_args* args, unsigned long long limit_ns, int withhold_full);

}  // namespace

extern "C" {

size_t sptp_paged_attn_prompt_workspace_size(int P, int M, int B, int Hq, int Hkv, int D) {
    if (check_heads(P, Hq, Hkv, D) != SPTP_OK || M < 0 || B < 0 || elems(P, M, Hq, D) < 0) return 0;
    return prompt_layout(M, Hq / Hkv, D, true).total;
}

int sptp_paged_attn_prompt(const sptp_paged_attn_prompt_args* args) { return attend_rows(args, kWaitLimitNs, -1); }

int sptp_paged_attn_prompt_wait_selftest(const sptp_paged_attn_prompt_args* args, int withhold_full,
                                         unsigned long long limit_ns) {
    if (!args) return SPTP_ERR_NULL;
    if (limit_ns == 0 || limit_ns > 10000000000ull || withhold_full < 0) return SPTP_ERR_SHAPE;
    if (args->dtype != SPTP_BF16) return SPTP_ERR_DTYPE;
    if (args->D <= 64 || args->D > 128 || args->cap != 0.f || args->slopes != nullptr || !(args->scale > 0.f))
        return SPTP_ERR_SHAPE;
    return attend_rows(args, limit_ns, withhold_full);
}

}  // extern "C"

namespace {

// sptp_paged_attn_prompt, and its self-test.
int attend_rows(const sptp_paged_attn_prompt_args* args, unsigned long long limit_ns, int withhold_full) {
    if (!args) return SPTP_ERR_NULL;
    const sptp_paged_attn_prompt_args& a = *args;
    const bool e4m3 = a.kv_type == SPTP_KV_E4M3;
    const bool some = a.M != 0 && a.B != 0;
    if (!a.k_cache || !a.v_cache || !a.workspace || (e4m3 && (!a.k_scale || !a.v_scale)) ||
        (some && (!a.q || !a.page_table || !a.seq_lens || !a.row_starts || !a.out)))
        return SPTP_ERR_NULL;
    int rc = check_cache(a.P, a.Hkv, a.D, a.B, a.max_pages, a.num_pages, a.page_size, a.dtype, a.kv_type);
    if (rc == SPTP_ERR_DTYPE) return rc;
    const int rc2 = check_heads(a.P, a.Hq, a.Hkv, a.D);
    if (rc2 != SPTP_OK || rc != SPTP_OK) return SPTP_ERR_SHAPE;
    if (a.M < 0 || a.B >= (1 << 30) || a.window < 0 || !std::isfinite(a.scale)) return SPTP_ERR_SHAPE;
    if (!score_cap_ok(a.cap)) return SPTP_ERR_SHAPE;
    const long long n = elems(a.P, a.M, a.Hq, a.D);
    if (n < 0) return SPTP_ERR_SHAPE;
    const sptp_dtype dtype = static_cast<sptp_dtype>(a.dtype);
    const size_t es = esize(dtype), rows = static_cast<size_t>(a.P) * a.num_pages * a.Hkv * a.page_size;
    const size_t cb = rows * a.D * (e4m3 ? 1 : es), sb = e4m3 ? rows * 4 : 0, qb = static_cast<size_t>(n) * es;
    const size_t need = sptp_paged_attn_prompt_workspace_size(a.P, a.M, a.B, a.Hq, a.Hkv, a.D);
    const size_t B = static_cast<size_t>(a.B);
    const Buf ins[] = {{a.q, qb, 16}, {a.k_cache, cb, 16}, {a.v_cache, cb, 16},
                       {e4m3 ? a.k_scale : nullptr, sb, 16}, {e4m3 ? a.v_scale : nullptr, sb, 16},
                       {a.page_table, B * a.max_pages * 4, 4}, {a.seq_lens, B * 4, 4}, {a.row_starts, (B + 1) * 4, 4},
                       {a.prefix_lens, B * 4, 4}, {a.slopes, static_cast<size_t>(a.P) * a.Hq * 4, 4}};
    const Buf outs[] = {{a.out, qb, 16}, {a.lse, static_cast<size_t>(a.P) * a.M * a.Hq * 4, 16}, {a.workspace, need, kAlign}};
    if ((rc = check_aligned(ins, 10)) != SPTP_OK || (rc = check_aligned(outs, 3)) != SPTP_OK) return rc;
    if (a.ws_bytes < need) return SPTP_ERR_WORKSPACE;
    if ((rc = check_alias(outs, 3, ins, 10)) != SPTP_OK) return rc;
    if (!some) return SPTP_OK;
    DevInfo di;
    if ((rc = device_info(&di)) != SPTP_OK) return rc;
    PromptParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = a.q;
    p.k = a.k_cache;
    p.v = a.v_cache;
    p.k_scale = static_cast<const float*>(a.k_scale);
    p.v_scale = static_cast<const float*>(a.v_scale);
    p.page_table = static_cast<const int*>(a.page_table);
    p.seq_lens = static_cast<const int*>(a.seq_lens);
    p.row_starts = static_cast<const int*>(a.row_starts);
    p.prefix_lens = static_cast<const int*>(a.prefix_lens);
    p.slopes = static_cast<const float*>(a.slopes);
    p.P = a.P;
    p.M = a.M;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.D = a.D;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.window = a.window;
    p.scale = a.scale;
    p.cap = a.cap;
    p.out = a.out;
    p.lse = static_cast<float*>(a.lse);
    p.wait_limit_ns = limit_ns;
    p.withhold_full = withhold_full;
    p.status = ws_status(a.workspace);
    const PromptLayout lay = prompt_layout(a.M, a.Hq / a.Hkv, a.D, dtype == SPTP_BF16);
    p.part_rows = lay.rows;
    p.parts = reinterpret_cast<PromptPart*>(mptr(a.workspace, lay.parts));
    p.part_ml = reinterpret_cast<float2*>(mptr(a.workspace, lay.ml));
    p.part_o = reinterpret_cast<float*>(mptr(a.workspace, lay.o));
    return cuda_status(launch_prompt_attn(p, dtype == SPTP_BF16, e4m3, di.sms, static_cast<cudaStream_t>(a.cuda_stream)));
}

}  // namespace
