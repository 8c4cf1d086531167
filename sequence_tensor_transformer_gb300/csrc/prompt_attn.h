// Declarations shared by the translation units of the attention of many rows
// per sequence over a paged key-value cache (sptp_paged_attn_prompt).
#pragma once

#include "attn.h"

namespace sptp {

constexpr int kPromptMaxCtas = 320;   // CTAs of one resident wave, at most
constexpr int kPromptWideCtas = 160;  // of the bf16 kernels, one an SM

// An item whose parts lie in several CTAs' shares, as each of these CTAs leaves
// it for the join; parts == 0: none.
struct PromptItem {
    int parts, first;     // CTAs first .. first + parts - 1 hold a part each
    int tokens, heads;    // rows are token * heads + head
    long long token0;     // shard * M + first token
    int head0;            // of the shard
    int pad;
};
struct alignas(16) PromptPart {
    PromptItem items[2];  // that began in an earlier share; that begins here and goes on in the next
    int status, where, info, pad;
};

struct PromptParams {
    CUtensorMap map_q;         // tensor-core kernels: q as [P * M][Hq][D], boxes of a row tile
    CUtensorMap map_k, map_v;  // and the pools as in PagedAttnParams
    const void* q;             // [P][M][Hq][D]
    const void* k;             // [P][num_pages][Hkv][page_size][D]
    const void* v;
    const float* k_scale;      // E4M3: [P][num_pages][Hkv][page_size]
    const float* v_scale;
    const int* page_table;     // [B][max_pages]
    const int* seq_lens;       // [B]
    const int* row_starts;     // [B + 1]
    const int* prefix_lens;    // [B] or nullptr
    const float* slopes;       // [P][Hq] or nullptr
    int P, M, B, Hq, Hkv, D;
    int max_pages, num_pages, page_size, window;
    int box_rows;
    uint32_t page_mul;         // as in PagedAttnParams
    int page_shift;
    int heads, head_blocks;    // query heads of an item; items per key/value head
    int tokens;                // tokens of an item: a block
    int items_per_block;       // P * Hkv * head_blocks
    float scale, cap;
    void* out;                 // [P][M][Hq][D]
    float* lse;                // [P][M][Hq] or nullptr
    unsigned long long wait_limit_ns;
    int withhold_full;         // self-test: tile of CTA 0 that is not loaded (-1: none)
    int part_rows;             // rows of a part, at most
    DeviceStatus* status;
    PromptPart* parts;         // [CTAs]
    float2* part_ml;           // [CTAs][2][part_rows]: maximum (in units of log 2) and sum
    float* part_o;             // [CTAs][2][part_rows][D]
};

// Rows of an item, at most, by head size and element type.
constexpr int prompt_item_rows(int D, bool bf16) { return !bf16 ? 64 : D <= 128 ? 256 : 128; }

// One each for plain scores (scale > 0), with a cap, with a bias and with both: an
// instruction cache holds the code of one.
using PromptLaunch = cudaError_t(PromptParams& p, int num_sms, int* ctas, cudaStream_t s);
PromptLaunch launch_prompt_bf16, launch_prompt_bf16_cap, launch_prompt_bf16_bias, launch_prompt_bf16_cap_bias;
PromptLaunch launch_prompt_e4m3, launch_prompt_e4m3_cap, launch_prompt_e4m3_bias, launch_prompt_e4m3_cap_bias;
PromptLaunch launch_prompt_f32;
// The self-test's form of it, on two CTAs; 64 < D <= 128, plain scores.
cudaError_t launch_prompt_test(PromptParams& p, bool e4m3, int* ctas, cudaStream_t s);
cudaError_t launch_prompt_attn(PromptParams& p, bool bf16, bool e4m3, int num_sms, cudaStream_t s);
// The split of the heads and rows into items of at most `rows` rows whose tiles
// hold `tile_rows`, and the division by the page size.
void plan_prompt(PromptParams& p, int rows, int tile_rows);
// CTAs of a launch: one resident wave of `most`, or a CTA per tile of `tk` keys
// where there cannot be as many.
int prompt_grid(const PromptParams& p, int most, int tk);

}  // namespace sptp
