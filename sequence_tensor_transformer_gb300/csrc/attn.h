// Declarations shared by the attention sub-layer's translation units: rotary
// positions, the append to a paged key-value cache, and the attention of one
// token per sequence over it.
#pragma once

#include "sptp_internal.h"

namespace sptp {

// Launches `kernel` so that it may be scheduled while the kernel before it in
// the stream ends (a programmatic dependency); it waits for that kernel's
// results on the device (await_previous) before it touches memory.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), int grid, int block, size_t smem, cudaStream_t s, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

#ifdef __CUDACC__
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The kernel after this one may be scheduled once every block of this one
// runs or has ended.
__device__ __forceinline__ void admit_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

// what a status word of these calls names (DeviceStatus::where)
enum : int {
    kWhereKvSlot = 14,  // a token's sequence, position or page outside its range
    kWhereKvPage = 15,  // a sequence's length or page outside its range
    kWhereKvFull = 16,
    kWhereKvEmpty = 17,
    kWhereAdapter = 18,  // a row's adapter outside its range
    kWherePromptItem = 27,
    kWherePromptQuery = 28,
    kWherePromptScores = 29,
    kWherePromptWeights = 30,
    kWherePromptOutputs = 31,
    kWherePromptChecked = 32,
    kWherePromptMasked = 33,
};

// ---------------------------------------------------------------- rotary positions, paged cache
struct RopeParams {
    const void* x;                     // [P][M][H][D] (append: the QKV rows, H = Hq + 2 Hkv)
    const int* positions;              // [M]
    const unsigned long long* turns;   // [rot/2]
    int P, M, H, Hr, D, rot;           // heads [0, Hr) of a row are rotated
    int interleaved, transpose;
    float gain;
    void* out;                         // rope: [P][M][H][D]; append: q_out [P][M][Hq][D]
    // append only
    const int* seq_ids;                // [M]
    const int* page_table;             // [B][max_pages]
    int Hq, Hkv, B, max_pages, num_pages, page_size;
    void* k_cache;                     // [P][num_pages][Hkv][page_size][D]
    void* v_cache;
    float* k_scale;                    // E4M3: [P][num_pages][Hkv][page_size]
    float* v_scale;
    DeviceStatus* status;
};

cudaError_t launch_rope(const RopeParams& p, bool bf16, int num_sms, cudaStream_t s);
cudaError_t launch_rope_append(const RopeParams& p, bool bf16, bool e4m3, int num_sms, cudaStream_t s);

// What one CTA of the attention leaves for the join: its status, and the items
// whose parts lie in several shares that its share ends ([0]: the item began
// in an earlier share) or begins ([1]: it goes on in the next).
struct alignas(16) PagedAttnItem {
    int parts;       // shares that hold a part, 0: no such item
    int first;       // the first of them
    int heads;       // of the item
    int pad;
    long long qrow;  // row of q and out of its first head
    long long pad2;
};
struct PagedAttnPart {
    PagedAttnItem items[2];
    int status, where, info, pad;
};
constexpr int kPagedMaxCtas = 320;  // CTAs of one resident wave, at most

struct PagedAttnParams {
    CUtensorMap map_k, map_v;  // the pools as [P * num_pages * Hkv * page_size][D], boxes of box_rows rows
    const void* q;          // [P][B][Hq][D]
    const void* k;          // [P][num_pages][Hkv][page_size][D]
    const void* v;
    const float* k_scale;   // E4M3: [P][num_pages][Hkv][page_size]
    const float* v_scale;
    const int* page_table;  // [B][max_pages]
    const int* seq_lens;    // [B]
    int P, B, Hq, Hkv, D;
    int max_pages, num_pages, page_size, window;
    int box_rows;           // divides page_size and a tile
    uint32_t page_mul;      // key / page_size = (key * page_mul) >> (32 + page_shift) for 0 <= key < 2^31
    int page_shift;
    int heads_per_item, head_blocks;  // query heads of an item, items per key/value head
    int items_per_seq;      // P * Hkv * head_blocks
    float scale;
    float cap;              // on the scores, 0: none
    const float* slopes;    // [P][Hq], of the bias by distance, or nullptr
    void* out;              // [P][B][Hq][D]
    float* lse;             // [P][B][Hq] or nullptr
    unsigned long long wait_limit_ns;
    int withhold_full, withhold_empty;  // self-test: tiles of CTA 0 (-1: none)
    DeviceStatus* status;
    PagedAttnPart* parts;   // [CTAs]
    float2* part_ml;        // [CTAs][2][heads_per_item]: maximum (in units of log 2) and sum
    float* part_o;          // [CTAs][2][heads_per_item][D]
};

// The paged attention's tensor maps (attn_maps.cu): rows of `inner` elements of
// 1, 2 or 4 bytes (fp32), boxes of box_inner x box_rows; swizzle of 128 bytes,
// or of 64 where a box's rows have 64.
bool encode_map_rows(CUtensorMap* map, const void* base, int elem_bytes, uint64_t inner, uint64_t rows,
                     uint32_t box_inner, uint32_t box_rows);

// The queries of sptp_paged_attn_prompt, bf16 [P][M][Hq][D]: boxes of 64 elements
// of `heads` heads of `tokens` rows, swizzle of 128 bytes.
bool encode_map_queries(CUtensorMap* map, const void* base, int D, int Hq, int M, int P, int heads, int tokens);

// One launch per element type (paged_attn_{bf16,e4m3,f32}.cu), and one each for
// scores with a cap or a bias (.._ex.cu): fills in the maps, the boxes and the
// split of the heads.
cudaError_t launch_paged_attn_bf16(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s);
cudaError_t launch_paged_attn_e4m3(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s);
cudaError_t launch_paged_attn_f32(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s);
cudaError_t launch_paged_attn_bf16_ex(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s);
cudaError_t launch_paged_attn_e4m3_ex(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s);
cudaError_t launch_paged_attn_f32_ex(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s);
cudaError_t launch_paged_attn(PagedAttnParams& p, bool bf16, bool e4m3, int num_sms, cudaStream_t s);
// The self-test's form of it, on two CTAs; D <= 128.
constexpr int kSelftestCtas = 2;
cudaError_t launch_paged_attn_test(PagedAttnParams& p, bool bf16, bool e4m3, int* ctas, cudaStream_t s);

}  // namespace sptp
