// Declarations shared by the translation units of the low-rank adapters (sptp_lora).
#pragma once

#include "attn.h"

namespace sptp {

struct LoraParams {
    const void* x;        // [M][K], or rowwise [P][M][f], f = K / P
    const void* A;        // [adapters][R][K]
    const void* B;        // [adapters][N][R]
    const int* ids;       // [M]
    const float* gains;   // [adapters] or nullptr
    const void* base;     // [P][M][n]: n = N / P, or rowwise N
    void* out;            // like base; may be base
    float* t;             // [splits][rowwise ? P : 1][M][R]: gain-free products with A
    int P, M, K, N, R, adapters, rowwise;
    int f;                // elements of a row of x
    int n;                // columns of a row of out
    int splits, split_k;  // of a row of x: split s has elements [s * split_k, (s + 1) * split_k)
    DeviceStatus* status;
    int beside;           // the status is another call's too: only an id outside its range is recorded, where there is none yet
};

constexpr int kLoraMaxRank = 128;
// Rows below which the second launch has a block per row instead of one per 16 (measured at rank
// 16 with an adapter of its own for most rows; with one adapter for all of 16 rows, and at
// higher ranks, the block per row reads B more often than it need be).
constexpr int kLoraFew = 160;

// How the product with A is split along a row of f elements: pieces of *split_k,
// as many as make two blocks an SM (bf16: of 16 rows; fp32: of 8 warps with 8 rows
// and 8 elements each), but none below 128 elements.
inline int lora_splits(int M, int f, int R, int shards, bool bf16, int* split_k) {
    const long long tiles = (static_cast<long long>(M) + (bf16 ? 15 : 7)) / (bf16 ? 16 : 8) * shards;
    const long long blocks = bf16 ? tiles : (tiles * (R / 8) + 7) / 8;
    constexpr int kBlocks = 304, kLeast = 128;
    long long splits = blocks < 1 || blocks >= kBlocks ? 1 : (kBlocks + blocks - 1) / blocks;
    const int most = f <= kLeast ? 1 : f / kLeast;
    if (splits > most) splits = most;
    *split_k = ((f + static_cast<int>(splits) - 1) / static_cast<int>(splits) + 31) / 32 * 32;
    return (f + *split_k - 1) / *split_k;
}

cudaError_t launch_lora(LoraParams& p, bool bf16, int num_sms, cudaStream_t s);

}  // namespace sptp
