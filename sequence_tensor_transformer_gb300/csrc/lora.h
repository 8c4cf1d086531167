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
};

constexpr int kLoraMaxRank = 128;
// Rows from which on a tile has 64 rows (ranks above 32: 32) instead of 16, so
// that each reads its adapter once for four times as many.
constexpr int kLoraMany = 2048;

// How the product with A is split along a row of f elements: pieces of *split_k,
// as many as make two blocks an SM of it, but none below 256 elements.
inline int lora_splits(int M, int f, int R, int shards, bool bf16, int* split_k) {
    const int rows = !bf16 ? 8 : M < kLoraMany ? 16 : R <= 32 ? 64 : 32;
    const long long tiles = (static_cast<long long>(M) + rows - 1) / rows * shards;
    constexpr int kBlocks = 304;
    long long splits = tiles >= kBlocks ? 1 : (kBlocks + tiles - 1) / tiles;
    const int most = f <= 256 ? 1 : f / 256;
    if (splits > most) splits = most;
    *split_k = ((f + static_cast<int>(splits) - 1) / static_cast<int>(splits) + 31) / 32 * 32;
    return (f + *split_k - 1) / *split_k;
}

cudaError_t launch_lora(LoraParams& p, bool bf16, int num_sms, cudaStream_t s);

}  // namespace sptp
