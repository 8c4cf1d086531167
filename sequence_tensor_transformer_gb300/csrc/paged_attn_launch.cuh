// Launch of the paged attention with one consumer class.
#pragma once

#include <atomic>

#include "paged_attn.cuh"

namespace sptp {
namespace paged {
namespace {  // internal: a process may load the library and its checked build, each with `done` of its own

template <class C, bool TEST = false>
cudaError_t launch(PagedAttnParams& p, int num_sms, int* ctas, cudaStream_t s) {
    // heads of a group, in equal blocks of at most HEADS
    const int group = p.Hq / p.Hkv;
    p.head_blocks = (group + Smem<C>::HEADS - 1) / Smem<C>::HEADS;
    p.heads_per_item = (group + p.head_blocks - 1) / p.head_blocks;
    p.head_blocks = (group + p.heads_per_item - 1) / p.heads_per_item;
    p.items_per_seq = p.P * p.Hkv * p.head_blocks;
    // the largest boxes that never cross a page
    p.box_rows = 16;
    while (p.box_rows < C::TK && p.page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
    const uint64_t rows = static_cast<uint64_t>(p.P) * p.num_pages * p.Hkv * p.page_size;
    if (!encode_map_rows(&p.map_k, p.k, C::ELEM, p.D, rows, C::SPAN / C::ELEM, p.box_rows) ||
        !encode_map_rows(&p.map_v, p.v, C::ELEM, p.D, rows, C::SPAN / C::ELEM, p.box_rows))
        return cudaErrorInvalidValue;
    // division by the page size: with 2^(l-1) < d <= 2^l and mul = floor(2^(31+l) / d) + 1, the error
    // mul - 2^(31+l) / d <= 1 adds less than key / 2^(31+l) < 1 / d to the quotient
    int l = 0;
    while ((1ll << l) < p.page_size) ++l;
    p.page_mul = static_cast<uint32_t>((1ull << (31 + l)) / static_cast<uint32_t>(p.page_size) + 1);
    p.page_shift = l - 1;
    // once per device (the call costs half a microsecond; doing it twice is harmless)
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(paged_attn_kernel<C, TEST>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<C>::BYTES);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    // one resident wave, or a CTA per tile where the table cannot hold as many
    long long grid = static_cast<long long>(num_sms) * C::CTAS;
    const long long span = static_cast<long long>(p.max_pages) * p.page_size;
    const long long most = (span + C::TK - 1) / C::TK * p.B * p.items_per_seq;
    if (grid > most) grid = most;
    if (grid > kPagedMaxCtas) grid = kPagedMaxCtas;
    if (TEST && grid > kSelftestCtas) grid = kSelftestCtas;
    *ctas = static_cast<int>(grid);
    return launch_after(paged_attn_kernel<C, TEST>, *ctas, 32 * (kTeam * C::TEAMS + 1), Smem<C>::BYTES, s, p);
}

}  // namespace
}  // namespace paged
}  // namespace sptp
