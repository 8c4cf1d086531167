// How the work of sptp_paged_attn_prompt is dealt out.
//
// The rows of a sequence are cut into blocks of `tokens` rows; a block and the
// query heads of one key/value head of one shard (up to `heads` of them) make an
// item of tokens * heads query rows, which sees a run of its sequence's keys, in
// tiles of TK.  The tiles of all items, in order, are dealt out to the CTAs of
// one resident wave in contiguous shares of equal cost, so that every SM has the
// same work whatever the lengths, masks and counts of rows are: kTileCost a tile
// and ITEM_COST an item (of its loads, its first scores and its end).  An item that crosses a share's end leaves its parts'
// maxima, sums and outputs in the workspace, and a second launch joins them in a
// fixed order.  Every CTA works out its own share from the lengths.
//
// Blocks are numbered without a pass over the sequences: block i of sequence b
// is number row_starts[b] / tokens + b + i.  Since floor((s + n) / t) + 1 - floor(s
// / t) >= ceil(n / t), sequences do not overlap; a number between them that no
// block has costs nothing.
#pragma once

#include "prompt_attn.h"
#include "sptp_ptx.cuh"

namespace sptp {
namespace prompt {

constexpr int kTileCost = 4;

struct Block {
    int b;        // sequence
    int row0, n;  // rows [row0, row0 + n) of the batch
    int pos0;     // position of row0 in its sequence
    int len;      // keys of the sequence
    int prefix;   // of them, that every row sees
    int lo, hi;   // keys that any row sees
    int tiles;    // TK-wide tiles that hold them, 1 if there are none; 0: no such block
};

__device__ __forceinline__ int row_start(const PromptParams& p, int b) {
    return max(0, min(p.M, __ldg(p.row_starts + b)));
}

__device__ __forceinline__ long long block_numbers(const PromptParams& p) {
    return row_start(p, p.B) / p.tokens + p.B;
}

// Keys [lo, hi) that the row at position pos sees.
__device__ __forceinline__ int first_key(const PromptParams& p, int pos) {
    return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}
__device__ __forceinline__ int end_key(int pos, int prefix) { return pos < 0 ? 0 : max(pos + 1, prefix); }

template <int TK>
__device__ __forceinline__ Block block_of(const PromptParams& p, long long number, int b) {
    Block k;
    k.b = b;
    // (what is outside its range is cut to it here, and reported by the join)
    const int s = row_start(p, b), e = max(s, row_start(p, b + 1));
    k.len = max(0, min(p.max_pages * p.page_size, __ldg(p.seq_lens + b)));
    k.prefix = p.prefix_lens != nullptr ? max(0, min(k.len, __ldg(p.prefix_lens + b))) : 0;
    const long long i = number - (s / p.tokens + b);
    k.tiles = 0;
    if (i < 0 || i * p.tokens >= e - s) return k;
    const int t0 = static_cast<int>(i) * p.tokens;
    k.row0 = s + t0;
    k.n = min(p.tokens, e - s - t0);
    k.pos0 = k.len - (e - s) + t0;
    k.lo = first_key(p, k.pos0);
    k.hi = end_key(k.pos0 + k.n - 1, k.prefix);
    k.tiles = k.hi > k.lo ? (k.hi + TK - 1) / TK - k.lo / TK : 1;
    return k;
}

// The sequence that a block number belongs to.
__device__ __forceinline__ int sequence_of(const PromptParams& p, long long number) {
    int lo = 0, hi = p.B;  // the last b in [0, B) whose first number is not above
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row_start(p, mid) / p.tokens + mid <= number)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Position in the list of tiles: tile t of item j of block `number`, whose cost
// begins at `at`.
template <int TK, int ITEM_COST>
struct Cursor {
    long long at, number;
    int j, t;
    Block k;

    __device__ __forceinline__ long long item_cost() const {
        return static_cast<long long>(k.tiles) * kTileCost + ITEM_COST;
    }
    __device__ __forceinline__ int key0() const { return (k.lo / TK + t) * TK; }
    __device__ __forceinline__ long long tile_at() const { return at + static_cast<long long>(t) * kTileCost; }
    // To the next item; false behind the last one.
    __device__ __forceinline__ bool next_item(const PromptParams& p, long long numbers) {
        at += item_cost();
        t = 0;
        if (++j < p.items_per_block) return true;
        j = 0;
        for (++number; number < numbers; ++number) {
            int b = k.b;
            while (b + 1 < p.B && row_start(p, b + 1) / p.tokens + b + 1 <= number) ++b;
            k = block_of<TK>(p, number, b);
            if (k.tiles != 0) return true;
        }
        return false;
    }
};

struct Share {
    long long begin, end, size;
};

// This CTA's share, by all its THREADS threads; `warp_cost` [THREADS / 32] and
// `at` are shared memory.  at->k.tiles == 0 afterwards: an empty share.
template <int THREADS, int TK, int ITEM_COST>
__device__ __forceinline__ Share find_share(const PromptParams& p, long long* warp_cost, Cursor<TK, ITEM_COST>* at) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long numbers = block_numbers(p);
    const long long run = (numbers + THREADS - 1) / THREADS;
    const long long n0 = min(numbers, tid * run), n1 = min(numbers, n0 + run);
    long long mine = 0;
    int b = n0 < n1 ? sequence_of(p, n0) : 0;
    const int b0 = b;
    for (long long n = n0; n < n1; ++n) {
        while (b + 1 < p.B && row_start(p, b + 1) / p.tokens + b + 1 <= n) ++b;
        const Block k = block_of<TK>(p, n, b);
        if (k.tiles != 0) mine += static_cast<long long>(k.tiles) * kTileCost + ITEM_COST;
    }
    mine *= p.items_per_block;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) warp_cost[warp] = incl;
    if (tid == 0) at->k.tiles = 0;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += warp_cost[w];
        total += warp_cost[w];
    }
    // A tile belongs to the share in which its cost begins; a share is at least
    // one tile's cost, so that an item's parts lie in successive shares.
    Share s;
    s.size = max(static_cast<long long>(kTileCost), (total + gridDim.x - 1) / gridDim.x);
    s.begin = s.size * blockIdx.x;
    s.end = s.begin + s.size;
    if (s.begin >= before && s.begin < before + mine) {
        Cursor<TK, ITEM_COST> c;
        c.at = before;
        int q = b0;
        for (c.number = n0;; ++c.number) {
            while (q + 1 < p.B && row_start(p, q + 1) / p.tokens + q + 1 <= c.number) ++q;
            c.k = block_of<TK>(p, c.number, q);
            if (c.k.tiles == 0) continue;
            const long long n = c.item_cost() * p.items_per_block;
            if (s.begin < c.at + n) break;
            c.at += n;
        }
        c.j = static_cast<int>((s.begin - c.at) / c.item_cost());
        c.at += c.j * c.item_cost();
        c.t = static_cast<int>((s.begin - c.at + kTileCost - 1) / kTileCost);
        bool more = true;
        if (c.t >= c.k.tiles) more = c.next_item(p, numbers);
        if (more && c.tile_at() < s.end) *at = c;
    }
    __syncthreads();
    return s;
}

// What a CTA does of one item: tiles [t, t + here) of it.
struct Piece {
    int here;
    bool begins, ends;           // the item's own first and last tile are among them
    int shard, kvh, head0, heads;
    long long token0;            // shard * M + first row
};

template <int TK, int ITEM_COST>
__device__ __forceinline__ Piece piece_of(const PromptParams& p, const Cursor<TK, ITEM_COST>& c, const Share& s) {
    Piece r;
    const long long room = (s.end - c.tile_at() + kTileCost - 1) / kTileCost;
    r.here = static_cast<int>(min(static_cast<long long>(c.k.tiles - c.t), room));
    r.begins = c.t == 0;
    r.ends = c.t + r.here == c.k.tiles;
    const int group = p.Hq / p.Hkv;
    const int hb = c.j % p.head_blocks, sk = c.j / p.head_blocks;
    r.shard = sk / p.Hkv;
    r.kvh = sk - r.shard * p.Hkv;
    r.head0 = r.kvh * group + hb * p.heads;
    r.heads = min(p.heads, group - hb * p.heads);
    r.token0 = static_cast<long long>(r.shard) * p.M + c.k.row0;
    return r;
}

// The item for the join, if it does not both begin and end in this share.
template <int TK, int ITEM_COST>
__device__ __forceinline__ PromptItem split_item(const Cursor<TK, ITEM_COST>& c, const Piece& r, const Share& s) {
    PromptItem it;
    it.first = static_cast<int>(c.at / s.size);
    it.parts = static_cast<int>((c.at + static_cast<long long>(c.k.tiles - 1) * kTileCost) / s.size) - it.first + 1;
    it.tokens = c.k.n;
    it.heads = r.heads;
    it.token0 = r.token0;
    it.head0 = r.head0;
    it.pad = 0;
    return it;
}

// Pool row of key `key` of sequence b for (shard, kvh); -1: its page is outside the pool.
__device__ __forceinline__ long long pool_row(const PromptParams& p, int b, int shard, int kvh, int key) {
    const int index = static_cast<int>(__umulhi(static_cast<uint32_t>(key), p.page_mul) >> p.page_shift);
    const int page = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + index);
    if (page < 0 || page >= p.num_pages) return -1;
    return ((static_cast<long long>(shard) * p.num_pages + page) * p.Hkv + kvh) * p.page_size + key - index * p.page_size;
}

}  // namespace prompt
}  // namespace sptp
