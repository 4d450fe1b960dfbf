// moe_plan.h -- layout of a grouping of rows by expert (the plan that
// nvfp4_moe_route and nvfp4_moe_plan write, include/nvfp4.h).
// Host and device arithmetic only: plain C++.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace nvfp4 {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxK = 32;
constexpr int64_t kMoeMaxSlots = 1LL << 24;
constexpr int kMoeBlock = 128;      // every expert's rows begin on a multiple of this in the quantised operands
constexpr int kMoeChunk = 32768;    // slots of a CTA at most (16-bit counters)
constexpr int kMoeHeader = 16;      // 32-bit words

// Words of the header.
enum MoeHeaderWord : int { kMoeRows = 0, kMoeBlocks = 1, kMoeTiles = 2 };

// Rows of a product's tile.  The weights are read once for each tile of an
// expert, so as far as tiles go (256) one holds what an expert has on average and
// some more.  64 at least: the tensor cores take a tile's scales from an even
// column (32 rows a column).
//
// 64 rows are streamed, with the weights on their way while the rows are
// quantised, 128 and 256 go to CTA pairs.  The layer in bf16, us at 64 / 128 / 256
// for experts with 8, 40, 64 rows on average (two of E for a token): 16 of 2048 x
// 2048 10.3 / 10.9 / 13.6, 10.8 / 11.0 / 14.1, 14.0 / 11.4 / 14.3; 128 of 1536 x 4096
// 73.3 / 78.0 / 79.9, 82.7 / 84.0 / 85.3, 95.8 / 88.5 / 90.1; 60 of 2600 x 3584 55.3 /
// 53.7 / 56.4, 62.3 / 57.8 / 58.9, 70.7 / 59.7 / 60.7; 8 of 14336 x 4096 44.7 / 44.7 /
// 46.8, 46.8 / 46.0 / 48.1, 55.6 / 46.6 / 48.7.  The product alone at 96, 128, 192 rows,
// 128 / 256: the 128 experts 79.2 / 80.2, 82.6 / 83.2, 96.3 / 90.7; the 8 45.3 / 46.1,
// 53.4 / 47.6, 59.5 / 50.5.  An expert far above the average only costs its own weights'
// reads again: 32 rows on average and 630 in one of 128, 81.3 / 81.3 / 83.6.
inline int moe_tile_rows(int64_t slots, int experts)
{
    const int64_t mean = slots / std::min<int64_t>(slots, experts);
    return mean <= 40 ? 64 : mean <= 96 ? 128 : 256;
}

// Where things are in the plan's buffer, in 32-bit words; every part begins on
// a multiple of four.
struct MoeLayout {
    int64_t slots;      // T k
    int experts;
    int tile_rows;
    int64_t max_blocks, max_tiles;
    int ctas;           // of the counting kernels; 1: everything in one
    int64_t offsets, first_block, position, order, padded, blocks, tiles, counts, total;

    MoeLayout(int64_t T, int64_t k, int E)
    {
        slots = T * k;
        experts = E;
        tile_rows = moe_tile_rows(slots, E);
        const int64_t some = std::min<int64_t>(slots, E);   // experts with rows, at most
        max_blocks = slots / kMoeBlock + some;
        max_tiles = slots / tile_rows + some;
        // one for every 1024 slots (a thread each), up to one for each of the chip's 152 SMs
        ctas = (int)std::max<int64_t>(std::min<int64_t>(152, (slots + 1023) / 1024), (slots + kMoeChunk - 1) / kMoeChunk);
        int64_t at = kMoeHeader;
        auto take = [&](int64_t words) {
            const int64_t p = at;
            at += (words + 3) / 4 * 4;
            return p;
        };
        offsets = take(E + 1);
        first_block = take(E + 1);
        position = take(slots);
        order = take(slots);
        padded = take(slots);
        blocks = take(4 * max_blocks);
        tiles = take(4 * max_tiles);
        counts = take(ctas > 1 ? (int64_t)ctas * E : 0);
        total = at;
    }
    int64_t padded_rows() const { return max_blocks * kMoeBlock; }
};

inline bool moe_sizes_ok(int64_t T, int64_t k, int64_t E)
{
    return T >= 1 && T <= kMoeMaxSlots && k >= 1 && k <= kMoeMaxK && E >= 1 && E <= kMoeMaxExperts && T * k <= kMoeMaxSlots;
}

}  // namespace nvfp4
