// How embedding_bwd cuts a gradient: host arithmetic, of sizes alone.
#pragma once

#include "wgs_sizes.h"

namespace wgs {

namespace {

// ------------------------------------------------------------------- sizes --

constexpr int kSortThreads = 512;      // of the sort's blocks
constexpr int kRounds = 4;             // indices of a thread at a time
constexpr int kSortTile = kSortThreads * kRounds;
// Blocks of a tile or less each, twice as many before a block takes more: every block
// reads all blocks' counts.  131040 indices into 24 and 32768 rows and 131040 rows once
// each, whole calls: 22.2, 57.9 and 52.1 us, with 32 blocks 24.8, 65.9 and 56.8, with 128
// 22.3, 56.3 and 55.0.
constexpr int kSortBlocks = 64;

constexpr int kSumThreads = 256;       // of the sums' blocks
// Of a block: the slots' ends are joined one after another.
constexpr int kMostSlots = 32;
constexpr int kMostPiece = 2048;       // indices of a block

constexpr int kFew = 1024;             // indices that every block sorts
static_assert(kFew <= kSortTile, "a tile of the sort");
constexpr int kFewCols = 64;           // threads of a row there, 16 bytes each: a block's part of it
constexpr int kTileBlocks = 152;       // of tiles: one an SM

// -------------------------------------------------------------------- plan --

// How a gradient is cut, and where its parts lie in the workspace.
struct Plan {
    bool few;                        // one launch
    int tile, tile_blocks;           // or two, in tiles of so many indices (0: not so)
    int passes, bits, sort_blocks;   // of the sort
    int64_t range;
    int slices, cols, slots, each, piece;
    int64_t pieces;
    int count_bytes;
    int64_t keys[2], at[2], counts, part, bytes;
};

// v: values of a thread
inline Plan plan_of(int64_t n, int64_t n_rows, int32_t width, int v) {
    Plan z = {};
    int bits = 1;
    while (bits < 31 && n_rows >> bits) ++bits;     // keys are 0 ... n_rows
    z.passes = static_cast<int>(ceil_div(bits, 9));
    z.bits = static_cast<int>(ceil_div(bits, z.passes));
    if (z.bits < 4) z.bits = 4;      // whole 16 bytes of a block's counts
    // whole rounds of a block's threads; twice the blocks where a tile each is too little
    int64_t rounds = ceil_div(ceil_div(n, kSortThreads), kSortBlocks);
    if (rounds > kRounds) {
        rounds = ceil_div(ceil_div(n, kSortThreads), 2 * kSortBlocks);
        if (rounds < kRounds) rounds = kRounds;
    }
    z.range = rounds * kSortThreads;
    z.sort_blocks = n ? static_cast<int>(ceil_div(n, z.range)) : 0;
    z.count_bytes = z.range < 65536 ? 2 : 4;
    const int parts = static_cast<int>(ceil_div(width, v));
    z.few = n <= kFew;
    // a tile an SM (or the largest ones), of four indices for each 16 bytes of a column of
    // the table at least, so that the blocks' tables, written and read, are an eighth of
    // the gradients' bytes at most
    const int64_t tile = ceil_div(n, kTileBlocks) < kSortTile ? ceil_div(n, kTileBlocks) : kSortTile;
    if (!z.few && n_rows > 0 && 4 * n_rows * v <= tile) {
        z.tile = static_cast<int>(tile);
        z.tile_blocks = static_cast<int>(ceil_div(n, tile));
    }
    z.slices = static_cast<int>(ceil_div(parts, z.few ? kFewCols : z.tile ? kSortThreads : kSumThreads));
    z.cols = static_cast<int>(ceil_div(parts, z.slices));
    if (z.few || z.tile) {
        z.bytes = z.tile ? 4ll * z.tile_blocks * n_rows * width : n ? 16 : 0;
        return z;
    }
    z.slots = kSumThreads / z.cols < kMostSlots ? kSumThreads / z.cols : kMostSlots;
    // some six blocks an SM, of slots of 8 to 64 indices (131040 indices into 24 rows of
    // 192: 22.2 us a call, with four 25.1, with eight 23.8, with twelve 26.1)
    const int64_t want = ceil_div(n, static_cast<int64_t>(z.slots) * 912);
    z.each = want < 8 ? 8 : want > 64 ? 64 : static_cast<int>(want);
    z.piece = z.slots * z.each;
    z.pieces = ceil_div(n, z.piece);
    int64_t at = 0;
    auto place = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 15) / 16 * 16;
        return here;
    };
    for (int i = 0; i < 2; ++i) {
        if (i < z.passes) z.keys[i] = place(4 * n), z.at[i] = place(4 * n);
    }
    z.counts = place(1ll * z.passes * z.sort_blocks * z.count_bytes << z.bits);
    z.part = place(z.pieces * 8 * width);
    z.bytes = at;
    return z;
}

// A thread's values are four or eight with grad's format, which cuts more or fewer
// pieces.
inline int64_t workspace_of(int64_t n, int64_t n_rows, int32_t width) {
    const int64_t four = plan_of(n, n_rows, width, 4).bytes, eight = plan_of(n, n_rows, width, 8).bytes;
    return four > eight ? four : eight;
}

// The table's zeros that the sort's launch of pass `pass` (-1: the counts before the
// first) writes beside its own work, and the blocks that do: 64 bytes a thread or more, by
// as many blocks as are resident beside the sort's (with 88 blocks 57 us in place of 53
// for 32768 rows of 384 FP32), and at least one where the sort's own fill a device of few
// SMs.  Zeros in the rows alone that no index names, written by blocks of the sums'
// launch, took those 6 us longer and spared the sort 5.
struct ZeroShare {
    int64_t first, bytes, blocks;
};

inline ZeroShare zero_share(const Plan &z, int pass, int64_t bytes, int sms) {
    const int64_t each = ceil_div(ceil_div(bytes, 1 + z.passes), 16) * 16, first = (pass + 1) * each;
    const int64_t here = bytes - first < each ? bytes - first : each;
    if (here <= 0) return {0, 0, 0};
    const int64_t want = ceil_div(here, 64 * kSortThreads);
    const int64_t room = 2 * sms - z.sort_blocks < 1 ? 1 : 2 * sms - z.sort_blocks;
    return {first, here, want < room ? want : room};
}

}  // namespace

}  // namespace wgs
