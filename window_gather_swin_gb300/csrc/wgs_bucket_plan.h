// Layout of the bucket plan: the inverse of a bucket map (pair -> bucket),
// built on the host and read by position_bias_bwd's kernels.
//
// The pairs (i, j) of a map, numbered i * n_k + j, are cut into tiles of
// kPlanTile consecutive pairs.  Inside a tile the pairs that hold a bucket
// are grouped by bucket, in increasing order within one; a group is a slot.  A slot's
// destination is its place among all slots sorted by bucket, so the slots of
// one bucket are neighbours there, in tile order.
//
// int32 words, every section starting on a multiple of four words:
//   header[8]              kPlanMagic, n_pairs, n_buckets, n_tiles, n_slots, 0...
//   tile_slot[n_tiles + 1] first slot of each tile
//   slot[n_slots]          two words: the slot's first entry in its tile's
//                          order and the number of entries << 16; its destination
//   bucket_dest[n_buckets + 1]  first destination of each bucket
//   order                  uint16 [n_tiles * kPlanTile]: per tile, the
//                          tile's pairs grouped by bucket, as offsets into it
#pragma once

#include <cstdint>

namespace wgs {

constexpr int32_t kPlanMagic = 0x57425031;
constexpr int32_t kPlanTile = 4096;
constexpr int32_t kPlanHeader = 8;

struct PlanLayout {
    int64_t tile_slot, slot, bucket_dest, order, words;
};

inline int64_t plan_round4(int64_t v) { return (v + 3) / 4 * 4; }

inline int64_t ceil_tiles(int64_t n_pairs) { return (n_pairs + kPlanTile - 1) / kPlanTile; }

inline PlanLayout plan_layout(int64_t n_pairs, int64_t n_buckets, int64_t n_slots) {
    const int64_t n_tiles = ceil_tiles(n_pairs);
    PlanLayout p;
    p.tile_slot = kPlanHeader;
    p.slot = p.tile_slot + plan_round4(n_tiles + 1);
    p.bucket_dest = p.slot + plan_round4(2 * n_slots);
    p.order = p.bucket_dest + plan_round4(n_buckets + 1);
    p.words = p.order + n_tiles * (kPlanTile / 2);
    return p;
}

}  // namespace wgs
