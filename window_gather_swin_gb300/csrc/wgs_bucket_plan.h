// Layout of the bucket plan: the inverse of a bucket map (pair -> bucket),
// built on the host and read by position_bias_bwd's kernels.
//
// The pairs (i, j) of a map, numbered i * n_k + j, are cut into tiles of
// kPlanTile consecutive pairs.  A tile's order lists its pairs that hold a
// bucket, grouped by bucket (in the order of the buckets' first pairs, and
// within a bucket in increasing order).  Lane l of kPlanLanes takes the
// entries 32 l ... 32 l + 31; a slot is a run of one bucket's entries within
// a lane.  Slots are numbered along the order, tile by tile.
//
// int32 words, every section starting on a multiple of four words:
//   header[8]              kPlanMagic, n_pairs, n_buckets, n_tiles, n_slots, 0...
//   lane[n_tiles * kPlanLanes]  two words: the lane's entries that end a slot, a
//                          bit each, and its first slot
//   bucket_first[n_buckets + 1]  first place of each bucket in bucket_slot
//   bucket_slot[n_slots]   the slots of each bucket, in increasing order
//   order                  uint16 [n_tiles][4][kPlanLanes][8]: eight entries at a
//                          time of each lane, each the place (plan_place) of
//                          its pair among the tile's
#pragma once

#include <cstdint>

namespace wgs {

constexpr int32_t kPlanMagic = 0x57425032;
constexpr int32_t kPlanTile = 4096;
constexpr int32_t kPlanLanes = kPlanTile / 32;
constexpr int32_t kPlanHeader = 8;

// Where pair i of a tile lies among the tile's sums in shared memory: in its
// block of 32, but on another bank in each, because the lanes of a warp read
// the i-th entries of runs that often lie 32 pairs apart.
#ifdef __CUDACC__
__host__ __device__
#endif
inline constexpr int plan_place(int i) { return i ^ ((i >> 5) & 31); }

struct PlanLayout {
    int64_t lane, bucket_first, bucket_slot, order, words;
};

inline int64_t plan_round4(int64_t v) { return (v + 3) / 4 * 4; }
inline int64_t ceil_tiles(int64_t n_pairs) { return (n_pairs + kPlanTile - 1) / kPlanTile; }

inline PlanLayout plan_layout(int64_t n_pairs, int64_t n_buckets, int64_t n_slots) {
    const int64_t n_tiles = ceil_tiles(n_pairs);
    PlanLayout p;
    p.lane = kPlanHeader;
    p.bucket_first = p.lane + 2 * kPlanLanes * n_tiles;
    p.bucket_slot = p.bucket_first + plan_round4(n_buckets + 1);
    p.order = p.bucket_slot + plan_round4(n_slots);
    p.words = p.order + n_tiles * (kPlanTile / 2);
    return p;
}

}  // namespace wgs
