// Host-side construction of bucket maps (query-key pair -> row of a learned
// position-bias table) and of their inverse, the bucket plan.  The readings
// are stated in wgs.h; the plan's layout in wgs_bucket_plan.h.
#include "wgs.h"
#include "wgs_bucket_plan.h"

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

namespace {

// Buckets of axis k: one per (query, key) position pair when the axis is
// absolute, one per signed difference when it is relative.
int64_t axis_buckets(int32_t extent, bool absolute) {
    return absolute ? static_cast<int64_t>(extent) * extent : 2 * static_cast<int64_t>(extent) - 1;
}

// Cells and buckets of a window, or false for extents below 1, an unknown
// axis bit, or counts past INT32_MAX (buckets, and the pairs of two cells).
bool window_counts(const int32_t window[3], int32_t absolute_axes, int64_t *cells,
                   int64_t *buckets) {
    if (absolute_axes < 0 || absolute_axes > 7) return false;
    int64_t n = 1, b = 1;
    for (int k = 0; k < 3; ++k) {
        if (window[k] < 1 || window[k] > 46340) return false;  // extent^2 fits in int32
        n *= window[k];
        b *= axis_buckets(window[k], (absolute_axes >> k) & 1);
        if (n > 46340 || b > INT32_MAX) return false;
    }
    *cells = n;
    *buckets = b;
    return true;
}

// Groups of a tile: buckets in the order of their first pairs, and how many
// pairs each has.  count holds n_buckets zeros before and after walk().
struct Tile {
    std::vector<int32_t> count, mine;

    explicit Tile(int32_t n_buckets) : count(static_cast<size_t>(n_buckets), 0) {}

    // group(bucket, first entry in the order, entries) for each group of the
    // pairs [p0, p1); false for a value outside [-1, n_buckets)
    template <typename Group>
    bool walk(const int32_t *bucket, int64_t p0, int64_t p1, Group group) {
        bool ok = true;
        mine.clear();
        for (int64_t p = p0; p < p1; ++p) {
            const int32_t b = bucket[p];
            if (b < -1 || b >= static_cast<int64_t>(count.size())) {
                ok = false;
                break;
            }
            if (b >= 0 && count[static_cast<size_t>(b)]++ == 0) mine.push_back(b);
        }
        int32_t entry = 0;
        for (int32_t b : mine) {
            int32_t &n = count[static_cast<size_t>(b)];
            if (ok) group(b, entry, n);
            entry += n;
            n = 0;
        }
        return ok;
    }
};

int64_t tile_end(int64_t tile, int64_t n_pairs) {
    const int64_t p = (tile + 1) * wgs::kPlanTile;
    return p < n_pairs ? p : n_pairs;
}

// Slots of a map; false for a value outside [-1, n_buckets).
bool count_slots(const int32_t *bucket, int64_t n_pairs, int32_t n_buckets, int64_t *n_slots) {
    Tile tile(n_buckets);
    int64_t slots = 0;
    for (int64_t t = 0; t < wgs::ceil_tiles(n_pairs); ++t)
        if (!tile.walk(bucket, t * wgs::kPlanTile, tile_end(t, n_pairs), [&](int32_t, int32_t entry, int32_t n) {
                slots += (entry + n - 1) / 32 - entry / 32 + 1;
            }))
            return false;
    *n_slots = slots;
    return true;
}

bool plan_sizes_ok(int64_t n_pairs, int32_t n_buckets) {
    return n_pairs >= 0 && n_pairs <= INT32_MAX - wgs::kPlanTile && n_buckets >= 1 &&
           n_buckets < INT32_MAX;
}

}  // namespace

extern "C" int64_t wgs_window_bucket_count(const int32_t window[3], int32_t absolute_axes) {
    int64_t cells, buckets;
    if (!window || !window_counts(window, absolute_axes, &cells, &buckets)) return -1;
    return buckets;
}

extern "C" wgs_status wgs_build_window_buckets(const int32_t window[3], int32_t absolute_axes,
                                               int32_t *out_host, int64_t out_len) {
    if (!window || !out_host) return WGS_ERR_NULL;
    int64_t n, buckets;
    if (!window_counts(window, absolute_axes, &n, &buckets)) return WGS_ERR_SHAPE;
    if (out_len < n * n) return WGS_ERR_SHAPE;
    const int64_t hw = static_cast<int64_t>(window[1]) * window[2];
    for (int64_t i = 0; i < n; ++i) {
        const int64_t qi[3] = {i / hw, i / window[2] % window[1], i % window[2]};
        for (int64_t j = 0; j < n; ++j) {
            const int64_t kj[3] = {j / hw, j / window[2] % window[1], j % window[2]};
            int64_t b = 0;
            for (int k = 0; k < 3; ++k) {
                const bool absolute = (absolute_axes >> k) & 1;
                b = b * axis_buckets(window[k], absolute) +
                    (absolute ? qi[k] * window[k] + kj[k] : qi[k] - kj[k] + window[k] - 1);
            }
            out_host[i * n + j] = static_cast<int32_t>(b);
        }
    }
    return WGS_OK;
}

extern "C" wgs_status wgs_build_distance_buckets(int64_t n_q, int64_t n_k, int64_t q_start,
                                                 int32_t n_buckets, int32_t max_distance,
                                                 int32_t bidirectional, int32_t *out_host,
                                                 int64_t out_len) {
    if (n_q < 0 || n_k < 0 || q_start < 0 || n_q > INT32_MAX || n_k > INT32_MAX ||
        q_start > INT32_MAX || (bidirectional != 0 && bidirectional != 1))
        return WGS_ERR_SHAPE;
    const int32_t half = bidirectional ? n_buckets / 2 : n_buckets;
    const int32_t exact = half / 2;
    if (exact < 1 || (bidirectional && n_buckets % 2 != 0) || max_distance <= exact)
        return WGS_ERR_SHAPE;
    if (n_q == 0 || n_k == 0) return WGS_OK;
    if (!out_host) return WGS_ERR_NULL;
    if (n_k > INT64_MAX / n_q || out_len < n_q * n_k) return WGS_ERR_SHAPE;
    // the bucket depends on the distance alone; beyond max_distance it is the last.
    // No pair is farther apart than `far`
    const int64_t behind = n_q - 1 + q_start, ahead = n_k - 1;
    const int64_t most = behind > ahead ? behind : ahead, far = most < max_distance ? most : max_distance;
    std::vector<int32_t> of;
    try {
        of.resize(static_cast<size_t>(far) + 1);
    } catch (const std::bad_alloc &) {
        return WGS_ERR_TOO_LARGE;
    }
    const double scale = (half - exact) / std::log(static_cast<double>(max_distance) / exact);
    for (int64_t d = 0; d <= far; ++d) {
        int64_t b = d;
        if (d >= exact) {
            b = exact + static_cast<int64_t>(
                            std::floor(std::log(static_cast<double>(d) / exact) * scale + 1e-9));
            if (b > half - 1) b = half - 1;
        }
        of[static_cast<size_t>(d)] = static_cast<int32_t>(b);
    }
    for (int64_t i = 0; i < n_q; ++i)
        for (int64_t j = 0; j < n_k; ++j) {
            const int64_t d = j - (i + q_start);  // key minus query position
            int32_t b = -1;
            if (d <= 0 || bidirectional) {
                const int64_t away = d < 0 ? -d : d;
                b = of[static_cast<size_t>(away < far ? away : far)] +
                    (d > 0 ? half : 0);
            }
            out_host[i * n_k + j] = b;
        }
    return WGS_OK;
}

extern "C" int64_t wgs_bucket_plan_words(const int32_t *bucket_host, int64_t n_pairs,
                                         int32_t n_buckets, int64_t *n_slots) {
    if (!plan_sizes_ok(n_pairs, n_buckets) || (n_pairs > 0 && !bucket_host)) return -1;
    try {
        int64_t slots;
        if (!count_slots(bucket_host, n_pairs, n_buckets, &slots)) return -1;
        if (n_slots) *n_slots = slots;
        return wgs::plan_layout(n_pairs, n_buckets, slots).words;
    } catch (const std::bad_alloc &) {
        return -1;
    }
}

extern "C" wgs_status wgs_build_bucket_plan(const int32_t *bucket_host, int64_t n_pairs,
                                            int32_t n_buckets, int32_t *plan_host,
                                            int64_t plan_words) {
    if (!plan_sizes_ok(n_pairs, n_buckets)) return WGS_ERR_SHAPE;
    if (!plan_host || (n_pairs > 0 && !bucket_host)) return WGS_ERR_NULL;
    try {
        const size_t nb = static_cast<size_t>(n_buckets);
        int64_t slots;
        if (!count_slots(bucket_host, n_pairs, n_buckets, &slots)) return WGS_ERR_INDEX;
        const wgs::PlanLayout at = wgs::plan_layout(n_pairs, n_buckets, slots);
        if (plan_words < at.words) return WGS_ERR_SHAPE;
        const int64_t n_tiles = wgs::ceil_tiles(n_pairs);
        std::vector<int32_t> next(nb);  // entry of the next pair of each bucket
        std::vector<int32_t> of_slot;   // the bucket of each slot
        of_slot.reserve(static_cast<size_t>(slots));

        std::memset(plan_host, 0, static_cast<size_t>(at.words) * sizeof(int32_t));
        const int32_t head[5] = {wgs::kPlanMagic, static_cast<int32_t>(n_pairs), n_buckets,
                                 static_cast<int32_t>(n_tiles), static_cast<int32_t>(slots)};
        std::memcpy(plan_host, head, sizeof(head));
        int32_t *first = plan_host + at.bucket_first, *bucket_slot = plan_host + at.bucket_slot;
        Tile tile(n_buckets);
        for (int64_t t = 0; t < n_tiles; ++t) {
            int32_t *lane = plan_host + at.lane + t * 2 * wgs::kPlanLanes;
            uint16_t *order = reinterpret_cast<uint16_t *>(plan_host + at.order) + t * wgs::kPlanTile;
            const int64_t p0 = t * wgs::kPlanTile, p1 = tile_end(t, n_pairs);
            tile.walk(bucket_host, p0, p1, [&](int32_t b, int32_t entry, int32_t n) {
                next[static_cast<size_t>(b)] = entry;
                for (int32_t e = entry; e < entry + n;) {
                    const int32_t l = e / 32, end = (l + 1) * 32 < entry + n ? (l + 1) * 32 : entry + n;
                    if (e % 32 == 0) lane[2 * l + 1] = static_cast<int32_t>(of_slot.size());
                    const uint32_t bit = uint32_t{1} << (end - 1) % 32;
                    lane[2 * l] = static_cast<int32_t>(static_cast<uint32_t>(lane[2 * l]) | bit);
                    of_slot.push_back(b);
                    ++first[static_cast<size_t>(b) + 1];
                    e = end;
                }
            });
            for (int64_t p = p0; p < p1; ++p) {
                if (bucket_host[p] < 0) continue;
                const int32_t e = next[static_cast<size_t>(bucket_host[p])]++;
                order[(e % 32 / 8 * wgs::kPlanLanes + e / 32) * 8 + e % 8] =
                    static_cast<uint16_t>(wgs::plan_place(static_cast<int>(p - p0)));
            }
        }
        for (size_t b = 0; b < nb; ++b) first[b + 1] += first[b];
        std::vector<int32_t> place(first, first + nb);
        for (size_t s = 0; s < of_slot.size(); ++s)
            bucket_slot[place[static_cast<size_t>(of_slot[s])]++] = static_cast<int32_t>(s);
        return WGS_OK;
    } catch (const std::bad_alloc &) {
        return WGS_ERR_TOO_LARGE;
    }
}
