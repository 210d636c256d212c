// Learned position bias by buckets and its gradient (sm_103a).
//
// A shifted-window block adds a learned bias to its attention logits.  What
// is learned is a table with one value per window type, bucket and head; a
// bucket map sends every (query, key) pair to a row of the table, or to -1
// for a pair that has none.  With p numbering the n_q * n_k pairs,
//     bias[t, h, p]       = table[t, bucket[p], h]        (0 for bucket -1)
//     grad_table[t, b, h] = sum over windows w of type t and pairs p with
//                           bucket[p] = b of grad[w, h, p]
// The first is what window_bias_mask_add reads as its `bias`; the second
// takes the gradient of the logits, through which the bias addition passes
// unchanged.
#include <type_traits>

#include "wgs_bucket_plan.h"
#include "wgs_common.cuh"

namespace wgs {

namespace {

// Set (never cleared by a kernel) when a bucket lies outside [-1, n_buckets),
// a window type outside [0, n_types), or a plan does not belong to the sizes
// it came with (bit 0), or a block gave up waiting for its own copies (bit 1);
// read and cleared by wgs_check_error.
__device__ unsigned int g_bucket_error;

}  // namespace

// As bias_mask_error_take, for the position-bias error word.
wgs_status position_bias_error_take(unsigned int *seen, cudaStream_t stream) {
    static const unsigned int cleared = 0;
    if (cudaMemcpyFromSymbolAsync(seen, g_bucket_error, sizeof(*seen), 0, cudaMemcpyDeviceToHost,
                                  stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_bucket_error, &cleared, sizeof(cleared), 0,
                                cudaMemcpyHostToDevice, stream) != cudaSuccess) {
        cudaGetLastError();  // clear this thread's error
        return WGS_ERR_CUDA;
    }
    return WGS_OK;
}

namespace {

constexpr int kThreads = 256;

struct F32 {};

template <typename T>
constexpr int kBytes = std::is_same<T, F32>::value ? 4 : 2;

// One table or gradient element as FP32 (exact).
template <typename T>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if constexpr (std::is_same<T, F32>::value)
        return static_cast<const float *>(p)[i];
    else
        return T::to_f2(static_cast<const uint16_t *>(p)[i]).x;
}

template <typename T>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
    if constexpr (std::is_same<T, F32>::value)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(T::from_f2(v, 0.f));
}

// HC neighbouring table values in one load, as their words: FP32 values, or
// 16-bit values in pairs (one alone in the low half).
template <typename T, int HC>
struct Heads {
    static constexpr int kWords = kBytes<T> == 4 ? HC : (HC + 1) / 2;
    uint32_t w[kWords];

    __device__ void zero() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = 0u;
    }
    __device__ void load(const char *p) {
        if constexpr (HC * kBytes<T> == 16) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
            w[0] = q.x, w[1] = q.y, w[kWords - 2] = q.z, w[kWords - 1] = q.w;
        } else if constexpr (HC * kBytes<T> == 8) {
            const uint2 q = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = q.x, w[kWords - 1] = q.y;
        } else if constexpr (HC * kBytes<T> == 4) {
            w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
        } else {
            w[0] = __ldg(reinterpret_cast<const uint16_t *>(p));
        }
    }
    __device__ float value(int k) const {
        if constexpr (kBytes<T> == 4) {
            return __uint_as_float(w[k]);
        } else {
            const float2 f = T::to_f2(w[k / 2]);
            return k & 1 ? f.y : f.x;
        }
    }
};

// Head k's values of eight pairs as outputs at a 16-byte aligned address:
// copied where table and output have one format, else rounded once, to
// nearest even.
template <typename O, typename T, int HC>
__device__ __forceinline__ void store8(void *p, const Heads<T, HC> (&v)[8], int k) {
    uint4 *q = static_cast<uint4 *>(p);
    if constexpr (kBytes<O> == 4) {
        st_stream(q, make_uint4(v[0].w[k], v[1].w[k], v[2].w[k], v[3].w[k]));
        st_stream(q + 1, make_uint4(v[4].w[k], v[5].w[k], v[6].w[k], v[7].w[k]));
    } else if constexpr (std::is_same<O, T>::value) {
        const uint32_t pick = k & 1 ? 0x7632 : 0x5410;  // the halves of two words
        uint4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) set_word(o, j, __byte_perm(v[2 * j].w[k / 2], v[2 * j + 1].w[k / 2], pick));
        st_stream(q, o);
    } else {
        uint4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) set_word(o, j, O::from_f2(v[2 * j].value(k), v[2 * j + 1].value(k)));
        st_stream(q, o);
    }
}

// ---------------------------------------------------------------- forward --

struct ExpandArgs {
    const void *table;      // [n_types, n_buckets, heads]
    const int32_t *bucket;  // [n_pairs]
    void *bias;             // [n_types, heads, n_pairs]
    int64_t n_pairs;
    int32_t n_buckets, heads;
    int32_t pair_blocks;    // blocks of kThreads * 8 pairs
    int32_t head_blocks;    // blocks of head_step heads
    int32_t head_step;
};

// Pairs in eights: the map is 16-byte aligned and every (type, head) slab of
// the output starts on 16 bytes.  A thread keeps the buckets of its eight
// pairs in registers and, HC heads at a time, gathers the heads of each
// bucket in one load (they are neighbours in the table) and stores eight
// outputs a head.  Neighbouring pairs name neighbouring or equal table rows,
// so the gather stays in L1; the stores, whole lines a warp, are the cost.  64
// types of 6 heads and 144 x 144 pairs, FP32 tables to fp16: 9.6 us for 16 MB
// written and the tables read.
template <typename O, typename T, int HC>
__global__ void __launch_bounds__(kThreads) bias_expand_eights(ExpandArgs a) {
    pdl_prologue();
    uint32_t blk = blockIdx.x;
    const uint32_t pb = blk % a.pair_blocks;
    blk /= a.pair_blocks;
    const uint32_t hb = blk % a.head_blocks;
    const int64_t type = blk / a.head_blocks;
    const int64_t p = (static_cast<int64_t>(pb) * kThreads + threadIdx.x) * 8;
    if (p >= a.n_pairs) return;
    int32_t row[8];
    const int4 lo = __ldg(reinterpret_cast<const int4 *>(a.bucket + p));
    const int4 hi = __ldg(reinterpret_cast<const int4 *>(a.bucket + p) + 1);
    row[0] = lo.x, row[1] = lo.y, row[2] = lo.z, row[3] = lo.w;
    row[4] = hi.x, row[5] = hi.y, row[6] = hi.z, row[7] = hi.w;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        bad |= row[e] < -1 || row[e] >= a.n_buckets;
        if (row[e] >= a.n_buckets) row[e] = -1;
    }
    if (bad) atomicOr(&g_bucket_error, 1u);
    // byte offsets of the rows from the type's table
    uint32_t at[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) at[e] = static_cast<uint32_t>(max(row[e], 0)) * a.heads * kBytes<T>;
    const char *table = static_cast<const char *>(a.table) + type * a.n_buckets * a.heads * kBytes<T>;
    const int32_t h1 = min(a.heads, static_cast<int32_t>((hb + 1) * a.head_step));
    for (int32_t h = hb * a.head_step; h < h1; h += HC) {
        Heads<T, HC> v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e].zero();
            if (row[e] >= 0) v[e].load(table + h * kBytes<T> + at[e]);
        }
#pragma unroll
        for (int k = 0; k < HC; ++k)
            store8<O>(static_cast<char *>(a.bias) + ((type * a.heads + h + k) * a.n_pairs + p) * kBytes<O>, v, k);
    }
}

// 16 bytes of a row in shared memory, from `lead` elements past the aligned `p` on
// (lead * kB below 16, the same for all threads).
template <int kB>
__device__ __forceinline__ uint4 shifted16(const char *p, int lead) {
    const uint4 lo = reinterpret_cast<const uint4 *>(p)[0];
    if (lead == 0) return lo;
    const uint4 hi = reinterpret_cast<const uint4 *>(p)[1];
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int words = lead * kB / 4;
    uint32_t v[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) {
        const uint32_t near = words & 1 ? w[j + 1] : w[j];
        const uint32_t far = j + 3 > 7 ? 0u : words & 1 ? w[j + 3] : w[j + 2];
        v[j] = words & 2 ? far : near;
    }
    if (kB == 2 && lead & 1)
        return make_uint4(__byte_perm(v[0], v[1], 0x5432), __byte_perm(v[1], v[2], 0x5432),
                          __byte_perm(v[2], v[3], 0x5432), __byte_perm(v[3], v[4], 0x5432));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Any pair count or alignment.  As above up to the stores: the eight outputs of
// a head go to shared memory, HC heads at a time, and from there to the slab
// in 16 bytes cut where the output's address is a multiple of 16, which differs
// from head to head; neighbouring threads store neighbours.
// 16 heads of 2047 x 2047 pairs, bf16: 30 us for 151 MB (5.0 TB/s; in words instead
// of 16 bytes 35, bound by issue).
template <typename O, typename T, int HC>
__global__ void __launch_bounds__(kThreads) bias_expand_any(ExpandArgs a) {
    constexpr int kSpan = kThreads * 8, kB = kBytes<O>, kEach = 16 / kB;
    // kept twice, so that one barrier a step does
    __shared__ __align__(16) char rows[2][HC][kSpan * kB + 16];
    pdl_prologue();
    uint32_t blk = blockIdx.x;
    const uint32_t pb = blk % a.pair_blocks;
    blk /= a.pair_blocks;
    const uint32_t hb = blk % a.head_blocks;
    const int64_t type = blk / a.head_blocks;
    const int64_t p0 = static_cast<int64_t>(pb) * kSpan;
    const int32_t count = static_cast<int32_t>(min(a.n_pairs - p0, static_cast<int64_t>(kSpan)));
    const int32_t mine = static_cast<int32_t>(threadIdx.x) * 8;
    int32_t row[8];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        row[e] = mine + e < count ? __ldg(a.bucket + p0 + mine + e) : -1;
        bad |= row[e] < -1 || row[e] >= a.n_buckets;
        if (row[e] >= a.n_buckets) row[e] = -1;
    }
    if (bad) atomicOr(&g_bucket_error, 1u);
    uint32_t at[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) at[e] = static_cast<uint32_t>(max(row[e], 0)) * a.heads * kBytes<T>;
    const char *table = static_cast<const char *>(a.table) + type * a.n_buckets * a.heads * kBytes<T>;
    const int32_t h1 = min(a.heads, static_cast<int32_t>((hb + 1) * a.head_step));
    int turn = 0;
    for (int32_t h = hb * a.head_step; h < h1; h += HC, turn ^= 1) {
        Heads<T, HC> v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e].zero();
            if (row[e] >= 0) v[e].load(table + h * kBytes<T> + at[e]);
        }
#pragma unroll
        for (int k = 0; k < HC; ++k) store8<O>(rows[turn][k] + mine * kB, v, k);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < HC; ++k) {
            char *to = static_cast<char *>(a.bias) + ((type * a.heads + h + k) * a.n_pairs + p0) * kB;
            const char *from = rows[turn][k];
            // elements before the first whole 16 bytes, whole ones, elements behind
            const int32_t lead = min(static_cast<int32_t>((16 - (reinterpret_cast<uintptr_t>(to) & 15)) & 15) / kB, count);
            const int32_t whole = (count - lead) / kEach, behind = count - lead - whole * kEach;
            for (int32_t i = threadIdx.x; i < whole; i += kThreads)
                st_stream(reinterpret_cast<uint4 *>(to + lead * kB) + i, shifted16<kB>(from + i * 16, lead));
            // the odd elements by threads of their own
            const int32_t e = static_cast<int32_t>(threadIdx.x);
            const int32_t odd = e < lead ? e : count - 1 - (e - lead);
            if (e < lead + behind) {
                if constexpr (kB == 4)
                    reinterpret_cast<uint32_t *>(to)[odd] = reinterpret_cast<const uint32_t *>(from)[odd];
                else
                    reinterpret_cast<uint16_t *>(to)[odd] = reinterpret_cast<const uint16_t *>(from)[odd];
            }
        }
    }
}

// Blocks to aim for when the heads are split over blocks: eight on each of
// 152 SMs.
constexpr int64_t kExpandBlocks = 1216;

template <typename O, typename T>
wgs_status launch_expand(ExpandArgs a, int32_t n_types, cudaStream_t stream) {
    const bool eights = a.n_pairs % 8 == 0 && aligned16(a.bucket) && aligned16(a.bias);
    int hc = 1;
    for (int c = 4; c > 1; c /= 2)
        if (a.heads % c == 0 && reinterpret_cast<uintptr_t>(a.table) % (c * kBytes<T>) == 0) {
            hc = c;
            break;
        }
    if (!eights && kBytes<O> == 4 && hc > 2) hc = 2;  // FP32 rows in 48 KB of shared memory
    const int64_t pair_blocks = ceil_div(a.n_pairs, kThreads * 8);
    // all heads in one block (the map is read once), unless that leaves the GPU idle
    const int64_t want = ceil_div(kExpandBlocks, pair_blocks * n_types);
    const int64_t steps = ceil_div(a.heads, hc);
    a.head_step = static_cast<int32_t>(ceil_div(steps, want < steps ? want : steps)) * hc;
    a.head_blocks = static_cast<int32_t>(ceil_div(a.heads, a.head_step));
    a.pair_blocks = static_cast<int32_t>(pair_blocks);
    const int64_t grid = pair_blocks * a.head_blocks * n_types;
    if (grid > INT32_MAX) return WGS_ERR_SHAPE;
    constexpr int kAny = kBytes<O> == 4 ? 2 : 4;
    auto kernel = eights ? (hc == 4   ? bias_expand_eights<O, T, 4>
                            : hc == 2 ? bias_expand_eights<O, T, 2>
                                      : bias_expand_eights<O, T, 1>)
                         : (hc == 4   ? bias_expand_any<O, T, kAny>
                            : hc == 2 ? bias_expand_any<O, T, 2>
                                      : bias_expand_any<O, T, 1>);
    return launch(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a);
}

// --------------------------------------------------------------- backward --

struct GradArgs {
    const char *grad;         // [n_win, heads, n_pairs]
    int64_t grad_bytes;
    const int32_t *plan;      // wgs_bucket_plan.h
    const int32_t *win_type;  // [n_win] or NULL
    float *partial;           // [slabs, n_types, heads, n_slots]
    void *table;              // grad_table [n_types, n_buckets, heads]
    PlanLayout at;
    int64_t n_pairs;
    int32_t n_win, heads, n_types, n_buckets, n_tiles, n_slots, slabs;
    int32_t units;            // n_tiles * n_types * slabs * heads
    bool early;               // pass 2: pass 1 of the call is the launch before, see start_table
};

// The plan's header against the sizes of the call (a plan of another map
// would name other places).
__device__ __forceinline__ bool plan_matches(const GradArgs &a, bool early = false) {  // early: see start_table
    const int4 *head = reinterpret_cast<const int4 *>(a.plan);
    const int4 v = early ? __ldcg(head) : __ldg(head), w = early ? __ldcg(head + 1) : __ldg(head + 1);
    return v.x == kPlanMagic && v.y == a.n_pairs && v.z == a.n_buckets && v.w == a.n_tiles && w.x == a.n_slots;
}

// The first of `count` things of the i-th of `parts` equal shares.
__device__ __forceinline__ int32_t share_start(int32_t count, int32_t parts, int32_t i) {
    return count / parts * i + min(i, count % parts);
}

// A unit of pass 1: a tile of pairs of one type, slab of windows and head,
// heads first, so that neighbouring units read the same part of the plan and
// list the same windows.
struct Unit {
    int32_t tile, type, slab, head;
    __device__ Unit(const GradArgs &a, int32_t u) {
        head = u % a.heads;
        u /= a.heads;
        slab = u % a.slabs;
        u /= a.slabs;
        type = u % a.n_types;
        tile = u / a.n_types;
    }
    __device__ void next(const GradArgs &a) {
        if (++head < a.heads) return;
        head = 0;
        if (++slab < a.slabs) return;
        slab = 0;
        if (++type < a.n_types) return;
        type = 0;
        ++tile;
    }
};

// Warps of a block: four add windows up, four add the sums up by slot, one copies.
constexpr int kAdders = 128, kSlotters = kPlanLanes;
constexpr int kGradThreads = kAdders + kSlotters + 32;
constexpr int kListed = 1024;                 // windows looked over at a time
// Blocks of an SM, and stages of a block's ring (48 KB).  960 windows of 6 heads and
// 144 x 144 pairs, fp16: two blocks of six stages 59 us, of four 60, one block 84
// (49 now, with slots added by lanes).
constexpr int kGradCtas = 2;
template <typename E>
constexpr int kGradStages = std::is_same<E, F32>::value ? 4 : 6;
template <typename E>
constexpr int kStageBytes = kPlanTile * kBytes<E> + 16;  // a tile that starts between 16-byte borders

// Windows that are added to one FP32 register in a row, in both kernels of pass
// 1; their sum then goes to a second one.  A single register's rounding errors grow
// with a unit's windows, which have no bound: 20,000 gradients of 0.1 were off by
// 1.7e-4.
constexpr int kRun = 128;

// What the copying warp says of a stage.
constexpr int kData = 8, kDirect = 16, kEnd = 32, kRunEnd = 64;  // | elements before the tile's first (0 ... 7)

template <typename E>
struct GradShared {
    alignas(16) char stage[kGradStages<E>][kStageBytes<E>];
    alignas(16) float sums[2][kPlanTile];  // of a unit, and of the next
    int32_t list[kListed];
    int32_t counts[8];
    int32_t said[kGradStages<E>];    // of the stage's window, see kData
    int32_t window[kGradStages<E>];
    alignas(8) uint64_t full[kGradStages<E>], empty[kGradStages<E>];
    uint64_t summed[2], read[2];     // the sums are there, have been added up
};

// The slot of the ring that a side of it is at.
template <int kStages>
struct RingPlace {
    int stage = 0;
    uint32_t phase = 0;
    bool wrapped = false;
    __device__ void next() {
        if (++stage == kStages) stage = 0, phase ^= 1, wrapped = true;
    }
};

__device__ __forceinline__ void must_wait(const uint64_t *bar, uint32_t parity) {
    if (!bar_wait(shared_address(bar), parity)) atomicOr(&g_bucket_error, 2u);
}

// The copying warp: the tiles of each unit's windows into the ring, in order.
// One lane does it, in as few steps a window as can be: a window's latency
// here bounds what the block takes in.
template <typename E, bool kVec>
__device__ void copy_units(const GradArgs &a, GradShared<E> &sh, Unit u, int32_t units, int32_t listed, int lane) {
    constexpr int kES = kBytes<E>, kRing = kGradStages<E>;
    const uint64_t policy = l2_policy(true);
    const uint32_t full = shared_address(sh.full), empty = shared_address(sh.empty), slots = shared_address(sh.stage);
    const char *end = a.grad + a.grad_bytes;
    int stage = 0;
    uint32_t phase = 1;  // of the wait for an empty stage: a new barrier's counts as past
    int32_t listed_type = listed >= 0 ? u.type : -1, listed_slab = u.slab;  // of the list
    int32_t slab = -1, w0 = 0, w1 = 0;
    for (; units > 0; --units, u.next(a)) {
        if (u.slab != slab) {
            slab = u.slab;
            w0 = share_start(a.n_win, a.slabs, slab), w1 = share_start(a.n_win, a.slabs, slab + 1);
        }
        const int64_t p0 = static_cast<int64_t>(u.tile) * kPlanTile;
        const uint32_t bytes = static_cast<uint32_t>(min(a.n_pairs - p0, static_cast<int64_t>(kPlanTile))) * kES;
        const char *tile0 = a.grad + (static_cast<int64_t>(u.head) * a.n_pairs + p0) * kES;
        const int64_t stride = static_cast<int64_t>(a.heads) * a.n_pairs * kES;
        auto advance = [&] {
            if (++stage == kRing) stage = 0, phase ^= 1;
        };
        uint32_t sent = 0;
        // `count` windows, the n-th window(n)
        auto send = [&](int32_t count, bool ends, auto window) {
            if (lane != 0) return;
            for (int32_t n = 0; n < count; ++n) {
                const int32_t w = window(n);
                const char *from = tile0 + w * stride;
                if (!bar_wait(empty + 8 * stage, phase)) atomicOr(&g_bucket_error, 2u);
                uint32_t size = bytes;
                int said = kData;
                if (ends && n + 1 == count) said |= kEnd;
                if (++sent % kRun == 0) said |= kRunEnd;
                if constexpr (!kVec) {
                    // the 16-byte lines that hold the tile; at the tensor's ends they
                    // hold other bytes too, and the tile is read directly
                    const uintptr_t first = reinterpret_cast<uintptr_t>(from);
                    const char *lo = reinterpret_cast<const char *>(first & ~uintptr_t{15});
                    const char *hi = reinterpret_cast<const char *>((first + bytes + 15) & ~uintptr_t{15});
                    said |= static_cast<int>(first & 15) / kES;
                    size = static_cast<uint32_t>(hi - lo);
                    from = lo;
                    if (lo < a.grad || hi > end) {
                        sh.window[stage] = w;
                        size = 0;
                        said |= kDirect;
                    }
                }
                sh.said[stage] = said;
                const uint32_t bar = full + 8 * stage;
                if (size) {
                    bar_expect(bar, size);
                    bulk_copy(slots + stage * kStageBytes<E>, from, size, bar, policy);
                } else {
                    bar_arrive(bar);
                }
                advance();
            }
            if (count == 0 && ends) {  // a stage without a window
                if (!bar_wait(empty + 8 * stage, phase)) atomicOr(&g_bucket_error, 2u);
                sh.said[stage] = kEnd;
                bar_arrive(full + 8 * stage);
                advance();
            }
        };
        if (!a.win_type) {
            send(u.type == 0 ? w1 - w0 : 0, true, [&](int32_t n) { return w0 + n; });
            continue;
        }
        const bool one = w1 - w0 <= kListed;  // the list holds the slab's
        const bool kept = one && listed_type == u.type && listed_slab == u.slab;
        for (int32_t w = w0; w < w1; w += kListed) {
            if (!kept) {
                // the windows of this type among the next kListed, in order
                constexpr int kBatch = 32;
                const int32_t stop = min(w1, w + kListed);
                listed = 0;
                __syncwarp();  // the list has been read
                for (int32_t part = w; part < stop; part += 32 * kBatch) {
                    int32_t t[kBatch];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const int32_t at = part + 32 * k + lane;
                        t[k] = at < stop ? __ldg(a.win_type + at) : u.type - 1;
                        if (at < stop && (t[k] < 0 || t[k] >= a.n_types)) atomicOr(&g_bucket_error, 1u);
                    }
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const int32_t at = part + 32 * k + lane;
                        const bool hit = at < stop && t[k] == u.type;
                        const unsigned hits = __ballot_sync(0xffffffffu, hit);
                        if (hit) sh.list[listed + __popc(hits & ((1u << lane) - 1u))] = at;
                        listed += __popc(hits);
                    }
                }
                __syncwarp();
                listed_type = u.type, listed_slab = u.slab;
            }
            send(listed, one, [&](int32_t n) { return sh.list[n]; });
        }
        if (!one || w0 == w1) send(0, true, [](int32_t) { return 0; });
    }
}

// The adding warps: a unit's windows pair by pair into FP32 registers, the
// sums into shared memory (where those of several runs of windows meet).
template <typename E, bool kVec>
__device__ void add_units(const GradArgs &a, GradShared<E> &sh, Unit u, int32_t units) {
    constexpr bool k32 = std::is_same<E, F32>::value;
    constexpr int kN = kVec ? (k32 ? 4 : 8) : 1;       // neighbouring pairs of a thread
    constexpr int kOwn = kPlanTile / (kAdders * kN);   // runs of them
    const int tid = threadIdx.x;
    const uint32_t full = shared_address(sh.full), empty = shared_address(sh.empty);
    RingPlace<kGradStages<E>> ring;
    RingPlace<2> out;
    for (; units > 0; --units, u.next(a)) {
        float acc[kOwn * kN];
        const int64_t p0 = static_cast<int64_t>(u.tile) * kPlanTile;
        const int32_t len = static_cast<int32_t>(min(a.n_pairs - p0, static_cast<int64_t>(kPlanTile)));
        int said;
        bool later = false;  // the sums hold a run
    next_run:
#pragma unroll
        for (int k = 0; k < kOwn * kN; ++k) acc[k] = 0.f;
        do {
            if (!bar_wait(full + 8 * ring.stage, ring.phase)) atomicOr(&g_bucket_error, 2u);
            said = sh.said[ring.stage];
            const char *at = sh.stage[ring.stage];
            if (!kVec && (said & kDirect)) {
                const int64_t first = (static_cast<int64_t>(sh.window[ring.stage]) * a.heads + u.head) * a.n_pairs + p0;
#pragma unroll
                for (int k = 0; k < kOwn; ++k)
#pragma unroll
                    for (int j = 0; j < kN; ++j) {
                        const int e = (tid + k * kAdders) * kN + j;
                        if (e < len) acc[k * kN + j] += load1<E>(a.grad, first + e);
                    }
            } else if (said & kData) {
                // (a short tile's last runs may add what an earlier one left: no slot names it)
                if constexpr (kVec) {
#pragma unroll
                    for (int k = 0; k < kOwn; ++k) {
                        const uint4 v = reinterpret_cast<const uint4 *>(at)[tid + k * kAdders];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (k32) {
                                acc[k * 4 + j] += __uint_as_float(word(v, j));
                            } else {
                                float *s = acc + k * 8 + 2 * j;
                                const float2 r = E::widen_add2(word(v, j), make_float2(s[0], s[1]));
                                s[0] = r.x, s[1] = r.y;
                            }
                        }
                    }
                } else {
                    using Raw = std::conditional_t<k32, float, uint16_t>;
                    const Raw *q = reinterpret_cast<const Raw *>(at) + (said & 7) + tid;
                    Raw v[kOwn];  // all under way before the first is added
#pragma unroll
                    for (int k = 0; k < kOwn; ++k) v[k] = q[k * kAdders];
#pragma unroll
                    for (int k = 0; k < kOwn; ++k) acc[k] += load1<E>(&v[k], 0);
                }
            }
            __syncwarp();
            if ((tid & 31) == 0) bar_arrive(empty + 8 * ring.stage);
            ring.next();
        } while (!(said & (kEnd | kRunEnd)));
        float *sums = sh.sums[out.stage];
        if (__builtin_expect(later, 0)) {
            const float *runs = sums;
            asm("" : "+l"(runs));  // addresses of its own, which the store below does not keep
#pragma unroll
            for (int k = 0; k < kOwn; ++k)
#pragma unroll
                for (int j = 0; j < kN; ++j) acc[k * kN + j] += runs[plan_place((tid + k * kAdders) * kN + j)];
        } else if (out.wrapped) {
            must_wait(&sh.read[out.stage], out.phase ^ 1);
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
#pragma unroll
            for (int j = 0; j < kN; ++j) sums[plan_place((tid + k * kAdders) * kN + j)] = acc[k * kN + j];
        if (__builtin_expect(!(said & kEnd), 0)) {
            later = true;
            goto next_run;
        }
        __syncwarp();
        if ((tid & 31) == 0) bar_arrive(shared_address(&sh.summed[out.stage]));
        out.next();
    }
}

// Where bit e of `ends` says that a slot ends: its sum to *to, and on to the next.
template <int e>
__device__ __forceinline__ void end_slot(uint32_t ends, float *&to, float &sum) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 t;\n\tand.b32 t, %2, %3;\n\tsetp.ne.u32 p, t, 0;\n\t"
                 "@p st.global.f32 [%0], %1;\n\t@p add.s64 %0, %0, 4;\n\t@p mov.f32 %1, 0f00000000;\n\t}"
                 : "+l"(to), "+f"(sum) : "r"(ends), "n"(1u << e) : "memory");
}
template <int e>
__device__ __forceinline__ void add_entries(const float (&v)[32], uint32_t ends, float *&to, float &sum) {
    if constexpr (e < 32) {
        sum += v[e];
        end_slot<e>(ends, to, sum);
        add_entries<e + 1>(v, ends, to, sum);
    }
}

// The slot warps: a unit's sums slot by slot, while the next unit's windows are
// added up.  A thread is a lane of the plan: 32 entries of the tile's order,
// whose sums it adds from slot end to slot end.  (A thread a slot took
// several times as long: slots are short and long, and named by loads.)
template <typename E>
__device__ void slot_units(const GradArgs &a, GradShared<E> &sh, Unit u, int32_t units, int tid) {
    RingPlace<2> in;
    int32_t tile = -1;
    uint32_t at[32];  // the entries' bytes among the sums
    int2 lane;
    const bool ok = plan_matches(a);  // else nothing of it is followed
    if (!ok && tid == 0) atomicOr(&g_bucket_error, 1u);
    for (; units > 0; --units, u.next(a)) {
        if (u.tile != tile && ok) {
            tile = u.tile;
            const uint4 *oq = reinterpret_cast<const uint4 *>(a.plan + a.at.order) + tile * (kPlanTile / 8);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 o = __ldg(oq + k * kPlanLanes + tid);
#pragma unroll
                for (int j = 0; j < 8; ++j) at[8 * k + j] = (word(o, j / 2) >> (j & 1 ? 16 : 0) & (kPlanTile - 1)) * 4;
            }
            lane = __ldg(reinterpret_cast<const int2 *>(a.plan + a.at.lane) + tile * kPlanLanes + tid);
            // no slot but the map's
            if (lane.y < 0 || lane.y > a.n_slots - __popc(lane.x)) lane.x = lane.y = 0;
        }
        float *to = a.partial + ((static_cast<int64_t>(u.slab) * a.n_types + u.type) * a.heads + u.head) * a.n_slots;
        must_wait(&sh.summed[in.stage], in.phase);
        const char *sums = reinterpret_cast<const char *>(sh.sums[in.stage]);
        if (ok) {
            float v[32];  // all under way before the first is added
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = *reinterpret_cast<const float *>(sums + at[e]);
            // without branches: lanes end their slots at different entries
            float sum = 0.f;
            to += lane.y;
            add_entries<0>(v, lane.x, to, sum);
        }
        __syncwarp();
        if ((tid & 31) == 0) bar_arrive(shared_address(&sh.read[in.stage]));
        in.next();
    }
}

// Pass 1.  Two resident blocks an SM share the units out; in each a warp copies
// the tiles of the units' windows in bulk (TMA) into a ring of stages, ahead
// across units, four warps add them up and four add the last unit's sums up by
// slot.  Every gradient is read once; what leaves is one value per slot.  The
// order of all additions is fixed by the sizes and the plan.
// 960 windows of 6 heads and 144 x 144 pairs in 64 types, fp16: 43 us of the call's
// 50 for 239 MB (5.6 TB/s, bound by DRAM).  Where a unit has one window the way
// of its sums through shared memory bounds it: 16 heads of 2047 x 2047 pairs, 134
// MB, 60 us (1.1 us a unit and block).
template <typename E, bool kVec>
__global__ void __launch_bounds__(kGradThreads, kGradCtas) bias_grad_tiles(GradArgs a) {
    extern __shared__ __align__(16) char smem[];
    GradShared<E> &sh = *reinterpret_cast<GradShared<E> *>(smem);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kGradStages<E>; ++i) {
            bar_init(shared_address(&sh.full[i]), 1);
            bar_init(shared_address(&sh.empty[i]), kAdders / 32);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(shared_address(&sh.summed[i]), kAdders / 32);
            bar_init(shared_address(&sh.read[i]), kSlotters / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_prologue();
    const int32_t u0 = share_start(a.units, gridDim.x, blockIdx.x);
    const int32_t units = share_start(a.units, gridDim.x, blockIdx.x + 1) - u0;
    const Unit u(a, u0);
    const int tid = threadIdx.x;
    int32_t listed = -1;
    if (a.win_type) {
        // the first unit's windows by eight warps at once: nothing is copied before
        const int32_t w0 = share_start(a.n_win, a.slabs, u.slab), w1 = share_start(a.n_win, a.slabs, u.slab + 1);
        if (w1 - w0 <= kListed) {
            constexpr int kEach = kListed / 8;
            const int warp = tid >> 5, lane = tid & 31;
            unsigned hits[kEach / 32];
            int32_t count = 0;
            if (warp < 8) {
                int32_t t[kEach / 32];
#pragma unroll
                for (int k = 0; k < kEach / 32; ++k) {
                    const int32_t at = w0 + warp * kEach + 32 * k + lane;
                    t[k] = at < w1 ? __ldg(a.win_type + at) : u.type - 1;
                    if (at < w1 && (t[k] < 0 || t[k] >= a.n_types)) atomicOr(&g_bucket_error, 1u);
                }
#pragma unroll
                for (int k = 0; k < kEach / 32; ++k) {
                    const int32_t at = w0 + warp * kEach + 32 * k + lane;
                    hits[k] = __ballot_sync(0xffffffffu, at < w1 && t[k] == u.type);
                    count += __popc(hits[k]);
                }
                if (lane == 0) sh.counts[warp] = count;
            }
            __syncthreads();
            listed = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (q == warp) count = listed;  // this warp's first place
                listed += sh.counts[q];
            }
            if (warp < 8)
#pragma unroll
                for (int k = 0; k < kEach / 32; ++k) {
                    if (hits[k] >> lane & 1)
                        sh.list[count + __popc(hits[k] & ((1u << lane) - 1u))] = w0 + warp * kEach + 32 * k + lane;
                    count += __popc(hits[k]);
                }
            __syncthreads();
        }
    }
    if (tid < kAdders)
        add_units<E, kVec>(a, sh, u, units);
    else if (tid < kAdders + kSlotters)
        slot_units<E>(a, sh, u, units, tid - kAdders);
    else
        copy_units<E, kVec>(a, sh, u, units, listed, tid - kAdders - kSlotters);
}

// Pass 1 of small maps, where a tile of one head is too little to copy: a block
// takes several heads of a slab's windows of one type, which lie side by side,
// window by window, groups of threads the windows in turn.  A thread keeps the
// sums of the same kOwn words (of kW pairs) of each of its windows; the groups'
// are added in order in shared memory, and from there by slot, as above.  4096
// windows, fp16, us of the call (by tiles): 1 pair of 32 heads 5 (134), 16 pairs of
// 32 heads 7 (83), 256 pairs of 16 heads, 34 MB, 14 (45).  Latency bounds it.
constexpr int kSmallThreads = 512, kSmallValues = 4096;

template <typename E, int kW, int kOwn>
__global__ void __launch_bounds__(kSmallThreads, 2) bias_grad_small(GradArgs a, int32_t head_step) {
    constexpr bool k32 = std::is_same<E, F32>::value;
    constexpr int kAhead = 8 / kOwn < 2 ? 2 : 8 / kOwn;  // windows in flight a thread
    __shared__ int32_t list[kListed];
    __shared__ int32_t counts[kSmallThreads / 32];
    // by group, or (one group) by place
    __shared__ float parts[kOwn == 1 ? kSmallThreads * kW : 1];
    __shared__ float sums[kSmallValues];
    pdl_prologue();
    const bool ok = plan_matches(a);
    if (!ok && threadIdx.x == 0) atomicOr(&g_bucket_error, 1u);
    const int tid = threadIdx.x;
    const int32_t chunks = (a.heads + head_step - 1) / head_step;
    int32_t u = blockIdx.x;
    const int32_t h0 = u % chunks * head_step, heads = min(head_step, a.heads - h0);
    u /= chunks;
    const int32_t slab = u % a.slabs, type = u / a.slabs;
    const int32_t w0 = share_start(a.n_win, a.slabs, slab), w1 = share_start(a.n_win, a.slabs, slab + 1);
    const int32_t pairs = static_cast<int32_t>(a.n_pairs), padded = (pairs + 31) / 32 * 32;
    const int32_t words = heads * pairs / kW;
    // groups of threads, of which each window has one: by the pairs, so that the order
    // of additions does not depend on the alignment
    const int32_t groups = kOwn == 1 ? max(kSmallThreads / (heads * pairs), 1) : 1;
    const int32_t group = kOwn == 1 ? tid / words : 0, j = kOwn == 1 ? tid - group * words : tid;
    const int64_t stride = static_cast<int64_t>(a.heads) * a.n_pairs;
    const char *base = a.grad + (static_cast<int64_t>(h0) * a.n_pairs + static_cast<int64_t>(j) * kW) * kBytes<E>;
    using Raw = std::conditional_t<k32 || kW == 2, uint32_t, uint16_t>;
    float acc[kOwn * kW], total[kOwn * kW];  // a run of windows, the runs
#pragma unroll
    for (int k = 0; k < kOwn * kW; ++k) acc[k] = total[k] = 0.f;
    auto end_run = [&] {
#pragma unroll
        for (int k = 0; k < kOwn * kW; ++k) total[k] += acc[k], acc[k] = 0.f;
    };
    // `count` windows, the n-th window(n); runs end with them
    auto add = [&](int32_t count, auto window) {
        if (group >= groups) return;
        static_assert(kRun % kAhead == 0, "a run ends where the loads in flight do");
        int32_t n = group;
        for (int32_t stop; n < count; end_run()) {
            stop = min(count, n + kRun * groups);
#pragma unroll 2  // (4096 windows of 256 pairs and 32 heads 19.5 us, without 21.6)
            for (; n < stop; n += kAhead * groups) {
                Raw v[kAhead][kOwn];
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    const bool live = n + q * groups < count;
                    const char *from = base + (live ? window(n + q * groups) * stride : 0) * kBytes<E>;
#pragma unroll
                    for (int k = 0; k < kOwn; ++k)
                        v[q][k] = live && j + k * kSmallThreads < words
                            ? __ldcs(reinterpret_cast<const Raw *>(from + k * (kSmallThreads * kW * kBytes<E>))) : Raw(0);
                }
#pragma unroll
                for (int q = 0; q < kAhead; ++q)
#pragma unroll
                    for (int k = 0; k < kOwn; ++k) {
                        if constexpr (k32) {
                            acc[k] += __uint_as_float(v[q][k]);
                        } else {
                            const float2 f = E::to_f2(v[q][k]);
                            acc[k * kW] += f.x;
                            if constexpr (kW == 2) acc[k * kW + 1] += f.y;
                        }
                    }
            }
        }
    };
    if (!a.win_type) {
        add(type == 0 ? w1 - w0 : 0, [&](int32_t n) { return w0 + n; });
    } else {
        constexpr int kWarps = kSmallThreads / 32, kEach = kListed / kSmallThreads;
        const int warp = tid >> 5, lane = tid & 31;
        for (int32_t w = w0; w < w1; w += kListed) {
            // the windows of this type among the next kListed, in order
            unsigned hits[kEach];
            int32_t count = 0;
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int32_t at = w + (warp * kEach + k) * 32 + lane;
                const int32_t t = at < w1 ? __ldg(a.win_type + at) : type - 1;
                if (at < w1 && (t < 0 || t >= a.n_types)) atomicOr(&g_bucket_error, 1u);
                hits[k] = __ballot_sync(0xffffffffu, at < w1 && t == type);
                count += __popc(hits[k]);
            }
            if (lane == 0) counts[warp] = count;
            __syncthreads();  // (the last list has been read, too)
            int32_t before = 0, listed = 0;
            for (int q = 0; q < kWarps; ++q) {
                if (q == warp) before = listed;
                listed += counts[q];
            }
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                if (hits[k] >> lane & 1)
                    list[before + __popc(hits[k] & ((1u << lane) - 1u))] = w + (warp * kEach + k) * 32 + lane;
                before += __popc(hits[k]);
            }
            __syncthreads();
            add(listed, [&](int32_t n) { return list[n]; });
        }
    }
    // pair i of head h at h * padded + plan_place(i)
    auto place = [&](int32_t e) {
        const int32_t h = e / pairs;
        return h * padded + plan_place(e - h * pairs);
    };
    if constexpr (kOwn == 1) {
        if (group < groups)
#pragma unroll
            for (int q = 0; q < kW; ++q) parts[(group * words + j) * kW + q] = total[q];
        __syncthreads();
        for (int32_t e = tid; e < words * kW; e += kSmallThreads) {
            float t = parts[e];
            for (int32_t g = 1; g < groups; ++g) t += parts[g * words * kW + e];
            sums[place(e)] = t;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (j + k * kSmallThreads < words)
#pragma unroll
                for (int q = 0; q < kW; ++q) sums[place((j + k * kSmallThreads) * kW + q)] = total[k * kW + q];
    }
    __syncthreads();
    if (!ok) return;
    const int32_t lanes = padded / 32;  // of the plan that can have entries
    for (int32_t i = tid; i < heads * lanes; i += kSmallThreads) {
        const int32_t h = i / lanes, l = i - h * lanes;
        int2 lane = __ldg(reinterpret_cast<const int2 *>(a.plan + a.at.lane) + l);
        if (lane.y < 0 || lane.y > a.n_slots - __popc(lane.x)) lane.x = lane.y = 0;
        float *to = a.partial + ((static_cast<int64_t>(slab) * a.n_types + type) * a.heads + h0 + h) * a.n_slots + lane.y;
        const uint4 *oq = reinterpret_cast<const uint4 *>(a.plan + a.at.order) + l;
        float v[32], sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 o = __ldg(oq + k * kPlanLanes);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[8 * k + q] = sums[h * padded + min(static_cast<int32_t>(word(o, q / 2) >> (q & 1 ? 16 : 0) & 0xffff), padded - 1)];
        }
        add_entries<0>(v, lane.x, to, sum);
    }
}

// Pass 2 after pass 1: all that came before on the stream is done when it starts
// (pass 1 has waited for it), so the plan may be read at once; the sums are there
// after wait_for_slots.  What is read before that comes from L2, as everywhere in
// the library: L1 may hold an older line.  A large grid waits first, see
// kEarlyBlocks.  (1 to 2 us of a call: 1024 x 1024 pairs of 8 heads, 2 windows 17.2 us
// on the device, 18.1 waiting first.)
__device__ __forceinline__ void start_table(const GradArgs &a) {
#if WGS_PDL
    if (!a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#endif
}
__device__ __forceinline__ void wait_for_slots(const GradArgs &a) {
#if WGS_PDL
    if (a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
#endif
}

// A word of the plan, from L2 or through L1.
__device__ __forceinline__ int32_t plan_word(const GradArgs &a, int64_t i, bool l2) {
    return l2 ? __ldcg(a.plan + i) : __ldg(a.plan + i);
}

// The places of bucket b in the buckets' lists of slots, [x, y).
__device__ __forceinline__ int2 places_of(const GradArgs &a, int32_t b) {
    return make_int2(max(plan_word(a, a.at.bucket_first + b, a.early), 0),
                     min(plan_word(a, a.at.bucket_first + b + 1, a.early), a.n_slots));
}

// The d-th slot of the buckets' lists.
template <bool kL2>
__device__ __forceinline__ int32_t slot_of(const GradArgs &a, int32_t d) {
    return min(max(plan_word(a, a.at.bucket_slot + d, kL2), 0), a.n_slots - 1);
}

// The sum of a bucket's values of one (type, head), n slots from d0 on in every
// slab: those of lane `lane` of `lanes`, of the slabs one after another.
__device__ __forceinline__ float add_bucket(const GradArgs &a, int32_t type, int32_t b, int32_t head, int32_t lane,
                                            int32_t lanes) {
    const int2 places = places_of(a, b);
    const int32_t d0 = places.x, n = places.y - d0;
    if (n <= 0) {
        wait_for_slots(a);
        return 0.f;
    }
    const int64_t step = static_cast<int64_t>(a.n_types) * a.heads * a.n_slots;
    const float *p = a.partial + (static_cast<int64_t>(type) * a.heads + head) * a.n_slots;
    const int32_t by_slabs = lanes / n, by_slots = lanes - by_slabs * n;
    int32_t s = lane / n, d = lane - s * n;
    float sum = 0.f;
    constexpr int kAhead = 8;  // loads in flight
    auto batch = [&](auto early) {
        const float *q[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            q[k] = s < a.slabs ? p + s * step + slot_of<decltype(early)::value>(a, d0 + d) : nullptr;
            s += by_slabs, d += by_slots;
            if (d >= n) d -= n, ++s;
        }
        if (decltype(early)::value) wait_for_slots(a);
        float v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v[k] = q[k] ? __ldcg(q[k]) : 0.f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) sum += v[k];
    };
    if (a.early) batch(std::true_type{});
    while (s < a.slabs) batch(std::false_type{});
    return sum;
}

// Pass 2: LANES lanes a (type, bucket, head) add the bucket's slots over the
// slabs and round once to the table's format.  Heads are neighbours, as in the
// table.
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads) bias_grad_table(GradArgs a, int32_t blocks) {
    start_table(a);
    const bool ok = plan_matches(a, a.early);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_bucket_error, 1u);
    const int32_t type = blockIdx.x / blocks;
    const int32_t i = ((blockIdx.x - type * blocks) * kThreads + static_cast<int32_t>(threadIdx.x)) / LANES;
    const int32_t lane = threadIdx.x % LANES;
    const int32_t b = i / a.heads, head = i - b * a.heads;
    float v = 0.f;
    if (ok && b < a.n_buckets)
        v = add_bucket(a, type, b, head, lane, LANES);
    else
        wait_for_slots(a);
    v = group_sum<LANES>(v);
    if (b < a.n_buckets && lane == 0)
        store1<T>(a.table, (static_cast<int64_t>(type) * a.n_buckets + b) * a.heads + head, v);
}

// Pass 2 where buckets have many slots: a block a (type, bucket, head).  The
// largest bucket bounds it, two rounds to L2 for 16 values a thread: 512 outputs
// of 158,323 slots 17 us.  (A cluster of blocks an output: 175.)
constexpr int kBlockThreads = 1024;

template <typename T>
__global__ void __launch_bounds__(kBlockThreads) bias_grad_block(GradArgs a) {
    __shared__ float part[kBlockThreads / 32];
    __shared__ int32_t known[3];  // the bucket's places and whether the plan is the call's
    start_table(a);
    const int32_t head = blockIdx.x % a.heads, tb = blockIdx.x / a.heads;
    const int32_t type = tb / a.n_buckets, b = tb - type * a.n_buckets;
    bool ok;
    int2 places;
    auto look = [&] {
        ok = plan_matches(a, a.early);
        places = ok ? places_of(a, b) : make_int2(0, 0);
    };
    if (a.early) {  // by one thread: L2 would take these words thousands of times
        if (threadIdx.x == 0) {
            look();
            known[0] = places.x, known[1] = places.y, known[2] = ok;
        }
        __syncthreads();
        places = make_int2(known[0], known[1]), ok = known[2];
    } else {
        look();
    }
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_bucket_error, 1u);
    float v = 0.f;
    const int32_t first = places.x + static_cast<int32_t>(threadIdx.x), d1 = places.y;  // (none without a plan)
    const int64_t step = static_cast<int64_t>(a.n_types) * a.heads * a.n_slots;
    const float *p = a.partial + (static_cast<int64_t>(type) * a.heads + head) * a.n_slots;
    constexpr int kAhead = 16, kStep = kAhead * kBlockThreads;  // loads in flight
    auto batch = [&](int32_t d, auto early) {
        int32_t slot[kAhead];
        float q[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            slot[k] = d1 - d > k * kBlockThreads ? slot_of<decltype(early)::value>(a, d + k * kBlockThreads) : -1;
        if (decltype(early)::value) wait_for_slots(a);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) q[k] = slot[k] >= 0 ? __ldcg(p + slot[k]) : 0.f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v += q[k];
    };
    auto next = [&](int32_t d) { return d1 - d > kStep ? d + kStep : d1; };  // (no step past 2^31 - 1)
    int32_t d = first;
    if (a.early) batch(d, std::true_type{}), d = next(d);
    for (int32_t s = 0; s < a.slabs; ++s, p += step, d = first)
        for (; d < d1; d = next(d)) batch(d, std::false_type{});
    v = group_sum<32>(v);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = group_sum<32>(part[threadIdx.x]);
        if (threadIdx.x == 0) store1<T>(a.table, blockIdx.x, v);
    }
}

// Pass 2 where a bucket has few values: a thread a (type, bucket) for all
// heads, whose slots it looks up once; the threads' slots are neighbours.
template <typename T>
__global__ void __launch_bounds__(kThreads) bias_grad_rows(GradArgs a, int32_t blocks) {
    start_table(a);
    const bool ok = plan_matches(a, a.early);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_bucket_error, 1u);
    const int32_t type = blockIdx.x / blocks;
    const int32_t b = (blockIdx.x - type * blocks) * kThreads + static_cast<int32_t>(threadIdx.x);
    const bool mine = ok && b < a.n_buckets;
    const int2 places = mine ? places_of(a, b) : make_int2(0, 0);
    const int32_t d0 = places.x, d1 = places.y;
    const int32_t slot0 = d0 < d1 ? (a.early ? slot_of<true>(a, d0) : slot_of<false>(a, d0)) : 0;
    wait_for_slots(a);
    if (b >= a.n_buckets) return;
    const int64_t step = static_cast<int64_t>(a.n_types) * a.heads * a.n_slots;
    const float *p = a.partial + static_cast<int64_t>(type) * a.heads * a.n_slots;
    const int64_t out = (static_cast<int64_t>(type) * a.n_buckets + b) * a.heads;
    constexpr int kHeads = 8;  // at a time: loads in flight
    for (int32_t h0 = 0; h0 < a.heads; h0 += kHeads) {
        float v[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) v[k] = 0.f;
        for (int32_t d = d0; d < d1; ++d) {
            const float *q = p + static_cast<int64_t>(h0) * a.n_slots + (d == d0 ? slot0 : slot_of<false>(a, d));
            for (int32_t s = 0; s < a.slabs; ++s, q += step) {
                float t[kHeads];
#pragma unroll
                for (int k = 0; k < kHeads; ++k)
                    t[k] = h0 + k < a.heads ? __ldcg(q + static_cast<int64_t>(k) * a.n_slots) : 0.f;
#pragma unroll
                for (int k = 0; k < kHeads; ++k) v[k] += t[k];
            }
        }
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
            if (h0 + k < a.heads) store1<T>(a.table, out + h0 + k, v[k]);
    }
}

// Blocks of pass 1 at most: two on each of 152 SMs.
constexpr int64_t kGradBlocks = 152 * kGradCtas;
// Windows of a type in a slab at least, on average.
constexpr int64_t kSlabWindows = 4;

// Slabs of windows: the fewest with which the blocks' shares of the units, whole
// ones, leave at most a tenth of them out, where the units are as many as the
// blocks' shares could hold.  (A map's last tile counts as a full one, so with a
// short one blocks that hold more full tiles take longer.)  Depends on the sizes
// alone, so results do not depend on the device.
int64_t grad_slabs(int64_t n_win, int64_t heads, int64_t n_types, int64_t n_tiles) {
    const int64_t base = heads * n_types * (n_tiles > 0 ? n_tiles : 1);
    const int64_t most = n_win / (n_types * kSlabWindows);
    if (base >= 16 * kGradBlocks || most <= 1) return 1;
    int64_t best = 1;
    double best_use = 0;
    for (int64_t s = 1; s <= most && s * base <= 16 * kGradBlocks; ++s) {
        const int64_t units = s * base;
        const double use = static_cast<double>(units) / (ceil_div(units, kGradBlocks) * kGradBlocks);
        if (use > best_use) best_use = use, best = s;
        if (use >= 0.9) break;
    }
    return best;
}

// Maps that bias_grad_small takes, and how it is cut: maps of 1024 pairs still
// gain (900 pairs, 16 heads, 1024 windows of 4 types: 13 us, by tiles 30), tiles of
// one head are as good from there on.  At most one wave of blocks, and 16 rounds of
// windows each on average: with 4 rounds 15 and 22 us where these take 9 and 15
// (16 pairs of 32 heads, 256 pairs of 16 heads; 4096 windows).
constexpr int64_t kSmallPairs = 1024, kSmallRounds = 16;
bool small_map(int64_t n_pairs) { return n_pairs > 0 && n_pairs <= kSmallPairs; }
int64_t small_heads(int64_t heads, int64_t n_pairs) {
    const int64_t most = kSmallValues / ((n_pairs + 31) / 32 * 32);
    return heads < most ? heads : most;
}
int64_t small_slabs(int64_t n_win, int64_t heads, int64_t n_types, int64_t n_pairs) {
    const int64_t step = small_heads(heads, n_pairs), base = ceil_div(heads, step) * n_types;
    const int64_t groups = step * n_pairs < kSmallThreads ? kSmallThreads / (step * n_pairs) : 1;
    const int64_t room = kGradBlocks / base, most = n_win / (n_types * groups * kSmallRounds);
    const int64_t s = room < most ? room : most;
    return s > 1 ? s : 1;
}
// Slabs of a call.
int64_t slabs_of(int64_t n_win, int64_t heads, int64_t n_types, int64_t n_pairs) {
    return small_map(n_pairs) ? small_slabs(n_win, heads, n_types, n_pairs)
                              : grad_slabs(n_win, heads, n_types, ceil_tiles(n_pairs));
}

template <typename E>
wgs_status launch_small(const GradArgs &a, cudaStream_t stream) {
    const int32_t step = static_cast<int32_t>(small_heads(a.heads, a.n_pairs));
    const int64_t blocks = ceil_div(a.heads, step) * a.n_types * a.slabs;
    if (blocks > INT32_MAX) return WGS_ERR_SHAPE;
    constexpr bool k32 = std::is_same<E, F32>::value;
    const bool two = !k32 && a.heads * a.n_pairs % 2 == 0 && step * a.n_pairs % 2 == 0 && aligned4(a.grad);
    const bool one = step * a.n_pairs / (two ? 2 : 1) <= kSmallThreads;
    auto kernel = one ? bias_grad_small<E, 1, 1> : bias_grad_small<E, 1, 8>;
    if constexpr (!k32)
        if (two) kernel = one ? bias_grad_small<E, 2, 1> : bias_grad_small<E, 2, 4>;
    return launch(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kSmallThreads), 0, stream, a, step);
}

template <typename E, bool kVec>
wgs_status launch_tiles(const GradArgs &a, cudaStream_t stream) {
    auto kernel = bias_grad_tiles<E, kVec>;
    // More than 48 KB needs the runtime's leave, which belongs to the context;
    // asking on every call needs no record of it.
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(GradShared<E>))) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    const unsigned grid = static_cast<unsigned>(a.units < kGradBlocks ? a.units : kGradBlocks);
    return launch(kernel, dim3(grid), dim3(kGradThreads), sizeof(GradShared<E>), stream, a);
}

template <typename E>
wgs_status launch_tiles_any(const GradArgs &a, cudaStream_t stream) {
    if (small_map(a.n_pairs)) return launch_small<E>(a, stream);
    constexpr int n = std::is_same<E, F32>::value ? 4 : 8;
    return a.n_pairs % n == 0 && aligned16(a.grad) ? launch_tiles<E, true>(a, stream)
                                                    : launch_tiles<E, false>(a, stream);
}

// Blocks of pass 2 with which it starts early, of kThreads and of kBlockThreads.
// Later ones have nothing to hide, and miss what L1 holds: 16 types of 32 buckets and
// 32 heads, 16,384 blocks, 159 us, starting early 238; 512 blocks 69.7, waiting 71.3.
constexpr int64_t kEarlyBlocks = 8 * 152, kEarlyLarge = 4 * 152;

template <typename T>
wgs_status launch_table(GradArgs a, cudaStream_t stream) {
    const int64_t outputs = static_cast<int64_t>(a.n_types) * a.n_buckets * a.heads;
    const int64_t mean = static_cast<int64_t>(a.n_slots) * a.slabs / a.n_buckets;  // values of a bucket
    if (mean < 4 && outputs >= int64_t{32} * kThreads * a.heads) {
        const int64_t blocks = ceil_div(a.n_buckets, kThreads);
        if (blocks * a.n_types > INT32_MAX) return WGS_ERR_SHAPE;
        a.early = a.early && blocks * a.n_types <= kEarlyBlocks;
        return launch(bias_grad_rows<T>, dim3(static_cast<unsigned>(blocks * a.n_types)), dim3(kThreads), 0,
                      stream, a, static_cast<int32_t>(blocks));
    }
    if (a.n_slots / a.n_buckets >= 64 && outputs <= INT32_MAX) {
        a.early = a.early && outputs <= kEarlyLarge;
        return launch(bias_grad_block<T>, dim3(static_cast<unsigned>(outputs)), dim3(kBlockThreads), 0, stream, a);
    }
    // more lanes where outputs are few: a bucket can hold many times the mean (32
    // buckets of 2047 pairs in 77 slots, 32 heads: 5 us, a lane each 30)
    const int lanes = mean >= 64 || outputs <= 8192 ? 32 : mean >= 8 || outputs <= 32768 ? 8 : 1;
    const int64_t blocks = ceil_div(static_cast<int64_t>(a.heads) * a.n_buckets * lanes, kThreads);
    if (blocks * a.n_types > INT32_MAX) return WGS_ERR_SHAPE;
    a.early = a.early && blocks * a.n_types <= kEarlyBlocks;
    auto kernel = lanes == 1 ? bias_grad_table<T, 1> : lanes == 8 ? bias_grad_table<T, 8> : bias_grad_table<T, 32>;
    return launch(kernel, dim3(static_cast<unsigned>(blocks * a.n_types)), dim3(kThreads), 0, stream, a,
                  static_cast<int32_t>(blocks));
}

// a * b for non-negative a and b, or false past 2^62.
bool times(int64_t a, int64_t b, int64_t *out) {
    if (b > 0 && a > (int64_t{1} << 62) / b) return false;
    *out = a * b;
    return true;
}

// Slabs, units and bytes of workspace of a gradient call, sizes not negative;
// false where they pass what its kernels can count.
bool grad_sizes(int64_t n_win, int64_t heads, int64_t n_types, int64_t n_pairs, int64_t n_slots, int64_t *slabs,
                int64_t *units, int64_t *part_bytes) {
    // (the kernels step past the last window by at most 65536)
    if (n_pairs > INT32_MAX - kPlanTile || n_slots > n_pairs || n_win > INT32_MAX - 65536) return false;
    const int64_t n_tiles = ceil_tiles(n_pairs);
    int64_t th;
    if (!times(n_types, heads, &th) || !times(th, n_tiles, units) || *units > INT32_MAX) return false;
    *slabs = slabs_of(n_win, heads, n_types, n_pairs);
    *units *= *slabs;
    return *units <= INT32_MAX && times(th, *slabs, &th) && times(th, n_slots * 4, part_bytes);
}

bool dtype_ok(wgs_dtype d) { return d == WGS_F32 || d == WGS_F16 || d == WGS_BF16; }
int64_t bytes_of(wgs_dtype d) { return d == WGS_F32 ? 4 : 2; }
bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

}  // namespace wgs

using namespace wgs;

extern "C" wgs_status position_bias(const void *table, const int32_t *bucket, void *bias,
                                    int32_t n_types, int32_t heads, int64_t n_pairs,
                                    int32_t n_buckets, wgs_dtype table_dtype, wgs_dtype dtype,
                                    cudaStream_t stream) {
    if (!dtype_ok(dtype) || !dtype_ok(table_dtype)) return WGS_ERR_DTYPE;
    if (table_dtype != WGS_F32 && table_dtype != dtype) return WGS_ERR_DTYPE;
    if (n_types < 0 || heads < 0 || n_pairs < 0 || n_buckets < 0) return WGS_ERR_SHAPE;
    if (n_types == 0 || heads == 0 || n_pairs == 0) return WGS_OK;
    if (n_buckets < 1 || n_pairs > INT32_MAX - kPlanTile) return WGS_ERR_SHAPE;
    int64_t slabs, out_n, table_n;
    if (!times(n_types, heads, &slabs) || !times(slabs, n_pairs * bytes_of(dtype), &out_n) ||
        !times(slabs, n_buckets * bytes_of(table_dtype), &table_n) ||
        static_cast<int64_t>(heads) * n_buckets > INT32_MAX / 32)
        return WGS_ERR_SHAPE;
    if (!table || !bucket || !bias) return WGS_ERR_NULL;
    if (!aligned_to(table, bytes_of(table_dtype)) || !aligned4(bucket) ||
        !aligned_to(bias, bytes_of(dtype)))
        return WGS_ERR_ALIGN;
    if (overlap(bias, out_n, table, table_n) || overlap(bias, out_n, bucket, n_pairs * 4))
        return WGS_ERR_ALIAS;
    DeviceInfo dev;
    const wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    const ExpandArgs a = {table, bucket, bias, n_pairs, n_buckets, heads, 0, 0, 0};
    if (dtype == WGS_F32) return launch_expand<F32, F32>(a, n_types, stream);
    if (dtype == WGS_F16)
        return table_dtype == WGS_F32 ? launch_expand<Fp16, F32>(a, n_types, stream)
                                      : launch_expand<Fp16, Fp16>(a, n_types, stream);
    return table_dtype == WGS_F32 ? launch_expand<Bf16, F32>(a, n_types, stream)
                                  : launch_expand<Bf16, Bf16>(a, n_types, stream);
}

extern "C" size_t wgs_position_bias_bwd_workspace_bytes(int64_t n_win, int32_t heads,
                                                        int32_t n_types, int64_t n_pairs,
                                                        int64_t n_slots) {
    int64_t slabs, units, part_bytes;
    if (n_win < 0 || heads < 1 || n_types < 1 || n_pairs < 0 || n_slots < 0 ||
        !grad_sizes(n_win, heads, n_types, n_pairs, n_slots, &slabs, &units, &part_bytes))
        return 0;
    return static_cast<size_t>(part_bytes);
}

extern "C" wgs_status position_bias_bwd(const void *grad, const int32_t *plan,
                                        const int32_t *win_type, void *grad_table, void *workspace,
                                        size_t workspace_bytes, int64_t n_win, int32_t heads,
                                        int64_t n_pairs, int32_t n_buckets, int64_t n_slots,
                                        int32_t n_types, wgs_dtype dtype, wgs_dtype table_dtype,
                                        cudaStream_t stream) {
    if (!dtype_ok(dtype) || !dtype_ok(table_dtype)) return WGS_ERR_DTYPE;
    if (table_dtype != WGS_F32 && table_dtype != dtype) return WGS_ERR_DTYPE;
    if (n_win < 0 || heads < 0 || n_pairs < 0 || n_buckets < 0 || n_types < 0 || n_slots < 0)
        return WGS_ERR_SHAPE;
    if (n_types == 0 || heads == 0 || n_buckets == 0) return WGS_OK;
    const int64_t n_tiles = ceil_tiles(n_pairs);
    int64_t slabs, units, grad_bytes, table_bytes, part_bytes;
    if (static_cast<int64_t>(heads) * n_buckets > INT32_MAX / 32 ||
        !grad_sizes(n_win, heads, n_types, n_pairs, n_slots, &slabs, &units, &part_bytes) ||
        !times(n_win * heads, n_pairs * bytes_of(dtype), &grad_bytes) ||
        !times(static_cast<int64_t>(n_types) * heads, n_buckets * bytes_of(table_dtype), &table_bytes))
        return WGS_ERR_SHAPE;
    if (!plan || !grad_table || (grad_bytes > 0 && !grad) || (part_bytes > 0 && !workspace))
        return WGS_ERR_NULL;
    if (workspace_bytes < static_cast<size_t>(part_bytes)) return WGS_ERR_SHAPE;
    if (!aligned16(plan) || !aligned16(workspace) || !aligned4(win_type) ||
        !aligned_to(grad, bytes_of(dtype)) || !aligned_to(grad_table, bytes_of(table_dtype)))
        return WGS_ERR_ALIGN;
    const PlanLayout at = plan_layout(n_pairs, n_buckets, n_slots);
    const void *out[2] = {grad_table, workspace};
    const int64_t out_bytes[2] = {table_bytes, part_bytes};
    for (int k = 0; k < 2; ++k)
        if (overlap(out[k], out_bytes[k], grad, grad_bytes) ||
            overlap(out[k], out_bytes[k], plan, at.words * 4) ||
            (win_type && overlap(out[k], out_bytes[k], win_type, n_win * 4)))
            return WGS_ERR_ALIAS;
    if (overlap(grad_table, table_bytes, workspace, part_bytes)) return WGS_ERR_ALIAS;
    DeviceInfo dev;
    wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    GradArgs a = {static_cast<const char *>(grad), grad_bytes, plan, win_type,
                  static_cast<float *>(workspace), grad_table, at, n_pairs,
                  static_cast<int32_t>(n_win), heads, n_types, n_buckets,
                  static_cast<int32_t>(n_tiles), static_cast<int32_t>(n_slots),
                  static_cast<int32_t>(slabs), static_cast<int32_t>(units), units > 0};
    if (units > 0) {
        st = dtype == WGS_F32   ? launch_tiles_any<F32>(a, stream)
             : dtype == WGS_F16 ? launch_tiles_any<Fp16>(a, stream)
                                : launch_tiles_any<Bf16>(a, stream);
        if (st != WGS_OK) return st;
    }
    return table_dtype == WGS_F32   ? launch_table<F32>(a, stream)
           : table_dtype == WGS_F16 ? launch_table<Fp16>(a, stream)
                                    : launch_table<Bf16>(a, stream);
}
