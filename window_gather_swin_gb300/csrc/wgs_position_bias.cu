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
// it came with; read and cleared by wgs_check_error.
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

// HC neighbouring table values in one load.
template <typename T, int HC>
__device__ __forceinline__ void load_heads(const void *table, int64_t i, float (&v)[HC]) {
    if constexpr (HC == 1) {
        v[0] = load1<T>(table, i);
    } else if constexpr (std::is_same<T, F32>::value) {
        const float *p = static_cast<const float *>(table) + i;
        if constexpr (HC == 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
            const float2 q = *reinterpret_cast<const float2 *>(p);
            v[0] = q.x, v[1] = q.y;
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(table) + i;
        if constexpr (HC == 4) {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            const float2 a = T::to_f2(q.x), b = T::to_f2(q.y);
            v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
        } else {
            const float2 a = T::to_f2(*reinterpret_cast<const uint32_t *>(p));
            v[0] = a.x, v[1] = a.y;
        }
    }
}

// Eight consecutive outputs at a 16-byte aligned address, each rounded once
// (to nearest even) to the output's format.
template <typename O>
__device__ __forceinline__ void store8(void *p, const float (&v)[8]) {
    uint4 *q = static_cast<uint4 *>(p);
    if constexpr (std::is_same<O, F32>::value) {
        st_stream(q, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                __float_as_uint(v[2]), __float_as_uint(v[3])));
        st_stream(q + 1, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]),
                                    __float_as_uint(v[6]), __float_as_uint(v[7])));
    } else {
        st_stream(q, make_uint4(O::from_f2(v[0], v[1]), O::from_f2(v[2], v[3]),
                                O::from_f2(v[4], v[5]), O::from_f2(v[6], v[7])));
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
// so the gather stays in L1; the stores, whole lines a warp, are the cost.
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
    const int32_t h1 = min(a.heads, static_cast<int32_t>((hb + 1) * a.head_step));
    for (int32_t h = hb * a.head_step; h < h1; h += HC) {
        float v[8][HC];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int k = 0; k < HC; ++k) v[e][k] = 0.f;
            if (row[e] >= 0)
                load_heads<T, HC>(a.table, (type * a.n_buckets + row[e]) * a.heads + h, v[e]);
        }
#pragma unroll
        for (int k = 0; k < HC; ++k) {
            const float o[8] = {v[0][k], v[1][k], v[2][k], v[3][k], v[4][k], v[5][k], v[6][k], v[7][k]};
            store8<O>(static_cast<char *>(a.bias) +
                          ((type * a.heads + h + k) * a.n_pairs + p) * kBytes<O>, o);
        }
    }
}

// Any pair count or alignment.  The outputs of a (type, head) slab are cut
// where the address is a multiple of eight elements, so all but the slab's
// two ends are stored 16 bytes at a time wherever the slab starts; the
// block's buckets wait in shared memory (nine words for eight pairs, which
// keeps the lanes' stride of eight off the same bank) because the cut moves
// from head to head.
template <typename O, typename T>
__global__ void __launch_bounds__(kThreads) bias_expand_any(ExpandArgs a) {
    constexpr int kSpan = kThreads * 8;
    __shared__ int32_t rows[(kSpan + 8) / 8 * 9];
    pdl_prologue();
    uint32_t blk = blockIdx.x;
    const uint32_t pb = blk % a.pair_blocks;
    blk /= a.pair_blocks;
    const uint32_t hb = blk % a.head_blocks;
    const int64_t type = blk / a.head_blocks;
    const int64_t first = static_cast<int64_t>(pb) * kSpan - 8;
    bool bad = false;
    for (int i = threadIdx.x; i < kSpan + 8; i += kThreads) {
        const int64_t p = first + i;
        int32_t r = p >= 0 && p < a.n_pairs ? __ldg(a.bucket + p) : -1;
        bad |= r < -1 || r >= a.n_buckets;
        if (r >= a.n_buckets) r = -1;
        rows[i + i / 8] = r;
    }
    if (bad) atomicOr(&g_bucket_error, 1u);
    __syncthreads();
    const uint64_t base = reinterpret_cast<uint64_t>(a.bias) / kBytes<O>;
    const int32_t h1 = min(a.heads, static_cast<int32_t>((hb + 1) * a.head_step));
    for (int32_t h = hb * a.head_step; h < h1; ++h) {
        const int64_t slab = (type * a.heads + h) * a.n_pairs;
        const int shift = static_cast<int>((base + static_cast<uint64_t>(slab)) & 7);
        const int i0 = static_cast<int>(threadIdx.x) * 8 + 8 - shift;
        const int64_t p = first + i0;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int32_t r = rows[i0 + e + (i0 + e) / 8];
            v[e] = r >= 0 ? load1<T>(a.table, (type * a.n_buckets + r) * a.heads + h) : 0.f;
        }
        if (p >= 0 && p + 8 <= a.n_pairs) {
            store8<O>(static_cast<char *>(a.bias) + (slab + p) * kBytes<O>, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (p + e >= 0 && p + e < a.n_pairs) store1<O>(a.bias, slab + p + e, v[e]);
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
    if (eights)
        for (int c = 4; c > 1; c /= 2)
            if (a.heads % c == 0 && reinterpret_cast<uintptr_t>(a.table) % (c * kBytes<T>) == 0) {
                hc = c;
                break;
            }
    // the slab's cut moves the pairs of a block by up to seven
    const int64_t pair_blocks = ceil_div(a.n_pairs + (eights ? 0 : 7), kThreads * 8);
    // all heads in one block (the map is read once), unless that leaves the GPU idle
    const int64_t want = ceil_div(kExpandBlocks, pair_blocks * n_types);
    const int64_t steps = ceil_div(a.heads, hc);
    a.head_step = static_cast<int32_t>(ceil_div(steps, want < steps ? want : steps)) * hc;
    a.head_blocks = static_cast<int32_t>(ceil_div(a.heads, a.head_step));
    a.pair_blocks = static_cast<int32_t>(pair_blocks);
    const int64_t grid = pair_blocks * a.head_blocks * n_types;
    if (grid > INT32_MAX) return WGS_ERR_SHAPE;
    auto kernel = !eights   ? bias_expand_any<O, T>
                  : hc == 4 ? bias_expand_eights<O, T, 4>
                  : hc == 2 ? bias_expand_eights<O, T, 2>
                            : bias_expand_eights<O, T, 1>;
    return launch(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a);
}

// --------------------------------------------------------------- backward --

struct GradArgs {
    const void *grad;         // [n_win, heads, n_pairs]
    const int32_t *plan;      // wgs_bucket_plan.h
    const int32_t *win_type;  // [n_win] or NULL
    float *partial;           // [slabs, n_types, heads, n_slots]
    void *table;              // grad_table [n_types, n_buckets, heads]
    PlanLayout at;
    int64_t n_win, n_pairs;
    int32_t heads, n_types, n_buckets, n_tiles, n_slots, slabs;
};

// The plan's header against the sizes of the call (a plan of another map
// would name other places).
__device__ __forceinline__ bool plan_matches(const GradArgs &a) {
    return a.plan[0] == kPlanMagic && a.plan[1] == a.n_pairs && a.plan[2] == a.n_buckets &&
           a.plan[3] == a.n_tiles && a.plan[4] == a.n_slots;
}

constexpr int kListed = 1024;  // windows looked over at a time

// Pass 1: a block takes one tile of pairs of one (slab of windows, type,
// head).  It adds the windows' gradients pair by pair in FP32 registers,
// puts the sums into shared memory and adds them there by slot, LANES
// neighbouring lanes a slot.  Every gradient is read once, 16 bytes a load;
// what leaves is one value per slot.  The order of all additions is fixed by
// the sizes and the plan.
template <typename E, bool kVec, int LANES>
__global__ void __launch_bounds__(kThreads, 4) bias_grad_tiles(GradArgs a) {
    constexpr bool k32 = std::is_same<E, F32>::value;
    constexpr int kN = kVec ? (k32 ? 4 : 8) : 1;        // elements of a load
    constexpr int kOwn = kPlanTile / (kThreads * kN);   // loads a window
    constexpr int kAhead = kVec ? 8 / kOwn : 1;         // windows in flight
    __shared__ __align__(16) float sums[kPlanTile];
    __shared__ __align__(16) uint16_t order[kPlanTile];
    __shared__ int32_t list[kListed];
    __shared__ int32_t warp_count[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_prologue();
    uint32_t blk = blockIdx.x;
    const int32_t tile = static_cast<int32_t>(blk % a.n_tiles);
    blk /= a.n_tiles;
    const int32_t head = static_cast<int32_t>(blk % a.heads);
    blk /= a.heads;
    const int32_t type = static_cast<int32_t>(blk % a.n_types);
    const int32_t slab = static_cast<int32_t>(blk / a.n_types);
    if (!plan_matches(a)) {
        if (tid == 0) atomicOr(&g_bucket_error, 1u);
        return;
    }
    const int64_t p0 = static_cast<int64_t>(tile) * kPlanTile;
    const int32_t len = static_cast<int32_t>(min(a.n_pairs - p0, static_cast<int64_t>(kPlanTile)));
    float acc[kOwn * kN];
#pragma unroll
    for (int i = 0; i < kOwn * kN; ++i) acc[i] = 0.f;

    const int64_t stride = a.heads * a.n_pairs;  // elements from window to window
    const char *src = static_cast<const char *>(a.grad) + (head * a.n_pairs + p0) * kBytes<E>;
    // the gradients of windows win(0) ... win(count - 1)
    auto add = [&](int count, auto win) {
        int i = 0;
        if constexpr (kVec) {
            for (; i + kAhead <= count; i += kAhead) {
                uint4 v[kAhead][kOwn];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const uint4 *q = reinterpret_cast<const uint4 *>(src + win(i + u) * stride * kBytes<E>);
#pragma unroll
                    for (int k = 0; k < kOwn; ++k)
                        if ((tid + k * kThreads) * kN < len) v[u][k] = ld_stream(q + tid + k * kThreads);
                        else v[u][k] = make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
#pragma unroll
                    for (int k = 0; k < kOwn; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t w = word(v[u][k], j);
                            if constexpr (k32) {
                                acc[k * 4 + j] += __uint_as_float(w);
                            } else {
                                float *s = acc + k * 8 + 2 * j;
                                const float2 r = E::widen_add2(w, make_float2(s[0], s[1]));
                                s[0] = r.x, s[1] = r.y;
                            }
                        }
            }
        }
        for (; i < count; ++i) {
            const char *q = src + win(i) * stride * kBytes<E>;
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                const int e = (tid + k * kThreads) * kN;
                if (e < len)
#pragma unroll
                    for (int j = 0; j < kN; ++j) acc[k * kN + j] += load1<E>(q, e + j);
            }
        }
    };
    const int64_t w0 = a.n_win * slab / a.slabs, w1 = a.n_win * (slab + 1) / a.slabs;
    if (!a.win_type) {
        if (type == 0)
            for (int64_t w = w0; w < w1; w += kListed)
                add(static_cast<int>(min(w1 - w, static_cast<int64_t>(kListed))),
                    [&](int i) { return w + i; });
    } else {
        for (int64_t w = w0; w < w1; w += kListed) {
            // the windows of this type among the next kListed, in order
            int found = 0;
            for (int part = 0; part < kListed && w + part < w1; part += kThreads) {
                const int64_t mine = w + part + tid;
                const int32_t t = mine < w1 ? __ldg(a.win_type + mine) : type - 1;
                const bool hit = mine < w1 && t == type;
                if (mine < w1 && (t < 0 || t >= a.n_types)) atomicOr(&g_bucket_error, 1u);
                const unsigned hits = __ballot_sync(0xffffffffu, hit);
                if (lane == 0) warp_count[warp] = __popc(hits);
                __syncthreads();
                int before = found;
#pragma unroll
                for (int q = 0; q < kThreads / 32; ++q) {
                    if (q < warp) before += warp_count[q];
                    found += warp_count[q];
                }
                if (hit) list[before + __popc(hits & ((1u << lane) - 1u))] = part + tid;
                __syncthreads();
            }
            add(found, [&](int i) { return w + list[i]; });
            __syncthreads();  // the list is free
        }
    }

    // the tile's sums and its order into shared memory
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
#pragma unroll
        for (int j = 0; j < kN; ++j) sums[(tid + k * kThreads) * kN + j] = acc[k * kN + j];
    const uint4 *oq = reinterpret_cast<const uint4 *>(a.plan + a.at.order) + tile * (kPlanTile / 8);
    for (int i = tid; i < kPlanTile / 8; i += kThreads)
        reinterpret_cast<uint4 *>(order)[i] = __ldg(oq + i);
    __syncthreads();
    const int32_t s0 = max(a.plan[a.at.tile_slot + tile], 0);
    const int32_t s1 = min(a.plan[a.at.tile_slot + tile + 1], a.n_slots);
    float *out = a.partial + ((static_cast<int64_t>(slab) * a.n_types + type) * a.heads + head) * a.n_slots;
    constexpr int kSlots = kThreads / LANES;  // at a time
    for (int32_t s = s0; s < s1; s += kSlots) {
        const int32_t mine = s + tid / LANES;
        float v = 0.f;
        if (mine < s1) {
            const uint32_t span = static_cast<uint32_t>(__ldg(a.plan + a.at.slot_span + mine));
            const int begin = span & 0xffffu, end = min(begin + static_cast<int>(span >> 16), kPlanTile);
            for (int k = begin + tid % LANES; k < end; k += LANES)
                v += sums[order[k] & (kPlanTile - 1)];
        }
        v = group_sum<LANES>(v);
        if (mine < s1 && tid % LANES == 0) {
            const int32_t d = __ldg(a.plan + a.at.slot_dest + mine);
            if (d >= 0 && d < a.n_slots) out[d] = v;
        }
    }
}

// Pass 2: LANES lanes a (type, head, bucket) add the bucket's slots over the
// slabs and round once to the table's format.
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads) bias_grad_table(GradArgs a) {
    pdl_prologue();
    const int64_t total = static_cast<int64_t>(a.n_types) * a.heads * a.n_buckets;
    const bool ok = plan_matches(a);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_bucket_error, 1u);
    const int64_t lane_of = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t i = lane_of / LANES;
    const int32_t lane = static_cast<int32_t>(lane_of % LANES);
    const int64_t th = i / a.n_buckets;
    const int32_t b = static_cast<int32_t>(i - th * a.n_buckets);
    float v = 0.f;
    if (ok && i < total) {
        const int32_t d0 = max(__ldg(a.plan + a.at.bucket_dest + b), 0);
        const int32_t d1 = min(__ldg(a.plan + a.at.bucket_dest + b + 1), a.n_slots);
        const int64_t step = static_cast<int64_t>(a.n_types) * a.heads * a.n_slots;
        for (int32_t d = d0 + lane; d < d1; d += LANES) {
            const float *p = a.partial + th * a.n_slots + d;
#pragma unroll 8
            for (int32_t s = 0; s < a.slabs; ++s) v += __ldcg(p + s * step);
        }
    }
    v = group_sum<LANES>(v);
    if (i < total && lane == 0) {
        const int64_t type = th / a.heads, head = th - type * a.heads;
        store1<T>(a.table, (type * a.n_buckets + b) * a.heads + head, v);
    }
}

// Slabs of windows: enough blocks for five on each of 152 SMs, but about
// four windows of a type in a slab (a block's slot sums cost about as much
// as reading two).  Depends on the sizes alone, so results do not depend on
// the device.
constexpr int64_t kGradBlocks = 1520;
constexpr int64_t kSlabWindows = 4;

int64_t grad_slabs(int64_t n_win, int64_t heads, int64_t n_types, int64_t n_tiles) {
    const int64_t units = heads * n_types * (n_tiles > 0 ? n_tiles : 1);
    int64_t s = ceil_div(kGradBlocks, units);
    const int64_t most = n_win / (n_types * kSlabWindows);
    if (s > most) s = most;
    return s > 1 ? s : 1;
}

template <typename E, bool kVec>
wgs_status launch_tiles(const GradArgs &a, unsigned grid, cudaStream_t stream) {
    // lanes a slot by the slots' average length
    const int64_t mean = a.n_slots > 0 ? a.n_pairs / a.n_slots : 0;
    auto kernel = mean < 8    ? bias_grad_tiles<E, kVec, 1>
                  : mean < 64 ? bias_grad_tiles<E, kVec, 8>
                              : bias_grad_tiles<E, kVec, 32>;
    return launch(kernel, dim3(grid), dim3(kThreads), 0, stream, a);
}

template <typename E>
wgs_status launch_tiles_any(const GradArgs &a, unsigned grid, cudaStream_t stream) {
    constexpr int n = std::is_same<E, F32>::value ? 4 : 8;
    return a.n_pairs % n == 0 && aligned16(a.grad) ? launch_tiles<E, true>(a, grid, stream)
                                                    : launch_tiles<E, false>(a, grid, stream);
}

template <typename T>
wgs_status launch_table(const GradArgs &a, cudaStream_t stream) {
    const int64_t mean = a.n_slots / a.n_buckets;
    const int lanes = mean < 8 ? 1 : mean < 64 ? 8 : 32;
    const int64_t grid = ceil_div(static_cast<int64_t>(a.n_types) * a.heads * a.n_buckets * lanes, kThreads);
    if (grid > INT32_MAX) return WGS_ERR_SHAPE;
    auto kernel = lanes == 1 ? bias_grad_table<T, 1> : lanes == 8 ? bias_grad_table<T, 8> : bias_grad_table<T, 32>;
    return launch(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a);
}

// a * b for non-negative a and b, or false past 2^62.
bool times(int64_t a, int64_t b, int64_t *out) {
    if (b > 0 && a > (int64_t{1} << 62) / b) return false;
    *out = a * b;
    return true;
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
        !times(slabs, n_buckets * bytes_of(table_dtype), &table_n))
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
    if (n_win < 0 || heads < 1 || n_types < 1 || n_pairs < 0 || n_slots < 0) return 0;
    return static_cast<size_t>(grad_slabs(n_win, heads, n_types, ceil_tiles(n_pairs))) * n_types *
           heads * static_cast<size_t>(n_slots) * sizeof(float);
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
    if (n_pairs > INT32_MAX - kPlanTile || n_slots > n_pairs || n_win > INT32_MAX)
        return WGS_ERR_SHAPE;
    const int64_t n_tiles = ceil_tiles(n_pairs);
    const int64_t slabs = grad_slabs(n_win, heads, n_types, n_tiles);
    int64_t th, units, grad_bytes, table_bytes, part_bytes;
    if (!times(n_types, heads, &th) || !times(th * slabs, n_tiles, &units) || units > INT32_MAX ||
        !times(n_win * heads, n_pairs * bytes_of(dtype), &grad_bytes) ||
        !times(th, n_buckets * bytes_of(table_dtype), &table_bytes) ||
        !times(th * slabs, n_slots * 4, &part_bytes))
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
    GradArgs a = {grad, plan, win_type, static_cast<float *>(workspace), grad_table, at,
                  n_win, n_pairs, heads, n_types, n_buckets, static_cast<int32_t>(n_tiles),
                  static_cast<int32_t>(n_slots), static_cast<int32_t>(slabs)};
    if (units > 0) {
        const unsigned grid = static_cast<unsigned>(units);
        st = dtype == WGS_F32   ? launch_tiles_any<F32>(a, grid, stream)
             : dtype == WGS_F16 ? launch_tiles_any<Fp16>(a, grid, stream)
                                : launch_tiles_any<Bf16>(a, grid, stream);
        if (st != WGS_OK) return st;
    }
    return table_dtype == WGS_F32   ? launch_table<F32>(a, stream)
           : table_dtype == WGS_F16 ? launch_table<Fp16>(a, stream)
                                    : launch_table<Bf16>(a, stream);
}
