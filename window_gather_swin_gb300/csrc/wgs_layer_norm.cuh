// What layer norm's forward and backward kernels share: how rows belong to
// threads, how they reach them, and how a call is cut.
//
// A row belongs to a unit: 4, 8, 16 or 32 lanes of a warp, or several warps.  It is
// read in chunks of 16 bytes on 16-byte boundaries of memory, chunk c of a unit's
// thread t being the row's (c threads + t)-th.  A width that is no whole number of
// chunks makes rows start anywhere in a chunk (`lead` elements after its boundary),
// but every `period`-th row starts at the same place: a block takes rows of one
// such class, so that a thread holds the same columns of all its rows whatever the
// width is.  What a row's first and last chunk hold of its neighbours counts as
// zero and is not written.
//
// Rows come through slots in shared memory that each thread fills for itself with
// asynchronous copies, `stages` passes ahead of its own use: nothing waits for
// another thread, and the copies in flight take no registers.  Tensors whose rows
// do not start at the same place in a chunk (views at odd offsets) are copied
// element by element into the same slots.
#pragma once

#include <type_traits>

#include "wgs_common.cuh"
#include "wgs_layer_norm_plan.h"

namespace wgs {

namespace {

struct F32 {};

static_assert(kExchangeBytes == 2 * kMeet * sizeof(float2), "two places of the units' sums");

struct LayerNormArgs {
    const char *in[3];   // forward: x, branch; backward: x, grad_y, grad_residual
    char *out;           // y or grad_x
    char *total;         // residual_out
    const void *weight, *bias;
    float *mean, *rstd;
    float *part;         // backward: [blocks][2][width]
    int64_t rows, closing;   // closing: the first row whose chunks may end behind the tensor
    int tensors;         // of in
    int width, chunks;   // chunks: of a row, at most
    int lead, period;    // of row 0, in elements; rows that start at the same place
    int stages, team_warps;
    int kept_bytes;      // of shared memory before the slots
    float eps, inv;      // inv: 1 / width
    bool p32;            // weight and bias are FP32
    bool together;       // all tensors' rows start at the same place in a chunk
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// FP32 pairs on the packed pipe: each half the correctly rounded operation.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

template <typename E>
constexpr int kBytes = std::is_same<E, F32>::value ? 4 : 2;

template <typename E>
__device__ __forceinline__ float widen(const char *p) {
    if constexpr (std::is_same<E, F32>::value)
        return *reinterpret_cast<const float *>(p);
    else
        return E::to_f2(*reinterpret_cast<const uint16_t *>(p)).x;
}

__device__ __forceinline__ uint4 load_shared(uint32_t at) {
    uint4 q;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}
__device__ __forceinline__ void store_shared(uint32_t at, const uint4 &q) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}
// 16-byte asynchronous copy of the first `bytes` bytes at gmem, zeros behind.
__device__ __forceinline__ void copy_part(uint32_t slot, const char *gmem, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot), "l"(gmem), "r"(bytes) : "memory");
}

// A thread's place: its unit, the unit's rows and the thread's columns of them.
// kC: chunks of a row that a thread holds.  kTeam: lanes of a row, or 0 for units
// of several warps.  kWhole: rows are whole chunks.
template <typename E, int kC, int kTeam, bool kWhole>
struct Place {
    static constexpr bool kMulti = kTeam == 0;
    static constexpr int kV = 16 / kBytes<E>;       // elements of a chunk
    static constexpr int kHalf = kV / 2;            // pairs of a chunk
    static constexpr int kPairs = kC * kHalf;       // of a thread's part of a row
    static constexpr int kRowsPerPass = kMulti ? 1 : 32 / kTeam;

    const LayerNormArgs &a;
    int warps, index, thread;   // of the unit, in the block, of its unit
    int lead;
    int64_t row, row_step;      // this thread's row of the present pass; from pass to pass
    int64_t at, step;           // the same in bytes, of its first chunk
    int64_t pass, passes, pass_step;
    uint32_t slots, stage_bytes, present, coming;   // this thread's; stages read and filled next
    int64_t next_row, next_at;  // to be fetched
    uint32_t held_bits = 0, full_bits = 0;      // of a ragged row's chunks, see held() and full()
    bool first_here, last_here; // a ragged row's partial first and last chunk are this warp's (team's)
    float2 (*meet)[kMeet];      // [2][places]: sums of the units' warps
    int turn = 0;

    __device__ Place(const LayerNormArgs &args, float2 (*exchange)[kMeet], uint32_t ring) : a(args), meet(exchange) {
        warps = kMulti ? a.team_warps : 1;
        const int warp = threadIdx.x >> 5;
        index = kMulti ? warp / warps : warp;
        thread = kMulti ? threadIdx.x - index * warps * 32 : threadIdx.x & 31;
        const int units = blockDim.x / (warps * 32);
        const int kind = kWhole ? 0 : blockIdx.x % a.period;      // the block's class of rows
        const int period = kWhole ? 1 : a.period;
        lead = kWhole ? 0 : (a.lead + kind * a.width) & (kV - 1);
        const int64_t rows = (a.rows - kind + period - 1) / period;
        const int blocks = (gridDim.x - kind + period - 1) / period;
        pass = static_cast<int64_t>(blockIdx.x / period) * units + index;
        pass_step = static_cast<int64_t>(blocks) * units;
        passes = (rows + kRowsPerPass - 1) / kRowsPerPass;
        row = kind + (pass * kRowsPerPass + (kMulti ? 0 : thread / kTeam)) * period;
        row_step = pass_step * kRowsPerPass * period;
        at = (row * a.width - lead) * kBytes<E> + column_thread() * 16;
        step = row_step * a.width * kBytes<E>;
        next_row = row, next_at = at;
        // a warp's slots side by side: [stage][tensor][chunk][lane]
        stage_bytes = a.tensors * kC * 512;
        slots = ring + warp * a.stages * stage_bytes + (threadIdx.x & 31) * 16;
        present = coming = 0;
        if constexpr (!kWhole) {
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int col = column(c);
                held_bits |= static_cast<uint32_t>(col < a.width) << c;
                full_bits |= static_cast<uint32_t>(col >= 0 && col + kV <= a.width) << c;
            }
            const unsigned firsts = __ballot_sync(0xffffffffu, column(0) < 0);
            const unsigned lasts = __ballot_sync(0xffffffffu, last_chunk() < kC);
            const unsigned mine = kMulti || kTeam == 32 ? 0xffffffffu : ((1u << (kTeam & 31)) - 1) << ((threadIdx.x & 31) / kTeam_or_32() * kTeam);
            first_here = (firsts & mine) != 0, last_here = (lasts & mine) != 0;
        }
    }
    __device__ static constexpr int kTeam_or_32() { return kMulti ? 32 : kTeam; }
    // This thread's chunk that ends behind the row but begins in it (kC: none).
    __device__ int last_chunk() const {
        int which = kC;
#pragma unroll
        for (int c = 0; c < kC; ++c)
            if (column(c) >= 0 && column(c) < a.width && column(c) + kV > a.width) which = c;
        return which;
    }
    __device__ int column_thread() const { return kMulti ? thread : thread & (kTeam - 1); }
    __device__ int column_threads() const { return kMulti ? warps * 32 : kTeam; }
    __device__ int capacity() const { return kC * column_threads(); }     // chunks of a unit
    __device__ int chunk(int c) const { return c * column_threads() + column_thread(); }
    __device__ int column(int c) const { return chunk(c) * kV - lead; }   // of its first element
    __device__ bool held(int c) const { return kWhole ? column(c) < a.width : (held_bits >> c & 1u) != 0; }
    __device__ bool full(int c) const { return (full_bits >> c & 1u) != 0; }
    __device__ bool there() const { return row < a.rows; }
    __device__ void advance() {
        pass += pass_step, row += row_step, at += step;
        present += stage_bytes;
        if (present == a.stages * stage_bytes) present = 0;
    }

    // Both sums over a row's threads, in a fixed order; every thread gets them.
    __device__ float2 sum(float2 v) {
#pragma unroll
        for (int o = (kMulti ? 32 : kTeam) / 2; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        return across(v);
    }
    __device__ float sum(float v) {
#pragma unroll
        for (int o = (kMulti ? 32 : kTeam) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return kMulti ? across(make_float2(v, 0.f)).x : v;
    }
    __device__ float2 across(float2 v) {
        if constexpr (kMulti) {
            // two places in turn: a warp that is here again has passed the other's barrier.
            // Two warps' sums a read; a unit of an odd number has a place of zeros behind.
            const int even = (warps + 1) / 2 * 2;
            float2 *place = meet[turn] + index * even;
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) {
                place[thread >> 5] = v;
                if (thread == 0 && even > warps) place[warps] = both(0.f);
            }
            asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(warps * 32) : "memory");
            v = both(0.f);
#pragma unroll
            for (int w = 0; w < kWarps; w += 2) {
                if (w >= warps) break;
                const float4 q = *reinterpret_cast<const float4 *>(place + w);
                v = add2(v, add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
            }
        }
        return v;
    }

    // Copy the coming row of every tensor into the coming stage; zeros where there is
    // none.  A row's first chunk may begin before the row, and before the tensor where
    // that begins inside a chunk: in the same 16 bytes of memory as the tensor's first
    // element.  Behind the tensor nothing is read.
    __device__ void fetch() {
        const uint32_t to = slots + coming;
        const bool is_there = next_row < a.rows;
        // (a copy of no bytes names 16 bytes' boundary all the same)
        const int64_t from_at = is_there ? next_at : kWhole || !a.together ? 0 : -a.lead * kBytes<E>;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k >= a.tensors) break;
            const char *from = a.in[k] + from_at;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                if (!held(c)) continue;
                const char *p = from + c * column_threads() * 16;
                const uint32_t slot = to + (k * kC + c) * 512;
                if constexpr (kWhole) {
                    copy_part(slot, p, is_there ? 16 : 0);
                } else if (a.together) {
                    int bytes = is_there ? 16 : 0;
                    if (next_row >= a.closing && is_there && !full(c)) {
                        const int left = (static_cast<int>(a.rows - next_row) * a.width - column(c)) * kBytes<E>;
                        if (left < bytes) bytes = left;
                    }
                    copy_part(slot, p, bytes);
                } else {
                    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < kV; ++j) {
                        if (!is_there || column(c) + j >= a.width) continue;
                        if constexpr (kV == 4)
                            w[j] = *reinterpret_cast<const uint32_t *>(p + 4 * j);
                        else
                            w[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p + 2 * j)) << (j & 1) * 16;
                    }
                    store_shared(slot, make_uint4(w[0], w[1], w[2], w[3]));
                }
            }
        }
        cp_async_commit();
        next_row += row_step, next_at += step;
        coming += stage_bytes;
        if (coming == a.stages * stage_bytes) coming = 0;
    }
    // Before the wait for the previous grid: L2 may look for the first rows' lines.
    __device__ void look_ahead() const {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k >= a.tensors) break;
#pragma unroll
            for (int c = 0; c < kC; ++c)
                if (there() && held(c) && column(c) >= 0) prefetch_l2(a.in[k] + at + c * column_threads() * 16);
        }
    }
    // Before the first fetch: the slots of chunks past the row's end hold zeros for good.
    __device__ void clear_slots() const {
        for (uint32_t s = 0; s < a.stages * stage_bytes; s += stage_bytes)
            for (int k = 0; k < a.tensors; ++k)
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    if (!held(c)) store_shared(slots + s + (k * kC + c) * 512, make_uint4(0u, 0u, 0u, 0u));
    }
    // Until the present stage has arrived.
    __device__ void arrived() const {
        if (a.stages == 4) cp_async_wait<3>();
        else if (a.stages == 3) cp_async_wait<2>();
        else if (a.stages == 2) cp_async_wait<1>();
        else cp_async_wait<0>();
    }
    // The thread's part of the present row of tensor k, widened; outside the row zeros, or
    // the bits `fill`:
    // `masks` are keep_edges', looked up by the chunks that are not full, or with kAll
    // keep_masks', for all chunks alike.  (The backward has no registers for the former:
    // [5000, 8191] bf16 85 us, so 78; the forward no shared memory to spare for the latter:
    // 51, so 87.)
    template <bool kAll>
    __device__ void load(int k, uint32_t masks, float2 (&v)[kPairs], uint32_t fill = 0u) const {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            uint4 q = load_shared(slots + present + (k * kC + c) * 512);
            if (!kWhole && (kAll || !full(c))) {
                const uint4 m = load_shared(masks + (kAll ? chunk(c) : kind(c)) * 16);
                q.x = (q.x & m.x) | (fill & ~m.x), q.y = (q.y & m.y) | (fill & ~m.y);
                q.z = (q.z & m.z) | (fill & ~m.z), q.w = (q.w & m.w) | (fill & ~m.w);
            }
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                if constexpr (kV == 4)
                    v[c * 2 + i] = make_float2(__uint_as_float(word(q, 2 * i)), __uint_as_float(word(q, 2 * i + 1)));
                else
                    v[c * 4 + i] = E::to_f2(word(q, i));
            }
        }
    }
    // A word of load()'s that holds `value` in every place, rounded to the tensors' format.
    __device__ static uint32_t filled(float value) {
        if constexpr (kV == 4)
            return __float_as_uint(value);
        else
            return E::from_f2(value, value);
    }
    // Rounds each value once, to nearest even, into the present row.  A ragged row's
    // first and last chunk go to shared memory (`edges`: two chunks a row of a warp), from
    // where the row's lanes write an element each.
    __device__ void store(char *base, uint32_t edges, const float2 (&v)[kPairs]) const {
        const int lane = threadIdx.x & 31, team = kMulti ? 0 : lane / kTeam_or_32();
        const uint32_t edge = edges + ((threadIdx.x >> 5) * 8 + team) * 32;
        const bool is_there = there();
        if (!kWhole) __syncwarp();   // the edges' last readers
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            char *p = base + at + c * column_threads() * 16;
            uint4 q;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kV == 4)
                    set_word(q, i, __float_as_uint(i & 1 ? v[c * 2 + i / 2].y : v[c * 2 + i / 2].x));
                else
                    set_word(q, i, E::from_f2(v[c * 4 + i].x, v[c * 4 + i].y));
            }
            if constexpr (kWhole) {
                if (is_there && held(c)) st_stream(p, q);
            } else if (!a.together) {
#pragma unroll
                for (int j = 0; j < kV; ++j)
                    if (is_there && column(c) + j < a.width) put(p, j, word(q, j * kBytes<E> / 4));
            } else if (full(c)) {
                if (is_there) st_stream(p, q);
            } else if (held(c)) {
                store_shared(edge + (column(c) < 0 ? 0 : 16), q);
            }
        }
        if (kWhole || !a.together) return;
        __syncwarp();
        if (!is_there) return;
        char *row_at = base + at - column_thread() * 16;     // the row's first chunk
#pragma unroll
        for (int j0 = 0; j0 < kV; j0 += kTeam_or_32()) {
            const int j = j0 + (kMulti ? lane : lane & (kTeam_or_32() - 1));
            if (j >= kV) break;
            if (first_here) {
                const int col = j - lead;
                if (col >= 0 && col < a.width) put(row_at, j, element(edge, j));
            }
            if (last_here) {
                const int first = (lead + a.width) / kV * kV;     // of the last chunk
                if (first + j - lead < a.width) put(row_at + first * kBytes<E>, j, element(edge + 16, j));
            }
        }
    }
    __device__ static void put(char *p, int j, uint32_t w) {
        if constexpr (kV == 4)
            *reinterpret_cast<uint32_t *>(p + 4 * j) = w;
        else
            *reinterpret_cast<uint16_t *>(p + 2 * j) = static_cast<uint16_t>(w >> (j & 1) * 16);
    }
    __device__ static uint32_t element(uint32_t chunk_at, int j) {
        uint32_t w;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(chunk_at + j * kBytes<E> / 4 * 4) : "memory");
        return w;
    }

    // Values of all columns in shared memory as the threads hold columns, zeros outside
    // the row: the first four elements of all chunks, then the other four (so that
    // neighbouring threads' 16 bytes lie side by side).  value(col): of a column in the
    // row; four(col, v): of four from col on, false where they cannot be had at once.
    template <typename Value, typename Four>
    __device__ void keep(float *to, Value value, Four four) const {
        constexpr int kQuads = kV / 4;       // of a chunk
        const int all = capacity();
#pragma unroll 4
        for (int i = threadIdx.x; i < all * kQuads; i += blockDim.x) {
            const int col = i * 4 - lead;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!(col >= 0 && col + 4 <= a.width && four(col, v))) {
                if (col >= 0 && col < a.width) v.x = value(col);
                if (col + 1 >= 0 && col + 1 < a.width) v.y = value(col + 1);
                if (col + 2 >= 0 && col + 2 < a.width) v.z = value(col + 2);
                if (col + 3 >= 0 && col + 3 < a.width) v.w = value(col + 3);
            }
            *reinterpret_cast<float4 *>(to + (i % kQuads * all + i / kQuads) * 4) = v;
        }
    }
    // weight or bias, widened
    __device__ void keep_param(float *to, const void *from, float other) const {
        const char *p = static_cast<const char *>(from);
        if (!from) {
            keep(to, [&](int) { return other; }, [&](int, float4 &v) { return v = make_float4(other, other, other, other), true; });
        } else if (a.p32) {
            const bool whole = (reinterpret_cast<uintptr_t>(p) + 16 - lead * 4) % 16 == 0;     // at columns of whole quads
            keep(to, [&](int col) { return __ldg(reinterpret_cast<const float *>(p) + col); },
                 [&](int col, float4 &v) {
                     if (whole) v = __ldg(reinterpret_cast<const float4 *>(p + col * 4));
                     return whole;
                 });
        } else {
            keep(to, [&](int col) { return widen<E>(p + static_cast<size_t>(col) * kBytes<E>); },
                 [](int, float4 &) { return false; });
        }
    }
    __device__ void kept(const float *from, int c, float2 (&w)[kHalf]) const {
#pragma unroll
        for (int h = 0; h < kV / 4; ++h) {
            const float4 q = *reinterpret_cast<const float4 *>(from + (h * capacity() + chunk(c)) * 4);
            w[2 * h] = make_float2(q.x, q.y), w[2 * h + 1] = make_float2(q.z, q.w);
        }
    }
    // What of a chunk that is not full is the row's: of the first one, the last one and one
    // behind the row, as bits and as a factor for every element.
    static constexpr int kKeptEdges = kept_edges(kBytes<E>);
    __device__ int kind(int c) const { return column(c) < 0 ? 0 : held(c) ? 1 : 2; }
    __device__ void keep_edges(char *to) const {
        const int i = threadIdx.x;
        if (i >= kEdgeKinds * kV) return;
        const int k = i / kV, j = i % kV;
        const int at = k == 0 ? -lead : k == 1 ? (lead + a.width) / kV * kV - lead : a.width, col = at + j;
        const bool in = col >= 0 && col < a.width;
        if constexpr (kV == 4)
            reinterpret_cast<uint32_t *>(to)[i] = in ? 0xffffffffu : 0u;
        else
            reinterpret_cast<uint16_t *>(to)[i] = in ? 0xffffu : 0u;
        reinterpret_cast<float *>(to + kEdgeKinds * 16)[i] = in ? 1.f : 0.f;
    }
    // The bits of each chunk that are the row's.
    __device__ void keep_masks(char *to) const {
        for (int i = threadIdx.x; i < capacity() * 4; i += blockDim.x) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < kV / 4; ++j) {
                const int col = i * (kV / 4) + j - lead;
                if (col >= 0 && col < a.width) m |= kV == 4 ? 0xffffffffu : 0xffffu << 16 * j;
            }
            reinterpret_cast<uint32_t *>(to)[i] = m;
        }
    }
    __device__ void inside(const char *edges, int c, float2 (&in)[kHalf]) const {
        const float *from = reinterpret_cast<const float *>(edges + kEdgeKinds * 16) + kind(c) * kV;
#pragma unroll
        for (int h = 0; h < kV / 4; ++h) {
            const float4 q = *reinterpret_cast<const float4 *>(from + 4 * h);
            in[2 * h] = make_float2(q.x, q.y), in[2 * h + 1] = make_float2(q.z, q.w);
        }
    }
};

// -------------------------------------------------------------------- host --

inline int64_t bytes_of(wgs_dtype d) { return d == WGS_F32 ? 4 : 2; }
inline bool dtype_ok(wgs_dtype d) { return d == WGS_F32 || d == WGS_F16 || d == WGS_BF16; }
inline bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Rows of `width` values of up to 4 bytes that can be addressed.
inline bool sizes_ok(int64_t rows, int32_t width) {
    return rows >= 0 && width > 0 && rows <= INT64_MAX / 16 / width;
}

// Where rows start in their chunks, and whether all tensors' do at the same place.
// True where rows are whole chunks.
template <typename E>
bool place_rows(LayerNormArgs *a) {
    constexpr int kV = 16 / kBytes<E>;
    const uintptr_t first = reinterpret_cast<uintptr_t>(a->out);
    a->together = !a->total || (reinterpret_cast<uintptr_t>(a->total) - first) % 16 == 0;
    for (int k = 0; k < a->tensors; ++k)
        a->together = a->together && (reinterpret_cast<uintptr_t>(a->in[k]) - first) % 16 == 0;
    a->lead = a->together ? static_cast<int>(first % 16 / kBytes<E>) : 0;
    a->period = 1;
    while (a->together && a->period < kV && a->width * a->period % kV != 0) a->period *= 2;
    const bool whole = a->together && a->period == 1 && a->lead == 0;
    a->chunks = static_cast<int>(ceil_div(a->width + (whole || !a->together ? 0 : kV - 1), kV));
    a->closing = a->rows - ceil_div(kV - 1, a->width);
    a->inv = 1.0f / static_cast<float>(a->width);
    return whole;
}

// No output may share a byte with another or with an input, but for those that may
// be an input's own buffer.
struct Buffer {
    const void *p;
    int64_t bytes;
    bool in_place;   // an output that may be one of the rows' inputs
    bool rows;       // an input that such an output may be
};

inline bool buffers_ok(const Buffer *outs, int n_outs, const Buffer *ins, int n_ins) {
    for (int i = 0; i < n_outs; ++i) {
        if (!outs[i].p) continue;
        for (int k = 0; k < n_ins; ++k) {
            if (!ins[k].p) continue;
            if (outs[i].in_place && ins[k].rows && outs[i].p == ins[k].p) continue;
            if (overlap(outs[i].p, outs[i].bytes, ins[k].p, ins[k].bytes)) return false;
        }
        for (int k = 0; k < i; ++k)
            if (outs[k].p && overlap(outs[i].p, outs[i].bytes, outs[k].p, outs[k].bytes)) return false;
    }
    return true;
}

}  // namespace

}  // namespace wgs
