// Embedding lookup with scaling and its gradient by sorted indices (sm_103a).
//
//     out[i] = scale * table[idx[i]]                    (0 for idx -1)
//     grad_table[r] = scale * sum of grad[i] over the i with idx[i] == r
//
// The lookup is a stream of rows: bound by the bytes of its output, and of the
// table's rows that are named (which L2 keeps between namings).
//
// The gradient.  Adding to the table by atomics would make the sums' order, and
// their last bits, change from run to run, and would wait at rows that many
// indices name.  Instead the indices are sorted by row, positions in order within
// a row (a stable counting sort by digits), and cut into equal pieces of the
// sorted order, whatever rows they fall on: a block sums its piece's runs of equal
// rows, writes those that end inside it, and leaves what reaches over its ends to
// a last launch, which adds a run's pieces up.  So the work is even if one row has
// most of the indices, and the order of additions is fixed.  Few indices, or few rows
// of the table, take one or two launches in which blocks sort for themselves.
#include <type_traits>

#include "wgs_common.cuh"
#include "wgs_embedding_plan.h"

namespace wgs {

namespace {

// Set (never cleared by a kernel) when an index lies outside [-1, n_rows); read
// and cleared by wgs_check_error.
__device__ unsigned int g_embedding_error;

struct F32 {};

constexpr int kMaxWidth = 32768;

template <typename E>
constexpr int kBytes = std::is_same<E, F32>::value ? 4 : 2;

// One value through L1.
template <typename E>
__device__ __forceinline__ float load_kept(const char *p) {
    if constexpr (std::is_same<E, F32>::value)
        return __ldg(reinterpret_cast<const float *>(p));
    else
        return E::to_f2(__ldg(reinterpret_cast<const uint16_t *>(p))).x;
}

template <typename E, int kV>
__device__ __forceinline__ void store_values(char *p, const float (&v)[kV]) {
    if constexpr (kV == 1) {
        if constexpr (std::is_same<E, F32>::value)
            *reinterpret_cast<float *>(p) = v[0];
        else
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(E::from_f2(v[0], 0.f));
    } else if constexpr (std::is_same<E, F32>::value) {
#pragma unroll
        for (int i = 0; i < kV / 4; ++i)
            *reinterpret_cast<float4 *>(p + 16 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint4 q;
#pragma unroll
        for (int j = 0; j < 4; ++j) set_word(q, j, E::from_f2(v[2 * j], v[2 * j + 1]));
        st_stream(p, q);
    }
}

// ------------------------------------------------------------------ lookup --

// Chunks of 16 bytes of the table's rows, those of a block's threads side by side,
// are taken in steps of the whole grid; a thread has its next step's chunk on its way
// into a slot of its own in shared memory, and the index of the one after that in a
// register, so that neither the index nor the row that it names is waited for at
// full length.  The copies go through L1, which keeps the rows that many indices
// name: past it, a skewed sequence's rows were asked of the same L2 lines by all SMs
// at once (131040 of 384, FP32 to bf16: 128 us, through L1 33).  Of those 33 us issue is
// at 71 % of its peak (77 instructions a chunk of a warp), L1 at 63 and L2 at 30, from
// which 150 MB of the 201 of the named rows come: instructions bound it first.  22 us from
// and to fp16; 47 us in FP32.
constexpr int kLookupThreads = 256;
constexpr int kLookupBlocksPerSm = 8;

struct LookupArgs {
    const char *table;
    const int32_t *idx;
    char *out;
    int64_t n, n_rows;
    int row_chunks, width;
    float scale;
};

// The table row of index r, seen by its row's first element as `first`: -1 for none.
__device__ __forceinline__ int32_t row_of_index(const LookupArgs &a, int64_t r, bool first) {
    if (r >= a.n) return -1;
    const int32_t k = __ldg(a.idx + r);
    if (k >= 0 && k < a.n_rows) return k;
    if (k != -1 && first) atomicOr(&g_embedding_error, 1u);
    return -1;
}

// T: the table's format, E: the output's.
template <typename T, typename E>
__global__ void __launch_bounds__(kLookupThreads, kLookupBlocksPerSm) embedding_lookup(const LookupArgs a) {
    constexpr int kIn = 16, kV = kIn / kBytes<T>, kOut = kV * kBytes<E>;    // of a chunk
    __shared__ uint4 slots[2][kLookupThreads];
    pdl_prologue();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kLookupThreads, row_step = step / a.row_chunks;
    const int col_step = static_cast<int>(step - row_step * a.row_chunks);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kLookupThreads + threadIdx.x;
    int64_t row = first / a.row_chunks;
    int col = static_cast<int>(first - row * a.row_chunks);
    auto advance = [&](int64_t &r, int &c) {
        r += row_step, c += col_step;
        if (c >= a.row_chunks) c -= a.row_chunks, ++r;
    };
    auto fetch = [&](int s, int32_t from, int c) {
        if (from >= 0) cp_async16_ca(&slots[s][threadIdx.x], a.table + (static_cast<int64_t>(from) * a.row_chunks + c) * kIn);
        cp_async_commit();
    };
    int64_t next_row = row;
    int next_col = col;
    int32_t now = row_of_index(a, row, col == 0);
    advance(next_row, next_col);
    fetch(0, now, col);
    int32_t next = row_of_index(a, next_row, next_col == 0);
    for (int s = 0; row < a.n; s ^= 1) {
        fetch(s ^ 1, next, next_col);
        int64_t later_row = next_row;
        int later_col = next_col;
        advance(later_row, later_col);
        const int32_t later = row_of_index(a, later_row, later_col == 0);
        float v[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = 0.f;
        cp_async_wait<1>();
        if (now >= 0) {
            const uint4 q = slots[s][threadIdx.x];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (kV == 4) {
                    v[k] = __uint_as_float(word(q, k)) * a.scale;
                } else {
                    const float2 f = T::to_f2(word(q, k));
                    v[2 * k] = f.x * a.scale, v[2 * k + 1] = f.y * a.scale;
                }
            }
        }
        char *p = a.out + (row * a.row_chunks + col) * kOut;
        if constexpr (kOut == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(E::from_f2(v[0], v[1]), E::from_f2(v[2], v[3]));
        else
            store_values<E, kV>(p, v);
        row = next_row, col = next_col, now = next;
        next_row = later_row, next_col = later_col, next = later;
    }
}

// Rows of other widths, or at other places: the output as one run of elements, 16 bytes
// of it a thread (single elements where it does not start on 16), which may span rows;
// the table's elements one by one, through L1.
template <typename T, typename E>
__global__ void __launch_bounds__(kLookupThreads, kLookupBlocksPerSm) embedding_lookup_ragged(const LookupArgs a) {
    constexpr int kV = 16 / kBytes<E>;
    pdl_prologue();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kLookupThreads * kV, row_step = step / a.width;
    const int col_step = static_cast<int>(step - row_step * a.width);
    const int64_t all = a.n * a.width;
    int64_t at = (static_cast<int64_t>(blockIdx.x) * kLookupThreads + threadIdx.x) * kV, row = at / a.width;
    int col = static_cast<int>(at - row * a.width);
    int32_t now = row_of_index(a, row, col == 0);
    while (at < all) {
        int64_t next_row = row + row_step;
        int next_col = col + col_step;
        if (next_col >= a.width) next_col -= a.width, ++next_row;
        const int32_t next = row_of_index(a, next_row, next_col == 0);
        float v[kV];
        const char *from = a.table + static_cast<int64_t>(now) * a.width * kBytes<T>;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            if (col == a.width) {
                col = 0, now = row_of_index(a, ++row, true);
                from = a.table + static_cast<int64_t>(now) * a.width * kBytes<T>;
            }
            v[j] = now >= 0 ? load_kept<T>(from + col * kBytes<T>) * a.scale : 0.f;     // (a pad is +0)
            ++col;
        }
        char *p = a.out + at * kBytes<E>;
        if (at + kV <= all && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
            store_values<E, kV>(p, v);
        } else {
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const float one[1] = {v[j]};
                if (at + j < all) store_values<E, 1>(p + j * kBytes<E>, one);
            }
        }
        at += step, row = next_row, col = next_col, now = next;
    }
}

// Zeros over n bytes at p; `unit` bytes of an element divide both.
__device__ void write_zeros(char *p, int64_t n, int unit, int64_t thread, int64_t threads) {
    int64_t lead = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15;
    if (lead > n) lead = n;
    const int64_t whole = (n - lead) / 16, rest = n - lead - whole * 16;
    for (int64_t i = thread; i < whole; i += threads) st_stream(p + lead + 16 * i, make_uint4(0u, 0u, 0u, 0u));
    if (thread < 16) {
        const int64_t i = thread * unit;
        char *end = p + lead + whole * 16;
        for (int side = 0; side < 2; ++side) {
            char *q = side ? end : p;
            if (i >= (side ? rest : lead)) continue;
            if (unit == 4)
                *reinterpret_cast<uint32_t *>(q + i) = 0u;
            else
                *reinterpret_cast<uint16_t *>(q + i) = 0;
        }
    }
}

// -------------------------------------------------------------------- sort --

// A stable counting sort by digits of up to 9 bits, from the lowest, a launch a
// pass and one before the first: each is bound by the time that a launch and a few
// dependent reads take, so the fewer the better.  A block has a range of the order
// so far; it adds up all blocks' counts of every digit, to know where its own
// indices of each go, ranks them, and lays them into shared memory in their order,
// from where runs of a digit leave side by side.  As it knows where an index goes, it
// counts it there for the next pass too (whole numbers, so the order of these
// atomics does not matter).  Each launch has blocks besides that write a share of
// the table's gradient's zeros.
//
// A warp ranks 32 indices at a time: lanes set their bits in a word of their digit
// and read it back.  (Measured for 8190 indices an SM: 3.0 to 4.0 thousand cycles, 10
// with a ballot for every bit of the digit, 16 with match.any.)  One cluster of 16
// blocks with its barriers in place of launches was slower, 35 us for two passes
// over 131040 indices: 16 SMs rank and place longer than launches take.
constexpr int kBins = 512;
constexpr int kSortWarps = kSortThreads / 32;

struct SortArgs {
    const int32_t *idx;          // first pass: the call's indices
    const int32_t *keys, *at;    // later passes: sorted by the lower digits
    int32_t *keys_out, *at_out;
    void *counts, *next;         // [blocks][bins], of this pass and the next
    int64_t n, range;            // indices; of a block
    int64_t clear_words;         // from next on, cleared by the first launch
    int32_t n_rows;
    int shift, bits, blocks;
    bool last;
    char *zeros;                 // to be written as such by the blocks behind `blocks`
    int64_t zero_bytes;
    int zero_unit;
};

// The row that index i names; n_rows, sorted behind all, for none.
__device__ __forceinline__ int32_t key_of(const SortArgs &a, int64_t i) {
    if (!a.idx) return __ldcg(a.keys + i);
    const int32_t k = __ldg(a.idx + i);
    return k >= 0 && k < a.n_rows ? k : a.n_rows;
}

__device__ __forceinline__ bool zeros_instead(const SortArgs &a) {
    const int block = static_cast<int>(blockIdx.x) - a.blocks;
    if (block < 0) return false;
    write_zeros(a.zeros, a.zero_bytes, a.zero_unit, static_cast<int64_t>(block) * kSortThreads + threadIdx.x,
                static_cast<int64_t>(gridDim.x - a.blocks) * kSortThreads);
    return true;
}

// The first pass's counts, zeros in the others', and the indices' check.  C: of a
// count, 16 bits where a block's range allows.
template <typename C>
__global__ void __launch_bounds__(kSortThreads) sort_count(const SortArgs a) {
    __shared__ int32_t count[kBins];
    pdl_prologue();
    if (zeros_instead(a)) return;
    count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * a.range, end = first + a.range < a.n ? first + a.range : a.n;
    const uint32_t mask = (1u << a.bits) - 1;
    bool bad = false;
#pragma unroll 4
    for (int64_t i = first + threadIdx.x; i < end; i += kSortThreads) {
        const int32_t k = __ldg(a.idx + i);
        bad |= k < -1 || k >= a.n_rows;
        atomicAdd(&count[static_cast<uint32_t>(k >= 0 && k < a.n_rows ? k : a.n_rows) & mask], 1);
    }
    if (bad) atomicOr(&g_embedding_error, 1u);
    __syncthreads();
    if (threadIdx.x <= mask) static_cast<C *>(a.counts)[(blockIdx.x << a.bits) + threadIdx.x] = static_cast<C>(count[threadIdx.x]);
    for (int64_t i = blockIdx.x * kSortThreads + threadIdx.x; i < a.clear_words; i += a.blocks * kSortThreads)
        static_cast<uint32_t *>(a.next)[i] = 0u;
}

// What a block of kSortThreads needs to sort a tile by a digit.
struct Ranker {
    uint32_t *lanes, *counts;       // [warps][bins]: lanes of a digit; counts of the warps
    int32_t *warp_sums;             // [warps]
    uint32_t *base;                 // [bins]: where a digit begins in the tile
    static constexpr int kTableBytes = kSortWarps * kBins * 8;

    __device__ Ranker(char *tables, int32_t *sums, uint32_t *bases)
        : lanes(reinterpret_cast<uint32_t *>(tables)), counts(lanes + kSortWarps * kBins), warp_sums(sums), base(bases) {}
    // the first use of the tables for digits of so many bins
    __device__ void clear(int bins) const {
        for (int i = threadIdx.x & 31; i < bins; i += 32) lanes[(threadIdx.x >> 5) * kBins + i] = 0u;
        __syncwarp();
    }
    // Exclusive sums over the threads' values, in the threads' order.
    __device__ int32_t scan(int32_t v) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int32_t s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        __syncthreads();   // warp_sums' last readers
        if (lane == 31) warp_sums[warp] = s;
        __syncthreads();
        int32_t before = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) before += w < warp ? warp_sums[w] : 0;
        return before + s - v;
    }
    __device__ static int first() { return (threadIdx.x >> 5) * 32 * kRounds + (threadIdx.x & 31); }
    // The n values at first() + 32 j, round j, go to `pairs` in the order of the digit
    // above `shift`, equal ones in theirs.  Returns the count of digit threadIdx.x.
    __device__ uint32_t place(const uint32_t (&key)[kRounds], const uint32_t (&at)[kRounds], int n, int shift, int bits,
                              uint2 *pairs) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits, bin = threadIdx.x;
        const uint32_t mask = bins - 1, lower = (1u << lane) - 1;
        uint32_t *lane_bits = lanes + warp * kBins, *mine = counts + warp * kBins;
        for (int i = lane; i < bins; i += 32) mine[i] = 0u;
        __syncwarp();
        uint32_t rank[kRounds];
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            const bool valid = first() + 32 * j < n;
            const uint32_t d = key[j] >> shift & mask;
            if (valid) atomicOr(&lane_bits[d], 1u << lane);
            __syncwarp();
            const uint32_t same = lane_bits[d], had = mine[d], before = __popc(same & lower);
            __syncwarp();
            if (valid && before == 0) lane_bits[d] = 0u, mine[d] = had + __popc(same);
            __syncwarp();
            rank[j] = had + before;
        }
        __syncthreads();
        // counts of the warps before, and of the digits before: places in the tile
        uint32_t run = 0;
        if (bin < bins) {
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = counts[w * kBins + bin];
                counts[w * kBins + bin] = run;
                run += c;
            }
        }
        base[bin] = static_cast<uint32_t>(scan(static_cast<int32_t>(run)));
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            if (first() + 32 * j >= n) continue;
            const uint32_t d = key[j] >> shift & mask;
            pairs[base[d] + mine[d] + rank[j]] = make_uint2(key[j], at[j]);
        }
        __syncthreads();
        return run;
    }
};

template <typename C>
__global__ void __launch_bounds__(kSortThreads) sort_place(const SortArgs a) {
    extern __shared__ __align__(16) char shared[];
    uint2 *pairs = reinterpret_cast<uint2 *>(shared);                          // [tile]: row, position
    __shared__ int32_t to_base[kBins], warp_sums[kSortWarps];
    __shared__ uint32_t local_base[kBins];
    const Ranker ranker(shared + kSortTile * 8, warp_sums, local_base);
    pdl_prologue();
    if (zeros_instead(a)) return;
    const int me = blockIdx.x, bin = threadIdx.x, bins = 1 << a.bits;
    const uint32_t mask = bins - 1;
    ranker.clear(bins);
    const int64_t first = me * a.range, end = first + a.range < a.n ? first + a.range : a.n;
    uint32_t key[kRounds], at[kRounds];
    auto load = [&](int64_t tile) {
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            const int64_t i = tile + Ranker::first() + 32 * j;
            key[j] = at[j] = 0u;
            if (i < end) {
                key[j] = static_cast<uint32_t>(key_of(a, i));
                at[j] = a.idx ? static_cast<uint32_t>(i) : static_cast<uint32_t>(__ldcg(a.at + i));
            }
        }
    };
    load(first);

    // Where this block's indices of digit `bin` go: behind all of lower digits and
    // those of the blocks before.  Groups of threads each read some blocks' counts, 16
    // bytes of digits a thread; the groups' sums meet in the ranks' tables.
    {
        constexpr int kEach = 16 / sizeof(C), kMostGroups = 16;
        const int across = bins / kEach, groups = kSortThreads / across < kMostGroups ? kSortThreads / across : kMostGroups;
        const int group = threadIdx.x / across, part = threadIdx.x - group * across;
        const C *counts = static_cast<const C *>(a.counts) + part * kEach;
        int32_t *sums = reinterpret_cast<int32_t *>(ranker.counts);    // [groups][2][bins]: no more than that holds
        if (group < groups) {
            int32_t all[kEach] = {}, before[kEach] = {};
#pragma unroll 1
            for (int from = group; from < a.blocks; from += 8 * groups) {
                uint4 q[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const int b = from + g * groups;
                    q[g] = b < a.blocks ? __ldcg(reinterpret_cast<const uint4 *>(counts + b * bins)) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int g = 0; g < 8; ++g) {
#pragma unroll
                    for (int j = 0; j < kEach; ++j) {
                        const int32_t c = sizeof(C) == 4 ? word(q[g], j) : word(q[g], j / 2) >> 16 * (j & 1) & 0xffff;
                        all[j] += c;
                        before[j] += from + g * groups < me ? c : 0;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kEach; j += 4) {
                *reinterpret_cast<int4 *>(sums + group * 2 * bins + part * kEach + j) =
                    make_int4(all[j], all[j + 1], all[j + 2], all[j + 3]);
                *reinterpret_cast<int4 *>(sums + (group * 2 + 1) * bins + part * kEach + j) =
                    make_int4(before[j], before[j + 1], before[j + 2], before[j + 3]);
            }
        }
        __syncthreads();
        int32_t total = 0, mine_before = 0;
        if (bin < bins) {
#pragma unroll 8
            for (int g = 0; g < groups; ++g) {
                total += sums[g * 2 * bins + bin];
                mine_before += sums[(g * 2 + 1) * bins + bin];
            }
        }
        to_base[bin] = ranker.scan(total) + mine_before;      // (with a barrier, after which the table is free)
    }
    for (int64_t tile = first; tile < end; tile += kSortTile) {
        const int n_here = static_cast<int>(end - tile < kSortTile ? end - tile : kSortTile);
        if (tile > first) load(tile);
        const uint32_t run = ranker.place(key, at, n_here, a.shift, a.bits, pairs);
        for (int i = threadIdx.x; i < n_here; i += kSortThreads) {
            const uint2 v = pairs[i];
            const uint32_t d = v.x >> a.shift & mask;
            const int64_t to = to_base[d] + (i - static_cast<int>(local_base[d]));
            a.keys_out[to] = static_cast<int32_t>(v.x);
            a.at_out[to] = static_cast<int32_t>(v.y);
            if (!a.last) {
                const uint32_t place = static_cast<uint32_t>(to) / static_cast<uint32_t>(a.range) * bins +
                                       (v.x >> (a.shift + a.bits) & mask);
                if constexpr (sizeof(C) == 4)
                    atomicAdd(static_cast<uint32_t *>(a.next) + place, 1u);
                else
                    atomicAdd(static_cast<uint32_t *>(a.next) + place / 2, 1u << 16 * (place & 1));
            }
        }
        __syncthreads();
        to_base[bin] += static_cast<int32_t>(run);
        __syncthreads();
    }
}

// -------------------------------------------------------------------- sums --

// A slot's rows are copied eight ahead of its sums (rows scattered over memory, bound
// by how many are in flight and by the instructions a row takes), a thread each 16
// bytes of columns.  131040 rows of 384 bf16 into 32768 rows: 27 to 29 us of 58 for the
// call, 4.3 TB/s read and written (floor of the call 22.3); of 192 fp16 into 24 rows 12.5
// of 20.7 (7.5); rows of 383 take 87 us.  Four rows ahead with five blocks an SM in place
// of four 60 and 21.4 us; six 64 and 22.1.
constexpr int kAhead = 8;              // rows that a thread has in flight

struct SumArgs {
    const char *grad;
    const int32_t *keys, *at;    // sorted
    char *out;
    float *part;                 // [pieces][2][width]: what reaches over a piece's ends
    int64_t n, pieces;
    int32_t n_rows;
    int width, cols;             // cols: threads of a row
    int each, piece;             // indices of a slot and of a block
    int64_t out_step;            // bytes from a tile's table to the next one's
    float scale;
};

template <typename P>
__device__ __forceinline__ void write_one(char *out, int64_t at, float v) {
    if constexpr (std::is_same<P, F32>::value)
        reinterpret_cast<float *>(out)[at] = v;
    else
        reinterpret_cast<uint16_t *>(out)[at] = static_cast<uint16_t>(P::from_f2(v, 0.f));
}

// A thread's columns of a row's part that a block takes, kV of them: neighbouring
// ones where rows are whole 16-byte chunks; else every cols-th of single FP32 values or
// pairs of 16-bit ones, so that neighbouring threads' copies of 4 bytes lie side by
// side.  Pairs of a row that starts between two words are cut from two words each.
template <typename E, typename P, bool kChunks>
struct RowPart {
    static constexpr int kV = 16 / kBytes<E>;
    static constexpr int kWords = kChunks || kV == 4 ? 4 : 8;    // of a slot
    int thread, cols, start, width;    // start: of the block's part

    __device__ RowPart(int t, int c, int slice, int w) : thread(t), cols(c), start(slice * c * kV), width(w) {}
    // from the part's start, of value i
    __device__ int offset(int i) const {
        return kChunks ? thread * kV + i : kV == 4 ? thread + i * cols : 2 * (thread + i / 2 * cols) + (i & 1);
    }
    __device__ int col(int i) const { return start + offset(i); }
    __device__ bool any() const { return col(0) < width; }

    // Copies of the thread's part of the row at `row` into its slot: words `step` bytes
    // apart, from ring on.  end: of the tensor.
    __device__ void fetch(const char *row, const char *end, uint32_t ring, uint32_t step) const {
        if constexpr (kChunks) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring), "l"(row + col(0) * kBytes<E>) : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = col(kV == 4 ? i : 2 * i);
                if (at >= width) break;
                const char *p = row + at * kBytes<E>;
                if constexpr (kV == 4) {
                    copy_word(ring + i * step, p, 4);
                } else if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
                    copy_word(ring + 2 * i * step, p, end - p < 4 ? 2 : 4);
                } else {
                    copy_word(ring + 2 * i * step, p - 2, 4);
                    if (at + 1 < width) copy_word(ring + (2 * i + 1) * step, p + 2, end - p < 6 ? 2 : 4);
                }
            }
        }
    }
    __device__ static void copy_word(uint32_t to, const char *from, int bytes) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    }
    // What fetch() copied of that row, widened.
    __device__ void take(const char *row, uint32_t ring, uint32_t step, float2 (&v)[kV / 2]) const {
        if constexpr (kChunks) {
            uint4 q;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(ring) : "memory");
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) {
                if constexpr (kV == 4)
                    v[i] = make_float2(__uint_as_float(word(q, 2 * i)), __uint_as_float(word(q, 2 * i + 1)));
                else
                    v[i] = E::to_f2(word(q, i));
            }
        } else if constexpr (kV == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[i] = make_float2(__uint_as_float(load_word(ring + 2 * i * step)), __uint_as_float(load_word(ring + (2 * i + 1) * step)));
        } else {
            // columns are even, so all pairs of a row lie alike
            const bool between = (reinterpret_cast<uintptr_t>(row) & 2) != 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t low = load_word(ring + 2 * i * step);
                v[i] = E::to_f2(between ? __funnelshift_r(low, load_word(ring + (2 * i + 1) * step), 16) : low);
            }
        }
    }
    __device__ static uint32_t load_word(uint32_t at) {
        uint32_t w;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
        return w;
    }
    __device__ void store(char *row, const float (&v)[kV]) const {
        if constexpr (kChunks) {
            store_values<P, kV>(row + col(0) * kBytes<P>, v);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (col(i) < width) write_one<P>(row, col(i), v[i]);
        }
    }
};

// The first of [from, to) that is so, where all behind it are; `to` for none.
template <typename F>
__device__ __forceinline__ int first_of(int from, int to, F so) {
    while (from < to) {
        const int middle = (from + to) / 2;
        if (so(middle)) to = middle; else from = middle + 1;
    }
    return from;
}

// How a block lays out its shared memory for sums: slots of rows on their way, 16 or
// 32 bytes a thread, kAhead or half as many; then [slots][2][wide] sums of the slots' ends.
template <typename E, bool kChunks>
struct SumLayout {
    static constexpr int kWords = RowPart<E, E, kChunks>::kWords;
    static constexpr int kDeep = kWords == 8 ? kAhead / 2 : kAhead;
    __host__ __device__ static constexpr int ring_bytes(int threads) { return kDeep * threads * kWords * 4; }
};

// The sums of `count` tokens (row, position) in their rows' order, `each` by each to
// the block's slots: runs that end inside a slot are written, the others' parts left in
// head (of a run that began before the slot) and tail (of one that began in it).
// tokens[-1] and tokens[count] are not of the same row as a run that is to end there.
template <typename E, typename P, bool kChunks, int kThreads>
__device__ void sum_slots(const SumArgs &a, const RowPart<E, P, kChunks> &part, const int2 *tokens, int count, int slot,
                          int each, uint32_t ring, float *head, float *tail) {
    using Part = RowPart<E, P, kChunks>;
    constexpr int kV = Part::kV, kDeep = SumLayout<E, kChunks>::kDeep;
    // slots: [deep][words][threads], or 16 bytes a thread
    constexpr uint32_t kStep = kThreads * 4, kRingStep = kThreads * Part::kWords * 4;
    const int t0 = slot * each, mine_count = count - t0 < each ? count - t0 : each;
    if (mine_count <= 0 || !part.any()) return;
    const uint32_t row_bytes = static_cast<uint32_t>(a.width) * kBytes<E>, out_bytes = static_cast<uint32_t>(a.width) * kBytes<P>;
    const char *end = a.grad + a.n * row_bytes;
    const int2 *mine = tokens + t0;
    const int wide = a.cols * kV;
    float2 acc[kV / 2];
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) acc[i] = make_float2(0.f, 0.f);
    int32_t cur = mine[0].x;
    bool open = mine[-1].x == cur;    // the run began before this slot
    auto flush = [&](float *place) {
        if (place) {
#pragma unroll
            for (int i = 0; i < kV; ++i) place[slot * wide + part.offset(i)] = i & 1 ? acc[i / 2].y : acc[i / 2].x;
        } else {
            float v[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) v[i] = (i & 1 ? acc[i / 2].y : acc[i / 2].x) * a.scale;
            part.store(a.out + static_cast<int64_t>(cur) * out_bytes, v);
        }
    };
    int2 coming[kDeep];         // rows on their way
    auto row_at = [&](int32_t at) { return a.grad + static_cast<uint64_t>(static_cast<uint32_t>(at)) * row_bytes; };
    auto fetch = [&](int t, int j) {
        if (t < mine_count) {
            coming[j] = mine[t];
            part.fetch(row_at(coming[j].y), end, ring + j * kRingStep, kStep);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < kDeep; ++j) fetch(j, j);
    for (int t = 0; t < mine_count; t += kDeep) {
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            cp_async_wait<kDeep - 1>();
            if (t + j < mine_count) {
                float2 v[kV / 2];
                part.take(row_at(coming[j].y), ring + j * kRingStep, kStep, v);
                if (coming[j].x != cur) {
                    flush(open ? head : nullptr);
                    open = false;
                    cur = coming[j].x;
#pragma unroll
                    for (int i = 0; i < kV / 2; ++i) acc[i] = v[i];
                } else {
#pragma unroll
                    for (int i = 0; i < kV / 2; ++i) acc[i] = __fadd2_rn(acc[i], v[i]);
                }
            }
            fetch(t + j + kDeep, j);
        }
    }
    cp_async_wait<0>();
    flush(open ? head : mine[mine_count].x == cur ? tail : nullptr);
}

// The slots' ends, in their order, value f of the block's part of a row.  A run that
// began before the tokens, or goes on behind them, is left in `left` ([2][width]).
template <typename P>
__device__ void join_slots(const SumArgs &a, const int2 *tokens, int count, int slots, int each, const float *head,
                           const float *tail, int wide, int f, int c, float *left) {
    float run = 0.f;
    bool before = tokens[-1].x == tokens[0].x;      // the open run began before them
    for (int s = 0; s * each < count; ++s) {
        const int b = s * each, e = count - b < each ? count : b + each;
        const int32_t key = tokens[b].x, last = tokens[e - 1].x;
        const bool on = tokens[e].x == last;        // the slot's last run goes on behind it
        if (tokens[b - 1].x == key) {
            run += head[s * wide + f];
            if (on && last == key) continue;
            if (before) left[c] = run;
            else write_one<P>(a.out, key * static_cast<int64_t>(a.width) + c, run * a.scale);
            before = false;
            run = 0.f;
        }
        if (on) run = tail[s * wide + f];
    }
    if (tokens[count].x == tokens[count - 1].x) left[(before ? 0 : a.width) + c] = run;
}

// A block takes a piece of the sorted order.  E: grad's format, P: the table's
// gradient's.
template <typename E, typename P, bool kChunks>
__global__ void __launch_bounds__(kSumThreads) sum_runs(const SumArgs a) {
    extern __shared__ __align__(16) char memory[];
    using Layout = SumLayout<E, kChunks>;
    constexpr int kV = 16 / kBytes<E>;
    const int thread = threadIdx.x, slot = thread / a.cols, col_thread = thread - slot * a.cols;
    const int slots = a.piece / a.each, wide = a.cols * kV;
    const uint32_t ring = shared_address(memory) + thread * (kChunks ? 16 : 4);
    int2 *tokens = reinterpret_cast<int2 *>(memory + Layout::ring_bytes(kSumThreads)) + 1;    // [-1] ... [piece]
    float *head = reinterpret_cast<float *>(tokens + a.piece + 1), *tail = head + slots * wide;
    pdl_prologue();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * a.piece;
    // no row: before the first index, and behind the last that names one
    for (int i = thread - 1; i <= a.piece; i += blockDim.x) {
        const int64_t t = first + i;
        const int2 token = t >= 0 && t < a.n ? make_int2(__ldcg(a.keys + t), __ldcg(a.at + t)) : make_int2(a.n_rows, 0);
        tokens[i] = token.x < a.n_rows ? token : make_int2(-1, 0);
    }
    __syncthreads();
    // sorted, so those that name a row come first
    const int count = first_of(0, a.piece, [&](int i) { return tokens[i].x < 0; });
    if (count == 0) return;
    const RowPart<E, P, kChunks> part(col_thread, a.cols, blockIdx.y, a.width);
    if (slot < slots) sum_slots<E, P, kChunks, kSumThreads>(a, part, tokens, count, slot, a.each, ring, head, tail);
    __syncthreads();
    // what reaches over the piece's ends is for the last launch
    for (int f = thread; f < wide; f += blockDim.x) {
        const int c = blockIdx.y * wide + f;
        if (c >= a.width) break;
        join_slots<P>(a, tokens, count, slots, a.each, head, tail, wide, f, c, a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.width);
    }
}

// Runs that go over the end of the piece they began in: the sums of the pieces that
// each reaches into.  A block looks through some of the pieces for such beginnings.
// A run of a few pieces is a warp's, 128 columns at a time; a long one the block's,
// whose groups of threads add every groups-th piece's sums, and then the groups'.  (Run
// by the last of a run's blocks inside the sums' launch, told by counters, it cost more
// than this launch does: 22 us in place of 12.5 + 6.4 for 24 rows of 192.)
__device__ __forceinline__ float4 plus(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
// Four columns of row `row` of the pieces' sums.
__device__ __forceinline__ float4 part_of(const SumArgs &a, int64_t row, int quad) {
    const float *p = a.part + row * a.width + quad * 4;
    if ((a.width & 3) == 0) return __ldcg(reinterpret_cast<const float4 *>(p));
    const int left = a.width - quad * 4;
    return make_float4(__ldcg(p), left > 1 ? __ldcg(p + 1) : 0.f, left > 2 ? __ldcg(p + 2) : 0.f, left > 3 ? __ldcg(p + 3) : 0.f);
}
template <typename P>
__device__ __forceinline__ void write_quad(const SumArgs &a, int32_t k, int quad, float4 s) {
    const int64_t at = k * static_cast<int64_t>(a.width) + quad * 4;
    const int left = a.width - quad * 4;
    write_one<P>(a.out, at, s.x * a.scale);
    if (left > 1) write_one<P>(a.out, at + 1, s.y * a.scale);
    if (left > 2) write_one<P>(a.out, at + 2, s.z * a.scale);
    if (left > 3) write_one<P>(a.out, at + 3, s.w * a.scale);
}
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;
constexpr int kLongRun = 24;           // pieces behind the first

// The first of [from, to) that is so, where all behind it are, by a warp; `to` for none.
template <typename F>
__device__ __forceinline__ int64_t first_piece(int64_t from, int64_t to, F so) {
    const int lane = threadIdx.x & 31;
    while (from < to) {
        const int64_t part = (to - from + 31) / 32, i = from + (lane + 1) * part - 1;
        const int below = 32 - __popc(__ballot_sync(0xffffffffu, i >= to || so(i < to ? i : to - 1)));
        from += below * part;
        to = from + part - 1 < to ? from + part - 1 : to;
    }
    return from;
}

template <typename P>
__global__ void __launch_bounds__(kJoinThreads) join_runs(const SumArgs a) {
    __shared__ float4 sums[kJoinThreads];
    __shared__ int found[kJoinThreads], pieces[kJoinThreads], n_found;
    const int thread = threadIdx.x, lane = thread & 31, warp = thread >> 5;
    bool waited = false;
    // does the run of piece c's last index go on into the next, having begun in c?
    auto begins = [&](int64_t c) {
        const int64_t end = (c + 1) * a.piece;
        if (c >= a.pieces || end >= a.n) return false;
        const int32_t k = __ldcg(a.keys + end), last = __ldcg(a.keys + end - 1);
        const int32_t before = c > 0 ? __ldcg(a.keys + c * a.piece - 1) : a.n_rows;
        return k < a.n_rows && last == k && before != k;
    };
    for (int64_t round = 0; round * kJoinThreads * gridDim.x < a.pieces; ++round) {
        if (thread == 0) n_found = 0;
        __syncthreads();
        const int64_t c = (round * kJoinThreads + thread) * gridDim.x + blockIdx.x;
        if (begins(c)) found[atomicAdd(&n_found, 1)] = static_cast<int>(c);
        __syncthreads();
        const int runs = n_found;
        // pieces behind the first that each run reaches into
        for (int f = warp; f < runs; f += kJoinWarps) {
            const int64_t c0 = found[f];
            const int32_t k = __ldcg(a.keys + (c0 + 1) * a.piece);
            // up to before the first piece that begins behind it
            const int64_t behind = first_piece(c0 + 2, a.pieces, [&](int64_t p) { return __ldcg(a.keys + p * a.piece) > k; });
            const int more = static_cast<int>(behind - 1 - c0);
            if (lane == 0) pieces[f] = more;
        }
        // This launch may start while the sums' blocks end; those have waited for the
        // sort, so its order is there to be read, and only their parts are waited for.
        if (!waited) pdl_prologue();
        waited = true;
        __syncthreads();
        const int quads = (a.width + 3) / 4;     // four columns each
        const int blocks = (quads + 31) / 32;
        for (int t = warp; t < runs * blocks; t += kJoinWarps) {
            const int f = t / blocks, more = pieces[f], quad = (t - f * blocks) * 32 + lane;
            if (more > kLongRun || quad >= quads) continue;
            const int64_t c0 = found[f];
            const int32_t k = __ldcg(a.keys + (c0 + 1) * a.piece);
            float4 s = part_of(a, 2 * c0 + 1, quad);
#pragma unroll 8
            for (int p = 1; p <= more; ++p) s = plus(s, part_of(a, 2 * (c0 + p), quad));
            write_quad<P>(a, k, quad, s);
        }
        const int wide = quads < 512 ? quads : 512, groups = kJoinThreads / wide;
        const int group = thread / wide, lead = thread - group * wide;
        for (int f = 0; f < runs; ++f) {
            const int more = pieces[f];
            if (more <= kLongRun) continue;
            const int64_t c0 = found[f];
            const int32_t k = __ldcg(a.keys + (c0 + 1) * a.piece);
            for (int from = 0; from < quads; from += wide) {
                const int quad = from + lead;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                if (quad < quads && group < groups) {
                    if (group == 0) s = part_of(a, 2 * c0 + 1, quad);
#pragma unroll 8
                    for (int p = 1 + group; p <= more; p += groups) s = plus(s, part_of(a, 2 * (c0 + p), quad));
                }
                sums[thread] = s;
                __syncthreads();
                // the groups' sums, halved as often as it takes
                for (int g = groups; g > 1; g = (g + 1) / 2) {
                    const int half = (g + 1) / 2;
                    if (group + half < g) sums[thread] = plus(sums[thread], sums[thread + half * wide]);
                    __syncthreads();
                }
                if (group == 0 && quad < quads) write_quad<P>(a, k, quad, sums[thread]);
                __syncthreads();
            }
        }
    }
}

// ------------------------------------------------- few indices, few table rows --

// Where a block can sort all indices, every block does, and takes the runs that begin
// in its share of the order, whole ones, so that nothing is left for another launch:
// one in place of five.  The rows that no index names are a share of the table's rows,
// found with a bit for each in shared memory.  180 indices into 366 rows of 192 take
// 7.1 us so, 12.4 in five launches; 2048 into 300 rows 10.4 and 13.3, but all of them
// into one row, which is one block's, 21 and 13: half as many are even there.  A block
// takes 1 KB of a row's columns, so that wide rows are several blocks' whatever rows are
// named: 1024 indices into one row of 2048 and 32768 FP32 take 19 and 32 us so, 108 and 1660
// where a block takes all columns, 43 and 740 in five launches; into 300 rows, evenly, 9
// and 38, so 9 and 60, so 13 and 64.
//
// Where the table has few rows, a block does the same with a tile of neighbouring
// indices, whose gradients are one run of bytes (which L2 is asked for while the block
// sorts), into a table of its own; a second launch adds the blocks' tables.  131040
// indices into 24 rows of 192 fp16 take 18.8 us so, 20.6 by pieces of a sorted order,
// into one row 17 and 44; into 48 rows, with fewer and larger tiles, 24 and 23.
template <typename E, typename P, bool kChunks>
__global__ void __launch_bounds__(kSortThreads) sum_tile(const SumArgs args, const int32_t *idx, int passes, int bits,
                                                         int range) {
    extern __shared__ __align__(16) char memory[];
    __shared__ int32_t warp_sums[kSortWarps];
    __shared__ uint32_t base[kBins];
    using Layout = SumLayout<E, kChunks>;
    constexpr int kV = 16 / kBytes<E>;
    static_assert(Layout::ring_bytes(kSortThreads) <= Ranker::kTableBytes, "the ring takes the sort's tables' place");
    // range: of a block's tile; 0 where every block takes all indices
    const bool tiled = range > 0;
    SumArgs a = args;
    a.out += blockIdx.x * args.out_step;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * range;
    const int n = static_cast<int>(tiled && a.n - first > range ? range : a.n - first), thread = threadIdx.x;
    int2 *tokens = reinterpret_cast<int2 *>(memory) + 2;      // [-1] ... [n]
    char *tables = memory + ((tiled ? range : static_cast<int>(a.n)) + 5) / 2 * 16;
    uint2 *pairs = reinterpret_cast<uint2 *>(tokens);
    const Ranker ranker(tables, warp_sums, base);
    ranker.clear(1 << bits);
    pdl_prologue();
    uint32_t key[kRounds], at[kRounds];
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
        const int i = Ranker::first() + 32 * j;
        key[j] = at[j] = 0u;
        if (i < n) {
            const int32_t k = __ldg(idx + first + i);
            key[j] = static_cast<uint32_t>(k >= 0 && k < a.n_rows ? k : a.n_rows), at[j] = static_cast<uint32_t>(first + i);
            if ((k < -1 || k >= a.n_rows) && (tiled || blockIdx.x + blockIdx.y == 0)) atomicOr(&g_embedding_error, 1u);
        }
    }
    if (tiled) {
        // the tile's gradients, a piece a thread
        constexpr int kPiece = 16 << 10;
        const int64_t row_bytes = static_cast<int64_t>(a.width) * kBytes<E>;
        const uintptr_t from = (reinterpret_cast<uintptr_t>(a.grad) + first * row_bytes + 15) & ~uintptr_t(15);
        const uintptr_t to = (reinterpret_cast<uintptr_t>(a.grad) + (first + n) * row_bytes) & ~uintptr_t(15);
        for (uintptr_t p = from + static_cast<uintptr_t>(thread) * kPiece; p < to; p += static_cast<uintptr_t>(kSortThreads) * kPiece) {
            const uint32_t bytes = to - p < kPiece ? static_cast<uint32_t>(to - p) : kPiece;
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
        }
    }
    for (int pass = 0;;) {
        ranker.place(key, at, n, pass * bits, bits, pairs);
        if (++pass == passes) break;
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            const int i = Ranker::first() + 32 * j;
            if (i < n) key[j] = pairs[i].x, at[j] = pairs[i].y;
        }
    }
    const int named = first_of(0, n, [&](int i) { return tokens[i].x >= a.n_rows; });
    __syncthreads();
    if (thread == 0) tokens[-1].x = tokens[named].x = -1;
    __syncthreads();

    // the runs that begin in this block's share of the order
    const int blocks = tiled ? 1 : gridDim.x, block = tiled ? 0 : blockIdx.x;
    auto begin = [&](int64_t b) {
        const int i = static_cast<int>(b * named / blocks);
        if (i == 0 || i >= named || tokens[i].x != tokens[i - 1].x) return i;
        const int32_t k = tokens[i].x;
        return first_of(i, named, [&](int t) { return tokens[t].x > k; });
    };
    const int from = begin(block), count = begin(block + 1) - from;
    if (count > 0) {
        const int slots = kSortThreads / a.cols < kMostSlots ? kSortThreads / a.cols : kMostSlots;
        const int slot = thread / a.cols, wide = a.cols * kV;
        const int each = (count + slots - 1) / slots;
        const uint32_t ring = shared_address(tables) + thread * (kChunks ? 16 : 4);
        float *head = reinterpret_cast<float *>(tables + Ranker::kTableBytes), *tail = head + slots * wide;
        for (int slice = blockIdx.y; slice * wide < a.width; slice += gridDim.y) {
            const RowPart<E, P, kChunks> part(thread - slot * a.cols, a.cols, slice, a.width);
            if (slot < slots)
                sum_slots<E, P, kChunks, kSortThreads>(a, part, tokens + from, count, slot, each, ring, head, tail);
            __syncthreads();
            for (int f = thread; f < wide; f += kSortThreads) {
                const int c = slice * wide + f;
                if (c >= a.width) break;
                join_slots<P>(a, tokens + from, count, slots, each, head, tail, wide, f, c, nullptr);
            }
            __syncthreads();
        }
    }

    // the zeros: a bit for each of some rows, set where an index names it
    constexpr int64_t kBits = kBins * 32;
    const int shares = blocks * gridDim.y, share = block + blocks * blockIdx.y;
    const int64_t row0 = static_cast<int64_t>(a.n_rows) * share / shares, row1 = static_cast<int64_t>(a.n_rows) * (share + 1) / shares;
    const int lane = thread & 31, warp = thread >> 5;
    int lanes = 1;      // of a row
    while (lanes < 32 && lanes < (kChunks ? a.width * kBytes<P> / 16 : a.width)) lanes *= 2;
    const int rows_at_once = 32 / lanes;
    for (int64_t r0 = row0; r0 < row1; r0 += kBits) {
        const int64_t r1 = r0 + kBits < row1 ? r0 + kBits : row1;
        __syncthreads();
        base[thread] = 0u;
        __syncthreads();
        const int lo = first_of(0, named, [&](int i) { return tokens[i].x >= r0; });
        const int hi = first_of(lo, named, [&](int i) { return tokens[i].x >= r1; });
        for (int i = lo + thread; i < hi; i += kSortThreads) {
            const int bit = static_cast<int>(tokens[i].x - r0);
            atomicOr(&base[bit / 32], 1u << bit % 32);
        }
        __syncthreads();
        for (int64_t r = r0 + warp * rows_at_once + lane / lanes; r < r1; r += kSortWarps * rows_at_once) {
            const int bit = static_cast<int>(r - r0);
            if (base[bit / 32] >> bit % 32 & 1u) continue;
            char *row = a.out + r * a.width * kBytes<P>;
            if constexpr (kChunks) {
                for (int i = lane % lanes; i < a.width * kBytes<P> / 16; i += lanes) st_stream(row + 16 * i, make_uint4(0u, 0u, 0u, 0u));
            } else {
                for (int i = lane % lanes; i < a.width; i += lanes) write_one<P>(row, i, 0.f);
            }
        }
    }
}

// The blocks' tables added up: 32 values a block, 16 threads a value.
template <typename P>
__global__ void __launch_bounds__(512) add_tables(const float *part, int blocks, int64_t values, float scale, char *out) {
    __shared__ float sums[16][33];
    pdl_prologue();
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int64_t v = blockIdx.x * 32ll + lane;
    float s = 0.f;
    if (v < values) {
#pragma unroll 10
        for (int b = group; b < blocks; b += 16) s += __ldcg(part + b * values + v);
    }
    sums[group][lane] = s;
    __syncthreads();
    if (group > 0 || v >= values) return;
#pragma unroll
    for (int g = 1; g < 16; ++g) s += sums[g][lane];
    write_one<P>(out, v, s * scale);
}

__global__ void __launch_bounds__(256) fill_zeros(char *p, int64_t n, int bytes) {
    pdl_prologue();
    write_zeros(p, n, bytes, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, gridDim.x * 256ll);
}

// -------------------------------------------------------------------- host --

int64_t bytes_of(wgs_dtype d) { return d == WGS_F32 ? 4 : 2; }
bool dtype_ok(wgs_dtype d) { return d == WGS_F32 || d == WGS_F16 || d == WGS_BF16; }
bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool sizes_ok(int64_t n_idx, int64_t n_rows) {
    return n_idx >= 0 && n_rows >= 0 && n_idx < INT32_MAX && n_rows < INT32_MAX;
}

template <typename E, typename P, bool kChunks>
wgs_status run_sums(const SumArgs &a, const Plan &z, int sms, cudaStream_t stream) {
    constexpr int kV = 16 / kBytes<E>;
    using Layout = SumLayout<E, kChunks>;
    const int smem = Layout::ring_bytes(kSumThreads) + 8 * (z.piece + 2) + 8 * z.slots * z.cols * kV;
    static_assert(kMostPiece == 64 * kMostSlots &&
                      Layout::ring_bytes(kSumThreads) + 8 * (kMostPiece + 2) + 8 * kSumThreads * kV <= 66 << 10,
                  "shared memory of a block");
    auto kernel = sum_runs<E, P, kChunks>;
    // (as the layer norm's)
    if (smem > 47 << 10 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 66 << 10) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    const wgs_status st = launch(kernel, dim3(static_cast<unsigned>(z.pieces), z.slices), dim3(z.cols * z.slots),
                                 static_cast<size_t>(smem), stream, a);
    if (st != WGS_OK || z.pieces == 1) return st;
    const int64_t blocks = z.pieces < sms ? z.pieces : sms;
    return launch(join_runs<P>, dim3(static_cast<unsigned>(blocks)), dim3(kJoinThreads), 0, stream, a);
}

// Few indices, P the table's gradient's format; or a tile a block, P FP32.
template <typename E, typename P, bool kChunks>
wgs_status run_tile(const SumArgs &a, const int32_t *idx, const Plan &z, int sms, cudaStream_t stream) {
    constexpr int kV = 16 / kBytes<E>;
    const int slots = kSortThreads / z.cols < kMostSlots ? kSortThreads / z.cols : kMostSlots;
    const int tokens = ((z.tile ? z.tile : static_cast<int>(a.n)) + 5) / 2 * 16;
    const int smem = tokens + Ranker::kTableBytes + 8 * slots * z.cols * kV;
    auto kernel = sum_tile<E, P, kChunks>;
    // (as the layer norm's)
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kSortTile + 5) / 2 * 16 + Ranker::kTableBytes + 8 * kSortThreads * kV) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    int64_t blocks = z.tile_blocks;
    if (z.few) {
        // an index a slot, or 8 KB of zeros a block, and an SM for each at most
        const int64_t bytes = static_cast<int64_t>(a.n_rows) * a.width * kBytes<P>, most = sms < z.slices ? 1 : sms / z.slices;
        blocks = ceil_div(a.n, slots);
        if (blocks < ceil_div(bytes, 8192 * z.slices)) blocks = ceil_div(bytes, 8192 * z.slices);
        if (blocks > most) blocks = most;
    }
    return launch(kernel, dim3(static_cast<unsigned>(blocks), z.few ? z.slices : 1), dim3(kSortThreads), static_cast<size_t>(smem), stream, a, idx,
                  z.passes, z.bits, z.tile);
}

template <typename E, typename P, bool kChunks>
wgs_status run_tiles(SumArgs a, const int32_t *idx, const Plan &z, int sms, cudaStream_t stream) {
    const int64_t values = static_cast<int64_t>(a.n_rows) * a.width;
    const float scale = a.scale;
    char *out = a.out;
    a.out = reinterpret_cast<char *>(a.part), a.out_step = 4 * values, a.scale = 1.f;
    const wgs_status st = run_tile<E, F32, kChunks>(a, idx, z, sms, stream);
    if (st != WGS_OK) return st;
    return launch(add_tables<P>, dim3(static_cast<unsigned>(ceil_div(values, 32))), dim3(512), 0, stream,
                  static_cast<const float *>(a.part), z.tile_blocks, values, scale, out);
}

// 16 bytes of gradient at a time where all rows, and those of the output, start
// on as many.
bool in_chunks(const void *grad, const void *out, int32_t width, int64_t eb, int64_t ob) {
    return aligned16(grad) && aligned16(out) && width * eb % 16 == 0 && width * ob % 16 == 0;
}

template <typename E>
wgs_status run_format(const SumArgs &a, const int32_t *idx, const Plan &z, bool chunks, bool p32, int sms,
                      cudaStream_t stream) {
    if (z.few && chunks)
        return p32 ? run_tile<E, F32, true>(a, idx, z, sms, stream) : run_tile<E, E, true>(a, idx, z, sms, stream);
    if (z.few)
        return p32 ? run_tile<E, F32, false>(a, idx, z, sms, stream) : run_tile<E, E, false>(a, idx, z, sms, stream);
    if (z.tile && chunks)
        return p32 ? run_tiles<E, F32, true>(a, idx, z, sms, stream) : run_tiles<E, E, true>(a, idx, z, sms, stream);
    if (z.tile)
        return p32 ? run_tiles<E, F32, false>(a, idx, z, sms, stream) : run_tiles<E, E, false>(a, idx, z, sms, stream);
    if (chunks) return p32 ? run_sums<E, F32, true>(a, z, sms, stream) : run_sums<E, E, true>(a, z, sms, stream);
    return p32 ? run_sums<E, F32, false>(a, z, sms, stream) : run_sums<E, E, false>(a, z, sms, stream);
}

// Sorts s.idx; s.keys and s.at are the order.  Zeros go to `bytes` bytes at `out`.
wgs_status sort_indices(SortArgs &s, const Plan &z, char *ws, char *out, int64_t bytes, int unit, int sms,
                        cudaStream_t stream) {
    s.range = z.range, s.blocks = z.sort_blocks, s.bits = z.bits, s.zero_unit = unit;
    const int64_t counts = 1ll * z.sort_blocks * z.count_bytes << z.bits;   // of a pass
    auto count = z.count_bytes == 2 ? sort_count<uint16_t> : sort_count<uint32_t>;
    auto order = z.count_bytes == 2 ? sort_place<uint16_t> : sort_place<uint32_t>;
    const int smem = kSortTile * 8 + Ranker::kTableBytes;
    // (as the layer norm's)
    if (cudaFuncSetAttribute(order, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    for (int p = -1; p < z.passes; ++p) {
        const ZeroShare share = zero_share(z, p, bytes, sms);
        s.zeros = out + share.first, s.zero_bytes = share.bytes;
        const dim3 grid(static_cast<unsigned>(s.blocks + share.blocks));
        const int q = p < 0 ? 0 : p;
        s.shift = q * z.bits, s.last = q + 1 == z.passes;
        s.counts = ws + z.counts + q * counts;
        s.next = ws + z.counts + (q + 1) * counts;
        s.clear_words = (z.passes - 1) * counts / 4;
        wgs_status st;
        if (p < 0) {
            st = launch(count, grid, dim3(kSortThreads), 0, stream, s);
        } else {
            s.keys_out = reinterpret_cast<int32_t *>(ws + z.keys[p & 1]);
            s.at_out = reinterpret_cast<int32_t *>(ws + z.at[p & 1]);
            st = launch(order, grid, dim3(kSortThreads), static_cast<size_t>(smem), stream, s);
            s.idx = nullptr, s.keys = s.keys_out, s.at = s.at_out;
        }
        if (st != WGS_OK) return st;
    }
    return WGS_OK;
}

template <typename T, typename E>
wgs_status run_lookup(LookupArgs a, int32_t width, int sms, cudaStream_t stream) {
    constexpr int kV = 16 / kBytes<T>;
    const bool chunks = width % kV == 0 && aligned16(a.table) && aligned_to(a.out, kV * kBytes<E>);
    a.row_chunks = static_cast<int>(ceil_div(width, kV)), a.width = width;
    const int64_t blocks = chunks ? ceil_div(a.n * a.row_chunks, kLookupThreads)
                                  : ceil_div(a.n * width, kLookupThreads * (16 / kBytes<E>));
    const int64_t most = static_cast<int64_t>(sms) * kLookupBlocksPerSm;
    return launch(chunks ? embedding_lookup<T, E> : embedding_lookup_ragged<T, E>,
                  dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(kLookupThreads), 0, stream, a);
}

}  // namespace

}  // namespace wgs

// As bias_mask_error_take, for the embedding's error word.
wgs_status wgs::embedding_error_take(unsigned int *seen, cudaStream_t stream) {
    static const unsigned int cleared = 0;
    if (cudaMemcpyFromSymbolAsync(seen, g_embedding_error, sizeof(*seen), 0, cudaMemcpyDeviceToHost,
                                  stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_embedding_error, &cleared, sizeof(cleared), 0,
                                cudaMemcpyHostToDevice, stream) != cudaSuccess) {
        cudaGetLastError();  // clear this thread's error
        return WGS_ERR_CUDA;
    }
    return WGS_OK;
}

using namespace wgs;

extern "C" wgs_status embedding(const void *table, const int32_t *idx, void *out, int64_t n_idx, int64_t n_rows,
                                int32_t width, float scale, wgs_dtype table_dtype, wgs_dtype dtype,
                                cudaStream_t stream) {
    if (!dtype_ok(dtype) || (table_dtype != WGS_F32 && table_dtype != dtype)) return WGS_ERR_DTYPE;
    if (width < 1 || width > kMaxWidth) return WGS_ERR_WIDTH;
    if (!sizes_ok(n_idx, n_rows)) return WGS_ERR_SHAPE;
    if (n_idx == 0) return WGS_OK;
    if (!idx || !out || (n_rows > 0 && !table)) return WGS_ERR_NULL;
    const int64_t tb = bytes_of(table_dtype), eb = bytes_of(dtype);
    if (!aligned_to(table, tb) || !aligned_to(out, eb) || !aligned4(idx)) return WGS_ERR_ALIGN;
    const int64_t bytes = n_idx * width * eb;
    if (overlap(out, bytes, table, n_rows * width * tb) || overlap(out, bytes, idx, n_idx * 4)) return WGS_ERR_ALIAS;
    DeviceInfo dev;
    const wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    LookupArgs a = {};
    a.table = static_cast<const char *>(table), a.idx = idx, a.out = static_cast<char *>(out);
    a.n = n_idx, a.n_rows = n_rows, a.scale = scale;
    auto go = dtype == WGS_F32   ? run_lookup<F32, F32>
              : dtype == WGS_F16 ? (table_dtype == WGS_F32 ? run_lookup<F32, Fp16> : run_lookup<Fp16, Fp16>)
                                 : (table_dtype == WGS_F32 ? run_lookup<F32, Bf16> : run_lookup<Bf16, Bf16>);
    return go(a, width, dev.sm_count, stream);
}

extern "C" size_t wgs_embedding_bwd_workspace_bytes(int64_t n_idx, int64_t n_rows, int32_t width) {
    if (width < 1 || width > kMaxWidth || !sizes_ok(n_idx, n_rows)) return 0;
    return static_cast<size_t>(workspace_of(n_idx, n_rows, width));
}

extern "C" wgs_status embedding_bwd(const void *grad, const int32_t *idx, void *grad_table, void *workspace,
                                    size_t workspace_bytes, int64_t n_idx, int64_t n_rows, int32_t width,
                                    float scale, wgs_dtype dtype, wgs_dtype table_dtype, cudaStream_t stream) {
    if (!dtype_ok(dtype) || (table_dtype != WGS_F32 && table_dtype != dtype)) return WGS_ERR_DTYPE;
    if (width < 1 || width > kMaxWidth) return WGS_ERR_WIDTH;
    if (!sizes_ok(n_idx, n_rows)) return WGS_ERR_SHAPE;
    if (n_rows == 0 && n_idx == 0) return WGS_OK;
    if ((n_rows > 0 && !grad_table) || (n_idx > 0 && (!grad || !idx || !workspace))) return WGS_ERR_NULL;
    const int64_t need = workspace_of(n_idx, n_rows, width);
    if (n_idx > 0 && workspace_bytes < static_cast<size_t>(need)) return WGS_ERR_SHAPE;
    const int64_t eb = bytes_of(dtype), tb = bytes_of(table_dtype);
    if (!aligned_to(grad, eb) || !aligned_to(grad_table, tb) || !aligned4(idx) || !aligned16(workspace))
        return WGS_ERR_ALIGN;
    const int64_t gbytes = n_idx * width * eb, tbytes = n_rows * width * tb;
    if (overlap(grad_table, tbytes, grad, gbytes) || overlap(grad_table, tbytes, idx, n_idx * 4)) return WGS_ERR_ALIAS;
    if (n_idx > 0 && (overlap(workspace, need, grad, gbytes) || overlap(workspace, need, idx, n_idx * 4) ||
                      overlap(workspace, need, grad_table, tbytes)))
        return WGS_ERR_ALIAS;
    DeviceInfo dev;
    wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    const bool chunks = in_chunks(grad, grad_table, width, eb, tb);
    const Plan z = plan_of(n_idx, n_rows, width, static_cast<int>(16 / eb));
    if (tbytes > 0 && n_idx == 0) {
        const int64_t blocks = ceil_div(ceil_div(tbytes, 16), 256 * 8);
        const int64_t most = 8ll * dev.sm_count;
        st = launch(fill_zeros, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, stream,
                    static_cast<char *>(grad_table), tbytes, static_cast<int>(tb));
    }
    if (st != WGS_OK || n_idx == 0) return st;
    char *ws = static_cast<char *>(workspace);
    SortArgs s = {};
    s.idx = idx, s.n = n_idx, s.n_rows = static_cast<int32_t>(n_rows);
    if (!z.few && !z.tile)
        st = sort_indices(s, z, ws, static_cast<char *>(grad_table), tbytes, static_cast<int>(tb), dev.sm_count, stream);
    if (st != WGS_OK || (n_rows == 0 && !z.few)) return st;
    SumArgs a = {};
    a.grad = static_cast<const char *>(grad), a.keys = s.keys, a.at = s.at;
    a.out = static_cast<char *>(grad_table), a.part = reinterpret_cast<float *>(ws + z.part);
    a.n = n_idx, a.pieces = z.pieces, a.n_rows = static_cast<int32_t>(n_rows), a.width = width, a.cols = z.cols;
    a.each = z.each, a.piece = z.piece, a.scale = scale;
    const bool p32 = table_dtype == WGS_F32;
    if (dtype == WGS_F32) return run_format<F32>(a, idx, z, chunks, true, dev.sm_count, stream);
    if (dtype == WGS_F16) return run_format<Fp16>(a, idx, z, chunks, p32, dev.sm_count, stream);
    return run_format<Bf16>(a, idx, z, chunks, p32, dev.sm_count, stream);
}
