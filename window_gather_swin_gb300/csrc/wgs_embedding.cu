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
// most of the indices, and the order of additions is fixed.
#include <type_traits>

#include "wgs_common.cuh"

namespace wgs {

namespace {

// Set (never cleared by a kernel) when an index lies outside [-1, n_rows); read
// and cleared by wgs_check_error.
__device__ unsigned int g_embedding_error;

struct F32 {};

constexpr int kMaxWidth = 32768;

template <typename E>
constexpr int kBytes = std::is_same<E, F32>::value ? 4 : 2;

// kV neighbouring values at p, widened, and rounded back.
template <typename E, int kV>
__device__ __forceinline__ void load_values(const char *p, float (&v)[kV]) {
    if constexpr (kV == 1) {
        if constexpr (std::is_same<E, F32>::value)
            v[0] = __ldcg(reinterpret_cast<const float *>(p));
        else
            v[0] = E::to_f2(__ldcg(reinterpret_cast<const uint16_t *>(p))).x;
    } else if constexpr (std::is_same<E, F32>::value) {
#pragma unroll
        for (int i = 0; i < kV / 4; ++i) {
            const uint4 q = ld_stream(p + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(word(q, j));
        }
    } else {
        static_assert(kV == 8, "16 bytes of 16-bit values");
        const uint4 q = ld_stream(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = E::to_f2(word(q, j));
            v[2 * j] = f.x, v[2 * j + 1] = f.y;
        }
    }
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

// Chunks of the output, those of a block's threads side by side, are taken in steps
// of the whole grid; a thread has the table's chunks of its next step on their way
// into slots of its own in shared memory, and the indices of the one after that in
// registers, so that neither the index nor the row that it names is waited for at
// full length.  Rows that are not whole chunks are taken in parts of as many single
// elements, every row_chunks-th of the row.
constexpr int kLookupThreads = 256;
constexpr int kLookupChunks = 2;       // of a thread in a step
constexpr int kLookupBlocksPerSm = 5;

struct LookupArgs {
    const char *table;
    const int32_t *idx;
    char *out;
    int64_t n, n_rows;
    int row_chunks, width;
    float scale;
};

// T: the table's format, E: the output's.
template <typename T, typename E, bool kChunks>
__global__ void __launch_bounds__(kLookupThreads, kLookupBlocksPerSm) embedding_lookup(const LookupArgs a) {
    constexpr int kV = 16 / kBytes<E>, kIn = kV * kBytes<T>, kOut = 16;    // values, bytes of a chunk
    constexpr int kSlots = kIn / 16;
    __shared__ uint4 slots[kChunks ? 2 : 1][kChunks ? kLookupChunks * kSlots : 1][kChunks ? kLookupThreads : 1];
    pdl_prologue();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kLookupThreads * kLookupChunks;
    const int64_t row_step = step / a.row_chunks;
    const int col_step = static_cast<int>(step - row_step * a.row_chunks);
    int64_t row[kLookupChunks];
    int col[kLookupChunks];
#pragma unroll
    for (int j = 0; j < kLookupChunks; ++j) {
        const int64_t at = (static_cast<int64_t>(blockIdx.x) * kLookupChunks + j) * kLookupThreads + threadIdx.x;
        row[j] = at / a.row_chunks;
        col[j] = static_cast<int>(at - row[j] * a.row_chunks);
    }
    auto advance = [&](int64_t &r, int &c) {
        r += row_step, c += col_step;
        if (c >= a.row_chunks) c -= a.row_chunks, ++r;
    };
    // the table row of a chunk's index: -1 for none
    auto index = [&](int64_t r, int c) {
        if (r >= a.n) return -1;
        const int32_t k = __ldg(a.idx + r);
        if (k >= 0 && k < a.n_rows) return k;
        if (k != -1 && c == 0) atomicOr(&g_embedding_error, 1u);
        return -1;
    };
    auto fetch = [&](int s, const int32_t (&from)[kLookupChunks], const int (&c)[kLookupChunks]) {
        if constexpr (kChunks) {
#pragma unroll
            for (int j = 0; j < kLookupChunks; ++j)
                if (from[j] >= 0) {
                    const char *p = a.table + (static_cast<int64_t>(from[j]) * a.row_chunks + c[j]) * kIn;
#pragma unroll
                    for (int i = 0; i < kSlots; ++i) cp_async16_ca(&slots[s][j * kSlots + i][threadIdx.x], p + 16 * i);
                }
            cp_async_commit();
        }
    };
    int64_t next_row[kLookupChunks];
    int next_col[kLookupChunks];
    int32_t now[kLookupChunks], next[kLookupChunks];
#pragma unroll
    for (int j = 0; j < kLookupChunks; ++j) {
        now[j] = index(row[j], col[j]);
        next_row[j] = row[j], next_col[j] = col[j];
        advance(next_row[j], next_col[j]);
        next[j] = index(next_row[j], next_col[j]);
    }
    fetch(0, now, col);
    for (int s = 0; row[0] < a.n; s ^= 1) {
        fetch(s ^ 1, next, next_col);
        int32_t later[kLookupChunks];
        int64_t later_row[kLookupChunks];
        int later_col[kLookupChunks];
#pragma unroll
        for (int j = 0; j < kLookupChunks; ++j) {
            later_row[j] = next_row[j], later_col[j] = next_col[j];
            advance(later_row[j], later_col[j]);
            later[j] = index(later_row[j], later_col[j]);
        }
        if constexpr (kChunks) cp_async_wait<1>();
#pragma unroll
        for (int j = 0; j < kLookupChunks; ++j) {
            if (row[j] >= a.n) continue;
            float v[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) v[i] = 0.f;
            if (now[j] >= 0) {
                if constexpr (kChunks) {
#pragma unroll
                    for (int i = 0; i < kSlots; ++i) {
                        const uint4 q = slots[s][j * kSlots + i][threadIdx.x];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if constexpr (std::is_same<T, F32>::value) {
                                v[4 * i + k] = __uint_as_float(word(q, k));
                            } else {
                                const float2 f = T::to_f2(word(q, k));
                                v[2 * k] = f.x, v[2 * k + 1] = f.y;
                            }
                        }
                    }
                } else {
                    const char *p = a.table + static_cast<int64_t>(now[j]) * a.width * kBytes<T>;
#pragma unroll
                    for (int i = 0; i < kV; ++i) {
                        float one[1] = {0.f};
                        if (col[j] + i * a.row_chunks < a.width) load_values<T, 1>(p + (col[j] + i * a.row_chunks) * kBytes<T>, one);
                        v[i] = one[0];
                    }
                }
#pragma unroll
                for (int i = 0; i < kV; ++i) v[i] *= a.scale;
            }
            if constexpr (kChunks) {
                store_values<E, kV>(a.out + (row[j] * a.row_chunks + col[j]) * kOut, v);
            } else {
                char *p = a.out + row[j] * a.width * kBytes<E>;
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    const float one[1] = {v[i]};
                    if (col[j] + i * a.row_chunks < a.width) store_values<E, 1>(p + (col[j] + i * a.row_chunks) * kBytes<E>, one);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kLookupChunks; ++j) {
            row[j] = next_row[j], col[j] = next_col[j], now[j] = next[j];
            next_row[j] = later_row[j], next_col[j] = later_col[j], next[j] = later[j];
        }
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
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kRounds = 4;             // indices of a thread at a time
constexpr int kSortTile = kSortThreads * kRounds;
// At most: every block reads all blocks' counts, so these cost the square.  131040
// indices: KSORT
constexpr int kSortBlocks = 64;

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

template <typename C>
__global__ void __launch_bounds__(kSortThreads) sort_place(const SortArgs a) {
    extern __shared__ __align__(16) char shared[];
    uint2 *pairs = reinterpret_cast<uint2 *>(shared);                          // [tile]: row, position
    uint32_t *same_digit = reinterpret_cast<uint32_t *>(pairs + kSortTile);    // [warps][bins]: lanes
    uint32_t *warp_count = same_digit + kSortWarps * kBins;                    // [warps][bins]
    __shared__ int32_t to_base[kBins], warp_sums[kSortWarps];
    __shared__ uint32_t local_base[kBins];
    pdl_prologue();
    if (zeros_instead(a)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = blockIdx.x, bin = threadIdx.x;
    const int bins = 1 << a.bits;
    const uint32_t mask = bins - 1, lower = (1u << lane) - 1;
    uint32_t *lanes = same_digit + warp * kBins, *mine = warp_count + warp * kBins;
    for (int i = lane; i < bins; i += 32) lanes[i] = 0u;

    // Exclusive sums over the threads' values, in the threads' order.
    auto scan = [&](int32_t v) {
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
    };

    const int64_t first = me * a.range, end = first + a.range < a.n ? first + a.range : a.n;
    const int here = warp * 32 * kRounds + lane;
    uint32_t key[kRounds], at[kRounds];
    auto load = [&](int64_t tile) {
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            const int64_t i = tile + here + 32 * j;
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
        int32_t *sums = reinterpret_cast<int32_t *>(warp_count);       // [groups][2][bins]: at most the ranks' table
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
        to_base[bin] = scan(total) + mine_before;      // (with a barrier, after which the table is free)
    }
    for (int64_t tile = first; tile < end; tile += kSortTile) {
        for (int i = lane; i < bins; i += 32) mine[i] = 0u;
        __syncwarp();
        const int n_here = static_cast<int>(end - tile < kSortTile ? end - tile : kSortTile);
        if (tile > first) load(tile);
        uint32_t rank[kRounds];
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            const bool valid = here + 32 * j < n_here;
            const uint32_t d = key[j] >> a.shift & mask;
            if (valid) atomicOr(&lanes[d], 1u << lane);
            __syncwarp();
            const uint32_t same = lanes[d], had = mine[d], before = __popc(same & lower);
            __syncwarp();
            if (valid && before == 0) lanes[d] = 0u, mine[d] = had + __popc(same);
            __syncwarp();
            rank[j] = had + before;
        }
        __syncthreads();
        // counts of the warps before, and of the digits before: places in the tile
        uint32_t run = 0;
        if (bin < bins) {
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = warp_count[w * kBins + bin];
                warp_count[w * kBins + bin] = run;
                run += c;
            }
        }
        local_base[bin] = static_cast<uint32_t>(scan(static_cast<int32_t>(run)));
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            if (here + 32 * j >= n_here) continue;
            const uint32_t d = key[j] >> a.shift & mask;
            pairs[local_base[d] + mine[d] + rank[j]] = make_uint2(key[j], at[j]);
        }
        __syncthreads();
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

constexpr int kSumThreads = 256;
constexpr int kAhead = 8;              // rows that a thread has in flight
// Of a block: the slots' ends are joined one after another.
constexpr int kMostSlots = 32;
constexpr int kMostPiece = 2048;       // indices of a block

struct SumArgs {
    const char *grad;
    const int32_t *keys, *at;    // sorted
    char *out;
    float *part;                 // [pieces][2][width]: what reaches over a piece's ends
    int64_t n, pieces;
    int32_t n_rows;
    int width, cols;             // cols: threads of a row
    int each, piece;             // indices of a slot and of a block
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
// ones where rows are whole 16-byte chunks, else every cols-th, so that a warp's
// single elements are neighbours.
template <typename E, typename P, bool kChunks>
struct RowPart {
    static constexpr int kV = 16 / kBytes<E>;
    int first, step, width;

    __device__ RowPart(int thread, int cols, int slice, int w) : width(w) {
        first = slice * cols * kV + (kChunks ? thread * kV : thread);
        step = kChunks ? 1 : cols;
    }
    __device__ int col(int i) const { return first + i * step; }
    __device__ bool any() const { return first < width; }
    __device__ void load(const char *row, float (&v)[kV]) const {
        if constexpr (kChunks) {
            load_values<E, kV>(row + first * kBytes<E>, v);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                float one[1] = {0.f};
                if (col(i) < width) load_values<E, 1>(row + col(i) * kBytes<E>, one);
                v[i] = one[0];
            }
        }
    }
    __device__ void store(char *row, const float (&v)[kV]) const {
        if constexpr (kChunks) {
            store_values<P, kV>(row + first * kBytes<P>, v);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (col(i) < width) write_one<P>(row, col(i), v[i]);
        }
    }
};

// A block of cols x slots threads: a slot takes neighbouring indices of the piece, a
// thread a part of their rows' columns.  E: grad's format, P: the table's gradient's.
template <typename E, typename P, bool kChunks>
__global__ void __launch_bounds__(kSumThreads) sum_runs(const SumArgs a) {
    extern __shared__ __align__(16) char memory[];
    using Part = RowPart<E, P, kChunks>;
    constexpr int kV = Part::kV;
    const int slots = blockDim.y, wide = a.cols * kV;            // values of a row here
    const int thread = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    // slots of rows on their way: [ahead][threads], 16 bytes each (kChunks alone)
    constexpr int kRingStep = kSumThreads * 16;
    const uint32_t ring = shared_address(memory) + thread * 16;
    constexpr int kRingBytes = kChunks ? kAhead * kRingStep : 0;
    int2 *tokens = reinterpret_cast<int2 *>(memory + kRingBytes) + 1;    // [-1] ... [piece]: row, position
    float *head = reinterpret_cast<float *>(tokens + a.piece + 1);       // [slots][wide]
    float *tail = head + slots * wide;
    pdl_prologue();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * a.piece;
    for (int i = thread - 1; i <= a.piece; i += threads) {
        const int64_t t = first + i;
        // no row: before the first index, and from the first that names none
        const bool some = t >= 0 && t < a.n;
        tokens[i] = some ? make_int2(__ldcg(a.keys + t), __ldcg(a.at + t)) : make_int2(a.n_rows, 0);
    }
    __syncthreads();
    if (tokens[0].x >= a.n_rows) return;
    const Part part(threadIdx.x, a.cols, blockIdx.y, a.width);
    const uint32_t row_bytes = static_cast<uint32_t>(a.width) * kBytes<E>;
    const int t0 = threadIdx.y * a.each;
    if (tokens[t0].x < a.n_rows && part.any()) {
        const uint32_t out_bytes = static_cast<uint32_t>(a.width) * kBytes<P>;
        const int2 *mine = tokens + t0;
        float2 acc[kV / 2];
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) acc[i] = make_float2(0.f, 0.f);
        int32_t cur = mine[0].x;
        bool open = mine[-1].x == cur;    // the run began before this slot
        auto flush = [&](float *place) {
            if (place) {
#pragma unroll
                for (int i = 0; i < kV; ++i)
                    place[threadIdx.y * wide + (kChunks ? threadIdx.x * kV + i : threadIdx.x + i * a.cols)] =
                        i & 1 ? acc[i / 2].y : acc[i / 2].x;
            } else {
                float v[kV];
#pragma unroll
                for (int i = 0; i < kV; ++i) v[i] = (i & 1 ? acc[i / 2].y : acc[i / 2].x) * a.scale;
                part.store(a.out + static_cast<int64_t>(cur) * out_bytes, v);
            }
        };
        // the run of row k takes v, after the one before is ended
        auto take = [&](int32_t k, const float2 (&v)[kV / 2]) {
            if (k != cur) {
                flush(open ? head : nullptr);
                open = false;
                cur = k;
#pragma unroll
                for (int i = 0; i < kV / 2; ++i) acc[i] = v[i];
                return;
            }
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) acc[i] = __fadd2_rn(acc[i], v[i]);
        };
        if constexpr (kChunks) {
            const char *from = a.grad + part.first * kBytes<E>;
            int32_t key[kAhead];         // of the rows on their way; n_rows: none
            auto fetch = [&](int t, int j) {
                key[j] = a.n_rows;
                if (t < a.each) {
                    const int2 token = mine[t];
                    key[j] = token.x;
                    if (token.x < a.n_rows)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + j * kRingStep),
                                     "l"(from + static_cast<uint64_t>(static_cast<uint32_t>(token.y)) * row_bytes) : "memory");
                }
                cp_async_commit();
            };
#pragma unroll
            for (int j = 0; j < kAhead; ++j) fetch(j, j);
            for (int t = 0; t < a.each; t += kAhead) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    cp_async_wait<kAhead - 1>();
                    if (key[j] < a.n_rows) {
                        uint4 q;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(ring + j * kRingStep) : "memory");
                        float2 v[kV / 2];
#pragma unroll
                        for (int i = 0; i < kV / 2; ++i) {
                            if constexpr (kV == 4)
                                v[i] = make_float2(__uint_as_float(word(q, 2 * i)), __uint_as_float(word(q, 2 * i + 1)));
                            else
                                v[i] = E::to_f2(word(q, i));
                        }
                        take(key[j], v);
                    }
                    fetch(t + j + kAhead, j);
                }
            }
            cp_async_wait<0>();
        } else {
            constexpr int kBatch = 4;
            for (int t = 0; t < a.each; t += kBatch) {
                float v[kBatch][kV];
                int32_t k[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int2 token = t + j < a.each ? mine[t + j] : make_int2(a.n_rows, 0);
                    k[j] = token.x;
                    if (k[j] < a.n_rows)
                        part.load(a.grad + static_cast<uint64_t>(static_cast<uint32_t>(token.y)) * row_bytes, v[j]);
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (k[j] >= a.n_rows) continue;
                    float2 pairs[kV / 2];
#pragma unroll
                    for (int i = 0; i < kV / 2; ++i) pairs[i] = make_float2(v[j][2 * i], v[j][2 * i + 1]);
                    take(k[j], pairs);
                }
            }
        }
        flush(open ? head : mine[a.each].x == cur ? tail : nullptr);
    }
    __syncthreads();
    // The slots' ends, in their order.  A run that began before this piece, or
    // goes on after it, is left for the last launch.
    float *left = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
    for (int f = thread; f < wide; f += threads) {
        const int c = blockIdx.y * wide + f;
        if (c >= a.width) break;
        float run = 0.f;
        bool before = tokens[-1].x == tokens[0].x;      // the open run began before the piece
        for (int s = 0; s < slots; ++s) {
            const int b = s * a.each, e = b + a.each;
            if (tokens[b].x >= a.n_rows) break;
            const int32_t last = tokens[e - 1].x;
            if (tokens[b - 1].x == tokens[b].x) {
                run += head[s * wide + f];
                // does it end here?
                if (!(last == tokens[b].x && tokens[e].x == last)) {
                    if (before) left[c] = run;
                    else write_one<P>(a.out, tokens[b].x * static_cast<int64_t>(a.width) + c, run * a.scale);
                    before = false;
                    run = 0.f;
                } else {
                    continue;
                }
            }
            if (last < a.n_rows && tokens[e].x == last) run = tail[s * wide + f];
        }
        const int32_t last = tokens[a.piece - 1].x;
        if (last < a.n_rows && tokens[a.piece].x == last) left[(before ? 0 : a.width) + c] = run;
    }
}

// Runs that go over the end of the piece they began in: the sums of the pieces that
// each reaches into.  A block looks through some of the pieces for such beginnings.
// A run of a few pieces is a warp's, 128 columns at a time; a long one the block's,
// whose groups of threads add every groups-th piece's sums, and then the groups'.
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
constexpr int kJoinThreads = 1024, kJoinWarps = kJoinThreads / 32;
constexpr int kLongRun = 24;           // pieces behind the first

template <typename P>
__global__ void __launch_bounds__(kJoinThreads) join_runs(const SumArgs a) {
    __shared__ float4 sums[kJoinThreads];
    __shared__ int found[kJoinThreads], pieces[kJoinThreads], n_found;
    pdl_prologue();
    const int thread = threadIdx.x, lane = thread & 31, warp = thread >> 5;
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
            int more = 1;
            for (;;) {
                const int64_t next = (c0 + more + 1 + lane) * a.piece;
                const int on = __popc(__ballot_sync(0xffffffffu, next < a.n && __ldcg(a.keys + (next < a.n ? next : 0)) == k));
                more += on;
                if (on < 32) break;
            }
            if (lane == 0) pieces[f] = more;
        }
        __syncthreads();
        const int quads = (a.width + 3) / 4;     // four columns each
        const int blocks = (quads + 31) / 32;
        for (int t = warp; t < runs * blocks; t += kJoinWarps) {
            const int f = t / blocks, more = pieces[f], quad = (t - f * blocks) * 32 + lane;
            if (more > kLongRun || quad >= quads) continue;
            const int64_t c0 = found[f];
            const int32_t k = __ldcg(a.keys + (c0 + 1) * a.piece);
            float4 s = part_of(a, 2 * c0 + 1, quad);
#pragma unroll 4
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

// How a gradient is cut, and where its parts lie in the workspace.
struct Plan {
    int passes, bits, sort_blocks;   // of the sort
    int64_t range;
    int slices, cols, slots, each, piece;
    int64_t pieces;
    int count_bytes;
    int64_t keys[2], at[2], counts, part, bytes;
};

// v: values of a thread
Plan plan_of(int64_t n, int64_t n_rows, int32_t width, int v) {
    Plan z = {};
    int bits = 1;
    while (bits < 31 && n_rows >> bits) ++bits;     // keys are 0 ... n_rows
    z.passes = static_cast<int>(ceil_div(bits, 9));
    z.bits = static_cast<int>(ceil_div(bits, z.passes));
    if (z.bits < 4) z.bits = 4;      // whole 16 bytes of a block's counts
    // whole rounds of a block's threads
    z.range = ceil_div(ceil_div(n, kSortThreads), kSortBlocks) * kSortThreads;
    z.sort_blocks = n ? static_cast<int>(ceil_div(n, z.range)) : 0;
    z.count_bytes = z.range < 65536 ? 2 : 4;
    const int parts = static_cast<int>(ceil_div(width, v));
    z.slices = static_cast<int>(ceil_div(parts, kSumThreads));
    z.cols = static_cast<int>(ceil_div(parts, z.slices));
    z.slots = kSumThreads / z.cols < kMostSlots ? kSumThreads / z.cols : kMostSlots;
    // some six blocks an SM, of slots of 8 to 64 indices
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
int64_t workspace_of(int64_t n, int64_t n_rows, int32_t width) {
    const int64_t four = plan_of(n, n_rows, width, 4).bytes, eight = plan_of(n, n_rows, width, 8).bytes;
    return four > eight ? four : eight;
}

template <typename E, typename P, bool kChunks>
wgs_status run_sums(const SumArgs &a, const Plan &z, int sms, cudaStream_t stream) {
    const int wide = z.cols * (16 / kBytes<E>);
    const int smem = (kChunks ? kAhead * kSumThreads * 16 : 0) + 8 * (z.piece + 2) + 8 * z.slots * wide;
    static_assert(kMostPiece == 64 * kMostSlots &&
                      kAhead * kSumThreads * 16 + 8 * (kMostPiece + 2) + 8 * kSumThreads * 8 <= 66 << 10,
                  "shared memory of a block");
    auto kernel = sum_runs<E, P, kChunks>;
    // (as the layer norm's)
    if (smem > 47 << 10 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 66 << 10) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    const wgs_status st = launch(kernel, dim3(static_cast<unsigned>(z.pieces), z.slices), dim3(z.cols, z.slots),
                                 static_cast<size_t>(smem), stream, a);
    if (st != WGS_OK || z.pieces == 1) return st;
    const int64_t blocks = z.pieces < sms ? z.pieces : sms;
    return launch(join_runs<P>, dim3(static_cast<unsigned>(blocks)), dim3(kJoinThreads), 0, stream, a);
}

// 16 bytes of gradient at a time where all rows, and those of the output, start
// on as many.
bool in_chunks(const void *grad, const void *out, int32_t width, int64_t eb, int64_t ob) {
    return aligned16(grad) && aligned16(out) && width * eb % 16 == 0 && width * ob % 16 == 0;
}

template <typename E>
wgs_status run_format(const SumArgs &a, const Plan &z, bool chunks, bool p32, int sms, cudaStream_t stream) {
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
    // a share of the zeros in each launch, 64 bytes a thread or more
    const int64_t share = ceil_div(ceil_div(bytes, 1 + z.passes), 16) * 16, most = 4 * sms - z.sort_blocks;
    const int smem = kSortTile * 8 + kSortWarps * kBins * 8;
    // (as the layer norm's)
    if (cudaFuncSetAttribute(order, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    for (int p = -1; p < z.passes; ++p) {
        s.zeros = out + (p + 1) * share;
        s.zero_bytes = bytes - (p + 1) * share < share ? bytes - (p + 1) * share : share;
        if (s.zero_bytes < 0) s.zero_bytes = 0;
        int64_t more = ceil_div(s.zero_bytes, 64 * kSortThreads);
        if (more > most) more = most;
        const dim3 grid(static_cast<unsigned>(s.blocks + more));
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
    constexpr int kV = 16 / kBytes<E>;
    const bool chunks = in_chunks(a.table, a.out, width, kBytes<T>, kBytes<E>);
    a.row_chunks = static_cast<int>(ceil_div(width, kV)), a.width = width;
    const int64_t blocks = ceil_div(a.n * a.row_chunks, kLookupThreads * kLookupChunks);
    const int64_t most = static_cast<int64_t>(sms) * kLookupBlocksPerSm;
    return launch(chunks ? embedding_lookup<T, E, true> : embedding_lookup<T, E, false>,
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
    st = sort_indices(s, z, ws, static_cast<char *>(grad_table), tbytes, static_cast<int>(tb), dev.sm_count, stream);
    if (st != WGS_OK || n_rows == 0) return st;
    SumArgs a = {};
    a.grad = static_cast<const char *>(grad), a.keys = s.keys, a.at = s.at;
    a.out = static_cast<char *>(grad_table), a.part = reinterpret_cast<float *>(ws + z.part);
    a.n = n_idx, a.pieces = z.pieces, a.n_rows = static_cast<int32_t>(n_rows), a.width = width, a.cols = z.cols;
    a.each = z.each, a.piece = z.piece, a.scale = scale;
    const bool p32 = table_dtype == WGS_F32;
    if (dtype == WGS_F32) return run_format<F32>(a, z, chunks, true, dev.sm_count, stream);
    if (dtype == WGS_F16) return run_format<Fp16>(a, z, chunks, p32, dev.sm_count, stream);
    return run_format<Bf16>(a, z, chunks, p32, dev.sm_count, stream);
}
