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
#include <cooperative_groups.h>

#include <type_traits>

#include "wgs_common.cuh"

namespace wgs {

namespace {

namespace cg = cooperative_groups;

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

constexpr int kLookupThreads = 256, kLookupChunks = 4;   // chunks of a thread

// A block takes neighbouring chunks of the output.  T: the table's format, E: the
// output's.  magic: 2^32 / chunks of a row, rounded up (exact quotients for
// numbers below 2^16: those of a row and of a block's chunks).
template <typename T, typename E, int kV>
__global__ void __launch_bounds__(kLookupThreads) embedding_lookup(const char *table, const int32_t *idx, char *out,
                                                                   int64_t n, int64_t n_rows, int row_chunks,
                                                                   uint32_t magic, float scale) {
    pdl_prologue();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kLookupThreads * kLookupChunks);
    const int64_t row0 = first / row_chunks;
    const uint32_t over = static_cast<uint32_t>(first - row0 * row_chunks);
    int64_t row[kLookupChunks];
    int32_t from[kLookupChunks], col[kLookupChunks];
#pragma unroll
    for (int j = 0; j < kLookupChunks; ++j) {
        const uint32_t at = over + threadIdx.x + j * kLookupThreads;
        const uint32_t r = row_chunks == 1 ? at : __umulhi(at, magic);
        row[j] = row0 + r;
        col[j] = static_cast<int32_t>(at - r * row_chunks);
        from[j] = row[j] < n ? __ldg(idx + row[j]) : -1;
    }
    float v[kLookupChunks][kV];
#pragma unroll
    for (int j = 0; j < kLookupChunks; ++j) {
        if (from[j] >= 0 && from[j] < n_rows) {
            load_values<T, kV>(table + (static_cast<int64_t>(from[j]) * row_chunks + col[j]) * (kV * kBytes<T>), v[j]);
        } else {
            if (from[j] != -1 && col[j] == 0) atomicOr(&g_embedding_error, 1u);
            from[j] = -1;
        }
    }
#pragma unroll
    for (int j = 0; j < kLookupChunks; ++j) {
        if (row[j] >= n) continue;
#pragma unroll
        for (int i = 0; i < kV; ++i) v[j][i] = from[j] < 0 ? 0.f : v[j][i] * scale;
        store_values<E, kV>(out + (row[j] * row_chunks + col[j]) * (kV * kBytes<E>), v[j]);
    }
}

// -------------------------------------------------------------------- sort --

// A stable counting sort by digits of at most 8 bits, from the lowest.  A block
// counts the digits of its own range, the counts are summed up over the blocks
// before it, and it places its range's indices behind those.
constexpr int kBins = 256;
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr int kSortTile = 4096;        // indices a block ranks at a time
constexpr int kSortBlocks = 608;       // at most

struct SortArgs {
    const int32_t *idx;          // first pass: the call's indices
    const int32_t *keys, *at;    // later passes: sorted by the lower digits
    int32_t *keys_out, *at_out;
    int32_t *counts;             // [bins][blocks]
    int32_t *totals;             // [bins]
    int64_t n, range;            // indices; of a block
    int32_t n_rows;
    int shift, bits, blocks;
};

// The row that index i names; n_rows, sorted behind all, for none.
__device__ __forceinline__ int32_t key_of(const SortArgs &a, int64_t i) {
    if (!a.idx) return __ldcg(a.keys + i);
    const int32_t k = __ldg(a.idx + i);
    return k >= 0 && k < a.n_rows ? k : a.n_rows;
}

__global__ void __launch_bounds__(kSortThreads) sort_count(const SortArgs a) {
    __shared__ int32_t count[kBins];
    pdl_prologue();
    count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * a.range, end = first + a.range < a.n ? first + a.range : a.n;
    const uint32_t mask = (1u << a.bits) - 1;
    for (int64_t i = first + threadIdx.x; i < end; i += kSortThreads) {
        if (a.idx) {
            const int32_t k = __ldg(a.idx + i);
            if (k < -1 || k >= a.n_rows) atomicOr(&g_embedding_error, 1u);
        }
        atomicAdd(&count[static_cast<uint32_t>(key_of(a, i)) >> a.shift & mask], 1);
    }
    __syncthreads();
    if (threadIdx.x <= mask) a.counts[static_cast<int64_t>(threadIdx.x) * a.blocks + blockIdx.x] = count[threadIdx.x];
}

// Sum of v over the threads before this one, of a block of kSortThreads; *total
// of all.
__device__ __forceinline__ int32_t scan_before(int32_t v, int32_t *warp_sums, int32_t *total) {
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
    int32_t before = 0, all = 0;
    for (int w = 0; w < kSortWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + s - v;
}

// A digit's counts become the sums over the blocks before.
__global__ void __launch_bounds__(kSortThreads) sort_scan(int32_t *counts, int32_t *totals, int blocks) {
    __shared__ int32_t warp_sums[kSortWarps];
    pdl_prologue();
    int32_t *mine = counts + static_cast<int64_t>(blockIdx.x) * blocks;
    int32_t run = 0;
    for (int b0 = 0; b0 < blocks; b0 += kSortThreads) {
        const int b = b0 + threadIdx.x;
        int32_t total;
        const int32_t before = scan_before(b < blocks ? mine[b] : 0, warp_sums, &total);
        if (b < blocks) mine[b] = run + before;
        run += total;
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = run;
}

__global__ void __launch_bounds__(kSortThreads) sort_place(const SortArgs a) {
    __shared__ int32_t base[kBins], warp_base[kSortWarps][kBins], warp_sums[kSortWarps];
    pdl_prologue();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t mask = (1u << a.bits) - 1;
    const bool digit = threadIdx.x <= mask;
    int32_t total;
    const int32_t lower = scan_before(digit ? a.totals[threadIdx.x] : 0, warp_sums, &total);
    base[threadIdx.x] = lower + (digit ? a.counts[static_cast<int64_t>(threadIdx.x) * a.blocks + blockIdx.x] : 0);
    const int64_t first = blockIdx.x * a.range, end = first + a.range < a.n ? first + a.range : a.n;
    constexpr int kEach = kSortTile / kSortThreads;   // of a lane
    for (int64_t tile = first; tile < end; tile += kSortTile) {
        for (int w = 0; w < kSortWarps; ++w) warp_base[w][threadIdx.x] = 0;
        __syncthreads();
        const int64_t mine = tile + warp * (kSortTile / kSortWarps) + lane;
        int32_t key[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int64_t i = mine + 32 * j;
            key[j] = i < end ? key_of(a, i) : 0;
            if (i < end) atomicAdd(&warp_base[warp][static_cast<uint32_t>(key[j]) >> a.shift & mask], 1);
        }
        __syncthreads();
        int32_t run = base[threadIdx.x];
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = warp_base[w][threadIdx.x];
            warp_base[w][threadIdx.x] = run;
            run += c;
        }
        base[threadIdx.x] = run;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int64_t i = mine + 32 * j;
            const uint32_t d = static_cast<uint32_t>(key[j]) >> a.shift & mask;
            const unsigned same = __match_any_sync(0xffffffffu, i < end ? d : 0xffffffffu);
            const int rank = __popc(same & ((1u << lane) - 1));
            const int32_t to = warp_base[warp][d] + rank;
            __syncwarp();
            if (i < end) {
                if (rank == 0) warp_base[warp][d] += __popc(same);
                a.keys_out[to] = key[j];
                a.at_out[to] = a.idx ? static_cast<int32_t>(i) : __ldcg(a.at + i);
            }
            __syncwarp();
        }
        __syncthreads();
    }
}

// The same sort in one cluster of blocks, for as many indices as its registers and
// shared memory hold: a pass counts, exchanges the blocks' counts over distributed
// shared memory and places the indices there, behind cluster barriers instead of
// launches.  Digits have up to 9 bits, so two passes sort 2^18 rows.  Measured at
// 131040 indices into 32768 rows: 152 us for the whole gradient with six launches
// that sort, see below for what is left.  The grid's other clusters write the
// table's gradient's zeros meanwhile, which the sort leaves the memory idle for.
constexpr int kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32;
constexpr int kRounds = 12;            // indices of a thread, at most
constexpr int kMostCluster = 16;
constexpr int kMostClustered = kMostCluster * kRounds * kClusterThreads;
constexpr int kClusterBins = 512;

struct ClusterArgs {
    SortArgs s;
    int passes, tile, cluster;   // tile: indices of a block
    uint32_t magic;              // 2^32 / tile, rounded up
    char *zeros;                 // to be written as such
    int64_t zero_bytes;
    int zero_unit;               // bytes that its start and length are multiples of
};

__device__ void write_zeros(char *p, int64_t n, int bytes, int64_t thread, int64_t threads) {
    int64_t lead = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15;
    if (lead > n) lead = n;
    const int64_t whole = (n - lead) / 16, rest = n - lead - whole * 16;
    for (int64_t i = thread; i < whole; i += threads) st_stream(p + lead + 16 * i, make_uint4(0u, 0u, 0u, 0u));
    if (thread < 16) {
        const int64_t i = thread * bytes;
        char *end = p + lead + whole * 16;
        for (int side = 0; side < 2; ++side) {
            char *q = side ? end : p;
            if (i >= (side ? rest : lead)) continue;
            if (bytes == 4)
                *reinterpret_cast<uint32_t *>(q + i) = 0u;
            else
                *reinterpret_cast<uint16_t *>(q + i) = 0;
        }
    }
}

__global__ void __launch_bounds__(kClusterThreads, 1) sort_in_cluster(const ClusterArgs a) {
    extern __shared__ __align__(16) char shared[];
    __shared__ int32_t total[kClusterBins], base[kClusterBins], warp_sums[kClusterWarps];
    const SortArgs &s = a.s;
    uint2 *pairs = reinterpret_cast<uint2 *>(shared);                       // [tile]: row, position
    uint16_t *counts = reinterpret_cast<uint16_t *>(pairs + a.tile);        // [warps][bins]
    pdl_prologue();
    if (static_cast<int>(blockIdx.x) >= a.cluster) {
        const int64_t blocks = gridDim.x - a.cluster, block = blockIdx.x - a.cluster;
        write_zeros(a.zeros, a.zero_bytes, a.zero_unit, block * kClusterThreads + threadIdx.x, blocks * kClusterThreads);
        return;
    }
    cg::cluster_group cluster = cg::this_cluster();
    const int me = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int bins = 1 << s.bits, rounds = a.tile / kClusterThreads;
    const uint32_t mask = bins - 1, lower = (1u << lane) - 1;
    uint16_t *mine = counts + warp * bins;
    const int here = warp * rounds * 32 + lane, n_here = static_cast<int>(s.n) - me * a.tile;   // valid below n_here
    uint32_t key[kRounds], at[kRounds], rank[kRounds];
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
        const int i = here + 32 * j;
        key[j] = 0;
        if (j < rounds && i < n_here) {
            at[j] = static_cast<uint32_t>(me * a.tile + i);
            const int32_t k = __ldg(s.idx + at[j]);
            key[j] = static_cast<uint32_t>(k >= 0 && k < s.n_rows ? k : s.n_rows);
            if (k < -1 || k >= s.n_rows) atomicOr(&g_embedding_error, 1u);
        }
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * s.bits;
        for (int i = lane; i < bins / 2; i += 32) reinterpret_cast<uint32_t *>(mine)[i] = 0u;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            if (j >= rounds) break;
            const bool valid = here + 32 * j < n_here;
            const uint32_t d = key[j] >> shift & mask;
            const unsigned same = __match_any_sync(0xffffffffu, valid ? d : 0xffffffffu);
            const uint32_t before = __popc(same & lower), had = mine[d];
            __syncwarp();
            if (valid && before == 0) mine[d] = static_cast<uint16_t>(had + __popc(same));
            __syncwarp();
            rank[j] = had + before;
        }
        __syncthreads();
        const int d = threadIdx.x;
        if (d < bins) {
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < kClusterWarps; ++w) {
                const uint32_t c = counts[w * bins + d];
                counts[w * bins + d] = static_cast<uint16_t>(run);
                run += c;
            }
            total[d] = static_cast<int32_t>(run);
        }
        cluster.sync();
        // all blocks hold their indices in registers from here on
        int32_t all = 0, before = 0;
        if (d < bins) {
#pragma unroll 4
            for (int b = 0; b < a.cluster; ++b) {
                const int32_t c = *cluster.map_shared_rank(&total[d], b);
                all += c;
                if (b < me) before += c;
            }
        }
        int32_t sum = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        if (d < bins) {
            for (int w = 0; w < warp; ++w) before += warp_sums[w];
            base[d] = before + sum - all;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            if (j >= rounds) break;
            if (here + 32 * j >= n_here) continue;
            const uint32_t digit = key[j] >> shift & mask;
            const uint32_t to = base[digit] + mine[digit] + rank[j];
            if (pass + 1 == a.passes) {
                s.keys_out[to] = static_cast<int32_t>(key[j]);
                s.at_out[to] = static_cast<int32_t>(at[j]);
            } else {
                const uint32_t block = a.cluster == 1 ? 0 : __umulhi(to, a.magic);
                *cluster.map_shared_rank(&pairs[to - block * a.tile], block) = make_uint2(key[j], at[j]);
            }
        }
        cluster.sync();
        if (pass + 1 == a.passes) break;
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            const int i = here + 32 * j;
            if (j >= rounds) break;
            if (i < n_here) key[j] = pairs[i].x, at[j] = pairs[i].y;
        }
    }
}

// -------------------------------------------------------------------- sums --

constexpr int kSumThreads = 256;
constexpr int kAhead = 6;              // rows that a thread has in flight
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
    const uint32_t ring = shared_address(memory) + thread * 16;
    const int ring_bytes = kChunks ? kAhead * threads * 16 : 0;
    int32_t *keys = reinterpret_cast<int32_t *>(memory + ring_bytes) + 1;       // keys[-1] ... keys[piece]
    int32_t *at = keys + a.piece + 1;
    float *head = reinterpret_cast<float *>(at + a.piece);       // [slots][wide]
    float *tail = head + slots * wide;
    pdl_prologue();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * a.piece;
    for (int i = thread - 1; i <= a.piece; i += threads) {
        const int64_t t = first + i;
        // no row: before the first index, and from the first that names none
        keys[i] = t >= 0 && t < a.n ? __ldcg(a.keys + t) : a.n_rows;
        if (i >= 0 && i < a.piece && t < a.n) at[i] = __ldcg(a.at + t);
    }
    __syncthreads();
    if (keys[0] >= a.n_rows) return;
    const Part part(threadIdx.x, a.cols, blockIdx.y, a.width);
    const int64_t row_bytes = static_cast<int64_t>(a.width) * kBytes<E>;
    const int t0 = threadIdx.y * a.each, t1 = t0 + a.each;
    if (keys[t0] < a.n_rows && part.any()) {
        const int64_t out_bytes = static_cast<int64_t>(a.width) * kBytes<P>;
        float acc[kV] = {};
        int32_t cur = keys[t0];
        bool open = keys[t0 - 1] == cur;    // the run began before this slot
        auto flush = [&](float *place) {
            if (place) {
#pragma unroll
                for (int i = 0; i < kV; ++i) place[threadIdx.y * wide + (kChunks ? threadIdx.x * kV + i : threadIdx.x + i * a.cols)] = acc[i];
            } else {
#pragma unroll
                for (int i = 0; i < kV; ++i) acc[i] *= a.scale;
                part.store(a.out + cur * out_bytes, acc);
            }
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[i] = 0.f;
        };
        auto take = [&](int32_t k, const float (&v)[kV]) {
            if (k != cur) {
                flush(open ? head : nullptr);
                open = false;
                cur = k;
            }
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[i] += v[i];
        };
        if constexpr (kChunks) {
            const char *from = a.grad + part.first * kBytes<E>;
            const uint32_t around = kAhead * threads * 16;
            auto fetch = [&](int t, uint32_t slot) {
                if (t < t1 && keys[t] < a.n_rows)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + slot), "l"(from + at[t] * row_bytes) : "memory");
                cp_async_commit();
            };
            uint32_t slot = 0;
            for (int j = 0; j < kAhead; ++j) fetch(t0 + j, j * threads * 16);
            for (int t = t0; t < t1; ++t) {
                const int32_t k = keys[t];
                if (k >= a.n_rows) break;
                cp_async_wait<kAhead - 1>();
                uint4 q;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(ring + slot) : "memory");
                float v[kV];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (kV == 4) {
                        v[i] = __uint_as_float(word(q, i));
                    } else {
                        const float2 f = E::to_f2(word(q, i));
                        v[2 * i] = f.x, v[2 * i + 1] = f.y;
                    }
                }
                take(k, v);
                fetch(t + kAhead, slot);
                slot += threads * 16;
                if (slot == around) slot = 0;
            }
            cp_async_wait<0>();
        } else {
            constexpr int kBatch = 4;
            for (int t = t0; t < t1; t += kBatch) {
                float v[kBatch][kV];
                int32_t k[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    k[j] = t + j < t1 ? keys[t + j] : a.n_rows;
                    if (k[j] < a.n_rows) part.load(a.grad + at[t + j] * row_bytes, v[j]);
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (k[j] < a.n_rows) take(k[j], v[j]);
            }
        }
        flush(open ? head : keys[t1] == cur ? tail : nullptr);
    }
    __syncthreads();
    // The slots' ends, in their order.  A run that began before this piece, or
    // goes on after it, is left for the last launch.
    float *left = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
    for (int f = thread; f < wide; f += threads) {
        const int c = blockIdx.y * wide + f;
        if (c >= a.width) break;
        float run = 0.f;
        bool before = keys[-1] == keys[0];      // the open run began before the piece
        for (int s = 0; s < slots; ++s) {
            const int b = s * a.each, e = b + a.each;
            if (keys[b] >= a.n_rows) break;
            const int32_t last = keys[e - 1];
            if (keys[b - 1] == keys[b]) {
                run += head[s * wide + f];
                // does it end here?
                if (!(last == keys[b] && keys[e] == last)) {
                    if (before) left[c] = run;
                    else write_one<P>(a.out, keys[b] * static_cast<int64_t>(a.width) + c, run * a.scale);
                    before = false;
                    run = 0.f;
                } else {
                    continue;
                }
            }
            if (last < a.n_rows && keys[e] == last) run = tail[s * wide + f];
        }
        const int32_t last = keys[a.piece - 1];
        if (last < a.n_rows && keys[a.piece] == last) left[(before ? 0 : a.width) + c] = run;
    }
}

// Runs that go over the end of the piece they began in: the sums of the pieces that
// each reaches into.  A block looks through some of the pieces for such beginnings
// and takes their runs one after another; its groups of blockDim.x threads add every
// groups-th piece's sums, and then the groups'.
constexpr int kJoinThreads = 1024;

template <typename P>
__global__ void __launch_bounds__(kJoinThreads) join_runs(const SumArgs a) {
    __shared__ float sums[kJoinThreads];
    __shared__ int found[kJoinThreads], n_found;
    pdl_prologue();
    const int thread = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    // does the run of piece c's last index go on into the next, having begun in c?
    auto begins = [&](int64_t c) {
        const int64_t end = (c + 1) * a.piece;
        if (c >= a.pieces || end >= a.n) return false;
        const int32_t k = __ldcg(a.keys + end), last = __ldcg(a.keys + end - 1);
        const int32_t before = c > 0 ? __ldcg(a.keys + c * a.piece - 1) : a.n_rows;
        return k < a.n_rows && last == k && before != k;
    };
    for (int64_t round = 0; round * threads * gridDim.x < a.pieces; ++round) {
        if (thread == 0) n_found = 0;
        __syncthreads();
        const int64_t c = (round * threads + thread) * gridDim.x + blockIdx.x;
        if (begins(c)) found[atomicAdd(&n_found, 1)] = static_cast<int>(c);
        __syncthreads();
        const int runs = n_found;
        for (int f = 0; f < runs; ++f) {
            const int64_t c0 = found[f];
            const int32_t k = __ldcg(a.keys + (c0 + 1) * a.piece);
            int64_t more = 1;       // pieces behind c0 that the run reaches into
            for (;;) {
                const int64_t next = (c0 + more + 1 + thread) * a.piece;
                const int on = __syncthreads_count(next < a.n && __ldcg(a.keys + (next < a.n ? next : 0)) == k);
                more += on;
                if (on < threads) break;
            }
            for (int col = threadIdx.x; col - static_cast<int>(threadIdx.x) < a.width; col += blockDim.x) {
                float s = 0.f;
                if (col < a.width) {
                    const float *part = a.part + c0 * 2 * a.width + col;
                    if (threadIdx.y == 0) s = __ldcg(part + a.width);
#pragma unroll 8
                    for (int64_t p = 1 + threadIdx.y; p <= more; p += blockDim.y) s += __ldcg(part + p * 2 * a.width);
                }
                sums[thread] = s;
                __syncthreads();
                if (threadIdx.y == 0 && col < a.width) {
                    for (int g = 1; g < static_cast<int>(blockDim.y); ++g) s += sums[g * blockDim.x + threadIdx.x];
                    write_one<P>(a.out, k * static_cast<int64_t>(a.width) + col, s * a.scale);
                }
                __syncthreads();
            }
        }
    }
}

// Zeros over n bytes at p; `bytes` of an element divide both.
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
    bool clustered;
    int passes, bits;             // of the sort
    int sort_blocks;              // of one in launches
    int64_t range;
    int cluster, tile;            // of one in a cluster
    int slices, cols, slots, each, piece;
    int64_t pieces;
    int64_t keys[2], at[2], counts, totals, part, bytes;
};

// v: values of a thread
Plan plan_of(int64_t n, int64_t n_rows, int32_t width, int v) {
    Plan z = {};
    int bits = 1;
    while (bits < 31 && n_rows >> bits) ++bits;     // keys are 0 ... n_rows
    z.clustered = n <= kMostClustered;
    z.passes = static_cast<int>(ceil_div(bits, z.clustered ? 9 : 8));
    z.bits = static_cast<int>(ceil_div(bits, z.passes));
    const int64_t tiles = ceil_div(n, kSortTile);
    z.range = ceil_div(tiles, kSortBlocks) * kSortTile;
    z.sort_blocks = n ? static_cast<int>(ceil_div(n, z.range)) : 0;
    z.cluster = 1;
    while (z.cluster < kMostCluster && z.cluster * kClusterThreads < n) z.cluster *= 2;
    z.tile = static_cast<int>(ceil_div(ceil_div(n, z.cluster), kClusterThreads)) * kClusterThreads;
    const int parts = static_cast<int>(ceil_div(width, v));
    z.slices = static_cast<int>(ceil_div(parts, kSumThreads));
    z.cols = static_cast<int>(ceil_div(parts, z.slices));
    z.slots = kSumThreads / z.cols;
    // some six blocks an SM, of slots of 8 to 64 indices
    const int64_t want = ceil_div(n, static_cast<int64_t>(z.slots) * 912);
    z.each = want < 8 ? 8 : want > 64 ? 64 : static_cast<int>(want);
    if (z.each * z.slots > kMostPiece) z.each = kMostPiece / z.slots;
    z.piece = z.slots * z.each;
    z.pieces = ceil_div(n, z.piece);
    int64_t at = 0;
    auto place = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 15) / 16 * 16;
        return here;
    };
    for (int i = 0; i < (z.clustered ? 1 : 2); ++i) z.keys[i] = place(4 * n), z.at[i] = place(4 * n);
    if (!z.clustered) {
        z.counts = place(4ll * kBins * z.sort_blocks);
        z.totals = place(4 * kBins);
    }
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
    const int smem = (kChunks ? kAhead * z.cols * z.slots * 16 : 0) + 4 * (2 * z.piece + 2) + 8 * z.slots * wide;
    static_assert(kAhead * kSumThreads * 16 + 4 * (2 * kMostPiece + 2) + 8 * kSumThreads * 8 <= 60 << 10,
                  "shared memory of a block");
    auto kernel = sum_runs<E, P, kChunks>;
    // (as the layer norm's)
    if (smem > 47 << 10 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 60 << 10) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    const wgs_status st = launch(kernel, dim3(static_cast<unsigned>(z.pieces), z.slices), dim3(z.cols, z.slots),
                                 static_cast<size_t>(smem), stream, a);
    if (st != WGS_OK || z.pieces == 1) return st;
    // threads for all columns, at least four groups of them where the rows are many
    int cols = a.width < 256 ? static_cast<int>(ceil_div(a.width, 32)) * 32 : 256;
    const int64_t blocks = z.pieces < 2 * sms ? z.pieces : 2 * sms;
    return launch(join_runs<P>, dim3(static_cast<unsigned>(blocks)), dim3(cols, kJoinThreads / cols), 0, stream, a);
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

// The sort in launches: three a pass.
wgs_status sort_in_launches(SortArgs &s, const Plan &z, char *ws, cudaStream_t stream) {
    s.range = z.range, s.blocks = z.sort_blocks, s.bits = z.bits;
    s.counts = reinterpret_cast<int32_t *>(ws + z.counts), s.totals = reinterpret_cast<int32_t *>(ws + z.totals);
    for (int p = 0; p < z.passes; ++p) {
        wgs_status st;
        s.shift = p * z.bits;
        s.keys_out = reinterpret_cast<int32_t *>(ws + z.keys[p & 1]);
        s.at_out = reinterpret_cast<int32_t *>(ws + z.at[p & 1]);
        if ((st = launch(sort_count, dim3(s.blocks), dim3(kSortThreads), 0, stream, s)) != WGS_OK) return st;
        if ((st = launch(sort_scan, dim3(1u << z.bits), dim3(kSortThreads), 0, stream, s.counts, s.totals,
                         s.blocks)) != WGS_OK)
            return st;
        if ((st = launch(sort_place, dim3(s.blocks), dim3(kSortThreads), 0, stream, s)) != WGS_OK) return st;
        s.idx = nullptr, s.keys = s.keys_out, s.at = s.at_out;
    }
    return WGS_OK;
}

// The sort in one cluster, with the zeros of `bytes` bytes at `out`.
wgs_status sort_in_one_cluster(SortArgs &s, const Plan &z, char *ws, char *out, int64_t bytes, int unit,
                               cudaStream_t stream) {
    s.bits = z.bits;
    s.keys_out = reinterpret_cast<int32_t *>(ws + z.keys[0]), s.at_out = reinterpret_cast<int32_t *>(ws + z.at[0]);
    ClusterArgs c = {};
    c.s = s, c.passes = z.passes, c.tile = z.tile, c.cluster = z.cluster;
    c.magic = static_cast<uint32_t>(((1ull << 32) + z.tile - 1) / z.tile);
    c.zeros = out, c.zero_bytes = bytes, c.zero_unit = unit;
    // 64 bytes of zeros a thread, in whole clusters and up to 112 blocks
    int64_t more = ceil_div(ceil_div(bytes, 64 * kClusterThreads), z.cluster);
    if (more > 112 / z.cluster) more = 112 / z.cluster;
    const int smem = z.tile * 8 + kClusterWarps * (2 << z.bits);
    // As the layer norm's, and clusters beyond eight blocks need it too.
    if ((smem > 43 << 10 &&
         cudaFuncSetAttribute(sort_in_cluster, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kRounds * kClusterThreads * 8 + kClusterWarps * 2 * kClusterBins) != cudaSuccess) ||
        (z.cluster > 8 && cudaFuncSetAttribute(sort_in_cluster, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                              cudaSuccess)) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    s.keys = s.keys_out, s.at = s.at_out;
    return launch_clusters(sort_in_cluster, dim3(static_cast<unsigned>(z.cluster * (1 + more))), dim3(kClusterThreads),
                           z.cluster, static_cast<size_t>(smem), stream, c);
}

template <typename T, typename E>
wgs_status run_lookup(const char *table, const int32_t *idx, char *out, int64_t n, int64_t n_rows, int32_t width,
                      float scale, cudaStream_t stream) {
    constexpr int kV = 16 / kBytes<E>;
    const bool chunks = in_chunks(table, out, width, kBytes<T>, kBytes<E>);
    const int row_chunks = chunks ? width / kV : width;
    const int64_t blocks = ceil_div(n * row_chunks, kLookupThreads * kLookupChunks);
    if (blocks > INT32_MAX) return WGS_ERR_SHAPE;
    const uint32_t magic = static_cast<uint32_t>(((1ull << 32) + row_chunks - 1) / row_chunks);
    return launch(chunks ? embedding_lookup<T, E, kV> : embedding_lookup<T, E, 1>, dim3(static_cast<unsigned>(blocks)),
                  dim3(kLookupThreads), 0, stream, table, idx, out, n, n_rows, row_chunks, magic, scale);
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
    const char *t = static_cast<const char *>(table);
    char *o = static_cast<char *>(out);
    auto go = dtype == WGS_F32    ? run_lookup<F32, F32>
              : dtype == WGS_F16 ? (table_dtype == WGS_F32 ? run_lookup<F32, Fp16> : run_lookup<Fp16, Fp16>)
                                 : (table_dtype == WGS_F32 ? run_lookup<F32, Bf16> : run_lookup<Bf16, Bf16>);
    return go(t, idx, o, n_idx, n_rows, width, scale, stream);
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
    if (tbytes > 0 && (n_idx == 0 || !z.clustered)) {
        const int64_t blocks = ceil_div(ceil_div(tbytes, 16), 256 * 8);
        const int64_t most = 8ll * dev.sm_count;
        st = launch(fill_zeros, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, stream,
                    static_cast<char *>(grad_table), tbytes, static_cast<int>(tb));
    }
    if (st != WGS_OK || n_idx == 0) return st;
    char *ws = static_cast<char *>(workspace);
    SortArgs s = {};
    s.idx = idx, s.n = n_idx, s.n_rows = static_cast<int32_t>(n_rows);
    st = z.clustered ? sort_in_one_cluster(s, z, ws, static_cast<char *>(grad_table), tbytes, static_cast<int>(tb), stream)
                     : sort_in_launches(s, z, ws, stream);
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
