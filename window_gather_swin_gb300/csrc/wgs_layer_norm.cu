// Layer norm with weight and bias over rows of any width up to 8192, fused with
// the residual add before it, and its gradients (sm_103a).
//
// With a row's mean and rstd = 1 / sqrt(var + eps), h = (x - mean) rstd:
//     y = h w + b
// and for a gradient gy of y, g = gy w and M the mean over the row
//     grad_x = rstd (g - M(g) - h M(g h))  (+ the residual stream's gradient)
//     grad_w = sum gy h,   grad_b = sum gy   (all rows).
//
// Design.  A row belongs to a unit: 8, 16 or 32 lanes of a warp up to a width of
// 512, several warps beyond.  A thread holds the same columns of every row that
// its unit takes, so weights and the columns' sums stay in registers while rows
// stream past.  Rows reach the units through stages in shared memory: a tile of
// neighbouring rows is one run of bytes, copied in bulk (TMA) several tiles ahead
// and widened on its way to registers, whatever the width's remainder: the copy
// starts and ends on 16 bytes, and the few bytes at the tensor's own ends that a
// bulk copy cannot take are copied by the unit.  One block an SM; the units walk
// the tiles in a fixed order.  The columns' sums of a block meet in shared memory,
// those of all blocks in a second launch, all in a fixed order.
#include <type_traits>

#include "wgs_common.cuh"

namespace wgs {

namespace {

// Set (never cleared by a kernel) when a unit gave up waiting for its own
// copies; read and cleared by wgs_check_error.
__device__ unsigned int g_layer_norm_error;

struct F32 {};

constexpr int kMaxWidth = 8192;
constexpr int kWarps = 16;         // of a block, at most
constexpr int kMaxStages = 4;
constexpr int kRing = 200 << 10;   // shared memory of a block's stages, at most

struct LayerNormArgs {
    const char *in[3];   // forward: x, branch; backward: x, grad_y, grad_residual
    char *out;           // y or grad_x
    char *total;         // residual_out
    const void *weight, *bias;
    float *mean, *rstd;
    float *part;         // backward: [blocks][2][width]
    int64_t rows, tiles;
    int tensors;         // of in
    int width, tile_rows, tile_bytes, stages;
    int team_warps;      // of a unit
    float eps, inv;      // inv: 1 / width
    bool p32;            // weight and bias are FP32
};

// ------------------------------------------------------------------ values --

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// FP32 pairs on the packed pipe: each half the correctly rounded operation.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

template <typename E>
constexpr int kBytes = std::is_same<E, F32>::value ? 4 : 2;

template <typename E>
__device__ __forceinline__ float load_one(const char *p) {
    if constexpr (std::is_same<E, F32>::value) {
        return *reinterpret_cast<const float *>(p);
    } else {
        return E::to_f2(*reinterpret_cast<const uint16_t *>(p)).x;
    }
}

template <typename E>
__device__ __forceinline__ float load_param(const void *p, int i, bool p32) {
    return p32 ? __ldg(static_cast<const float *>(p) + i)
               : load_one<E>(static_cast<const char *>(p) + static_cast<size_t>(i) * kBytes<E>);
}

// A thread's columns of a row: kE values as pairs, in chunks of kV neighbouring
// ones, the chunks of a unit's threads side by side.
template <typename E, int kV, int kE>
struct Columns {
    static constexpr int kChunks = kE / kV;
    int first, step, width;   // the thread's first column, from chunk to chunk, and the row's end

    __device__ Columns(int thread, int threads, int w) : first(thread * kV), step(threads * kV), width(w) {}
    __device__ int at(int c) const { return first + c * step; }
    __device__ bool held(int c) const { return at(c) < width; }

    // v = the row's values, widened; 0 for columns past the end and rows that are not there
    __device__ void load(const char *row, bool there, float2 (&v)[kE / 2]) const {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const bool ok = there && held(c);
            const char *p = row + static_cast<size_t>(at(c)) * kBytes<E>;
            if constexpr (kV == 1) {
                const float f = ok ? load_one<E>(p) : 0.f;
                if (c & 1) v[c / 2].y = f; else v[c / 2].x = f;
            } else if constexpr (std::is_same<E, F32>::value) {
                const float4 q = ok ? *reinterpret_cast<const float4 *>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[2 * c] = make_float2(q.x, q.y), v[2 * c + 1] = make_float2(q.z, q.w);
            } else {
                const uint2 q = ok ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0u, 0u);
                v[2 * c] = E::to_f2(q.x), v[2 * c + 1] = E::to_f2(q.y);
            }
        }
    }
    // rounds each value once, to nearest even
    __device__ void store(char *row, bool there, const float2 (&v)[kE / 2]) const {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (!there || !held(c)) continue;
            char *p = row + static_cast<size_t>(at(c)) * kBytes<E>;
            if constexpr (kV == 1) {
                const float f = c & 1 ? v[c / 2].y : v[c / 2].x;
                if constexpr (std::is_same<E, F32>::value)
                    *reinterpret_cast<float *>(p) = f;
                else
                    *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(E::from_f2(f, 0.f));
            } else if constexpr (std::is_same<E, F32>::value) {
                *reinterpret_cast<float4 *>(p) = make_float4(v[2 * c].x, v[2 * c].y, v[2 * c + 1].x, v[2 * c + 1].y);
            } else {
                *reinterpret_cast<uint2 *>(p) = make_uint2(E::from_f2(v[2 * c].x, v[2 * c].y),
                                                           E::from_f2(v[2 * c + 1].x, v[2 * c + 1].y));
            }
        }
    }
    // as the residual stream holds them: rounded to the format and widened again
    __device__ static void round(float2 (&v)[kE / 2]) {
        if constexpr (!std::is_same<E, F32>::value) {
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) v[i] = E::to_f2(E::from_f2(v[i].x, v[i].y));
        }
    }
    __device__ void params(const void *p, bool p32, float other, float2 (&v)[kE / 2]) const {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const float f = !held(c) ? 0.f : p ? load_param<E>(p, at(c) + j, p32) : other;
                const int i = c * kV + j;
                if (i & 1) v[i / 2].y = f; else v[i / 2].x = f;
            }
    }
};

// ------------------------------------------------------------------- units --

// A unit's place in the block and its ring of stages.  kTeam: lanes of a row,
// or 0 for units of several warps.
template <int kTeam>
struct Unit {
    static constexpr bool kMulti = kTeam == 0;
    static constexpr int kRowsPerPass = kMulti ? 1 : 32 / kTeam;
    int warps, index, thread;   // of the unit, in the block, of its unit
    float2 (*meet)[kWarps];     // [2][warps]: sums of the unit's warps
    int turn = 0;

    __device__ Unit(int team_warps, float2 (*exchange)[kWarps]) {
        warps = kMulti ? team_warps : 1;
        const int warp = threadIdx.x >> 5;
        index = kMulti ? warp / warps : warp;
        thread = kMulti ? threadIdx.x - index * warps * 32 : threadIdx.x & 31;
        meet = exchange;
    }
    __device__ int column_thread() const { return kMulti ? thread : thread & (kTeam - 1); }
    __device__ int column_threads() const { return kMulti ? warps * 32 : kTeam; }
    __device__ int row_of_pass() const { return kMulti ? 0 : thread / kTeam; }

    __device__ void sync() const {
        if constexpr (kMulti)
            asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(warps * 32) : "memory");
        else
            __syncwarp();
    }
    // Both sums over a row's threads, in a fixed order; every thread gets them.
    __device__ float2 sum(float2 v) {
#pragma unroll
        for (int o = (kMulti ? 32 : kTeam) / 2; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        if constexpr (kMulti) {
            // two places in turn: a warp that is here again has passed the other's barrier
            float2 *place = meet[turn] + index * warps;
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) place[thread >> 5] = v;
            sync();
            v = place[0];
            for (int w = 1; w < warps; ++w) v = add2(v, place[w]);
        }
        return v;
    }
};

// A tile of a tensor: bytes [from, from + bytes) at `base`, laid into a stage so
// that a 16-byte boundary of memory is one of the stage.  A bulk copy takes what
// lies between such boundaries inside the tensor's `total` bytes, or runs over the
// tile's own ends up to the next one; at the tensor's ends some bytes are left over.
struct Piece {
    const char *begin;     // of the tile
    const char *bulk;      // first byte copied in bulk
    uint32_t bulk_bytes, bytes;

    __device__ Piece(const char *base, int64_t total, int64_t from, int64_t n) {
        begin = base + from;
        bytes = static_cast<uint32_t>(n);
        const uintptr_t b = reinterpret_cast<uintptr_t>(base), lo = (b + 15) & ~uintptr_t(15),
                        hi = (b + total) & ~uintptr_t(15), at = b + from;
        uintptr_t first = at & ~uintptr_t(15), last = (at + n + 15) & ~uintptr_t(15);
        if (first < lo) first = lo;
        if (last > hi) last = hi;
        bulk = reinterpret_cast<const char *>(first);
        bulk_bytes = last > first ? static_cast<uint32_t>(last - first) : 0u;
    }
    __device__ static uint32_t lead(const char *p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15); }
    // where in the stage a byte of memory of this tile lies
    __device__ uint32_t place(const char *p) const {
        return static_cast<uint32_t>(p - (begin - lead(begin)));
    }
    __device__ bool whole() const { return bulk_bytes > 0 && bulk <= begin && bulk + bulk_bytes >= begin + bytes; }
    __device__ void rest(char *stage, int thread, int threads) const {
        for (uint32_t i = thread; i < bytes; i += threads) {
            const char *p = begin + i;
            if (p < bulk || p >= bulk + bulk_bytes) stage[place(p)] = *p;
        }
    }
};

// The tiles of a unit: copies kept `stages` ahead of what is read.
template <typename E, int kTeam>
struct Tiles {
    const LayerNormArgs &a;
    const Unit<kTeam> &unit;
    char *ring;
    uint32_t bars;
    int64_t tile, step;
    int64_t issued;          // first tile not yet asked for (leader)
    int stage = 0, parity = 0, issue_stage = 0;
    bool leader, dead = false;

    __device__ Tiles(const LayerNormArgs &args, const Unit<kTeam> &u, char *r, uint64_t *b)
        : a(args), unit(u) {
        const int units = blockDim.x / (u.warps * 32);
        ring = r + static_cast<size_t>(u.index) * a.stages * a.tensors * a.tile_bytes;
        bars = shared_address(b + u.index * kMaxStages);
        tile = static_cast<int64_t>(blockIdx.x) * units + u.index;
        step = static_cast<int64_t>(gridDim.x) * units;
        issued = tile;
        leader = u.thread == 0;
        if (leader)
            for (int s = 0; s < a.stages; ++s) bar_init(bars + 8 * s, 1);
    }
    __device__ int64_t row_bytes() const { return static_cast<int64_t>(a.width) * kBytes<E>; }
    __device__ int rows_of(int64_t t) const {
        const int64_t left = a.rows - t * a.tile_rows;
        return left < a.tile_rows ? static_cast<int>(left) : a.tile_rows;
    }
    __device__ Piece piece(int64_t t, int k) const {
        return Piece(a.in[k], a.rows * row_bytes(), t * a.tile_rows * row_bytes(), rows_of(t) * row_bytes());
    }
    __device__ char *stage_of(int s, int k) const {
        return ring + (static_cast<size_t>(s) * a.tensors + k) * a.tile_bytes;
    }
    // Ask for the next tile, into the stage that was read longest ago.
    __device__ void issue() {
        if (!leader || dead || issued >= a.tiles) return;
        const uint32_t bar = bars + 8 * issue_stage;
        uint32_t bytes = 0;
        for (int k = 0; k < a.tensors; ++k) bytes += piece(issued, k).bulk_bytes;
        bar_expect(bar, bytes);
        for (int k = 0; k < a.tensors; ++k) {
            const Piece p = piece(issued, k);
            if (p.bulk_bytes)
                bulk_copy(shared_address(stage_of(issue_stage, k)) + p.place(p.bulk), p.bulk, p.bulk_bytes, bar,
                          l2_policy(true));
        }
        issued += step;
        issue_stage = issue_stage + 1 == a.stages ? 0 : issue_stage + 1;
    }
    __device__ void start() {
        for (int s = 0; s < a.stages; ++s) issue();
    }
    // Wait for the present tile and finish its ends.  A thread that gave up says so
    // and goes on without waiting: what it computes is not to be used, but every
    // barrier of the unit is met.
    __device__ void wait() {
        if (!dead && !bar_wait(bars + 8 * stage, parity)) {
            dead = true;
            atomicOr(&g_layer_norm_error, 1u);
        }
        const int64_t from = tile * a.tile_rows * row_bytes();
        if (from >= 16 && from + rows_of(tile) * row_bytes() <= a.rows * row_bytes() - 16) return;
        bool rest = false;
        for (int k = 0; k < a.tensors; ++k) {
            const Piece p = piece(tile, k);
            if (p.whole()) continue;
            p.rest(stage_of(stage, k), unit.thread, unit.warps * 32);
            rest = true;
        }
        if (rest) unit.sync();
    }
    // Row r of the present tile of tensor k.
    __device__ const char *row(int k, int r) const {
        return stage_of(stage, k) + Piece::lead(a.in[k] + tile * a.tile_rows * row_bytes()) + r * row_bytes();
    }
    // The present tile has been read by all threads: its stage takes another.
    __device__ void next() {
        unit.sync();
        issue();
        tile += step;
        if (++stage == a.stages) stage = 0, parity ^= 1;
    }
    // A leader that gave up leaves no copy of its own behind.
    __device__ void end() {
        if (!leader || !dead) return;
        for (int64_t t = tile; t < issued; t += step) {
            bar_wait(bars + 8 * stage, parity);
            if (++stage == a.stages) stage = 0, parity ^= 1;
        }
    }
};

template <int kE>
__device__ __forceinline__ float2 pair_total(const float2 (&v)[kE / 2]) {
    float2 s = v[0];
#pragma unroll
    for (int i = 1; i < kE / 2; ++i) s = add2(s, v[i]);
    return s;
}

// ----------------------------------------------------------------- forward --

// The row's statistics: with m = round(sum x / width) the distances d = x - m are
// small whatever the mean's size, and their own mean, which m's rounding leaves,
// comes off the variance and the result.
template <typename E, int kV, int kE, int kTeam>
__global__ void __launch_bounds__(kWarps * 32, 1) layer_norm_forward(const LayerNormArgs a) {
    extern __shared__ __align__(128) char ring[];
    __shared__ uint64_t bars[kWarps * kMaxStages];
    __shared__ float2 exchange[2][kWarps];
    Unit<kTeam> unit(a.team_warps, exchange);
    const Columns<E, kV, kE> cols(unit.column_thread(), unit.column_threads(), a.width);
    Tiles<E, kTeam> tiles(a, unit, ring, bars);
    __syncthreads();
    pdl_prologue();
    tiles.start();
    float2 w[kE / 2], b[kE / 2];
    cols.params(a.weight, a.p32, 1.f, w);
    cols.params(a.bias, a.p32, 0.f, b);

    const int64_t row_bytes = tiles.row_bytes();
    while (tiles.tile < a.tiles) {
        tiles.wait();
        const int64_t row0 = tiles.tile * a.tile_rows;
        const int rows = tiles.rows_of(tiles.tile);
        for (int r0 = 0; r0 < rows; r0 += unit.kRowsPerPass) {
            const int r = r0 + unit.row_of_pass();
            const bool there = r < rows;
            float2 x[kE / 2];
            cols.load(tiles.row(0, r), there, x);
            if (a.tensors == 2) {
                float2 add[kE / 2];
                cols.load(tiles.row(1, r), there, add);
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) x[i] = add2(x[i], add[i]);
                cols.round(x);
                cols.store(a.total + (row0 + r) * row_bytes, there, x);
            }
            const float2 s = pair_total<kE>(x);
            const float m = unit.sum(make_float2(s.x + s.y, 0.f)).x * a.inv;
            float2 q = both(0.f), p = both(0.f);
#pragma unroll
            for (int c = 0; c < cols.kChunks; ++c) {
                if constexpr (kV == 1) {
                    float &v = c & 1 ? x[c / 2].y : x[c / 2].x;
                    v = cols.held(c) ? v - m : 0.f;
                    p.x += v, q.x = fmaf(v, v, q.x);
                } else {
#pragma unroll
                    for (int i = c * kV / 2; i < (c + 1) * kV / 2; ++i) {
                        x[i] = cols.held(c) ? add2(x[i], both(-m)) : both(0.f);
                        p = add2(p, x[i]), q = fma2(x[i], x[i], q);
                    }
                }
            }
            const float2 t = unit.sum(make_float2(p.x + p.y, q.x + q.y));
            const float m1 = t.x * a.inv;
            float var = fmaf(t.y, a.inv, -m1 * m1);
            if (var < 0.f) var = 0.f;   // (NaN stays)
            const float rstd = __frsqrt_rn(var + a.eps);
#pragma unroll
            for (int i = 0; i < kE / 2; ++i)
                x[i] = fma2(mul2(add2(x[i], both(-m1)), both(rstd)), w[i], b[i]);
            cols.store(a.out + (row0 + r) * row_bytes, there, x);
            if (a.mean && there && unit.column_thread() == 0) {
                a.mean[row0 + r] = m + m1;
                a.rstd[row0 + r] = rstd;
            }
        }
        tiles.next();
    }
    tiles.end();
}

// ---------------------------------------------------------------- backward --

template <typename E, int kV, int kE, int kTeam>
__global__ void __launch_bounds__(kWarps * 32, 1) layer_norm_backward(const LayerNormArgs a) {
    extern __shared__ __align__(128) char ring[];
    __shared__ uint64_t bars[kWarps * kMaxStages];
    __shared__ float2 exchange[2][kWarps];
    Unit<kTeam> unit(a.team_warps, exchange);
    const Columns<E, kV, kE> cols(unit.column_thread(), unit.column_threads(), a.width);
    Tiles<E, kTeam> tiles(a, unit, ring, bars);
    __syncthreads();
    pdl_prologue();
    tiles.start();
    float2 w[kE / 2], gw[kE / 2], gb[kE / 2];
    cols.params(a.weight, a.p32, 1.f, w);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) gw[i] = gb[i] = both(0.f);

    // the statistics of two tiles ahead, a row a lane
    const int lane = threadIdx.x & 31;
    auto stats = [&](int64_t tile, float &m, float &r) {
        const int64_t row = tile * a.tile_rows + lane;
        const bool there = tile < a.tiles && lane < a.tile_rows && row < a.rows;
        m = there ? __ldg(a.mean + row) : 0.f;
        r = there ? __ldg(a.rstd + row) : 0.f;
    };
    float m0, r0s, m1, r1s;
    stats(tiles.tile, m0, r0s);
    stats(tiles.tile + tiles.step, m1, r1s);

    const int64_t row_bytes = tiles.row_bytes();
    while (tiles.tile < a.tiles) {
        float m2, r2s;
        stats(tiles.tile + 2 * tiles.step, m2, r2s);
        tiles.wait();
        const int64_t row0 = tiles.tile * a.tile_rows;
        const int rows = tiles.rows_of(tiles.tile);
        for (int base = 0; base < rows; base += unit.kRowsPerPass) {
            const int r = base + unit.row_of_pass();
            const bool there = r < rows;
            const float mean = __shfl_sync(0xffffffffu, m0, r & 31), rstd = __shfl_sync(0xffffffffu, r0s, r & 31);
            float2 h[kE / 2], g[kE / 2];
            cols.load(tiles.row(0, r), there, h);
            cols.load(tiles.row(1, r), there, g);
            float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) {
                h[i] = mul2(add2(h[i], both(-mean)), both(rstd));
                gb[i] = add2(gb[i], g[i]);
                gw[i] = fma2(g[i], h[i], gw[i]);
                g[i] = mul2(g[i], w[i]);
                s1 = add2(s1, g[i]);
                s2 = fma2(g[i], h[i], s2);
            }
            const float2 t = unit.sum(make_float2(s1.x + s1.y, s2.x + s2.y));
            const float2 c1 = both(-t.x * a.inv), c2 = both(-t.y * a.inv);
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) g[i] = mul2(fma2(h[i], c2, add2(g[i], c1)), both(rstd));
            if (a.tensors == 3) {
                float2 add[kE / 2];
                cols.load(tiles.row(2, r), there, add);
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) g[i] = add2(g[i], add[i]);
            }
            cols.store(a.out + (row0 + r) * row_bytes, there, g);
        }
        m0 = m1, r0s = r1s, m1 = m2, r1s = r2s;
        tiles.next();
    }
    tiles.end();
    if (!a.part) return;

    // The block's sums: a warp's rows, then the units, in their order.
    __syncthreads();
    if constexpr (!Unit<kTeam>::kMulti) {
#pragma unroll
        for (int i = 0; i < kE / 2; ++i)
#pragma unroll
            for (int o = 16; o >= kTeam; o >>= 1) {
                gw[i].x += __shfl_xor_sync(0xffffffffu, gw[i].x, o);
                gw[i].y += __shfl_xor_sync(0xffffffffu, gw[i].y, o);
                gb[i].x += __shfl_xor_sync(0xffffffffu, gb[i].x, o);
                gb[i].y += __shfl_xor_sync(0xffffffffu, gb[i].y, o);
            }
    }
    float *sums = reinterpret_cast<float *>(ring) + static_cast<size_t>(unit.index) * 2 * a.width;
    if (unit.row_of_pass() == 0) {
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            const int c = i / kV;
            if (!cols.held(c)) continue;
            const int at = cols.at(c) + i % kV;
            sums[at] = i & 1 ? gw[i / 2].y : gw[i / 2].x;
            sums[a.width + at] = i & 1 ? gb[i / 2].y : gb[i / 2].x;
        }
    }
    __syncthreads();
    const int units = blockDim.x / (unit.warps * 32);
    const float *all = reinterpret_cast<const float *>(ring);
    float *part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.width;
    for (int i = threadIdx.x; i < 2 * a.width; i += blockDim.x) {
        float s = all[i];
        for (int u = 1; u < units; ++u) s += all[static_cast<size_t>(u) * 2 * a.width + i];
        part[i] = s;
    }
}

// grad_weight (blockIdx.y 0) and grad_bias (1): the blocks' sums, 32 columns a
// block, 32 threads a column.
template <typename E>
__global__ void __launch_bounds__(1024) layer_norm_params(const float *part, int blocks, int width, void *grad_weight,
                                                          void *grad_bias, bool p32) {
    __shared__ float sums[32][33];
    pdl_prologue();
    const int col = blockIdx.x * 32 + threadIdx.x;
    const int64_t at = static_cast<int64_t>(blockIdx.y) * width + col;
    float s = 0.f;
    if (col < width) {
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += 32) s += __ldcg(part + b * 2ll * width + at);
    }
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y >= 32) return;
    const float t = group_sum<32>(sums[threadIdx.x][threadIdx.y]);
    const int out_col = blockIdx.x * 32 + threadIdx.y;
    void *out = blockIdx.y ? grad_bias : grad_weight;
    if (threadIdx.x != 0 || out_col >= width || !out) return;
    if (p32)
        static_cast<float *>(out)[out_col] = t;
    else if constexpr (!std::is_same<E, F32>::value)
        static_cast<uint16_t *>(out)[out_col] = static_cast<uint16_t>(E::from_f2(t, 0.f));
}

// -------------------------------------------------------------------- host --

int64_t bytes_of(wgs_dtype d) { return d == WGS_F32 ? 4 : 2; }
bool dtype_ok(wgs_dtype d) { return d == WGS_F32 || d == WGS_F16 || d == WGS_BF16; }
bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Rows of `width` values of up to 4 bytes that can be addressed.
bool sizes_ok(int64_t rows, int32_t width) {
    return rows >= 0 && width > 0 && rows <= INT64_MAX / 16 / width;
}

constexpr int kMostBlocks = 152;   // of a launch, and of the workspace's sums

template <typename E, int kV, int kE, int kTeam>
wgs_status run_unit(LayerNormArgs a, bool backward, cudaStream_t stream, int *blocks) {
    DeviceInfo dev;
    const wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    a.team_warps = kTeam == 0 ? static_cast<int>(ceil_div(a.width, 32 * kE)) : 1;
    const int per_pass = kTeam == 0 ? 1 : 32 / kTeam;
    const int64_t row_bytes = static_cast<int64_t>(a.width) * kBytes<E>;
    const int most_blocks = dev.sm_count < kMostBlocks ? dev.sm_count : kMostBlocks;
    int units = kWarps / a.team_warps;
    // rows of few units: one tile each, spread over the SMs
    const int64_t passes = ceil_div(a.rows, per_pass);
    if (passes < static_cast<int64_t>(units) * most_blocks)
        units = static_cast<int>(ceil_div(passes, most_blocks));
    // two passes a tile, one where the ring does not hold two stages of that
    auto tile_bytes = [&](int rows) { return (rows * row_bytes + 15) / 16 * 16 + 16; };
    const int64_t room = kRing / (units * a.tensors);
    a.tile_rows = per_pass * (2 * tile_bytes(2 * per_pass) <= room ? 2 : 1);
    if (passes <= static_cast<int64_t>(units) * most_blocks) a.tile_rows = per_pass;
    a.tile_bytes = static_cast<int>(tile_bytes(a.tile_rows));
    a.stages = static_cast<int>(room / a.tile_bytes);
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    a.tiles = ceil_div(a.rows, a.tile_rows);
    a.inv = 1.0f / static_cast<float>(a.width);
    const int64_t want = ceil_div(a.tiles, units);
    *blocks = static_cast<int>(want < most_blocks ? want : most_blocks);
    int64_t smem = static_cast<int64_t>(units) * a.tensors * a.stages * a.tile_bytes;
    if (backward && smem < 8ll * a.width * units) smem = 8ll * a.width * units;
    auto kernel = backward ? layer_norm_backward<E, kV, kE, kTeam> : layer_norm_forward<E, kV, kE, kTeam>;
    // Above 48 KB, its static barriers among them, a kernel needs the runtime's
    // leave, which belongs to the context; asking for the same amount on every
    // call needs no record of it.
    if (smem > 46 << 10 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    return launch(kernel, dim3(*blocks), dim3(units * a.team_warps * 32), static_cast<size_t>(smem), stream, a);
}

// The narrowest unit that holds a row in 16 columns a thread, and the fewest
// columns that do.
template <typename E, int kV>
wgs_status run_width(const LayerNormArgs &a, bool backward, cudaStream_t stream, int *blocks) {
    const int w = a.width;
    auto fits = [&](int lanes, int each) { return w <= lanes * each; };
    if (fits(8, 4)) return run_unit<E, kV, 4, 8>(a, backward, stream, blocks);
    if (fits(8, 8)) return run_unit<E, kV, 8, 8>(a, backward, stream, blocks);
    if (fits(8, 12)) return run_unit<E, kV, 12, 8>(a, backward, stream, blocks);
    if (fits(8, 16)) return run_unit<E, kV, 16, 8>(a, backward, stream, blocks);
    if (fits(16, 12)) return run_unit<E, kV, 12, 16>(a, backward, stream, blocks);
    if (fits(16, 16)) return run_unit<E, kV, 16, 16>(a, backward, stream, blocks);
    if (fits(32, 12)) return run_unit<E, kV, 12, 32>(a, backward, stream, blocks);
    if (fits(32, 16)) return run_unit<E, kV, 16, 32>(a, backward, stream, blocks);
    const int64_t w12 = ceil_div(w, 32 * 12), w16 = ceil_div(w, 32 * 16);
    if (w12 * 12 < w16 * 16 && w12 <= kWarps) return run_unit<E, kV, 12, 0>(a, backward, stream, blocks);
    return run_unit<E, kV, 16, 0>(a, backward, stream, blocks);
}

// Four neighbouring values at a time where every row of every tensor starts on
// as many, else single ones.
template <typename E>
wgs_status run_any(const LayerNormArgs &a, bool backward, cudaStream_t stream, int *blocks) {
    uintptr_t at = reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.total) |
                   (static_cast<uintptr_t>(a.width) * kBytes<E>);
    for (int k = 0; k < a.tensors; ++k) at |= reinterpret_cast<uintptr_t>(a.in[k]);
    return at % (4 * kBytes<E>) == 0 ? run_width<E, 4>(a, backward, stream, blocks)
                                     : run_width<E, 1>(a, backward, stream, blocks);
}

wgs_status run_dtype(const LayerNormArgs &a, wgs_dtype dtype, bool backward, cudaStream_t stream, int *blocks) {
    if (dtype == WGS_F32) return run_any<F32>(a, backward, stream, blocks);
    if (dtype == WGS_F16) return run_any<Fp16>(a, backward, stream, blocks);
    return run_any<Bf16>(a, backward, stream, blocks);
}

// No output may share a byte with another or with an input, but for y or grad_x
// and residual_out, which may each be an input's own buffer.
struct Buffer {
    const void *p;
    int64_t bytes;
    bool in_place;   // an output that may be one of the rows' inputs
    bool rows;       // an input that such an output may be
};

bool buffers_ok(const Buffer *outs, int n_outs, const Buffer *ins, int n_ins) {
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

wgs_status forward(const void *x, const void *branch, bool residual, const void *weight, const void *bias,
                   void *total, void *y, float *mean, float *rstd, int64_t rows, int32_t width, float eps,
                   wgs_dtype dtype, wgs_dtype param_dtype, cudaStream_t stream) {
    if (!dtype_ok(dtype) || (param_dtype != WGS_F32 && param_dtype != dtype)) return WGS_ERR_DTYPE;
    if (width < 1 || width > kMaxWidth) return WGS_ERR_WIDTH;
    if (!sizes_ok(rows, width)) return WGS_ERR_SHAPE;
    if (rows == 0) return WGS_OK;
    if (!x || !y || (residual && (!branch || !total)) || (bias && !weight) ||
        (mean == nullptr) != (rstd == nullptr))
        return WGS_ERR_NULL;
    const int64_t eb = bytes_of(dtype), pb = bytes_of(param_dtype);
    if (!aligned_to(x, eb) || !aligned_to(branch, eb) || !aligned_to(total, eb) || !aligned_to(y, eb) ||
        !aligned_to(weight, pb) || !aligned_to(bias, pb) || !aligned4(mean) || !aligned4(rstd))
        return WGS_ERR_ALIGN;
    const int64_t bytes = rows * width * eb, pbytes = width * pb;
    const Buffer outs[4] = {{y, bytes, true, false}, {total, bytes, true, false},
                            {mean, rows * 4, false, false}, {rstd, rows * 4, false, false}};
    const Buffer ins[4] = {{x, bytes, false, true}, {branch, bytes, false, true},
                           {weight, pbytes, false, false}, {bias, pbytes, false, false}};
    if (!buffers_ok(outs, 4, ins, 4)) return WGS_ERR_ALIAS;
    LayerNormArgs a = {};
    a.in[0] = static_cast<const char *>(x), a.in[1] = static_cast<const char *>(branch);
    a.tensors = residual ? 2 : 1;
    a.out = static_cast<char *>(y), a.total = static_cast<char *>(total);
    a.weight = weight, a.bias = bias, a.mean = mean, a.rstd = rstd;
    a.rows = rows, a.width = width, a.eps = eps, a.p32 = param_dtype == WGS_F32;
    int blocks;
    return run_dtype(a, dtype, false, stream, &blocks);
}

}  // namespace

}  // namespace wgs

// As bias_mask_error_take, for the layer norm's error word.
wgs_status wgs::layer_norm_error_take(unsigned int *seen, cudaStream_t stream) {
    static const unsigned int cleared = 0;
    if (cudaMemcpyFromSymbolAsync(seen, g_layer_norm_error, sizeof(*seen), 0, cudaMemcpyDeviceToHost,
                                  stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_layer_norm_error, &cleared, sizeof(cleared), 0,
                                cudaMemcpyHostToDevice, stream) != cudaSuccess) {
        cudaGetLastError();  // clear this thread's error
        return WGS_ERR_CUDA;
    }
    return WGS_OK;
}

using namespace wgs;

extern "C" wgs_status layer_norm(const void *x, const void *weight, const void *bias, void *y, float *mean,
                                 float *rstd, int64_t rows, int32_t width, float eps, wgs_dtype dtype,
                                 wgs_dtype param_dtype, cudaStream_t stream) {
    return forward(x, nullptr, false, weight, bias, nullptr, y, mean, rstd, rows, width, eps, dtype,
                   param_dtype, stream);
}

extern "C" wgs_status residual_add_layer_norm(const void *residual, const void *branch, const void *weight,
                                              const void *bias, void *residual_out, void *y, float *mean,
                                              float *rstd, int64_t rows, int32_t width, float eps,
                                              wgs_dtype dtype, wgs_dtype param_dtype, cudaStream_t stream) {
    return forward(residual, branch, true, weight, bias, residual_out, y, mean, rstd, rows, width, eps, dtype,
                   param_dtype, stream);
}

extern "C" size_t wgs_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t width) {
    if (width < 1 || width > kMaxWidth || !sizes_ok(rows, width)) return 0;
    return static_cast<size_t>(rows < kMostBlocks ? rows : kMostBlocks) * 8 * width;
}

extern "C" wgs_status layer_norm_bwd(const void *grad_y, const void *x, const float *mean, const float *rstd,
                                     const void *weight, const void *grad_residual, void *grad_x,
                                     void *grad_weight, void *grad_bias, void *workspace,
                                     size_t workspace_bytes, int64_t rows, int32_t width, wgs_dtype dtype,
                                     wgs_dtype param_dtype, cudaStream_t stream) {
    if (!dtype_ok(dtype) || (param_dtype != WGS_F32 && param_dtype != dtype)) return WGS_ERR_DTYPE;
    if (width < 1 || width > kMaxWidth) return WGS_ERR_WIDTH;
    if (!sizes_ok(rows, width)) return WGS_ERR_SHAPE;
    const bool params = grad_weight || grad_bias;
    if (rows == 0 && !params) return WGS_OK;
    const int64_t need = static_cast<int64_t>(wgs_layer_norm_bwd_workspace_bytes(rows, width));
    if (rows > 0 && (!grad_y || !x || !mean || !rstd || !grad_x || (params && !workspace))) return WGS_ERR_NULL;
    if (rows > 0 && params && workspace_bytes < static_cast<size_t>(need)) return WGS_ERR_SHAPE;
    const int64_t eb = bytes_of(dtype), pb = bytes_of(param_dtype);
    if (!aligned_to(grad_y, eb) || !aligned_to(x, eb) || !aligned_to(grad_residual, eb) ||
        !aligned_to(grad_x, eb) || !aligned_to(weight, pb) || !aligned_to(grad_weight, pb) ||
        !aligned_to(grad_bias, pb) || !aligned4(mean) || !aligned4(rstd) || !aligned16(workspace))
        return WGS_ERR_ALIGN;
    const int64_t bytes = rows * width * eb, pbytes = width * pb;
    const Buffer outs[4] = {{grad_x, bytes, true, false}, {grad_weight, pbytes, false, false},
                            {grad_bias, pbytes, false, false}, {params ? workspace : nullptr, need, false, false}};
    const Buffer ins[6] = {{grad_y, bytes, false, true}, {x, bytes, false, true},
                           {grad_residual, bytes, false, true}, {mean, rows * 4, false, false},
                           {rstd, rows * 4, false, false}, {weight, pbytes, false, false}};
    if (!buffers_ok(outs, 4, ins, 6)) return WGS_ERR_ALIAS;
    LayerNormArgs a = {};
    a.in[0] = static_cast<const char *>(x), a.in[1] = static_cast<const char *>(grad_y);
    a.in[2] = static_cast<const char *>(grad_residual);
    a.tensors = grad_residual ? 3 : 2;
    a.out = static_cast<char *>(grad_x);
    a.weight = weight;
    a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    a.part = params ? static_cast<float *>(workspace) : nullptr;
    a.rows = rows, a.width = width, a.p32 = param_dtype == WGS_F32;
    int blocks = 0;
    if (rows > 0) {
        const wgs_status st = run_dtype(a, dtype, true, stream, &blocks);
        if (st != WGS_OK) return st;
    } else {
        DeviceInfo dev;   // no rows: the launch that ends the (empty) sums alone
        const wgs_status st = current_device(&dev);
        if (st != WGS_OK) return st;
    }
    if (!params) return WGS_OK;
    auto kernel = dtype == WGS_F16 ? layer_norm_params<Fp16>
                  : dtype == WGS_BF16 ? layer_norm_params<Bf16> : layer_norm_params<F32>;
    return launch(kernel, dim3(static_cast<unsigned>(ceil_div(width, 32)), 2), dim3(32, 32), 0, stream,
                  static_cast<const float *>(a.part), blocks, width, grad_weight, grad_bias, a.p32);
}
