// Group norm with an activation over channels-last rows, and its gradients
// (sm_103a).
//
// x is [n, s, C]: n samples of s positions with C channels side by side; a
// group is C / groups neighbouring channels over all positions of a sample,
// m = s * C / groups values.  With the group's mean and rstd = 1 / sqrt(var +
// eps) and the channel's weight w and bias b,
//     h = (x - mean) rstd,   z = h w + b,   y = act(z)
// and for a gradient gy of y
//     dz = gy act'(z),   grad_b = sum dz,   grad_w = sum dz h   (all rows)
//     grad_x = rstd (dz w - M(dz w) - h M(dz w h)),  M: mean over the group.
//
// Design.  A sample is cut into slabs of rows, a block each; a thread owns one
// chunk of channels (16 bytes where rows consist of whole ones) and steps
// through the slab's rows, so that a block reads whole rows and a channel's
// weights and sums stay in registers.  Rows reach the block through stages in
// shared memory, copied in bulk several stages ahead.  Pass 1 sums, pass 2
// computes the result; between them the sums of a sample have to meet:
//   * each block of pass 1 leaves one pair of values a group in the workspace,
//     and every block of pass 2, a launch of its own, adds its sample's up;
//   * a small sample, or one of many, is taken through both passes in one
//     launch by a cluster of blocks, which add theirs over distributed shared
//     memory.
// Pass 2 walks its rows backwards: what pass 1 read last is still in L2.  Cutting
// a call into batches of samples that L2 holds, so that pass 2 finds all of
// them there, was measured slower, as launches of their own (the few
// microseconds that each pass takes to start and end) and as one resident
// launch whose blocks wait for one another batch by batch.
#include <cooperative_groups.h>

#include <type_traits>

#include "wgs_common.cuh"

namespace wgs {

namespace {

namespace cg = cooperative_groups;

// Set (never cleared by a kernel) when a block gave up waiting for its own
// copies; read and cleared by wgs_check_error.
__device__ unsigned int g_norm_error;

struct F32 {};

constexpr int kMaxChannels = 4096;
constexpr int kMaxGroups = 2048;
// Threads of a block at most, and blocks of a launch that cuts few samples into
// slabs: two blocks an SM for the forward, whose loops wait for the rows, one
// for the backward, whose threads need twice the registers and whose ring takes
// the shared memory of the SM.  Measured, in us: the forward at [1, 131040, 192]
// fp16 with SiLU and at [8, 32760, 384] bf16 with GELU, the backward at the same
// with 4 samples: 32, 102, 50, 94; with 608 blocks of half the threads 52, 104,
// 95, 122; with those for the forward's pass 2 alone 34 for the first.
constexpr int kThreadsFwd = 384, kBlocksFwd = 304;
constexpr int kThreadsBwd = 512, kBlocksBwd = 152;
// Rows of a thread a stage and stages of the ring: the forward's with one
// tensor, the backward's with two.  Same sizes: the forward with 2 x 6 36 and
// 108, with 1 x 10 46 and 127, with 8 x 2 32 and 102; the backward with 4 x 3
// 50 and 94, with 4 x 2 51 and 97, with 2 x 4 52 and 103, with 1 x 8 65 and
// 125.  The backward's third stage is left out where the values of many
// channels and groups or more blocks an SM need its room, and where each thread
// copies its own rows.
constexpr int kRowsFwd = 4, kStagesFwd = 3;
constexpr int kRowsBwd = 4, kStagesBwd = 2, kMostStages = 3;
// Of a block.  The most that a call needs is 208 KB (backward, 4096 channels
// of FP32 in 2048 groups); a third stage of the backward's fills what is left.
constexpr int kMaxSmem = 220 << 10;
constexpr int kBarBytes = 2 * kMostStages * static_cast<int>(sizeof(uint64_t));  // beside kMaxSmem
constexpr int kMaxCluster = 8;   // of a sample that one cluster holds

enum : int { kNone = 0, kSilu = 1, kGeluTanh = 2 };

// ------------------------------------------------------------ pairs, chunks --

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// FP32 pairs on the packed pipe: each half the correctly rounded operation.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// kV neighbouring elements in one register value, handled as pairs (a single
// element is the first of a pair).
template <typename E, int kV>
struct Chunk {
    static constexpr bool k32 = std::is_same<E, F32>::value;
    static constexpr int kBytes = kV * (k32 ? 4 : 2);
    static constexpr int kPairs = (kV + 1) / 2;
    using Raw = std::conditional_t<
        kBytes == 16, uint4,
        std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>>;

    __device__ static Raw load(const char *p) { return __ldcg(reinterpret_cast<const Raw *>(p)); }

    __device__ static Raw load_shared(uint32_t at) {
        Raw r;
        if constexpr (kBytes == 16)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
        else if constexpr (kBytes == 8)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
        else if constexpr (kBytes == 4)
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
        return r;
    }

    __device__ static uint32_t word_of(const Raw &r, int j) {
        if constexpr (kBytes == 16)
            return word(r, j);
        else if constexpr (kBytes == 8)
            return j == 0 ? r.x : r.y;
        else
            return r;
    }
    // pair p plus c (16-bit elements widen exactly; one rounding)
    __device__ static float2 plus(const Raw &r, int p, float2 c) {
        if constexpr (k32) {
            if constexpr (kV == 1)
                return make_float2(__uint_as_float(r) + c.x, 0.f);
            else
                return add2(make_float2(__uint_as_float(word_of(r, 2 * p)),
                                              __uint_as_float(word_of(r, 2 * p + 1))), c);
        } else {
            return E::widen_add2(word_of(r, p), c);
        }
    }
    __device__ static float2 wide(const Raw &r, int p) {
        if constexpr (k32) {
            if constexpr (kV == 1)
                return make_float2(__uint_as_float(r), 0.f);
            else
                return make_float2(__uint_as_float(word_of(r, 2 * p)), __uint_as_float(word_of(r, 2 * p + 1)));
        } else {
            return E::to_f2(word_of(r, p));
        }
    }
    // rounds each value once, to nearest even; `policy` says how L2 keeps the line
    __device__ static void store(char *p, const float2 (&v)[kPairs], uint64_t policy) {
        Raw r;
        if constexpr (k32) {
            if constexpr (kV == 4)
                r = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y),
                               __float_as_uint(v[1].x), __float_as_uint(v[1].y));
            else if constexpr (kV == 2)
                r = make_uint2(__float_as_uint(v[0].x), __float_as_uint(v[0].y));
            else
                r = __float_as_uint(v[0].x);
        } else if constexpr (kV == 8) {
            r = make_uint4(E::from_f2(v[0].x, v[0].y), E::from_f2(v[1].x, v[1].y),
                           E::from_f2(v[2].x, v[2].y), E::from_f2(v[3].x, v[3].y));
        } else {
            r = static_cast<Raw>(E::from_f2(v[0].x, v[0].y));
        }
        if constexpr (kBytes == 16)
            asm volatile("st.global.L2::cache_hint.v4.b32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "l"(policy) : "memory");
        else
            *reinterpret_cast<Raw *>(p) = r;
    }
};

// A weight or bias: FP32 or the tensor's own format; NULL is the default.
// Read from L2, as all that pass 2 reads before it waits: L1 may hold an older
// line.
template <typename E>
__device__ __forceinline__ float param(const void *p, int64_t c, bool p32, float otherwise) {
    if (!p) return otherwise;
    if (p32) return __ldcg(static_cast<const float *>(p) + c);
    if constexpr (std::is_same<E, F32>::value)
        return otherwise;  // FP32 tensors have FP32 weights
    else
        return E::to_f2(__ldcg(static_cast<const uint16_t *>(p) + c)).x;
}

template <typename E>
__device__ __forceinline__ void store_param(void *p, int64_t c, bool p32, float v) {
    if (p32) {
        static_cast<float *>(p)[c] = v;
    } else if constexpr (!std::is_same<E, F32>::value) {
        static_cast<uint16_t *>(p)[c] = static_cast<uint16_t>(E::from_f2(v, 0.f));
    }
}

constexpr float kTwoK = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kCubic = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-q)), q = z for SiLU and z (kTwoK + kTwoK kCubic z^2) for the
// GELU (0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u)), which does not cancel for
// negative z).  16-bit tensors take the hardware's exp2 and reciprocal
// (relative errors of a few 2^-22, and that of the argument's rounding: far
// below the output's half step), with log2(e) in the constants; FP32 tensors
// take expf and a division.
template <int kAct, bool k32>
__device__ __forceinline__ float2 gate(float2 z) {
    constexpr float m = k32 ? -1.0f : -kLog2e;
    float2 t;
    if constexpr (kAct == kSilu)
        t = mul2(z, both(m));
    else
        t = mul2(z, fma2(mul2(z, z), both(m * kTwoK * kCubic), both(m * kTwoK)));
    if constexpr (k32) {
        return make_float2(1.0f / (1.0f + expf(t.x)), 1.0f / (1.0f + expf(t.y)));
    } else {
        float2 e, s;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
        e = add2(e, both(1.0f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(e.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(e.y));
        return s;
    }
}

template <int kAct, bool k32>
__device__ __forceinline__ float2 act(float2 z) {
    if constexpr (kAct == kNone) return z;
    return mul2(z, gate<kAct, k32>(z));
}

// act'(z) = s + z s (1 - s) q', with s the gate.
template <int kAct, bool k32>
__device__ __forceinline__ float2 act_grad(float2 z) {
    if constexpr (kAct == kNone) return both(1.0f);
    const float2 s = gate<kAct, k32>(z);
    const float2 p = mul2(z, s);
    const float2 rest = fma2(s, both(-1.0f), both(1.0f));
    if constexpr (kAct == kSilu) {
        return fma2(p, rest, s);
    } else {
        // q' = kTwoK + 3 kTwoK kCubic z^2.  Far out z s (1 - s) is 0, and there
        // the slope may be infinite: it is cut to what a finite z^2 gives
        float2 z2 = mul2(z, z);
        z2 = make_float2(fminf(z2.x, 1e30f), fminf(z2.y, 1e30f));
        return fma2(mul2(p, rest), fma2(z2, both(3.0f * kTwoK * kCubic), both(kTwoK)), s);
    }
}

// max(v, 0) that keeps NaN.
__device__ __forceinline__ float not_below_zero(float v) { return v < 0.f ? 0.f : v; }

// -------------------------------------------------------------------- work --

// A sample's rows in `count` slabs of `rows`, one more in the first `longer`.
struct Slabs {
    int32_t count, rows, longer;
    // first row of slab s
    __device__ int32_t start(int32_t s) const { return s * rows + min(s, longer); }
    // rows of n slabs from slab s on
    __device__ int32_t of(int32_t s, int32_t n) const { return n * rows + max(min(longer - s, n), 0); }
};

struct NormArgs {
    const char *x, *gy;         // gy: backward
    const void *weight, *bias;  // [C] or NULL
    char *out;                  // y, or grad_x
    float *mean, *rstd;         // [n, groups]; written by the forward unless NULL
    float2 *groups_part;        // [n, clusters, groups]: (mean, M2), or the sums of (d, d h)
    float2 *chan_part;          // backward: [n, clusters, C]: the sums of (dz, dz h)
    void *grad_weight, *grad_bias;
    int64_t spatial;
    int32_t channels, groups, per_group;
    int32_t group_shift;        // log2 of the lanes that add a group's channels up
    int32_t chunks;             // of a row
    int32_t cluster, clusters;  // blocks of a cluster, clusters of a sample
    Slabs slabs1, slabs2;       // of the two passes
    int32_t ring;               // bytes of the slots
    int32_t stages;             // of rows copied in bulk
    int32_t behind;             // bytes before what pass 1 of the backward keeps of the groups
    int32_t passes;             // of the launch: 1, 2 or 3 (both)
    bool last_use;              // pass 2's lines need not stay in L2: the call is larger
    float eps;
    bool p32;                   // weight and bias are FP32
};

// The first launch of a call waits for what came before on the stream.  A
// launch of pass 2 follows one of pass 1 of the same call, which has waited
// for all that, and needs of it only the workspace's sums: it may read the
// call's inputs at once, and waits (wait_for_sums) before it reads the sums or
// writes.
__device__ __forceinline__ void start_launch(const NormArgs &a) {
#if WGS_PDL
    if (a.passes != 2) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#endif
}
__device__ __forceinline__ void wait_for_sums(const NormArgs &a) {
#if WGS_PDL
    if (a.passes == 2) asm volatile("griddepcontrol.wait;" ::: "memory");
#endif
}

// A block's work: a slab of a sample in pass 1 or 2; and what its thread is in
// it: chunk j and row group g of the columns x row groups that the block walks
// side by side.
struct Job {
    int64_t sample;
    int32_t cl, rank;  // cluster of the sample, block of the cluster (pass 1)
    int32_t r0, rows;  // first row, rows
    int j, g, columns, row_groups, tid, threads;
    __device__ explicit Job(const NormArgs &a) {
        const Slabs &slabs = a.passes & 1 ? a.slabs1 : a.slabs2;
        const int32_t slab = blockIdx.x;
        sample = blockIdx.y;
        rank = slab & (a.cluster - 1);  // clusters have a power of two
        cl = slab / a.cluster;
        r0 = slabs.start(slab);
        rows = slabs.of(slab, 1);
        j = threadIdx.x, g = threadIdx.y, columns = blockDim.x, row_groups = blockDim.y;
        tid = g * columns + j, threads = columns * row_groups;
    }
    // rows of this thread
    __device__ int32_t mine() const { return g < rows ? (rows - g + row_groups - 1) / row_groups : 0; }
};

// Rows of a thread after which run() calls between() first; then 8 times as many.
constexpr int32_t kMove = 8;
static_assert(kMove % kRowsFwd == 0 && kMove % kRowsBwd == 0, "between whole stages");
struct Nothing {
    __device__ void operator()(int32_t) const {}
};

// A slab's rows on their way through shared memory: kRows rows of every thread
// a stage, kStages stages, f(chunk of each tensor, its byte offset) for each
// of the thread's places in run(), and once the thread has had 8, 64, 512 ... rows
// between(their number), where it hides behind copies under way.
//
// Rows of whole 16-byte chunks: one thread copies a stage's rows in bulk (TMA;
// they are one piece of memory where the block walks whole rows), and an
// mbarrier a stage tells that they have come, another that every warp has
// read them.  A thread spends nothing on addresses and copies of its own.
struct Bars {
    uint32_t full, empty;  // of stage 0; 8 bytes a stage
    int stages;
    int stage;             // of the next use
    uint32_t phase;        // its parity
    bool used;             // a stage has been
};

template <typename C, int kTensors, int kRows, int kStages>  // stages, or 0: bars.stages
struct Bulk {
    const Job &job;
    Bars &bars;
    const char *src[kTensors];
    uint32_t ring;
    int64_t base;       // byte offset of the slab's first row, at the block's first chunk
    int64_t row_bytes;
    int32_t wide;       // chunks of a row that the block takes
    int32_t count;      // stages of the slab
    bool reverse;
    uint64_t policy;

    __device__ Bulk(const Job &job_, Bars &bars_) : job(job_), bars(bars_) {}
    __device__ static void wait(uint32_t bar, uint32_t parity) {
        if (!bar_wait(bar, parity)) atomicOr(&g_norm_error, 1u);
    }
    __device__ int stages() const { return kStages ? kStages : bars.stages; }
    __device__ uint32_t stage_bytes() const { return job.threads * C::kBytes * kTensors * kRows; }
    __device__ int32_t stage_rows() const { return job.row_groups * kRows; }

    // by one thread: the slab's i-th stage into slot `stage`
    __device__ void copy(int32_t i, int stage) const {
        const int32_t r0 = (reverse ? count - 1 - i : i) * stage_rows(), rows = min(stage_rows(), job.rows - r0);
        const uint32_t bar = bars.full + 8 * stage, to = ring + stage * stage_bytes();
        const uint32_t seg = wide * C::kBytes;
        bar_expect(bar, rows * seg * kTensors);
        const int64_t from = base + r0 * row_bytes;
#pragma unroll
        for (int t = 0; t < kTensors; ++t) {
            const uint32_t at = to + t * job.threads * C::kBytes * kRows;
            if (seg == row_bytes)
                bulk_copy(at, src[t] + from, rows * seg, bar, policy);
            else
                for (int32_t r = 0; r < rows; ++r)
                    bulk_copy(at + r * (job.columns * C::kBytes), src[t] + from + r * row_bytes, seg, bar, policy);
        }
    }
    // every slot has been read (the block has met at a barrier since)
    __device__ void start(const float2 *smem, int64_t base_, int64_t row_bytes_, int32_t wide_, bool reverse_,
                          uint64_t policy_) {
        ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
        base = base_, row_bytes = row_bytes_, wide = wide_, reverse = reverse_, policy = policy_;
        count = (job.rows + stage_rows() - 1) / stage_rows();
        if (job.tid == 0) {
            // what the block wrote to the slots comes before the copies
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            for (int i = 0; i < stages() - 1 && i < count; ++i)
                copy(i, bars.stage + i < stages() ? bars.stage + i : bars.stage + i - stages());
        }
    }
    template <typename Use, typename Between = Nothing>
    __device__ void run(Use f, Between between = {}) {
        int32_t move = kMove / kRows;
        const uint32_t stride = job.threads * C::kBytes;
        const int32_t step = static_cast<int32_t>(job.row_groups * row_bytes);
        int64_t at = base + job.g * row_bytes + job.j * C::kBytes;
        if (reverse) at += static_cast<int64_t>(count - 1) * kRows * step;
        for (int32_t i = 0; i < count; ++i) {
            if (job.tid == 0 && i + stages() - 1 < count) {
                // into the slot that was read last, when all warps have
                const int free = bars.stage == 0 ? stages() - 1 : bars.stage - 1;
                if (bars.used) wait(bars.empty + 8 * free, bars.stage == 0 ? bars.phase ^ 1 : bars.phase);
                copy(i + stages() - 1, free);
            }
            if (i == move) {
                between(i * kRows);
                move = move < INT32_MAX / 8 ? 8 * move : INT32_MAX;
            }
            wait(bars.full + 8 * bars.stage, bars.phase);
            const uint32_t slot = ring + bars.stage * stage_bytes() + job.tid * C::kBytes;
            auto load = [&](int u, typename C::Raw (&v)[kTensors]) {
#pragma unroll
                for (int t = 0; t < kTensors; ++t) v[t] = C::load_shared(slot + (t * kRows + u) * stride);
            };
            // only the slab's last stage can be short
            int32_t live = kRows * job.row_groups;
            if (i == (reverse ? 0 : count - 1)) live = job.rows - (count - 1) * live;
            live = job.j < wide ? live - job.g : 0;
            if (live > (kRows - 1) * job.row_groups) {
                typename C::Raw v[kRows][kTensors];
#pragma unroll
                for (int u = 0; u < kRows; ++u) load(u, v[u]);
#pragma unroll
                for (int u = 0; u < kRows; ++u) f(v[u], at + u * step);
            } else {
                for (int u = 0; u * job.row_groups < live; ++u) {
                    typename C::Raw v[kTensors];
                    load(u, v);
                    f(v, at + u * step);
                }
            }
            at += reverse ? -kRows * step : kRows * step;
            __syncwarp();
            if ((job.tid & 31) == 0) bar_arrive(bars.empty + 8 * bars.stage);
            bars.used = true;
            if (++bars.stage == stages()) bars.stage = 0, bars.phase ^= 1;
        }
    }
};

// Other rows: each thread copies its own chunks into its own slots
// (cp.async), which needs no barrier; 2-byte chunks, which cp.async does not
// know, are loaded several rows at a time.
template <typename C, int kTensors, int kRows, int kStages>
struct Own {
    static constexpr bool kAsync = C::kBytes >= 4;
    const Job &job;
    const char *src[kTensors];
    uint32_t slots, stride;  // address of the thread's first slot, bytes from slot to slot
    int64_t at;              // offset of the next chunk to use
    int32_t step, left;

    __device__ Own(const Job &job_, Bars &) : job(job_) {}

    __device__ void copy(uint32_t to, int64_t from, int32_t rows) const {
        if constexpr (kAsync) {
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                if (u < rows) {
#pragma unroll
                    for (int t = 0; t < kTensors; ++t)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + (u * kTensors + t) * stride), "l"(src[t] + from + u * step), "n"(C::kBytes) : "memory");
                }
            cp_async_commit();
        }
    }
    __device__ void start(const float2 *smem, int64_t base, int64_t row_bytes, int32_t wide, bool reverse, uint64_t) {
        slots = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + job.tid * C::kBytes;
        stride = job.threads * C::kBytes;
        left = job.j < wide ? job.mine() : 0;
        step = static_cast<int32_t>(job.row_groups * row_bytes);
        at = base + job.g * row_bytes + job.j * C::kBytes;
        if (reverse) at += static_cast<int64_t>(left - 1) * step, step = -step;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            copy(slots + i * kRows * kTensors * stride, at + i * kRows * step, left - i * kRows);
    }
    template <typename Use, typename Between = Nothing>
    __device__ void run(Use f, Between between = {}) {
        const int32_t all = left;
        int32_t move = kMove;
        auto moves = [&] {
            if (all - left != move) return;
            between(move);
            move = move < INT32_MAX / 8 ? 8 * move : INT32_MAX;
        };
        if constexpr (kAsync) {
            const uint32_t stage = kRows * kTensors * stride;
            const int32_t lead = (kStages - 1) * kRows * step;
            uint32_t use = slots, free = slots + (kStages - 1) * stage;
            for (; left > 0; left -= kRows, at += kRows * step) {
                cp_async_wait<kStages - 2>();
                typename C::Raw v[kRows][kTensors];
#pragma unroll
                for (int u = 0; u < kRows; ++u)
#pragma unroll
                    for (int t = 0; t < kTensors; ++t) v[u][t] = C::load_shared(use + (u * kTensors + t) * stride);
                copy(free, at + lead, left - (kStages - 1) * kRows);
                free = use;
                use = use == slots + (kStages - 1) * stage ? slots : use + stage;
                moves();
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    if (u < left) f(v[u], at + u * step);
            }
            cp_async_wait<0>();
        } else {
            constexpr int kAhead = 4;
            for (; left > 0; left -= kAhead, at += kAhead * step) {
                typename C::Raw v[kAhead][kTensors];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (u < left)
#pragma unroll
                        for (int t = 0; t < kTensors; ++t) v[u][t] = C::load(src[t] + at + u * step);
                moves();
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (u < left) f(v[u], at + u * step);
            }
        }
    }
};

template <typename C, int kTensors>
using Stream = std::conditional_t<
    C::kBytes == 16,
    std::conditional_t<kTensors == 1, Bulk<C, 1, kRowsFwd, kStagesFwd>, Bulk<C, 2, kRowsBwd, 0>>,
    std::conditional_t<kTensors == 1, Own<C, 1, kRowsFwd, kStagesFwd>, Own<C, 2, kRowsBwd, kStagesBwd>>>;

// The block's barriers, before its first job.
__device__ __forceinline__ Bars make_bars(uint64_t *storage, int stages) {
    Bars b;
    b.stages = stages;
    b.full = static_cast<uint32_t>(__cvta_generic_to_shared(storage));
    b.empty = b.full + 8 * kMostStages;
    b.stage = 0, b.phase = 0, b.used = false;
    if (threadIdx.x == 0 && threadIdx.y == 0) {
        for (int i = 0; i < stages; ++i) {
            bar_init(b.full + 8 * i, 1);
            bar_init(b.empty + 8 * i, (blockDim.x * blockDim.y + 31) / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    return b;
}

// Add the threads' pairs of sums (s1, s2) over the row groups, in order;
// done(element of the chunk, its channel, its sums) is called once a channel
// by a thread of the channel's chunk.  Every thread calls it.  In `red` a row group's
// values lie element by element of the chunk, so that neighbouring threads
// touch neighbouring words.
template <int kV, int kPairs, typename Done>
__device__ __forceinline__ void add_row_groups(float2 *red, const Job &job, int32_t c0, int wide,
                                               const float2 (&s1)[kPairs],
                                               const float2 (&s2)[kPairs], Done done) {
    __syncthreads();  // the slots that `red` lies over have been read
    if (job.j < wide) {
        float2 *mine = red + job.g * wide * kV + job.j;
#pragma unroll
        for (int e = 0; e < kV; ++e)
            mine[e * wide] = e & 1 ? make_float2(s1[e / 2].y, s2[e / 2].y) : make_float2(s1[e / 2].x, s2[e / 2].x);
    }
    __syncthreads();
    if (job.j < wide)
        for (int e = job.g; e < kV; e += job.row_groups) {
            const float2 *p = red + e * wide + job.j;
            float2 t = *p;
#pragma unroll 4
            for (int g = 1; g < job.row_groups; ++g) t = add2(t, p[g * wide * kV]);
            done(e, (c0 + job.j) * kV + e, t);
        }
    __syncthreads();
}

// Sum over the 2^shift neighbouring lanes of a group.
__device__ __forceinline__ float lanes_sum(float v, int shift) {
    for (int o = 1 << shift >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// For every group g: f(g, first lane, lanes) with all threads of full warps.
template <typename F>
__device__ __forceinline__ void each_group(const NormArgs &a, const Job &job, F f) {
    const int whole = job.threads & ~31;
    if (job.tid >= whole) return;
    const int at_a_time = whole >> a.group_shift;
    for (int g0 = 0; g0 < a.groups; g0 += at_a_time)
        f(g0 + (job.tid >> a.group_shift), job.tid & ((1 << a.group_shift) - 1), 1 << a.group_shift);
}

// Values of a group in `count` of pass 1's slabs from slab s on.
__device__ __forceinline__ float values_of(const NormArgs &a, int32_t s, int32_t count) {
    return static_cast<float>(a.slabs1.of(s, count)) * static_cast<float>(a.per_group);
}

// For every group g: the sum of its pairs over the parts, in a fixed order, to
// done(g, sum).  part[parts][groups].  Neighbouring threads take neighbouring groups, and the
// threads beyond the groups a share of the parts each.  smem holds a pair a
// thread.  then() runs once the first loads are under way: what it starts
// should not be ahead of them on the way to memory.
template <typename Then, typename Done>
__device__ __forceinline__ void add_parts(float2 *smem, const Job &job, const float2 *part, int groups, int parts,
                                          Then then, Done done) {
    constexpr int kFirst = 16;
    const int wide = min(groups, job.threads);
    const int lanes = job.threads / wide;
    const int l = job.tid / wide, j = job.tid - l * wide;
    for (int g0 = 0; g0 < groups; g0 += wide) {
        const int g = g0 + j;
        const bool live = l < lanes && g < groups;
        const float2 *q = part + (live ? g : 0);
        float2 v[kFirst];
#pragma unroll
        for (int k = 0; k < kFirst; ++k)
            if (live && l + k * lanes < parts) v[k] = __ldcg(q + (l + k * lanes) * groups);
        if (g0 == 0) then();
        float2 t = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kFirst; ++k)
            if (live && l + k * lanes < parts) t = add2(t, v[k]);
        if (live)
            for (int p = l + kFirst * lanes; p < parts; p += lanes) t = add2(t, __ldcg(q + p * groups));
        smem[job.tid] = t;
        __syncthreads();
        if (l == 0 && live) {
#pragma unroll 8
            for (int k = 1; k < min(lanes, parts); ++k) t = add2(t, smem[k * wide + j]);
            done(g, t);
        }
        __syncthreads();
    }
}

// A set of values: how many, their mean (here from some origin) and M2.
struct Stats {
    float n = 0.f, mean = 0.f, m2 = 0.f;
    // m > 0 more, whose mean is d further on: the joint mean is d m / (n + m)
    // further on, and M2 grows by theirs and d^2 n m / (n + m)
    __device__ void join(float m, float at, float more) {
        const float share = __fdividef(m, n + m), d = at - mean;
        m2 += fmaf(d * d, n * share, more);
        mean = fmaf(d, share, mean);
        n += m;
    }
};

// For every group the statistics of all parts, each a (mean, M2), as add_parts
// adds, joined one by one: a sum about one part's mean would cancel by a factor of
// the parts where that one lies far from all others (a slab of zeros before values
// 100 deviations off left rstd 6e-5 off, of 152 parts).  smem holds a pair and a
// count a thread.
template <typename Count, typename Then, typename Done>
__device__ __forceinline__ void join_parts(float2 *smem, const Job &job, const float2 *part, int groups, int parts,
                                            Count count, Then then, Done done) {
    if (parts == 1) {  // a sample of one cluster
        float2 v = __ldcg(part + min(job.tid, groups - 1));
        then();
        for (int g = job.tid; g < groups; g += job.threads) {
            if (g != job.tid) v = __ldcg(part + g);
            Stats t;
            t.mean = v.x, t.m2 = v.y;
            done(g, t);
        }
        __syncthreads();
        return;
    }
    constexpr int kAhead = 16, kMostLanes = 16;
    float *counts = reinterpret_cast<float *>(smem + job.threads);
    const int wide = min(groups, job.threads);
    const int lanes = min(min(job.threads / wide, kMostLanes), parts);
    const int l = job.tid / wide, j = job.tid - l * wide;
    for (int g0 = 0; g0 < groups; g0 += wide) {
        const int g = g0 + j;
        const bool live = l < lanes && g < groups;
        const float2 *q = part + (live ? g : 0);
        const float own = __ldcg(q).x;  // the origin
        Stats t;
        auto batch = [&](int first, auto started) {
            float2 v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                v[k] = live && first + k * lanes < parts ? __ldcg(q + (first + k * lanes) * groups) : make_float2(own, 0.f);
            started();
            // a part that is not there counts nothing (each lane has its first)
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int p = first + k * lanes;
                t.join(p < parts ? count(p) : 0.f, v[k].x - own, v[k].y);
            }
        };
        batch(l, [&] { if (g0 == 0) then(); });
        for (int p = l + kAhead * lanes; p < parts; p += kAhead * lanes) batch(p, [] {});
        smem[job.tid] = make_float2(t.mean, t.m2), counts[job.tid] = t.n;
        __syncthreads();
        if (l == 0 && live) {
#pragma unroll 4
            for (int k = 1; k < lanes; ++k) {
                const float2 more = smem[k * wide + j];
                t.join(counts[k * wide + j], more.x, more.y);
            }
            t.mean += own;
            done(g, t);
        }
        __syncthreads();
    }
}

// enter(group) at a chunk's first channel and where another group begins,
// f(element, channel) for each of its channels.
template <int kV, typename Enter, typename F>
__device__ __forceinline__ void each_channel(const NormArgs &a, int32_t chunk, Enter enter, F f) {
    int32_t g = chunk * kV / a.per_group, in_group = chunk * kV - g * a.per_group;
    enter(g);
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        if (in_group == a.per_group) {
            in_group = 0;
            enter(++g);
        }
        f(e);
        ++in_group;
    }
}

__device__ __forceinline__ void set_half(float2 *v, int e, float x) {
    if (e & 1) v[e / 2].y = x; else v[e / 2].x = x;
}

// Forward, pass 1 (reads x once; bound by DRAM): (mean, M2) of every group over
// the rows of a cluster, M2 the sum of the squared distances from the mean.  A
// thread sums x - k and its square, k first the channel's value in its first
// row and after 8, 64, 512 ... rows their mean: M2 = sum d^2 - (sum d)^2 / n then
// cancels by a small factor at most, whatever the mean and wherever a row lies
// far from all others.  (With one k for a slab such a row in its first place cost
// a factor of the slab's rows: rstd off by 1e-3 after 4096.)  Threads' parts are
// joined one by one, those of a cluster's blocks, 8 at most, about the first one's
// mean.
template <typename E, int kV>
__device__ void stats_pass(const NormArgs &a, const Job &job, Bars &bars, float2 *smem) {
    using C = Chunk<E, kV>;
    constexpr int kP = C::kPairs;
    float2 *ch = smem, *red = smem + a.channels;  // red holds the groups' results in the end
    float2 *ring = job.columns == a.chunks ? smem : red;
    const int64_t row_bytes = static_cast<int64_t>(a.chunks) * C::kBytes;
    const int64_t origin = (job.sample * a.spatial + job.r0) * row_bytes;
    for (int32_t c0 = 0; c0 < a.chunks; c0 += job.columns) {
        const int32_t wide = min(job.columns, a.chunks - c0), count = wide * kV;
        const int64_t o = origin + c0 * C::kBytes;
        // first the few values that the block starts with, before its copies
        // fill the way to memory
        typename C::Raw lead = {};
        if (job.j < wide && job.g < job.rows) lead = C::load(a.x + o + job.g * row_bytes + job.j * C::kBytes);
        Stream<C, 1> in(job, bars);
        in.src[0] = a.x;
        in.start(ring, o, row_bytes, wide, false, l2_policy(false));
        // row groups that have rows, and their rows: one more in the first `more`
        const int live = min(job.row_groups, job.rows), each = job.rows / job.row_groups;
        const int more = job.rows - each * job.row_groups;
        const float few = static_cast<float>(each);
        auto rows_of = [&](int g) { return g < more ? few + 1.f : few; };
        // Narrow rows have many row groups, which are joined in two steps, kShares
        // shares of them side by side: [1, 2000000, 8] fp16 25 us, in one step 30.
        constexpr int kShares = 8;
        const bool narrow = live >= max(kShares * kV, 64);
        auto rows_of_share = [&](int l) {
            const int with = max(more - l + kShares - 1, 0) / kShares;
            return fmaf(static_cast<float>((live - l + kShares - 1) / kShares), few, static_cast<float>(with));
        };
        const float inv = 1.0f / rows_of(job.g);
        float2 k[kP], s1[kP], s2[kP];  // -k
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            k[p] = C::wide(lead, p);
            k[p].x = -k[p].x, k[p].y = -k[p].y;
            s1[p] = s2[p] = both(0.f);
        }
        in.run(
            [&](const typename C::Raw (&v)[1], int64_t) {
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const float2 d = C::plus(v[0], p, k[p]);
                    s1[p] = add2(s1[p], d);
                    s2[p] = fma2(d, d, s2[p]);
                }
            },
            [&](int32_t rows) {
                // k moves by c: sum (d - c) = s1 - n c, sum (d - c)^2 = s2 - c (s1 + (s1 - n c))
                const float n = static_cast<float>(rows);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const float2 to = fma2(s1[p], both(-1.0f / n), k[p]);
                    const float2 c = add2(k[p], make_float2(-to.x, -to.y));
                    const float2 t = fma2(c, both(-n), s1[p]);
                    s2[p] = fma2(make_float2(-c.x, -c.y), add2(s1[p], t), s2[p]);
                    s1[p] = t, k[p] = to;
                }
            });
        // the row groups: the threads' (mean, M2) by chunk element, so that
        // neighbouring threads touch neighbouring words
        __syncthreads();  // the slots that `red` lies over have been read
        if (job.j < wide) {
            float2 *to = red + job.g * count + job.j;
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float2 m = job.g < live ? mul2(s1[p], both(inv)) : both(0.f);
                const float2 m2 = fma2(make_float2(-m.x, -m.y), s1[p], s2[p]);
                to[2 * p * wide] = make_float2(m.x - k[p].x, not_below_zero(m2.x));
                if constexpr (kV > 1) to[(2 * p + 1) * wide] = make_float2(m.y - k[p].y, not_below_zero(m2.y));
            }
        }
        __syncthreads();
        auto join = [&](const float2 *q, int first, int step, int end, auto rows) {
            const float2 own = q[first * count];
            Stats t;
            t.n = rows(first), t.m2 = own.y;
#pragma unroll 4
            for (int g = first + step; g < end; g += step) {
                const float2 v = q[g * count];
                t.join(rows(g), v.x - own.x, v.y);
            }
            return make_float2(own.x + t.mean, t.m2);
        };
        if (__builtin_expect(narrow, 0)) {
            const int e = job.g % kV, l = job.g / kV;
            float2 *q = red + e * wide + job.j;
            if (job.j < wide && l < kShares) q[l * count] = join(q, l, kShares, live, rows_of);
            __syncthreads();
            if (job.j < wide && l == 0) ch[(c0 + job.j) * kV + e] = join(q, 0, 1, kShares, rows_of_share);
        } else if (job.j < wide) {
            for (int e = job.g; e < kV; e += job.row_groups)
                ch[(c0 + job.j) * kV + e] = join(red + e * wide + job.j, 0, 1, live, rows_of);
        }
        __syncthreads();
    }
    float2 *out = a.groups_part + (job.sample * a.clusters + job.cl) * a.groups;
    // the channels of a group, in two steps: the mean, M2 about it
    each_group(a, job, [&](int g, int lane, int lanes) {
        const bool live = g < a.groups;
        const float2 *p = ch + (live ? g : 0) * a.per_group;
        const float ref = p[0].x;
        float mean = 0.f, m2 = 0.f;
        for (int i = lane; i < a.per_group; i += lanes) mean += p[i].x - ref;
        mean = ref + lanes_sum(mean, a.group_shift) / static_cast<float>(a.per_group);
        for (int i = lane; i < a.per_group; i += lanes) {
            const float d = p[i].x - mean;
            m2 += fmaf(static_cast<float>(job.rows) * d, d, p[i].y);
        }
        m2 = lanes_sum(m2, a.group_shift);
        if (live && lane == 0) (a.cluster == 1 ? out : red)[g] = make_float2(mean, m2);
    });
    if (a.cluster == 1) {
        __syncthreads();
        return;
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int32_t slab0 = job.cl * a.cluster;
    const float n_all = values_of(a, slab0, a.cluster);
    for (int g = job.rank * job.threads + job.tid; g < a.groups; g += a.cluster * job.threads) {
        const float ref = cluster.map_shared_rank(red, 0)[g].x;
        float s1 = 0.f, s2 = 0.f;
        for (int r = 0; r < a.cluster; ++r) {
            const float2 v = cluster.map_shared_rank(red, r)[g];
            const float n = values_of(a, slab0 + r, 1), d = n > 0.f ? v.x - ref : 0.f;
            s1 = fmaf(n, d, s1);
            s2 += fmaf(n * d, d, v.y);
        }
        const float m = s1 / n_all;
        out[g] = make_float2(ref + m, not_below_zero(fmaf(-m, s1, s2)));
    }
    cluster.sync();  // the others' shared memory has been read; the result is visible to them
}

// Forward, pass 2 (reads x again, writes y), the slab's last rows first.  The
// statistics of the groups lie behind the slots.  At [1, 131040, 192] fp16, 50
// MB, pass 1 reads x from DRAM and pass 2 finds all but 4 MB in L2; the call's
// 100 MB take 32 us, 3.1 TB/s, of which each pass spends a few us on its start
// and its last blocks, and pass 2 on the join.  At [8, 32760, 384] bf16, 201 MB,
// most of x comes from DRAM twice: 102 us for 403 MB (604 MB moved, 5.9 TB/s).
template <typename E, int kV, int kAct>
__device__ void apply_pass(const NormArgs &a, const Job &job, Bars &bars, float2 *smem) {
    using C = Chunk<E, kV>;
    constexpr int kP = C::kPairs;
    const int64_t row_bytes = static_cast<int64_t>(a.chunks) * C::kBytes;
    const int64_t base = (job.sample * a.spatial + job.r0) * row_bytes;
    const uint64_t policy = l2_policy(a.last_use);
    // behind the slots: the groups' (-mean, rstd), the channels' (weight, bias),
    // a pair and a count a thread
    float2 *stat = smem + a.ring / 8, *wb = stat + a.groups, *lanes = wb + a.channels;
    for (int c = job.tid; c < a.channels; c += job.threads)
        wb[c] = make_float2(param<E>(a.weight, c, a.p32, 1.f), param<E>(a.bias, c, a.p32, 0.f));
    Stream<C, 1> in(job, bars);
    in.src[0] = a.x;
    wait_for_sums(a);
    // (mean, rstd) of the sample's groups
    join_parts(
        lanes, job, a.groups_part + job.sample * a.clusters * a.groups, a.groups, a.clusters,
        [&](int c) { return values_of(a, c * a.cluster, a.cluster); },
        [&] { in.start(smem, base, row_bytes, min(job.columns, a.chunks), true, policy); },
        [&](int g, const Stats &t) {
            const float n = static_cast<float>(a.spatial) * static_cast<float>(a.per_group), mean = t.mean;
            const float rstd = 1.0f / sqrtf(not_below_zero(t.m2) / n + a.eps);
            stat[g] = make_float2(-mean, rstd);
            if (job.r0 == 0 && a.mean) {
                a.mean[job.sample * a.groups + g] = mean;
                a.rstd[job.sample * a.groups + g] = rstd;
            }
        });
    for (int32_t c0 = 0; c0 < a.chunks; c0 += job.columns) {
        const int32_t wide = min(job.columns, a.chunks - c0), c = c0 + min(job.j, wide - 1);
        if (c0 > 0) {
            __syncthreads();  // the slots have been read
            in.start(smem, base + c0 * C::kBytes, row_bytes, wide, true, policy);
        }
        float2 mean[kP], scale[kP], shift[kP], st;
        mean[kP - 1].y = scale[kP - 1].y = shift[kP - 1].y = 0.f;
        each_channel<kV>(a, c, [&](int32_t g) { st = stat[g]; }, [&](int e) {
            const float2 f = wb[c * kV + e];
            set_half(mean, e, st.x);
            set_half(scale, e, st.y * f.x);
            set_half(shift, e, f.y);
        });
        in.run([&](const typename C::Raw (&v)[1], int64_t o) {
            float2 y[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p)
                y[p] = act<kAct, C::k32>(fma2(C::plus(v[0], p, mean[p]), scale[p], shift[p]));
            C::store(a.out + o, y, policy);
        });
    }
}

template <typename E, int kV, int kAct>
__global__ void __launch_bounds__(kThreadsFwd, 2) norm_forward(NormArgs a) {
    extern __shared__ __align__(16) float2 smem[];
    __shared__ __align__(8) uint64_t storage[kBarBytes / sizeof(uint64_t)];
    Bars bars = make_bars(storage, a.stages);
    start_launch(a);
    const Job job(a);
    if (a.passes & 1) stats_pass<E, kV>(a, job, bars, smem);
    if (a.passes & 2) apply_pass<E, kV, kAct>(a, job, bars, smem);
}

// What the backward passes need of a thread's channels, from the groups'
// (-mean, rstd) and the channels' (weight, bias) in shared memory.
template <typename E, int kV>
struct Channels {
    static constexpr int kP = Chunk<E, kV>::kPairs;
    float2 mean[kP], scale[kP], shift[kP];  // -mean, rstd w, b
    __device__ void set(const NormArgs &a, int32_t c, const float2 *stat, const float2 *wb) {
        float2 st;
        mean[kP - 1].y = scale[kP - 1].y = shift[kP - 1].y = 0.f;
        each_channel<kV>(a, c, [&](int32_t g) { st = stat[g]; }, [&](int e) {
            const float2 f = wb[c * kV + e];
            set_half(mean, e, st.x);
            set_half(scale, e, st.y * f.x);
            set_half(shift, e, f.y);
        });
    }
};

// The block's copy of both.
template <typename E>
__device__ __forceinline__ void keep_inputs(const NormArgs &a, const Job &job, float2 *stat, float2 *wb) {
    for (int g = job.tid; g < a.groups; g += job.threads) {
        const int64_t at = job.sample * a.groups + g;
        stat[g] = make_float2(-__ldcg(a.mean + at), __ldcg(a.rstd + at));
    }
    for (int c = job.tid; c < a.channels; c += job.threads)
        wb[c] = make_float2(param<E>(a.weight, c, a.p32, 1.f), param<E>(a.bias, c, a.p32, 0.f));
}

// Backward, pass 1 (reads x and gy): the sums of dz and dz h a channel, and of d = dz w and d h
// a group, over the rows of a cluster.
template <typename E, int kV, int kAct>
__device__ void sums_pass(const NormArgs &a, const Job &job, Bars &bars, float2 *smem) {
    using C = Chunk<E, kV>;
    constexpr int kP = C::kPairs;
    float2 *ch = smem, *red = smem + a.channels, *stat = smem + a.behind / 8, *wb = stat + a.groups;
    float2 *ring = job.columns == a.chunks ? smem : red;
    const int64_t row_bytes = static_cast<int64_t>(a.chunks) * C::kBytes;
    keep_inputs<E>(a, job, stat, wb);
    __syncthreads();
    for (int32_t c0 = 0; c0 < a.chunks; c0 += job.columns) {
        const int32_t wide = min(job.columns, a.chunks - c0);
        Stream<C, 2> in(job, bars);
        in.src[0] = a.x, in.src[1] = a.gy;
        in.start(ring, (job.sample * a.spatial + job.r0) * row_bytes + c0 * C::kBytes, row_bytes, wide, false,
                 l2_policy(false));
        float2 s1[kP], s2[kP];
#pragma unroll
        for (int p = 0; p < kP; ++p) s1[p] = s2[p] = both(0.f);
        Channels<E, kV> t;
        t.set(a, c0 + min(job.j, wide - 1), stat, wb);
        in.run([&](const typename C::Raw (&v)[2], int64_t) {
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float2 xc = C::plus(v[0], p, t.mean[p]);
                const float2 dz = mul2(
                    C::wide(v[1], p), act_grad<kAct, C::k32>(fma2(xc, t.scale[p], t.shift[p])));
                s1[p] = add2(s1[p], dz);
                s2[p] = fma2(dz, xc, s2[p]);
            }
        });
        // h = (x - mean) rstd
        add_row_groups<kV>(red, job, c0, wide, s1, s2, [&](int, int c, float2 t) {
            t.y *= stat[c / a.per_group].y;
            ch[c] = t;
        });
    }
    const int64_t place = job.sample * a.clusters + job.cl;
    float2 *group_out = a.groups_part + place * a.groups;
    each_group(a, job, [&](int g, int lane, int lanes) {
        float m1 = 0.f, m2 = 0.f;
        if (g < a.groups)
            for (int i = lane; i < a.per_group; i += lanes) {
                const int c = g * a.per_group + i;
                const float w = wb[c].x;
                m1 = fmaf(w, ch[c].x, m1);
                m2 = fmaf(w, ch[c].y, m2);
            }
        m1 = lanes_sum(m1, a.group_shift);
        m2 = lanes_sum(m2, a.group_shift);
        if (g < a.groups && lane == 0) (a.cluster == 1 ? group_out : red)[g] = make_float2(m1, m2);
    });
    const bool weights = a.grad_weight || a.grad_bias;
    float2 *chan_out = a.chan_part + place * a.channels;
    if (a.cluster == 1) {
        if (weights)
            for (int c = job.tid; c < a.channels; c += job.threads) chan_out[c] = ch[c];
        __syncthreads();
        return;
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    // every block of the cluster ends its share of the values
    auto gather = [&](float2 *mine, float2 *out, int count) {
        for (int i = job.rank * job.threads + job.tid; i < count; i += a.cluster * job.threads) {
            float2 t = make_float2(0.f, 0.f);
            for (int r = 0; r < a.cluster; ++r) t = add2(t, cluster.map_shared_rank(mine, r)[i]);
            out[i] = t;
        }
    };
    gather(red, group_out, a.groups);
    if (weights) gather(ch, chan_out, a.channels);
    cluster.sync();
}

// Backward, pass 2 (reads x and gy again): grad_x = rstd w dz - rstd M1 -
// (x - mean) rstd^2 M2.  The gate is computed in both passes, two special
// functions an element: 10 us a pass at [1, 131040, 192] on that unit alone,
// beside 15 us for 100 MB from DRAM; keeping dz for pass 2 would be 50 MB to write
// and to read.  That size takes 50 us for 151 MB (3.0 TB/s; pass 2 finds 60 of
// its 100 MB in L2), [4, 32760, 384] bf16 94 us for 302 MB.
template <typename E, int kV, int kAct>
__device__ void grad_pass(const NormArgs &a, const Job &job, Bars &bars, float2 *smem) {
    using C = Chunk<E, kV>;
    constexpr int kP = C::kPairs;
    const int64_t row_bytes = static_cast<int64_t>(a.chunks) * C::kBytes;
    const int64_t base = (job.sample * a.spatial + job.r0) * row_bytes;
    const uint64_t policy = l2_policy(a.last_use);
    // behind the slots: the groups' (-mean, rstd) and what grad_x takes off, the
    // channels' (weight, bias), a pair a thread
    float2 *stat = smem + a.ring / 8, *coef = stat + a.groups, *wb = coef + a.groups, *lanes = wb + a.channels;
    keep_inputs<E>(a, job, stat, wb);
    Channels<E, kV> t;
    Stream<C, 2> in(job, bars);
    in.src[0] = a.x, in.src[1] = a.gy;
    wait_for_sums(a);
    add_parts(
        lanes, job, a.groups_part + job.sample * a.clusters * a.groups, a.groups, a.clusters,
        [&] { in.start(smem, base, row_bytes, min(job.columns, a.chunks), true, policy); },
        [&](int g, float2 v) {
            const float n = static_cast<float>(a.spatial) * static_cast<float>(a.per_group), rstd = stat[g].y;
            coef[g] = make_float2(-rstd * (v.x / n), -rstd * rstd * (v.y / n));
        });
    for (int32_t c0 = 0; c0 < a.chunks; c0 += job.columns) {
        const int32_t wide = min(job.columns, a.chunks - c0), c = c0 + min(job.j, wide - 1);
        if (c0 > 0) {
            __syncthreads();  // the slots have been read
            in.start(smem, base + c0 * C::kBytes, row_bytes, wide, true, policy);
        }
        t.set(a, c, stat, wb);
        float2 k1[kP], k2[kP], m;
        k1[kP - 1].y = k2[kP - 1].y = 0.f;
        each_channel<kV>(a, c, [&](int32_t g) { m = coef[g]; }, [&](int e) {
            set_half(k1, e, m.x);
            set_half(k2, e, m.y);
        });
        in.run([&](const typename C::Raw (&v)[2], int64_t o) {
            float2 y[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float2 xc = C::plus(v[0], p, t.mean[p]);
                const float2 dz = mul2(
                    C::wide(v[1], p), act_grad<kAct, C::k32>(fma2(xc, t.scale[p], t.shift[p])));
                y[p] = fma2(xc, k2[p], fma2(t.scale[p], dz, k1[p]));
            }
            C::store(a.out + o, y, policy);
        });
    }
}

template <typename E, int kV, int kAct>
__global__ void __launch_bounds__(kThreadsBwd, 1) norm_backward(NormArgs a) {
    extern __shared__ __align__(16) float2 smem[];
    __shared__ __align__(8) uint64_t storage[kBarBytes / sizeof(uint64_t)];
    Bars bars = make_bars(storage, a.stages);
    start_launch(a);
    const Job job(a);
    if (a.passes & 1) sums_pass<E, kV, kAct>(a, job, bars, smem);
    if (a.passes & 2) grad_pass<E, kV, kAct>(a, job, bars, smem);
}

// Backward, last: the weight's and bias's gradients over all samples'
// clusters; 128 lanes a channel, 8 channels a block, 16 loads in flight a thread
// (latency bounds it: a call leaves at least one pair a sample and channel).
template <typename E>
__global__ void __launch_bounds__(1024) norm_params(NormArgs a, int64_t parts) {
    constexpr int kChannels = 8, kLanes = 1024 / kChannels, kAhead = 16;
    __shared__ float2 red[kChannels][32 + 1];
    pdl_prologue();
    const int j = threadIdx.x % kChannels, l = threadIdx.x / kChannels, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t c0 = blockIdx.x * kChannels;
    float2 t = both(0.f);
    if (c0 + j < a.channels) {
        const float2 *q = a.chan_part + c0 + j;
        for (int64_t i = l; i < parts; i += kLanes * kAhead) {
            float2 v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                v[u] = i + kLanes * u < parts ? __ldcg(q + (i + kLanes * u) * a.channels) : both(0.f);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) t = add2(t, v[u]);
        }
    }
    for (int o = 16; o >= kChannels; o /= 2) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    }
    if (lane < kChannels) red[j][warp] = t;
    __syncthreads();
    // warp w ends channel w of the block
    if (warp >= kChannels) return;
    t = red[warp][lane];
    t.x = group_sum<32>(t.x);
    t.y = group_sum<32>(t.y);
    const int32_t mine = c0 + warp;
    if (lane == 0 && mine < a.channels) {
        if (a.grad_weight) store_param<E>(a.grad_weight, mine, a.p32, t.y);
        if (a.grad_bias) store_param<E>(a.grad_bias, mine, a.p32, t.x);
    }
}

// ------------------------------------------------------------------- host --

bool dtype_ok(wgs_dtype d) { return d == WGS_F32 || d == WGS_F16 || d == WGS_BF16; }
int64_t bytes_of(wgs_dtype d) { return d == WGS_F32 ? 4 : 2; }
bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Elements beyond which a call's tensors outgrow L2: pass 2 then marks its
// lines as the first to leave, so that rows not yet read stay.
constexpr int64_t kResident = int64_t{32} << 20;
// Rows that a slab has at least.
constexpr int64_t kMinSlabRows = 16;
// A sample of at most this many elements goes through both passes in one
// launch of a cluster, and so do samples that are many enough to fill the GPU
// with clusters; the larger ones of fewer samples are cut into slabs over the
// whole GPU ([8, 32760, 384] bf16 by clusters of 8 leaves SMs idle).
constexpr int64_t kOneLaunch = int64_t{1} << 19;

// Slabs of a sample in pass 1 at most: so many pairs a group come to pass 2 in
// one round of loads ([1, 131040, 192] fp16 forward: 32.4 us; with 304 33.5).
constexpr int64_t kMaxParts = 152;

// A sample's cluster grows to 8 blocks while the launch has fewer than
// kEnoughBlocks or a block would keep kShare elements: [1024, 256, 128] fp16 forward
// and backward by 1024 blocks 43 and 70 us, by 4096 62 and 95; [300, 1000, 512]
// by 1200 154 and 276, by 2400 163 and 288.
constexpr int64_t kEnoughBlocks = 608, kShare = 65536;
// See run().
constexpr int64_t kFewBlocksFwd = 304, kFewBlocksBwd = 100, kRowsMany = 32;
constexpr int kThreadsMany = 256;

struct Plan {
    int64_t x_bytes, group_part, chan_part;  // bytes
    int64_t slabs1, slabs2, cluster;
    bool one_launch;
};

// How a call is cut up: by its sizes alone, so that results do not depend on
// the device.  false for sizes that are negative, inconsistent or too large.
bool plan_of(int64_t n, int64_t spatial, int64_t channels, int64_t groups, int64_t elem,
             bool backward, Plan *z) {
    if (n < 0 || spatial < 0 || channels < 1 || groups < 1 || channels % groups != 0) return false;
    if (n > 65535 || spatial > INT32_MAX || channels > kMaxChannels || groups > kMaxGroups) return false;
    if (spatial > 0 && n > (int64_t{1} << 44) / spatial) return false;
    z->x_bytes = n * spatial * channels * elem;
    z->slabs1 = z->slabs2 = z->cluster = 1;
    z->one_launch = true;
    if (n > 0 && spatial > 0) {
        const int64_t most = ceil_div(spatial, kMinSlabRows);
        while (z->cluster < kMaxCluster && 2 * z->cluster <= most &&
               (n * z->cluster < kEnoughBlocks || spatial * channels >= 2 * z->cluster * kShare))
            z->cluster *= 2;
        z->slabs1 = z->slabs2 = z->cluster;
        z->one_launch = spatial * channels <= kOneLaunch || n * z->cluster >= 304;
        if (!z->one_launch) {
            z->cluster = 1;
            // the launch's blocks over the samples, no more than are resident
            auto share = [&](int64_t blocks) { return blocks / n < most ? blocks / n : most; };
            z->slabs2 = share(backward ? kBlocksBwd : kBlocksFwd);
            z->slabs1 = z->slabs2 < kMaxParts ? z->slabs2 : kMaxParts;
        }
    }
    const int64_t parts = n * (z->slabs1 / z->cluster);
    z->group_part = parts * groups * 8;
    z->chan_part = backward ? parts * channels * 8 : 0;
    return true;
}

// The launches of a call.
template <typename E, int kV>
wgs_status run(NormArgs a, const Plan &z, int act, bool backward, int64_t n, cudaStream_t stream) {
    using C = Chunk<E, kV>;
    a.chunks = a.channels / kV;
    a.cluster = static_cast<int32_t>(z.cluster);
    a.clusters = static_cast<int32_t>(z.slabs1 / z.cluster);
    auto slabs = [&](int64_t count) {
        return Slabs{static_cast<int32_t>(count), static_cast<int32_t>(a.spatial / count),
                     static_cast<int32_t>(a.spatial % count)};
    };
    a.slabs1 = slabs(z.slabs1), a.slabs2 = slabs(z.slabs2);
    a.last_use = n * a.spatial * a.channels > kResident;
    a.group_shift = 0;
    while (a.group_shift < 5 && 1 << a.group_shift < a.per_group) ++a.group_shift;
    auto kernel = backward ? (act == kSilu       ? norm_backward<E, kV, kSilu>
                              : act == kGeluTanh ? norm_backward<E, kV, kGeluTanh>
                                                 : norm_backward<E, kV, kNone>)
                           : (act == kSilu       ? norm_forward<E, kV, kSilu>
                              : act == kGeluTanh ? norm_forward<E, kV, kGeluTanh>
                                                 : norm_forward<E, kV, kNone>);
    int most = backward ? kThreadsBwd : kThreadsFwd;
    // Of the blocks that take a slab through both passes, more have to fit an SM
    // where there are more than the GPU holds of the largest: a block's way from
    // end to end is a chain of waits.  Threads halve to 64 as long as each has
    // kRowsMany rows of the slab at most.  (The backward's blocks of 512 fill an SM,
    // and clusters of 8 of those do not all find room beyond some 100 blocks.)
    // [4096, 49, 96] fp16: 42 and 63 us forward and backward, with 256 threads 75 and
    // 118; [1024, 256, 128] 41 and 63 (43 and 70); [16, 512, 320] backward 20, with
    // 512 threads 28; [12, 512, 512] of 96 blocks 18.6, with 256 threads 22.
    const int64_t blocks = n * z.cluster;
    if (z.one_launch && blocks > (backward ? kFewBlocksBwd : kFewBlocksFwd)) most = kThreadsMany;
    if (z.one_launch && blocks > kFewBlocksFwd) {
        const int64_t rows = ceil_div(a.spatial, z.cluster), want = ceil_div(rows, kRowsMany) * a.chunks;
        while (most > 64 && most / 2 >= want) most /= 2;
    }
    auto go = [&](int passes) {
        const int columns = a.chunks < most ? a.chunks : most;
        const int row_groups = most / columns;  // more than half of the threads, so whole warps
        const int threads = columns * row_groups;
        // Shared memory.  Pass 1: the channels' sums, and in one place the
        // slots, the row groups' sums and the groups'; where one walk covers
        // the row the channels' lie over the slots too.  Pass 2: the slots,
        // the groups' and channels' values, a pair a thread (and a count, forward).
        const int red = 8 * (threads * kV > a.groups ? threads * kV : a.groups), ch = 8 * a.channels;
        auto size = [&](int stages) {
            a.stages = stages;
            a.ring = C::kBytes < 4 ? 0 : threads * C::kBytes * (backward ? 2 * kRowsBwd : kRowsFwd) * stages;
            const int pass1 = columns == a.chunks ? (ch + red > a.ring ? ch + red : a.ring)
                                                  : ch + (red > a.ring ? red : a.ring);
            // (the backward's pass 1 keeps the groups' and channels' values behind that)
            a.behind = (pass1 + 15) / 16 * 16;
            const int one = passes & 1 ? a.behind + (backward ? 8 * (a.groups + a.channels) : 0) : 0;
            const int two = passes & 2 ? a.ring + 8 * ((backward ? 2 : 1) * a.groups + a.channels + threads) +
                                             (backward ? 0 : 4 * threads) : 0;
            return one > two ? one : two;
        };
        int smem = size(backward ? kStagesBwd : kStagesFwd);
        if (backward && C::kBytes == 16 && most == kThreadsBwd) {
            smem = size(kMostStages);
            if (smem > kMaxSmem) smem = size(kStagesBwd);
        }
        // Above 48 KB, its static barriers among them, a kernel needs the
        // runtime's leave, which belongs to the context; asking for the same
        // amount on every call needs no record of it.
        if (smem + kBarBytes > 48 << 10 &&
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) {
            cudaGetLastError();
            return WGS_ERR_LAUNCH;
        }
        a.passes = passes;
        const int64_t count = passes & 1 ? z.slabs1 : z.slabs2;
        return launch_clusters(kernel, dim3(static_cast<unsigned>(count), static_cast<unsigned>(n)),
                               dim3(columns, row_groups), a.cluster, static_cast<size_t>(smem), stream, a);
    };
    wgs_status st = WGS_OK;
    if (n > 0) {
        st = go(z.one_launch ? 3 : 1);
        if (st == WGS_OK && !z.one_launch) st = go(2);
    }
    if (st == WGS_OK && backward && (a.grad_weight || a.grad_bias))
        st = launch(norm_params<E>, dim3(static_cast<unsigned>(ceil_div(a.channels, 8))), dim3(1024), 0,
                    stream, a, n * a.clusters);
    return st;
}

// Chunks of 16 bytes when rows consist of whole ones and every tensor starts
// on 16 bytes; else pairs of elements where those fit, else single ones.
template <typename E>
wgs_status run_any(const NormArgs &a, const Plan &z, int act, bool backward, int64_t n,
                   cudaStream_t stream) {
    constexpr int es = std::is_same<E, F32>::value ? 4 : 2;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                         reinterpret_cast<uintptr_t>(a.gy) | (static_cast<uintptr_t>(a.channels) * es);
    if (at % 16 == 0) return run<E, 16 / es>(a, z, act, backward, n, stream);
    if (at % (2 * es) == 0) return run<E, 2>(a, z, act, backward, n, stream);
    return run<E, 1>(a, z, act, backward, n, stream);
}

wgs_status run_dtype(const NormArgs &a, const Plan &z, wgs_act act, wgs_dtype dtype, bool backward,
                     int64_t n, cudaStream_t stream) {
    const int t = act == WGS_ACT_SILU ? kSilu : act == WGS_ACT_GELU_TANH ? kGeluTanh : kNone;
    if (dtype == WGS_F32) return run_any<F32>(a, z, t, backward, n, stream);
    if (dtype == WGS_F16) return run_any<Fp16>(a, z, t, backward, n, stream);
    return run_any<Bf16>(a, z, t, backward, n, stream);
}

}  // namespace

}  // namespace wgs

// As bias_mask_error_take, for the group norm's error word.
wgs_status wgs::group_norm_error_take(unsigned int *seen, cudaStream_t stream) {
    static const unsigned int cleared = 0;
    if (cudaMemcpyFromSymbolAsync(seen, g_norm_error, sizeof(*seen), 0, cudaMemcpyDeviceToHost,
                                  stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_norm_error, &cleared, sizeof(cleared), 0,
                                cudaMemcpyHostToDevice, stream) != cudaSuccess) {
        cudaGetLastError();  // clear this thread's error
        return WGS_ERR_CUDA;
    }
    return WGS_OK;
}

using namespace wgs;

extern "C" size_t wgs_group_norm_act_workspace_bytes(int64_t n, int64_t spatial, int32_t channels,
                                                     int32_t groups) {
    Plan z;
    if (!plan_of(n, spatial, channels, groups, 4, false, &z)) return 0;
    return static_cast<size_t>(z.group_part);
}

extern "C" size_t wgs_group_norm_act_bwd_workspace_bytes(int64_t n, int64_t spatial,
                                                         int32_t channels, int32_t groups) {
    Plan z;
    if (!plan_of(n, spatial, channels, groups, 4, true, &z)) return 0;
    return static_cast<size_t>(z.group_part + z.chan_part);
}

extern "C" wgs_status group_norm_act(const void *x, const void *weight, const void *bias, void *y,
                                     float *mean, float *rstd, void *workspace,
                                     size_t workspace_bytes, int64_t n, int64_t spatial,
                                     int32_t channels, int32_t groups, float eps, wgs_act act,
                                     wgs_dtype dtype, wgs_dtype param_dtype, cudaStream_t stream) {
    if (!dtype_ok(dtype) || (param_dtype != WGS_F32 && param_dtype != dtype)) return WGS_ERR_DTYPE;
    if (act != WGS_ACT_NONE && act != WGS_ACT_SILU && act != WGS_ACT_GELU_TANH) return WGS_ERR_DTYPE;
    if (channels > kMaxChannels || groups > kMaxGroups) return WGS_ERR_WIDTH;
    Plan z;
    if (!plan_of(n, spatial, channels, groups, bytes_of(dtype), false, &z)) return WGS_ERR_SHAPE;
    if (n == 0 || spatial == 0) return WGS_OK;
    if (!x || !y || !workspace || (weight == nullptr) != (bias == nullptr) ||
        (mean == nullptr) != (rstd == nullptr))
        return WGS_ERR_NULL;
    if (workspace_bytes < static_cast<size_t>(z.group_part)) return WGS_ERR_SHAPE;
    if (!aligned_to(x, bytes_of(dtype)) || !aligned_to(y, bytes_of(dtype)) ||
        !aligned_to(weight, bytes_of(param_dtype)) || !aligned_to(bias, bytes_of(param_dtype)) ||
        !aligned4(mean) || !aligned4(rstd) || !aligned16(workspace))
        return WGS_ERR_ALIGN;
    const int64_t pbytes = channels * bytes_of(param_dtype), sbytes = n * groups * 4;
    if (!same_or_disjoint(y, x, z.x_bytes)) return WGS_ERR_ALIAS;
    const void *outs[4] = {y, mean, rstd, workspace};
    const int64_t obytes[4] = {z.x_bytes, mean ? sbytes : 0, rstd ? sbytes : 0, z.group_part};
    for (int i = 0; i < 4; ++i) {
        if (i > 0 && overlap(outs[i], obytes[i], x, z.x_bytes)) return WGS_ERR_ALIAS;
        if ((weight && overlap(outs[i], obytes[i], weight, pbytes)) ||
            (bias && overlap(outs[i], obytes[i], bias, pbytes)))
            return WGS_ERR_ALIAS;
        for (int k = 0; k < i; ++k)
            if (overlap(outs[i], obytes[i], outs[k], obytes[k])) return WGS_ERR_ALIAS;
    }
    DeviceInfo dev;
    const wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    NormArgs a = {};
    a.x = static_cast<const char *>(x), a.out = static_cast<char *>(y);
    a.weight = weight, a.bias = bias, a.mean = mean, a.rstd = rstd;
    a.groups_part = static_cast<float2 *>(workspace);
    a.spatial = spatial, a.channels = channels, a.groups = groups, a.per_group = channels / groups;
    a.eps = eps, a.p32 = param_dtype == WGS_F32;
    return run_dtype(a, z, act, dtype, false, n, stream);
}

extern "C" wgs_status group_norm_act_bwd(const void *grad_y, const void *x, const void *weight,
                                         const void *bias, const float *mean, const float *rstd,
                                         void *grad_x, void *grad_weight, void *grad_bias,
                                         void *workspace, size_t workspace_bytes, int64_t n,
                                         int64_t spatial, int32_t channels, int32_t groups,
                                         wgs_act act, wgs_dtype dtype, wgs_dtype param_dtype,
                                         cudaStream_t stream) {
    if (!dtype_ok(dtype) || (param_dtype != WGS_F32 && param_dtype != dtype)) return WGS_ERR_DTYPE;
    if (act != WGS_ACT_NONE && act != WGS_ACT_SILU && act != WGS_ACT_GELU_TANH) return WGS_ERR_DTYPE;
    if (channels > kMaxChannels || groups > kMaxGroups) return WGS_ERR_WIDTH;
    Plan z;
    if (!plan_of(n, spatial, channels, groups, bytes_of(dtype), true, &z)) return WGS_ERR_SHAPE;
    const bool empty = n == 0 || spatial == 0;
    if (empty && !grad_weight && !grad_bias) return WGS_OK;
    const int64_t need = z.group_part + z.chan_part;
    if (!empty && (!grad_y || !x || !mean || !rstd || !grad_x || !workspace)) return WGS_ERR_NULL;
    if ((weight == nullptr) != (bias == nullptr) || (!weight && (grad_weight || grad_bias)))
        return WGS_ERR_NULL;
    if (!empty && workspace_bytes < static_cast<size_t>(need)) return WGS_ERR_SHAPE;
    const int64_t eb = bytes_of(dtype), pb = bytes_of(param_dtype);
    if (!aligned_to(grad_y, eb) || !aligned_to(x, eb) || !aligned_to(grad_x, eb) ||
        !aligned_to(weight, pb) || !aligned_to(bias, pb) || !aligned_to(grad_weight, pb) ||
        !aligned_to(grad_bias, pb) || !aligned4(mean) || !aligned4(rstd) || !aligned16(workspace))
        return WGS_ERR_ALIGN;
    const int64_t pbytes = channels * pb, sbytes = n * groups * 4;
    if (!same_or_disjoint(grad_x, grad_y, z.x_bytes) || !same_or_disjoint(grad_x, x, z.x_bytes))
        return WGS_ERR_ALIAS;
    const void *ins[6] = {weight, bias, mean, rstd, grad_y, x};
    const int64_t ibytes[6] = {weight ? pbytes : 0, bias ? pbytes : 0, sbytes, sbytes, z.x_bytes, z.x_bytes};
    const void *outs[4] = {grad_x, grad_weight, grad_bias, workspace};
    const int64_t obytes[4] = {z.x_bytes, grad_weight ? pbytes : 0, grad_bias ? pbytes : 0,
                               empty ? 0 : need};
    for (int i = 0; i < 4; ++i) {
        for (int k = 0; k < (i == 0 ? 4 : 6); ++k)
            if (overlap(outs[i], obytes[i], ins[k], ibytes[k])) return WGS_ERR_ALIAS;
        for (int k = 0; k < i; ++k)
            if (overlap(outs[i], obytes[i], outs[k], obytes[k])) return WGS_ERR_ALIAS;
    }
    DeviceInfo dev;
    const wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    NormArgs a = {};
    a.x = static_cast<const char *>(x), a.gy = static_cast<const char *>(grad_y);
    a.out = static_cast<char *>(grad_x);
    a.weight = weight, a.bias = bias;
    a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    a.groups_part = static_cast<float2 *>(workspace);
    a.chan_part = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + z.group_part);
    a.grad_weight = grad_weight, a.grad_bias = grad_bias;
    a.spatial = spatial, a.channels = channels, a.groups = groups, a.per_group = channels / groups;
    a.p32 = param_dtype == WGS_F32;
    // no rows: no launch but the one that ends the (empty) sums
    return run_dtype(a, z, act, dtype, true, empty ? 0 : n, stream);
}
