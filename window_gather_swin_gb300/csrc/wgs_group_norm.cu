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
// weights and sums stay in registers.  Rows reach a thread through slots of
// its own in shared memory, filled by asynchronous copies several rows ahead:
// a slab is only some twenty rows a thread, so without them most of the time
// is the latency of its loads.  Pass 1 sums, pass 2 computes the result;
// between them the sums of a sample have to meet:
//   * the blocks of a cluster add theirs over distributed shared memory, and
//     one value pair per (cluster, group) goes to the workspace, where every
//     block of pass 2 adds those of its sample up;
//   * a sample that one cluster holds goes through both passes in one launch.
// Pass 2 finds what pass 1 read in L2 when few enough samples are worked on
// at a time, and walks its rows backwards, the latest first.  With more
// samples than that, one launch runs pass 2 of a batch of samples next to
// pass 1 of the following batch, so that reading, writing and arithmetic
// overlap.
#include <cooperative_groups.h>

#include <type_traits>

#include "wgs_common.cuh"

namespace wgs {

namespace {

namespace cg = cooperative_groups;

struct F32 {};

constexpr int kMaxChannels = 4096;
constexpr int kMaxGroups = 2048;
constexpr int kThreadsFwd = 512, kThreadsBwd = 384;  // two blocks an SM, of 64 and 80 registers a thread
constexpr int kMaxSmem = 112 << 10;                  // two blocks an SM
constexpr int kMaxCluster = 8;   // of a sample that one cluster holds
constexpr int kPairCluster = 2;  // of larger ones: a pair of blocks finds room on any GPC

enum : int { kNone = 0, kSilu = 1, kGeluTanh = 2 };

// ------------------------------------------------------------ pairs, chunks --

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

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
                return __fadd2_rn(make_float2(__uint_as_float(word_of(r, 2 * p)),
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
    // rounds each value once, to nearest even
    __device__ static void store(char *p, const float2 (&v)[kPairs]) {
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
        *reinterpret_cast<Raw *>(p) = r;
    }
};

// A weight or bias: FP32 or the tensor's own format; NULL is the default.
template <typename E>
__device__ __forceinline__ float param(const void *p, int64_t c, bool p32, float otherwise) {
    if (!p) return otherwise;
    if (p32) return __ldg(static_cast<const float *>(p) + c);
    if constexpr (std::is_same<E, F32>::value)
        return otherwise;  // FP32 tensors have FP32 weights
    else
        return E::to_f2(__ldg(static_cast<const uint16_t *>(p) + c)).x;
}

template <typename E>
__device__ __forceinline__ void store_param(void *p, int64_t c, bool p32, float v) {
    if (p32) {
        static_cast<float *>(p)[c] = v;
    } else if constexpr (!std::is_same<E, F32>::value) {
        static_cast<uint16_t *>(p)[c] = static_cast<uint16_t>(E::from_f2(v, 0.f));
    }
}

// 1 / (1 + exp(-t)).  For 16-bit tensors the hardware's exp2 and reciprocal
// (relative errors of a few 2^-22 and that of the product t log2(e)) are far
// below the output's half step; FP32 tensors take expf and a division.
template <bool k32>
__device__ __forceinline__ float2 sigmoid(float2 t) {
    if constexpr (k32) {
        return make_float2(1.0f / (1.0f + expf(-t.x)), 1.0f / (1.0f + expf(-t.y)));
    } else {
        const float2 w = __fmul2_rn(t, both(-1.4426950408889634f));
        float2 e, s;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(w.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(w.y));
        e = __fadd2_rn(e, both(1.0f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(e.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(e.y));
        return s;
    }
}

constexpr float kTwoK = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kCubic = 0.044715f;

// act(z); gelu_tanh(z) = 0.5 z (1 + tanh(u)) = z sigmoid(2u), which does not
// cancel for negative z.
template <int kAct, bool k32>
__device__ __forceinline__ float2 act(float2 z) {
    if constexpr (kAct == kSilu) return __fmul2_rn(z, sigmoid<k32>(z));
    if constexpr (kAct == kGeluTanh) {
        const float2 q = __ffma2_rn(__fmul2_rn(z, z), both(kTwoK * kCubic), both(kTwoK));
        return __fmul2_rn(z, sigmoid<k32>(__fmul2_rn(z, q)));
    }
    return z;
}

// act'(z) = s + z s (1 - s) q', with s the sigmoid's value and q its argument.
template <int kAct, bool k32>
__device__ __forceinline__ float2 act_grad(float2 z) {
    if constexpr (kAct == kSilu) {
        const float2 s = sigmoid<k32>(z);
        return __ffma2_rn(__fmul2_rn(z, s), __ffma2_rn(s, both(-1.0f), both(1.0f)), s);
    }
    if constexpr (kAct == kGeluTanh) {
        const float2 z2 = __fmul2_rn(z, z);
        const float2 q = __ffma2_rn(z2, both(kTwoK * kCubic), both(kTwoK));
        const float2 s = sigmoid<k32>(__fmul2_rn(z, q));
        const float2 p = __fmul2_rn(__fmul2_rn(z, s), __ffma2_rn(s, both(-1.0f), both(1.0f)));
        // q' = q + 2 kTwoK kCubic z^2.  Far out p is 0, and there the slope
        // may be infinite: it is cut to what a finite z^2 gives
        const float2 zc = make_float2(fminf(z2.x, 1e30f), fminf(z2.y, 1e30f));
        return __ffma2_rn(p, __ffma2_rn(zc, both(3.0f * kTwoK * kCubic), both(kTwoK)), s);
    }
    return both(1.0f);
}

// -------------------------------------------------------------------- work --

struct NormArgs {
    const char *x, *gy;         // gy: backward
    const void *weight, *bias;  // [C] or NULL
    char *out;                  // y, or grad_x
    float *mean, *rstd;         // [n, groups]; written by the forward unless NULL
    float2 *groups_part;        // [n, clusters, groups]: (mean, M2), or the sums of (d, d h)
    float2 *chan_part;          // backward: [n, clusters, C]: the sums of (dz, dz h)
    void *grad_weight, *grad_bias;
    int64_t spatial;
    int64_t first1, first2;     // first sample of pass 1 and of pass 2
    int32_t n1, n2;             // samples of pass 1 and of pass 2
    int32_t channels, groups, per_group;
    int32_t chunks;             // of a row
    int32_t columns;            // chunks a block walks side by side
    int32_t slabs, cluster;     // slabs of a sample, a multiple of the cluster size
    int32_t clusters;           // slabs / cluster
    int32_t slab_rows, longer;  // rows of a slab, one more in the first `longer`
    int32_t ring;               // bytes of the slots
    int32_t passes;             // 1 + 2 for a launch that takes its samples through both
    float eps;
    bool p32;                   // weight and bias are FP32
};

// First row of a slab.
__device__ __forceinline__ int32_t slab_start(const NormArgs &a, int32_t slab) {
    return slab * a.slab_rows + min(slab, a.longer);
}

// What a block is to do: its pass (1, 2 or 3 for both), sample and slab.
struct Job {
    int pass;
    int64_t sample;
    int32_t cl, rank;  // cluster of the sample, block of the cluster
    int32_t r0, rows;  // first row, rows
    __device__ explicit Job(const NormArgs &a) {
        const uint32_t per = static_cast<uint32_t>(a.clusters);
        uint32_t id = blockIdx.x / static_cast<uint32_t>(a.cluster);
        rank = static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(a.cluster));
        pass = a.passes;
        if (pass == 0) {
            // clusters of the two passes alternate while both have some
            const uint32_t c1 = per * a.n1, c2 = per * a.n2, m = min(c1, c2);
            if (id < 2 * m) {
                pass = id & 1 ? 1 : 2;
                id >>= 1;
            } else {
                pass = c1 > c2 ? 1 : 2;
                id -= m;
            }
        }
        sample = (pass == 2 ? a.first2 : a.first1) + id / per;
        cl = static_cast<int32_t>(id % per);
        const int32_t slab = cl * a.cluster + rank;
        r0 = slab_start(a, slab);
        rows = a.slab_rows + (slab < a.longer);
    }
};

// Thread (g, j) of a block of `columns` chunks x row groups.
struct Place {
    int j, g, row_groups;
    bool active;
    __device__ explicit Place(int columns) {
        row_groups = static_cast<int>(blockDim.x) / columns;
        j = static_cast<int>(threadIdx.x) % columns;
        g = static_cast<int>(threadIdx.x) / columns;
        active = g < row_groups;
    }
};

// The chunks of kTensors tensors at the byte offsets at, at + step, ... of a
// thread, kSlots - 1 places ahead of their use: each thread copies its own
// chunks into its own slots and needs no barrier.  The slot that a copy
// overwrites was read one place before.
template <typename C, int kTensors, int kSlots>
struct Stream {
    static constexpr bool kAsync = C::kBytes >= 4;  // the smallest asynchronous copy
    static constexpr int kLead = kSlots - 1;
    uint32_t slots;  // address of the thread's chunk of slot 0
    const char *src[kTensors];
    int64_t at;  // offset of the next chunk to use
    int32_t step, left;
    int next;    // its slot

    __device__ uint32_t slot(int s, int t) const { return slots + (s * kTensors + t) * (blockDim.x * C::kBytes); }
    // the chunk kLead places on, into slot s
    __device__ void copy(int s, int64_t from, bool live) const {
        if (live) {
#pragma unroll
            for (int t = 0; t < kTensors; ++t) {
                const uint32_t to = slot(s, t);
                if constexpr (C::kBytes == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src[t] + from) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src[t] + from), "n"(C::kBytes) : "memory");
            }
        }
        cp_async_commit();
    }
    __device__ void start(float2 *smem, int64_t first, int32_t step_, int32_t rows) {
        slots = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * C::kBytes;
        at = first;
        step = step_;
        left = rows;
        next = 0;
        if constexpr (kAsync)
#pragma unroll
            for (int i = 0; i < kLead; ++i) copy(i, at + i * step, i < left);
    }
    // f(chunk of each tensor, offset) for every place in order
    template <typename Use>
    __device__ void run(Use f) {
        if constexpr (kAsync) {
            for (; left > 0; --left) {
                cp_async_wait<kLead - 1>();
                typename C::Raw v[kTensors];
#pragma unroll
                for (int t = 0; t < kTensors; ++t) v[t] = C::load_shared(slot(next, t));
                copy(next == 0 ? kLead : next - 1, at + kLead * step, left > kLead);
                next = next == kLead ? 0 : next + 1;
                f(v, at);
                at += step;
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
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (u < left) f(v[u], at + u * step);
            }
        }
    }
};

constexpr int kSlotsFwd = 8, kSlotsBwd = 6;

// Add the threads' pairs of sums (s1, s2) over the row groups, in order;
// done(channel of the column block, its sums) is called once a channel.
// Every thread calls it.  In `red` a row group's values lie element by element of
// the chunk, so that neighbouring threads touch neighbouring words.
template <int kV, int kPairs, typename Done>
__device__ __forceinline__ void add_row_groups(float2 *red, const Place &at, int wide,
                                               const float2 (&s1)[kPairs],
                                               const float2 (&s2)[kPairs], Done done) {
    __syncthreads();  // the slots that `red` lies over have been read
    if (at.active && at.j < wide) {
        float2 *mine = red + at.g * wide * kV + at.j;
#pragma unroll
        for (int e = 0; e < kV; ++e)
            mine[e * wide] = e & 1 ? make_float2(s1[e / 2].y, s2[e / 2].y) : make_float2(s1[e / 2].x, s2[e / 2].x);
    }
    __syncthreads();
    const int cols = wide * kV;
    for (int i = threadIdx.x; i < cols; i += blockDim.x) {
        float2 t = red[i];
#pragma unroll 4
        for (int g = 1; g < at.row_groups; ++g) t = __fadd2_rn(t, red[g * cols + i]);
        done(i % wide * kV + i / wide, t);
    }
    __syncthreads();
}

// Values of a group in the slabs [s0, s1).
__device__ __forceinline__ float values_of(const NormArgs &a, int32_t s0, int32_t s1) {
    return static_cast<float>(slab_start(a, s1) - slab_start(a, s0)) * static_cast<float>(a.per_group);
}

// For every group g: the sum of value(part, g) over the parts [0, parts),
// in a fixed order, to done(g, sum).  Neighbouring threads take neighbouring
// groups, and the threads beyond the groups a share of the parts each.
template <typename Value, typename Done>
__device__ __forceinline__ void add_parts(float2 *smem, int groups, int parts, Value value, Done done) {
    const int wide = min(groups, static_cast<int>(blockDim.x));
    const int lanes = static_cast<int>(blockDim.x) / wide;
    const int j = static_cast<int>(threadIdx.x) % wide, l = static_cast<int>(threadIdx.x) / wide;
    for (int g0 = 0; g0 < groups; g0 += wide) {
        const int g = g0 + j;
        float2 t = make_float2(0.f, 0.f);
        if (l < lanes && g < groups)
#pragma unroll 4
            for (int p = l; p < parts; p += lanes) t = __fadd2_rn(t, value(p, g));
        smem[threadIdx.x] = t;
        __syncthreads();
        if (l == 0 && g < groups) {
            for (int q = 1; q < lanes && q < parts; ++q) t = __fadd2_rn(t, smem[q * wide + j]);
            done(g, t);
        }
        __syncthreads();
    }
}

// Forward, pass 1: (mean, M2) of every group over the rows of a cluster, M2
// the sum of the squared distances from the mean.  A thread sums x - k and
// its square, k the channel's value in the slab's first row.  With k one of
// the values, the cancellation in M2 = sum d^2 - (sum d)^2 / n costs at most
// a factor of the slab's rows in relative error, and that only where k is an
// outlier, whatever the mean.  Where parts are joined the same is done with
// the first part's mean as the reference.
template <typename E, int kV>
__device__ void stats_pass(const NormArgs &a, const Job &job, float2 *smem) {
    using C = Chunk<E, kV>;
    using One = Chunk<E, 1>;
    constexpr int kP = C::kPairs;
    float2 *ch = smem, *red = smem + a.channels;  // red holds the groups' results in the end
    float2 *ring = a.columns == a.chunks ? smem : red;
    const Place at(a.columns);
    const int64_t row_bytes = static_cast<int64_t>(a.chunks) * C::kBytes;
    const int32_t rows = job.rows;
    const float inv = rows > 0 ? 1.0f / static_cast<float>(rows) : 0.f;
    const char *lead = a.x + (job.sample * a.spatial + job.r0) * row_bytes;
    auto first = [&](int c) {  // the channel's value in the slab's first row
        return rows > 0 ? One::wide(One::load(lead + static_cast<int64_t>(c) * One::kBytes), 0).x : 0.f;
    };
    for (int32_t c0 = 0; c0 < a.chunks; c0 += a.columns) {
        const int32_t wide = min(a.columns, a.chunks - c0);
        const bool mine = at.active && at.j < wide && at.g < rows;
        Stream<C, 1, kSlotsFwd> in;
        in.src[0] = a.x;
        const int64_t o = (job.sample * a.spatial + job.r0 + at.g) * row_bytes + (c0 + at.j) * C::kBytes;
        in.start(ring, o, static_cast<int32_t>(at.row_groups * row_bytes),
                 mine ? (rows - at.g + at.row_groups - 1) / at.row_groups : 0);
        float2 k[kP], s1[kP], s2[kP];
#pragma unroll
        for (int p = 0; p < kP; ++p) k[p] = s1[p] = s2[p] = both(0.f);
        if (mine) {
            const typename C::Raw r = C::load(lead + (c0 + at.j) * C::kBytes);
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                k[p] = C::wide(r, p);
                k[p].x = -k[p].x, k[p].y = -k[p].y;
            }
        }
        // the value that this thread will need where it ends a channel
        const int ends = static_cast<int>(threadIdx.x) % wide * kV + static_cast<int>(threadIdx.x) / wide;
        const float ahead = static_cast<int>(threadIdx.x) < wide * kV ? first(c0 * kV + ends) : 0.f;
        in.run([&](const typename C::Raw (&v)[1], int64_t) {
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float2 d = C::plus(v[0], p, k[p]);
                s1[p] = __fadd2_rn(s1[p], d);
                s2[p] = __ffma2_rn(d, d, s2[p]);
            }
        });
        add_row_groups<kV>(red, at, wide, s1, s2, [&](int c, float2 t) {
            const float m = t.x * inv;
            ch[c0 * kV + c] = make_float2((c == ends ? ahead : first(c0 * kV + c)) + m,
                                          fmaxf(fmaf(-m, t.x, t.y), 0.f));
        });
    }
    // a warp a group, in two steps over its channels: the mean, M2 about it
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    for (int g = threadIdx.x / 32; g < a.groups; g += warps) {
        const float2 *p = ch + g * a.per_group;
        const float ref = p[0].x;
        float mean = 0.f, m2 = 0.f;
        for (int i = lane; i < a.per_group; i += 32) mean += p[i].x - ref;
        mean = ref + group_sum<32>(mean) / static_cast<float>(a.per_group);
        for (int i = lane; i < a.per_group; i += 32) {
            const float d = p[i].x - mean;
            m2 += fmaf(static_cast<float>(rows) * d, d, p[i].y);
        }
        m2 = group_sum<32>(m2);
        if (lane == 0) red[g] = make_float2(mean, m2);
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int32_t slab0 = job.cl * a.cluster;
    float2 *out = a.groups_part + (job.sample * a.clusters + job.cl) * a.groups;
    for (int g = job.rank * blockDim.x + threadIdx.x; g < a.groups; g += a.cluster * blockDim.x) {
        const float ref = cluster.map_shared_rank(red, 0)[g].x;
        float s1 = 0.f, s2 = 0.f;
        for (int r = 0; r < a.cluster; ++r) {
            const float2 v = cluster.map_shared_rank(red, r)[g];
            const float n = values_of(a, slab0 + r, slab0 + r + 1), d = n > 0.f ? v.x - ref : 0.f;
            s1 = fmaf(n, d, s1);
            s2 += fmaf(n * d, d, v.y);
        }
        const float m = s1 / values_of(a, slab0, slab0 + a.cluster);
        out[g] = make_float2(ref + m, fmaxf(fmaf(-m, s1, s2), 0.f));
    }
    cluster.sync();  // the others' shared memory has been read; the result is visible to them
}

// f(e, channel, group) for the elements of a chunk.
template <int kV, typename F>
__device__ __forceinline__ void each_channel(const NormArgs &a, int32_t chunk, F f) {
    int32_t g = chunk * kV / a.per_group, in_group = chunk * kV - g * a.per_group;
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        f(e, chunk * kV + e, g);
        if (++in_group == a.per_group) in_group = 0, ++g;
    }
}

__device__ __forceinline__ void set_half(float2 *v, int e, float x) {
    if (e & 1) v[e / 2].y = x; else v[e / 2].x = x;
}

// The rows of a pass 2: a thread's in the slab, and the offset of the last.
struct LastRows {
    int32_t left;
    int64_t last;
    __device__ LastRows(const NormArgs &a, const Job &job, const Place &at, int64_t row_bytes) {
        const int32_t rows = job.rows;
        left = at.active && at.g < rows ? (rows - at.g + at.row_groups - 1) / at.row_groups : 0;
        last = (job.sample * a.spatial + job.r0 + at.g + static_cast<int64_t>(left - 1) * at.row_groups) * row_bytes;
    }
};

// Forward, pass 2.  The first rows are on their way while the statistics of
// the groups, which lie behind the slots, are put together.
template <typename E, int kV, int kAct>
__device__ void apply_pass(const NormArgs &a, const Job &job, float2 *smem) {
    using C = Chunk<E, kV>;
    using In = Stream<C, 1, kSlotsFwd>;
    constexpr int kP = C::kPairs;
    const Place at(a.columns);
    const int64_t row_bytes = static_cast<int64_t>(a.chunks) * C::kBytes;
    const LastRows rows(a, job, at, row_bytes);
    const int32_t step = -static_cast<int32_t>(at.row_groups * row_bytes);
    float2 *stat = smem + a.ring / 8, *lanes = stat + a.groups;
    In in;
    in.src[0] = a.x;
    in.start(smem, rows.last + at.j * C::kBytes, step, rows.left);
    // (mean, rstd) of the sample's groups from its clusters'
    const int32_t clusters = a.clusters;
    const float2 *part = a.groups_part + job.sample * clusters * a.groups;
    add_parts(
        lanes, a.groups, clusters,
        [&](int c, int g) {
            const float2 v = __ldcg(part + static_cast<int64_t>(c) * a.groups + g);
            const int32_t s0 = c * a.cluster;
            const float n = values_of(a, s0, s0 + a.cluster), d = v.x - __ldcg(part + g).x;
            return make_float2(n * d, fmaf(n * d, d, v.y));
        },
        [&](int g, float2 t) {
            const float n = static_cast<float>(a.spatial) * a.per_group, m = t.x / n;
            const float mean = __ldcg(part + g).x + m;
            const float rstd = 1.0f / sqrtf(fmaxf(fmaf(-m, t.x, t.y), 0.f) / n + a.eps);
            stat[g] = make_float2(-mean, rstd);
            if (job.cl == 0 && job.rank == 0 && a.mean) {
                a.mean[job.sample * a.groups + g] = mean;
                a.rstd[job.sample * a.groups + g] = rstd;
            }
        });
    for (int32_t c = at.j; c < a.chunks; c += a.columns) {
        if (c != at.j) in.start(smem, rows.last + c * C::kBytes, step, rows.left);
        float2 mean[kP], scale[kP], shift[kP];
        each_channel<kV>(a, c, [&](int e, int32_t k, int32_t g) {
            const float2 st = stat[g];
            set_half(mean, e, st.x);
            set_half(scale, e, st.y * param<E>(a.weight, k, a.p32, 1.f));
            set_half(shift, e, param<E>(a.bias, k, a.p32, 0.f));
        });
        if (kV == 1) mean[0].y = scale[0].y = shift[0].y = 0.f;
        in.run([&](const typename C::Raw (&v)[1], int64_t o) {
            float2 y[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p)
                y[p] = act<kAct, C::k32>(__ffma2_rn(C::plus(v[0], p, mean[p]), scale[p], shift[p]));
            C::store(a.out + o, y);
        });
    }
}

template <typename E, int kV, int kAct>
__global__ void __launch_bounds__(kThreadsFwd, 2) norm_forward(NormArgs a) {
    extern __shared__ __align__(16) float2 smem[];
    pdl_prologue();
    const Job job(a);
    if (job.pass & 1) stats_pass<E, kV>(a, job, smem);
    if (job.pass & 2) apply_pass<E, kV, kAct>(a, job, smem);
}

// What the backward passes need of a thread's channels.
template <typename E, int kV>
struct Channels {
    static constexpr int kP = Chunk<E, kV>::kPairs;
    float2 mean[kP], scale[kP], shift[kP];  // -mean, rstd w, b
    __device__ void read(const NormArgs &a, int64_t sample, int32_t c) {
        each_channel<kV>(a, c, [&](int e, int32_t k, int32_t g) {
            set_half(mean, e, -__ldcg(a.mean + sample * a.groups + g));
            set_half(scale, e, __ldcg(a.rstd + sample * a.groups + g) * param<E>(a.weight, k, a.p32, 1.f));
            set_half(shift, e, param<E>(a.bias, k, a.p32, 0.f));
        });
        if (kV == 1) mean[0].y = scale[0].y = shift[0].y = 0.f;
    }
};

// Backward, pass 1: the sums of dz and dz h a channel, and of d = dz w and d h
// a group, over the rows of a cluster.
template <typename E, int kV, int kAct>
__device__ void sums_pass(const NormArgs &a, const Job &job, float2 *smem) {
    using C = Chunk<E, kV>;
    constexpr int kP = C::kPairs;
    float2 *ch = smem, *red = smem + a.channels;
    float2 *ring = a.columns == a.chunks ? smem : red;
    const Place at(a.columns);
    const int64_t row_bytes = static_cast<int64_t>(a.chunks) * C::kBytes;
    const int32_t rows = job.rows;
    for (int32_t c0 = 0; c0 < a.chunks; c0 += a.columns) {
        const int32_t wide = min(a.columns, a.chunks - c0);
        const bool mine = at.active && at.j < wide && at.g < rows;
        Stream<C, 2, kSlotsBwd> in;
        in.src[0] = a.x, in.src[1] = a.gy;
        in.start(ring, (job.sample * a.spatial + job.r0 + at.g) * row_bytes + (c0 + at.j) * C::kBytes,
                 static_cast<int32_t>(at.row_groups * row_bytes),
                 mine ? (rows - at.g + at.row_groups - 1) / at.row_groups : 0);
        float2 s1[kP], s2[kP];
#pragma unroll
        for (int p = 0; p < kP; ++p) s1[p] = s2[p] = both(0.f);
        if (mine) {
            Channels<E, kV> t;
            t.read(a, job.sample, c0 + at.j);
            in.run([&](const typename C::Raw (&v)[2], int64_t) {
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const float2 xc = C::plus(v[0], p, t.mean[p]);
                    const float2 dz = __fmul2_rn(
                        C::wide(v[1], p), act_grad<kAct, C::k32>(__ffma2_rn(xc, t.scale[p], t.shift[p])));
                    s1[p] = __fadd2_rn(s1[p], dz);
                    s2[p] = __ffma2_rn(dz, xc, s2[p]);
                }
            });
        }
        // h = (x - mean) rstd
        add_row_groups<kV>(red, at, wide, s1, s2, [&](int c, float2 t) {
            t.y *= __ldcg(a.rstd + job.sample * a.groups + (c0 * kV + c) / a.per_group);
            ch[c0 * kV + c] = t;
        });
    }
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    for (int g = threadIdx.x / 32; g < a.groups; g += warps) {
        float m1 = 0.f, m2 = 0.f;
        for (int i = lane; i < a.per_group; i += 32) {
            const int c = g * a.per_group + i;
            const float w = param<E>(a.weight, c, a.p32, 1.f);
            m1 = fmaf(w, ch[c].x, m1);
            m2 = fmaf(w, ch[c].y, m2);
        }
        m1 = group_sum<32>(m1);
        m2 = group_sum<32>(m2);
        if (lane == 0) red[g] = make_float2(m1, m2);
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int64_t place = job.sample * a.clusters + job.cl;
    auto gather = [&](float2 *mine, float2 *out, int count) {
        // every block of the cluster ends its share of the values
        for (int i = job.rank * blockDim.x + threadIdx.x; i < count; i += a.cluster * blockDim.x) {
            float2 t = make_float2(0.f, 0.f);
            for (int r = 0; r < a.cluster; ++r) t = __fadd2_rn(t, cluster.map_shared_rank(mine, r)[i]);
            out[i] = t;
        }
    };
    gather(red, a.groups_part + place * a.groups, a.groups);
    if (a.grad_weight || a.grad_bias) gather(ch, a.chan_part + place * a.channels, a.channels);
    cluster.sync();
}

// Backward, pass 2: grad_x = rstd w dz - rstd M1 - (x - mean) rstd^2 M2.
template <typename E, int kV, int kAct>
__device__ void grad_pass(const NormArgs &a, const Job &job, float2 *smem) {
    using C = Chunk<E, kV>;
    constexpr int kP = C::kPairs;
    const Place at(a.columns);
    const int64_t row_bytes = static_cast<int64_t>(a.chunks) * C::kBytes;
    const LastRows rows(a, job, at, row_bytes);
    const int32_t step = -static_cast<int32_t>(at.row_groups * row_bytes);
    float2 *coef = smem + a.ring / 8, *lanes = coef + a.groups;
    Stream<C, 2, kSlotsBwd> in;
    in.src[0] = a.x, in.src[1] = a.gy;
    in.start(smem, rows.last + at.j * C::kBytes, step, rows.left);
    const int32_t clusters = a.clusters;
    const float2 *part = a.groups_part + job.sample * clusters * a.groups;
    add_parts(
        lanes, a.groups, clusters,
        [&](int c, int g) { return __ldcg(part + static_cast<int64_t>(c) * a.groups + g); },
        [&](int g, float2 t) {
            const float count = static_cast<float>(a.spatial) * a.per_group;
            const float rstd = __ldcg(a.rstd + job.sample * a.groups + g);
            coef[g] = make_float2(-rstd * (t.x / count), -rstd * rstd * (t.y / count));
        });
    for (int32_t c = at.j; c < a.chunks; c += a.columns) {
        if (c != at.j) in.start(smem, rows.last + c * C::kBytes, step, rows.left);
        Channels<E, kV> t;
        t.read(a, job.sample, c);
        float2 k1[kP], k2[kP];
        each_channel<kV>(a, c, [&](int e, int32_t, int32_t g) {
            set_half(k1, e, coef[g].x);
            set_half(k2, e, coef[g].y);
        });
        if (kV == 1) k1[0].y = k2[0].y = 0.f;
        in.run([&](const typename C::Raw (&v)[2], int64_t o) {
            float2 y[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float2 xc = C::plus(v[0], p, t.mean[p]);
                const float2 dz = __fmul2_rn(
                    C::wide(v[1], p), act_grad<kAct, C::k32>(__ffma2_rn(xc, t.scale[p], t.shift[p])));
                y[p] = __ffma2_rn(xc, k2[p], __ffma2_rn(t.scale[p], dz, k1[p]));
            }
            C::store(a.out + o, y);
        });
    }
}

template <typename E, int kV, int kAct>
__global__ void __launch_bounds__(kThreadsBwd, 2) norm_backward(NormArgs a) {
    extern __shared__ __align__(16) float2 smem[];
    pdl_prologue();
    const Job job(a);
    if (job.pass & 1) sums_pass<E, kV, kAct>(a, job, smem);
    if (job.pass & 2) grad_pass<E, kV, kAct>(a, job, smem);
}

// Backward, last: the weight's and bias's gradients over all samples'
// clusters; 32 row lanes of 32 channels each.
template <typename E>
__global__ void __launch_bounds__(1024) norm_params(NormArgs a, int64_t parts) {
    __shared__ float2 red[32][33];
    pdl_prologue();
    const int j = threadIdx.x & 31, l = threadIdx.x >> 5;
    const int32_t c = blockIdx.x * 32 + j;
    float2 t = make_float2(0.f, 0.f);
    if (c < a.channels) {
#pragma unroll 4
        for (int64_t i = l; i < parts; i += 32) t = __fadd2_rn(t, __ldcg(a.chan_part + i * a.channels + c));
    }
    red[l][j] = t;
    __syncthreads();
    // warp l ends channel l of the block
    t = red[j][l];
    t.x = group_sum<32>(t.x);
    t.y = group_sum<32>(t.y);
    const int32_t mine = blockIdx.x * 32 + l;
    if (j == 0 && mine < a.channels) {
        if (a.grad_weight) store_param<E>(a.grad_weight, mine, a.p32, t.y);
        if (a.grad_bias) store_param<E>(a.grad_bias, mine, a.p32, t.x);
    }
}

// ------------------------------------------------------------------- host --

bool dtype_ok(wgs_dtype d) { return d == WGS_F32 || d == WGS_F16 || d == WGS_BF16; }
int64_t bytes_of(wgs_dtype d) { return d == WGS_F32 ? 4 : 2; }
bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Samples in a batch: as many as pass 2 still finds in L2, counted in
// elements that both passes read (48 MB of 16-bit ones).
constexpr int64_t kResident = int64_t{24} << 20;
// Blocks that fill the GPU: two on each of 152 SMs.
constexpr int64_t kBlocks = 304;
// Rows that a slab has at least.
constexpr int64_t kMinSlabRows = 16;
// A sample of at most this many elements goes through both passes in one
// launch of a cluster.
constexpr int64_t kOneLaunch = int64_t{1} << 19;

struct Plan {
    int64_t x_bytes, group_part, chan_part;  // bytes
    int64_t slabs, cluster, batch;
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
    z->slabs = z->cluster = z->batch = 1;
    z->one_launch = true;
    if (n > 0 && spatial > 0) {
        const int64_t most = ceil_div(spatial, kMinSlabRows);
        while (z->cluster < kMaxCluster && 2 * z->cluster <= most) z->cluster *= 2;
        z->one_launch = spatial * channels <= kOneLaunch || n * z->cluster >= kBlocks;
        if (z->one_launch) {
            z->batch = n;
            z->slabs = z->cluster;
        } else {
            if (z->cluster > kPairCluster) z->cluster = kPairCluster;
            const int64_t fit = kResident / (spatial * channels * (backward ? 2 : 1));
            z->batch = fit < 1 ? 1 : fit > n ? n : fit;
            // two batches share a launch when there are several
            const int64_t want = ceil_div(z->batch < n ? kBlocks / 2 : kBlocks, z->batch);
            z->slabs = ceil_div(want < most ? want : most, z->cluster) * z->cluster;
        }
    }
    const int64_t parts = n * (z->slabs / z->cluster);
    z->group_part = parts * groups * 8;
    z->chan_part = backward ? parts * channels * 8 : 0;
    return true;
}

// The launches of a call: batches of samples through pass 1 and pass 2.
template <typename E, int kV>
wgs_status run(NormArgs a, const Plan &z, int act, bool backward, int64_t n, cudaStream_t stream) {
    using C = Chunk<E, kV>;
    a.chunks = a.channels / kV;
    a.slabs = static_cast<int32_t>(z.slabs), a.cluster = static_cast<int32_t>(z.cluster);
    a.clusters = a.slabs / a.cluster;
    a.slab_rows = static_cast<int32_t>(a.spatial / a.slabs);
    a.longer = static_cast<int32_t>(a.spatial % a.slabs);
    // Shared memory.  Pass 1: the channels' sums, and in one place the slots,
    // the row groups' sums and the groups'; where one walk covers the row the
    // channels' lie over the slots too.  Pass 2: the slots, the groups'
    // values, a pair a thread.
    const int threads = backward ? kThreadsBwd : kThreadsFwd;
    a.columns = a.chunks < threads ? a.chunks : threads;
    a.ring = C::kBytes < 4 ? 0 : threads * C::kBytes * (backward ? 2 * kSlotsBwd : kSlotsFwd);
    const int red = 8 * (threads * kV > a.groups ? threads * kV : a.groups), ch = 8 * a.channels;
    const int pass1 = a.columns == a.chunks ? (ch + red > a.ring ? ch + red : a.ring)
                                            : ch + (red > a.ring ? red : a.ring);
    const int pass2 = a.ring + 8 * (a.groups + threads);
    const int smem = pass1 > pass2 ? pass1 : pass2;
    auto kernel = backward ? (act == kSilu       ? norm_backward<E, kV, kSilu>
                              : act == kGeluTanh ? norm_backward<E, kV, kGeluTanh>
                                                 : norm_backward<E, kV, kNone>)
                           : (act == kSilu       ? norm_forward<E, kV, kSilu>
                              : act == kGeluTanh ? norm_forward<E, kV, kGeluTanh>
                                                 : norm_forward<E, kV, kNone>);
    // Above 48 KB a kernel needs the runtime's leave, which belongs to the
    // context; asking for the same amount on every call needs no record of it.
    if (smem > 48 << 10 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    auto part = [&](int64_t i) { return static_cast<int32_t>(i < 0 || i >= n ? 0 : i + z.batch < n ? z.batch : n - i); };
    wgs_status st = WGS_OK;
    a.passes = z.one_launch ? 3 : 0;
    for (int64_t i = 0; i < (z.one_launch ? n : n + z.batch) && st == WGS_OK; i += z.batch) {
        a.first1 = i, a.n1 = part(i);
        a.first2 = i - z.batch, a.n2 = part(i - z.batch);
        if (z.one_launch) a.n2 = 0;
        const unsigned grid = static_cast<unsigned>((a.n1 + a.n2) * z.slabs);
        if (grid == 0) continue;
        st = launch_clusters(kernel, dim3(grid), dim3(threads), a.cluster, static_cast<size_t>(smem), stream, a);
    }
    if (st == WGS_OK && backward && (a.grad_weight || a.grad_bias))
        st = launch(norm_params<E>, dim3(static_cast<unsigned>(ceil_div(a.channels, 32))), dim3(1024), 0,
                    stream, a, n * (z.slabs / z.cluster));
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
