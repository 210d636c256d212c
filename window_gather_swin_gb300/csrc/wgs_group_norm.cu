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
// Both are streams: an element takes one pass for the sums and one for the
// result, and the second finds it in L2 when the samples worked on at a time
// fit there.  Rows are walked by column chunk: a thread owns one chunk of
// channels (16 bytes, or one element where rows do not consist of whole
// aligned chunks) and steps through the rows of its block's slab, so the
// channels' weights and statistics stay in registers.
#include <type_traits>

#include "wgs_common.cuh"

namespace wgs {

namespace {

struct F32 {};

constexpr int kThreads = 512;
constexpr int kMaxChannels = 4096;  // two FP32 sums a channel: 32 KB of shared memory
constexpr int kAhead = 4;           // rows in flight a thread

enum : int { kNone = 0, kSilu = 1, kGeluTanh = 2 };

// A chunk of kN elements: 16 bytes, or one element.
template <typename E, bool kVec>
struct Chunk {
    static constexpr bool k32 = std::is_same<E, F32>::value;
    static constexpr int kN = kVec ? (k32 ? 4 : 8) : 1;
    using Raw = std::conditional_t<kVec, uint4, std::conditional_t<k32, float, uint16_t>>;

    __device__ static Raw load(const void *p, int64_t i) {
        if constexpr (kVec)
            return ld_stream(static_cast<const uint4 *>(p) + i);
        else
            return __ldcg(static_cast<const Raw *>(p) + i);
    }
    __device__ static void widen(const Raw &r, float (&v)[kN]) {
        if constexpr (kVec && k32) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(word(r, k));
        } else if constexpr (kVec) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = E::to_f2(word(r, k));
                v[2 * k] = f.x, v[2 * k + 1] = f.y;
            }
        } else if constexpr (k32) {
            v[0] = r;
        } else {
            v[0] = E::to_f2(r).x;
        }
    }
    // rounds each value once, to nearest even
    __device__ static void store(void *p, int64_t i, const float (&v)[kN]) {
        if constexpr (kVec && k32) {
            st_stream(static_cast<uint4 *>(p) + i,
                      make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                 __float_as_uint(v[2]), __float_as_uint(v[3])));
        } else if constexpr (kVec) {
            st_stream(static_cast<uint4 *>(p) + i,
                      make_uint4(E::from_f2(v[0], v[1]), E::from_f2(v[2], v[3]),
                                 E::from_f2(v[4], v[5]), E::from_f2(v[6], v[7])));
        } else if constexpr (k32) {
            static_cast<float *>(p)[i] = v[0];
        } else {
            static_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(E::from_f2(v[0], 0.f));
        }
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

// 1 / (1 + exp(-t)).  For 16-bit tensors the hardware's exp2 and reciprocal
// (relative errors of a few 2^-22 and that of the product t log2(e)) are far
// below the output's half step; FP32 tensors take expf and a division.
template <bool k32>
__device__ __forceinline__ float sigmoid(float t) {
    if constexpr (k32) {
        return 1.0f / (1.0f + expf(-t));
    } else {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t * -1.4426950408889634f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
        return r;
    }
}

constexpr float kTwoK = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kCubic = 0.044715f;

// act(z); gelu_tanh(z) = 0.5 z (1 + tanh(u)) = z sigmoid(2u), which does not
// cancel for negative z.
template <int kAct, bool k32>
__device__ __forceinline__ float act(float z) {
    if constexpr (kAct == kSilu) return z * sigmoid<k32>(z);
    if constexpr (kAct == kGeluTanh)
        return z * sigmoid<k32>(z * fmaf(kTwoK * kCubic, z * z, kTwoK));
    return z;
}

// act'(z) = s + z s (1 - s) q', with s the sigmoid's value and q its argument.
template <int kAct, bool k32>
__device__ __forceinline__ float act_grad(float z) {
    if constexpr (kAct == kSilu) {
        const float s = sigmoid<k32>(z);
        return fmaf(z * s, 1.0f - s, s);
    }
    if constexpr (kAct == kGeluTanh) {
        const float z2 = z * z;
        const float s = sigmoid<k32>(z * fmaf(kTwoK * kCubic, z2, kTwoK));
        // far out s (1 - s) is 0 and the cubic's slope may be infinite
        const float p = z * s * (1.0f - s);
        return p == 0.f ? s : fmaf(p, fmaf(3.0f * kTwoK * kCubic, z2, kTwoK), s);
    }
    return 1.0f;
}

struct NormArgs {
    const void *x, *gy;          // gy: backward
    const void *weight, *bias;   // [C] or NULL
    void *out;                   // y, or grad_x
    float *mean, *rstd;          // [n, groups]
    float2 *partial;             // per sample, slab: [groups] (mean, M2), or [C] (sum dz, sum dz (x - mean))
    float2 *sums;                // backward: [n, C] (sum dz, sum dz h)
    float2 *coef;                // backward: [n, groups] (M(dz w), M(dz w h))
    void *grad_weight, *grad_bias;
    int64_t spatial, first;      // first: the launch's first sample
    int32_t n, channels, groups, per_group;
    int32_t chunks;              // of a row
    int32_t columns;             // chunks a block walks side by side
    int32_t slabs;
    float eps;
    bool p32;                    // weight and bias are FP32
};

// Thread (g, j) of a block of `columns` x row groups.
struct Place {
    int j, g, row_groups;
    bool active;
    __device__ explicit Place(int columns) {
        row_groups = kThreads / columns;
        j = static_cast<int>(threadIdx.x) % columns;
        g = static_cast<int>(threadIdx.x) / columns;
        active = g < row_groups;
    }
};

// Statistics (mean, M2 = sum of squared distances from it) of na and nb
// values joined: Chan, Golub & LeVeque, "Algorithms for computing the sample
// variance", 1983.
__device__ __forceinline__ void join(float &n, float &mean, float &m2, float nb, float meanb,
                                     float m2b) {
    if (nb > 0.f) {
        const float total = n + nb, d = meanb - mean, part = nb / total;
        mean = fmaf(d, part, mean);
        m2 += fmaf(d * d, n * part, m2b);
        n = total;
    }
}

// Forward, pass 1: (mean, M2) of every group over the rows of a slab.  A
// thread sums x - k and its square, k the first value of the channel that it
// meets (with k one of the values, the cancellation in M2 = sum d^2 - (sum
// d)^2 / n costs at most a factor n in relative error, for the few dozen
// rows of a thread, whatever the mean or the outliers); the block joins its
// row groups and then the channels of a group, in a fixed order.
template <typename E, bool kVec>
__global__ void __launch_bounds__(kThreads) norm_stats(NormArgs a) {
    using C = Chunk<E, kVec>;
    constexpr int kN = C::kN;
    extern __shared__ float2 smem[];
    const bool one = a.columns == a.chunks;
    float2 *ch = smem, *red = one ? smem : smem + a.channels;
    const Place at(a.columns);
    const int64_t sample = a.first + blockIdx.y;
    const int64_t r0 = a.spatial * blockIdx.x / a.slabs, r1 = a.spatial * (blockIdx.x + 1) / a.slabs;
    pdl_prologue();
    const int64_t G = at.row_groups;
    for (int32_t c0 = 0; c0 < a.chunks; c0 += a.columns) {
        const int32_t wide = min(a.columns, a.chunks - c0);
        float k[kN], s1[kN], s2[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) k[e] = s1[e] = s2[e] = 0.f;
        float count = 0.f;
        if (at.active && at.j < wide && r0 + at.g < r1) {
            const int64_t base = sample * a.spatial * a.chunks + c0 + at.j;
            C::widen(C::load(a.x, base + (r0 + at.g) * a.chunks), k);
            for (int64_t r = r0 + at.g; r < r1; r += kAhead * G) {
                typename C::Raw v[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (r + u * G < r1) v[u] = C::load(a.x, base + (r + u * G) * a.chunks);
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (r + u * G < r1) {
                        float f[kN];
                        C::widen(v[u], f);
#pragma unroll
                        for (int e = 0; e < kN; ++e) {
                            const float d = f[e] - k[e];
                            s1[e] += d;
                            s2[e] = fmaf(d, d, s2[e]);
                        }
                        count += 1.f;
                    }
            }
        }
        if (at.active && at.j < wide) {
            const float inv = count > 0.f ? 1.f / count : 0.f;
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const float d = s1[e] * inv;
                red[(at.g * wide + at.j) * kN + e] =
                    make_float2(k[e] + d, fmaxf(fmaf(-d, s1[e], s2[e]), 0.f));
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < wide * kN; c += kThreads) {
            float n = 0.f, mean = 0.f, m2 = 0.f;
            for (int g = 0; g < at.row_groups; ++g) {
                const int64_t rows = r1 - r0 - g;  // of row group g, before the step
                const float2 p = red[g * wide * kN + c];
                join(n, mean, m2, rows > 0 ? static_cast<float>((rows + G - 1) / G) : 0.f, p.x, p.y);
            }
            ch[c0 * kN + c] = make_float2(mean, m2);
        }
        __syncthreads();
    }
    // a warp a group: the channels' means have one weight each
    const int lane = threadIdx.x & 31;
    const float rows = static_cast<float>(r1 - r0);
    for (int g = threadIdx.x / 32; g < a.groups; g += kThreads / 32) {
        const float2 *p = ch + static_cast<int64_t>(g) * a.per_group;
        float mean = 0.f;
        const float lead = p[0].x;
        for (int c = lane; c < a.per_group; c += 32) mean += p[c].x - lead;
        mean = lead + group_sum<32>(mean) / static_cast<float>(a.per_group);
        float m2 = 0.f;
        for (int c = lane; c < a.per_group; c += 32) {
            const float d = p[c].x - mean;
            m2 += fmaf(rows * d, d, p[c].y);
        }
        m2 = group_sum<32>(m2);
        if (lane == 0)
            a.partial[(static_cast<int64_t>(sample) * a.slabs + blockIdx.x) * a.groups + g] =
                make_float2(mean, m2);
    }
}

// Forward, between the passes: a warp joins the slabs of one (sample, group).
__global__ void __launch_bounds__(128) norm_join(NormArgs a) {
    pdl_prologue();
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) / 32;
    const int lane = threadIdx.x & 31;
    if (i >= static_cast<int64_t>(a.n) * a.groups) return;
    const int64_t sample = a.first + i / a.groups, g = i % a.groups;
    float n = 0.f, mean = 0.f, m2 = 0.f;
    for (int32_t s = lane; s < a.slabs; s += 32) {
        const int64_t rows = a.spatial * (s + 1) / a.slabs - a.spatial * s / a.slabs;
        const float2 p = __ldcg(a.partial + (sample * a.slabs + s) * a.groups + g);
        join(n, mean, m2, static_cast<float>(rows) * a.per_group, p.x, p.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float nb = __shfl_down_sync(0xffffffffu, n, o);
        const float mb = __shfl_down_sync(0xffffffffu, mean, o);
        const float qb = __shfl_down_sync(0xffffffffu, m2, o);
        join(n, mean, m2, nb, mb, qb);
    }
    if (lane == 0) {
        a.mean[sample * a.groups + g] = mean;
        a.rstd[sample * a.groups + g] =
            1.0f / sqrtf(m2 / (static_cast<float>(a.spatial) * a.per_group) + a.eps);
    }
}

// Forward, pass 2.
template <typename E, bool kVec, int kAct>
__global__ void __launch_bounds__(kThreads) norm_apply(NormArgs a) {
    using C = Chunk<E, kVec>;
    constexpr int kN = C::kN;
    const Place at(a.columns);
    const int64_t sample = a.first + blockIdx.y;
    const int64_t r0 = a.spatial * blockIdx.x / a.slabs, r1 = a.spatial * (blockIdx.x + 1) / a.slabs;
    pdl_prologue();
    const int64_t G = at.row_groups;
    if (!at.active) return;
    for (int32_t c = at.j; c < a.chunks; c += a.columns) {
        float mean[kN], scale[kN], shift[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const int32_t k = c * kN + e;
            const int64_t g = sample * a.groups + k / a.per_group;
            mean[e] = __ldcg(a.mean + g);
            scale[e] = __ldcg(a.rstd + g) * param<E>(a.weight, k, a.p32, 1.f);
            shift[e] = param<E>(a.bias, k, a.p32, 0.f);
        }
        const int64_t base = sample * a.spatial * a.chunks + c;
        for (int64_t r = r0 + at.g; r < r1; r += kAhead * G) {
            typename C::Raw v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (r + u * G < r1) v[u] = C::load(a.x, base + (r + u * G) * a.chunks);
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (r + u * G < r1) {
                    float f[kN];
                    C::widen(v[u], f);
#pragma unroll
                    for (int e = 0; e < kN; ++e)
                        f[e] = act<kAct, C::k32>(fmaf(f[e] - mean[e], scale[e], shift[e]));
                    C::store(a.out, base + (r + u * G) * a.chunks, f);
                }
        }
    }
}

// Backward, pass 1: per channel the sums of dz and dz (x - mean) over the
// rows of a slab.
template <typename E, bool kVec, int kAct>
__global__ void __launch_bounds__(kThreads) norm_bwd_sums(NormArgs a) {
    using C = Chunk<E, kVec>;
    constexpr int kN = C::kN;
    constexpr int kRows = 2;
    extern __shared__ float2 smem[];
    const Place at(a.columns);
    const int64_t sample = a.first + blockIdx.y;
    const int64_t r0 = a.spatial * blockIdx.x / a.slabs, r1 = a.spatial * (blockIdx.x + 1) / a.slabs;
    pdl_prologue();
    const int64_t G = at.row_groups;
    float2 *out = a.partial + (sample * a.slabs + blockIdx.x) * a.channels;
    for (int32_t c0 = 0; c0 < a.chunks; c0 += a.columns) {
        const int32_t wide = min(a.columns, a.chunks - c0);
        float s1[kN], s2[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) s1[e] = s2[e] = 0.f;
        if (at.active && at.j < wide) {
            float mean[kN], scale[kN], shift[kN];
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const int32_t k = (c0 + at.j) * kN + e;
                const int64_t g = sample * a.groups + k / a.per_group;
                mean[e] = __ldcg(a.mean + g);
                scale[e] = __ldcg(a.rstd + g) * param<E>(a.weight, k, a.p32, 1.f);
                shift[e] = param<E>(a.bias, k, a.p32, 0.f);
            }
            const int64_t base = sample * a.spatial * a.chunks + c0 + at.j;
            for (int64_t r = r0 + at.g; r < r1; r += kRows * G) {
                typename C::Raw vx[kRows], vg[kRows];
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    if (r + u * G < r1) {
                        vx[u] = C::load(a.x, base + (r + u * G) * a.chunks);
                        vg[u] = C::load(a.gy, base + (r + u * G) * a.chunks);
                    }
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    if (r + u * G < r1) {
                        float f[kN], d[kN];
                        C::widen(vx[u], f);
                        C::widen(vg[u], d);
#pragma unroll
                        for (int e = 0; e < kN; ++e) {
                            const float xc = f[e] - mean[e];
                            const float dz = d[e] * act_grad<kAct, C::k32>(fmaf(xc, scale[e], shift[e]));
                            s1[e] += dz;
                            s2[e] = fmaf(dz, xc, s2[e]);
                        }
                    }
            }
#pragma unroll
            for (int e = 0; e < kN; ++e)
                smem[(at.g * wide + at.j) * kN + e] = make_float2(s1[e], s2[e]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < wide * kN; c += kThreads) {
            float2 t = smem[c];
            for (int g = 1; g < at.row_groups; ++g) {
                const float2 p = smem[g * wide * kN + c];
                t.x += p.x, t.y += p.y;
            }
            out[c0 * kN + c] = t;
        }
        __syncthreads();
    }
}

template <typename E>
__device__ __forceinline__ void store_param(void *p, int64_t c, bool p32, float v) {
    if (p32) {
        static_cast<float *>(p)[c] = v;
    } else if constexpr (!std::is_same<E, F32>::value) {
        static_cast<uint16_t *>(p)[c] = static_cast<uint16_t>(E::from_f2(v, 0.f));
    }
}

constexpr int kJoin = 256;

// Backward, between the passes: a block joins the slabs of one (sample,
// group): the channels' sums, then the group's two means.  With one sample
// the channels' sums are the weight's and bias's gradients already.
template <typename E>
__global__ void __launch_bounds__(kJoin) norm_bwd_join(NormArgs a, bool last) {
    __shared__ float2 part[kJoin];
    pdl_prologue();
    const int64_t sample = a.first + blockIdx.x / a.groups, g = blockIdx.x % a.groups;
    const int tid = threadIdx.x;
    const int wide = min(a.per_group, kJoin), lanes = kJoin / wide;
    const int j = tid % wide, l = tid / wide;
    const float rstd = __ldcg(a.rstd + sample * a.groups + g);
    float m1 = 0.f, m2 = 0.f;  // of the channels that this thread ends
    for (int32_t c0 = 0; c0 < a.per_group; c0 += wide) {
        const int32_t c = c0 + j;
        float2 t = make_float2(0.f, 0.f);
        if (l < lanes && c < a.per_group) {
            const float2 *p = a.partial + sample * a.slabs * a.channels + g * a.per_group + c;
#pragma unroll 4
            for (int32_t s = l; s < a.slabs; s += lanes) {
                const float2 v = __ldcg(p + static_cast<int64_t>(s) * a.channels);
                t.x += v.x, t.y += v.y;
            }
        }
        part[tid] = t;
        __syncthreads();
        if (l == 0 && c < a.per_group) {
            for (int q = 1; q < lanes; ++q) {
                const float2 v = part[q * wide + j];
                t.x += v.x, t.y += v.y;
            }
            t.y *= rstd;
            const int64_t k = g * a.per_group + c;
            const float w = param<E>(a.weight, k, a.p32, 1.f);
            m1 = fmaf(w, t.x, m1);
            m2 = fmaf(w, t.y, m2);
            if (!last) {
                a.sums[sample * a.channels + k] = t;
            } else {
                if (a.grad_weight) store_param<E>(a.grad_weight, k, a.p32, t.y);
                if (a.grad_bias) store_param<E>(a.grad_bias, k, a.p32, t.x);
            }
        }
        __syncthreads();
    }
    part[tid] = make_float2(m1, m2);
    __syncthreads();
    if (tid < 32) {
        float2 t = make_float2(0.f, 0.f);
        for (int q = tid; q < wide; q += 32) t.x += part[q].x, t.y += part[q].y;
        t.x = group_sum<32>(t.x);
        t.y = group_sum<32>(t.y);
        const float m = static_cast<float>(a.spatial) * a.per_group;
        if (tid == 0) a.coef[sample * a.groups + g] = make_float2(t.x / m, t.y / m);
    }
}

// Backward, last: the weight's and bias's gradients over the samples.
template <typename E>
__global__ void __launch_bounds__(128) norm_bwd_params(NormArgs a) {
    pdl_prologue();
    const int32_t c = blockIdx.x * 128 + threadIdx.x;
    if (c >= a.channels) return;
    float2 t = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int32_t i = 0; i < a.n; ++i) {
        const float2 v = __ldcg(a.sums + static_cast<int64_t>(i) * a.channels + c);
        t.x += v.x, t.y += v.y;
    }
    if (a.grad_weight) store_param<E>(a.grad_weight, c, a.p32, t.y);
    if (a.grad_bias) store_param<E>(a.grad_bias, c, a.p32, t.x);
}

// Backward, pass 2: grad_x = rstd w dz - rstd M1 - (x - mean) rstd^2 M2.
template <typename E, bool kVec, int kAct>
__global__ void __launch_bounds__(kThreads) norm_bwd_apply(NormArgs a) {
    using C = Chunk<E, kVec>;
    constexpr int kN = C::kN;
    constexpr int kRows = 2;
    const Place at(a.columns);
    const int64_t sample = a.first + blockIdx.y;
    const int64_t r0 = a.spatial * blockIdx.x / a.slabs, r1 = a.spatial * (blockIdx.x + 1) / a.slabs;
    pdl_prologue();
    const int64_t G = at.row_groups;
    if (!at.active) return;
    for (int32_t c = at.j; c < a.chunks; c += a.columns) {
        float mean[kN], scale[kN], shift[kN], k1[kN], k2[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const int32_t k = c * kN + e;
            const int64_t g = sample * a.groups + k / a.per_group;
            const float rstd = __ldcg(a.rstd + g);
            const float2 m = __ldcg(a.coef + g);
            mean[e] = __ldcg(a.mean + g);
            scale[e] = rstd * param<E>(a.weight, k, a.p32, 1.f);
            shift[e] = param<E>(a.bias, k, a.p32, 0.f);
            k1[e] = rstd * m.x;
            k2[e] = rstd * rstd * m.y;
        }
        const int64_t base = sample * a.spatial * a.chunks + c;
        for (int64_t r = r0 + at.g; r < r1; r += kRows * G) {
            typename C::Raw vx[kRows], vg[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                if (r + u * G < r1) {
                    vx[u] = C::load(a.x, base + (r + u * G) * a.chunks);
                    vg[u] = C::load(a.gy, base + (r + u * G) * a.chunks);
                }
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                if (r + u * G < r1) {
                    float f[kN], d[kN];
                    C::widen(vx[u], f);
                    C::widen(vg[u], d);
#pragma unroll
                    for (int e = 0; e < kN; ++e) {
                        const float xc = f[e] - mean[e];
                        const float dz = d[e] * act_grad<kAct, C::k32>(fmaf(xc, scale[e], shift[e]));
                        f[e] = fmaf(scale[e], dz, -k1[e]) - xc * k2[e];
                    }
                    C::store(a.out, base + (r + u * G) * a.chunks, f);
                }
        }
    }
}

// ------------------------------------------------------------------- host --

bool dtype_ok(wgs_dtype d) { return d == WGS_F32 || d == WGS_F16 || d == WGS_BF16; }
int64_t bytes_of(wgs_dtype d) { return d == WGS_F32 ? 4 : 2; }
bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Samples worked on at a time: as many as the second pass still finds in L2,
// counted in elements that both passes read (48 MB of 16-bit ones).
constexpr int64_t kResident = int64_t{24} << 20;

// Slabs a sample is cut into: blocks for two on each of 152 SMs, but 16
// rows or more a slab.  Both depend on the sizes alone, so results do not
// depend on the device.
constexpr int64_t kBlocks = 304;
constexpr int64_t kMinSlabRows = 16;

struct Sizes {
    int64_t x_bytes, partial, sums, coef, stats;  // bytes
    int64_t slabs, at_a_time;
};

// false for sizes that are negative, inconsistent or too large
bool sizes_of(int64_t n, int64_t spatial, int64_t channels, int64_t groups, int64_t elem,
              bool backward, Sizes *z) {
    if (n < 0 || spatial < 0 || channels < 1 || groups < 1 || channels % groups != 0) return false;
    if (n > 65535 || spatial > (int64_t{1} << 40) || channels > kMaxChannels) return false;
    if (spatial > 0 && n > (int64_t{1} << 44) / spatial) return false;
    z->x_bytes = n * spatial * channels * elem;
    z->slabs = z->at_a_time = 1;
    if (n > 0 && spatial > 0) {
        const int64_t fit = kResident / (spatial * channels * (backward ? 2 : 1));
        z->at_a_time = fit < 1 ? 1 : fit > n ? n : fit;
        const int64_t want = ceil_div(kBlocks, z->at_a_time), most = ceil_div(spatial, kMinSlabRows);
        z->slabs = want < most ? want : most;
    }
    z->partial = n * z->slabs * (backward ? channels : groups) * 8;
    z->sums = backward ? n * channels * 8 : 0;
    z->coef = backward ? n * groups * 8 : 0;
    z->stats = backward ? 0 : n * groups * 8;  // mean and rstd, where the caller keeps none
    return true;
}

template <typename E, bool kVec>
wgs_status forward(NormArgs a, int act, int64_t n, int64_t at_a_time, cudaStream_t stream) {
    constexpr int kN = Chunk<E, kVec>::kN;
    a.chunks = a.channels / kN;
    a.columns = a.chunks < kThreads ? a.chunks : kThreads;
    const size_t smem = sizeof(float2) * (a.columns == a.chunks
                                              ? (kThreads / a.columns) * a.channels
                                              : a.channels + kThreads * kN);
    for (int64_t i = 0; i < n; i += at_a_time) {
        a.first = i;
        a.n = static_cast<int32_t>(n - i < at_a_time ? n - i : at_a_time);
        const dim3 grid(a.slabs, a.n);
        wgs_status st = launch(norm_stats<E, kVec>, grid, dim3(kThreads), smem, stream, a);
        if (st != WGS_OK) return st;
        st = launch(norm_join, dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(a.n) * a.groups, 4))),
                    dim3(128), 0, stream, a);
        if (st != WGS_OK) return st;
        auto kernel = act == kSilu       ? norm_apply<E, kVec, kSilu>
                      : act == kGeluTanh ? norm_apply<E, kVec, kGeluTanh>
                                         : norm_apply<E, kVec, kNone>;
        st = launch(kernel, grid, dim3(kThreads), 0, stream, a);
        if (st != WGS_OK) return st;
    }
    return WGS_OK;
}

template <typename E, bool kVec>
wgs_status backward(NormArgs a, int act, int64_t n, int64_t at_a_time, cudaStream_t stream) {
    constexpr int kN = Chunk<E, kVec>::kN;
    a.chunks = a.channels / kN;
    a.columns = a.chunks < kThreads ? a.chunks : kThreads;
    const size_t smem = sizeof(float2) * (kThreads / a.columns) * a.columns * kN;
    auto sums = act == kSilu       ? norm_bwd_sums<E, kVec, kSilu>
                : act == kGeluTanh ? norm_bwd_sums<E, kVec, kGeluTanh>
                                   : norm_bwd_sums<E, kVec, kNone>;
    auto apply = act == kSilu       ? norm_bwd_apply<E, kVec, kSilu>
                 : act == kGeluTanh ? norm_bwd_apply<E, kVec, kGeluTanh>
                                    : norm_bwd_apply<E, kVec, kNone>;
    for (int64_t i = 0; i < n; i += at_a_time) {
        a.first = i;
        a.n = static_cast<int32_t>(n - i < at_a_time ? n - i : at_a_time);
        const dim3 grid(a.slabs, a.n);
        wgs_status st = launch(sums, grid, dim3(kThreads), smem, stream, a);
        if (st != WGS_OK) return st;
        st = launch(norm_bwd_join<E>, dim3(static_cast<unsigned>(a.n) * a.groups), dim3(kJoin), 0,
                    stream, a, n == 1);
        if (st != WGS_OK) return st;
        st = launch(apply, grid, dim3(kThreads), 0, stream, a);
        if (st != WGS_OK) return st;
    }
    if (n != 1 && (a.grad_weight || a.grad_bias)) {
        a.n = static_cast<int32_t>(n);
        return launch(norm_bwd_params<E>, dim3(static_cast<unsigned>(ceil_div(a.channels, 128))),
                      dim3(128), 0, stream, a);
    }
    return WGS_OK;
}

// Column chunks of 16 bytes when rows consist of whole ones and every tensor
// starts on 16 bytes, single elements otherwise.
bool vectors(int64_t channels, wgs_dtype dtype, const void *a, const void *b, const void *c) {
    return channels % (16 / bytes_of(dtype)) == 0 && aligned16(a) && aligned16(b) && aligned16(c);
}

}  // namespace

}  // namespace wgs

using namespace wgs;

extern "C" size_t wgs_group_norm_act_workspace_bytes(int64_t n, int64_t spatial, int32_t channels,
                                                     int32_t groups) {
    Sizes z;
    if (!sizes_of(n, spatial, channels, groups, 4, false, &z)) return 0;
    return static_cast<size_t>(z.partial + z.stats);
}

extern "C" size_t wgs_group_norm_act_bwd_workspace_bytes(int64_t n, int64_t spatial,
                                                         int32_t channels, int32_t groups) {
    Sizes z;
    if (!sizes_of(n, spatial, channels, groups, 4, true, &z)) return 0;
    return static_cast<size_t>(z.partial + z.sums + z.coef);
}

extern "C" wgs_status group_norm_act(const void *x, const void *weight, const void *bias, void *y,
                                     float *mean, float *rstd, void *workspace,
                                     size_t workspace_bytes, int64_t n, int64_t spatial,
                                     int32_t channels, int32_t groups, float eps, wgs_act act,
                                     wgs_dtype dtype, wgs_dtype param_dtype, cudaStream_t stream) {
    if (!dtype_ok(dtype) || (param_dtype != WGS_F32 && param_dtype != dtype)) return WGS_ERR_DTYPE;
    if (act != WGS_ACT_NONE && act != WGS_ACT_SILU && act != WGS_ACT_GELU_TANH) return WGS_ERR_DTYPE;
    if (channels > kMaxChannels) return WGS_ERR_WIDTH;
    Sizes z;
    if (!sizes_of(n, spatial, channels, groups, bytes_of(dtype), false, &z)) return WGS_ERR_SHAPE;
    if (n == 0 || spatial == 0) return WGS_OK;
    if (!x || !y || !workspace || (weight == nullptr) != (bias == nullptr) ||
        (mean == nullptr) != (rstd == nullptr))
        return WGS_ERR_NULL;
    if (workspace_bytes < static_cast<size_t>(z.partial + z.stats)) return WGS_ERR_SHAPE;
    if (!aligned_to(x, bytes_of(dtype)) || !aligned_to(y, bytes_of(dtype)) ||
        !aligned_to(weight, bytes_of(param_dtype)) || !aligned_to(bias, bytes_of(param_dtype)) ||
        !aligned4(mean) || !aligned4(rstd) || !aligned16(workspace))
        return WGS_ERR_ALIGN;
    const int64_t pbytes = channels * bytes_of(param_dtype), sbytes = n * groups * 4;
    if (!same_or_disjoint(y, x, z.x_bytes)) return WGS_ERR_ALIAS;
    const void *outs[4] = {y, mean, rstd, workspace};
    const int64_t obytes[4] = {z.x_bytes, mean ? sbytes : 0, rstd ? sbytes : 0, z.partial + z.stats};
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
    a.x = x, a.weight = weight, a.bias = bias, a.out = y;
    a.partial = static_cast<float2 *>(workspace);
    float *stats = reinterpret_cast<float *>(static_cast<char *>(workspace) + z.partial);
    a.mean = mean ? mean : stats;
    a.rstd = rstd ? rstd : stats + n * groups;
    a.spatial = spatial, a.channels = channels, a.groups = groups, a.per_group = channels / groups;
    a.slabs = static_cast<int32_t>(z.slabs), a.eps = eps, a.p32 = param_dtype == WGS_F32;
    const int64_t k = z.at_a_time;
    const bool vec = vectors(channels, dtype, x, y, x);
    const int t = act == WGS_ACT_SILU ? kSilu : act == WGS_ACT_GELU_TANH ? kGeluTanh : kNone;
    if (dtype == WGS_F32)
        return vec ? forward<F32, true>(a, t, n, k, stream) : forward<F32, false>(a, t, n, k, stream);
    if (dtype == WGS_F16)
        return vec ? forward<Fp16, true>(a, t, n, k, stream) : forward<Fp16, false>(a, t, n, k, stream);
    return vec ? forward<Bf16, true>(a, t, n, k, stream) : forward<Bf16, false>(a, t, n, k, stream);
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
    if (channels > kMaxChannels) return WGS_ERR_WIDTH;
    Sizes z;
    if (!sizes_of(n, spatial, channels, groups, bytes_of(dtype), true, &z)) return WGS_ERR_SHAPE;
    const bool empty = n == 0 || spatial == 0;
    if (empty && !grad_weight && !grad_bias) return WGS_OK;
    const int64_t need = z.partial + z.sums + z.coef;
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
    a.x = x, a.gy = grad_y, a.weight = weight, a.bias = bias, a.out = grad_x;
    a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    char *ws = static_cast<char *>(workspace);
    a.partial = reinterpret_cast<float2 *>(ws);
    a.sums = reinterpret_cast<float2 *>(ws + z.partial);
    a.coef = reinterpret_cast<float2 *>(ws + z.partial + z.sums);
    a.grad_weight = grad_weight, a.grad_bias = grad_bias;
    a.spatial = spatial, a.channels = channels, a.groups = groups, a.per_group = channels / groups;
    a.slabs = static_cast<int32_t>(z.slabs), a.p32 = param_dtype == WGS_F32;
    if (empty) n = 0;  // the gradients of no rows: zeros
    const int64_t k = z.at_a_time;
    const bool vec = vectors(channels, dtype, x, grad_y, grad_x);
    const int t = act == WGS_ACT_SILU ? kSilu : act == WGS_ACT_GELU_TANH ? kGeluTanh : kNone;
    if (dtype == WGS_F32)
        return vec ? backward<F32, true>(a, t, n, k, stream) : backward<F32, false>(a, t, n, k, stream);
    if (dtype == WGS_F16)
        return vec ? backward<Fp16, true>(a, t, n, k, stream) : backward<Fp16, false>(a, t, n, k, stream);
    return vec ? backward<Bf16, true>(a, t, n, k, stream) : backward<Bf16, false>(a, t, n, k, stream);
}
