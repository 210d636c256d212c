// Layer norm with weight and bias over rows of any width up to 8192, and the
// residual add fused before it (sm_103a).
//
//     mean = sum x / width,  rstd = 1 / sqrt(var + eps),  y = (x - mean) rstd w + b
//
// Design.  A stream of rows: bound by their bytes.  A row stays in the registers of
// its unit between load, both sums and store; weight and bias are in shared memory
// in the threads' own order, read again for every row (16 bytes a lane, the lanes
// of a warp's rows the same ones).
//
// Measured, us a call in a row of calls, and of the copy rate: [131040, 192] fp16 16.9
// (6.0 TB/s, 88 %), FP32 33 (89 %); [32761, 768] bf16 with residual 33.5 (89 %), [32761,
// 771] 45 (66 %); [5000, 8192] FP32 63 (76 %), bf16 37 (65 %).  24 warps an SM issue in
// half of their cycles, some 290 instructions for four rows of 192: the start (weights,
// first rows) and the last rows' way through are the rest.  Ragged rows take 890
// instructions a row of 771 where 482 do for 768, most of them for the ends.
//
// Rows in tiles copied in bulk (TMA) into a ring of each warp, with two sums a row
// from shared memory, took 31 us for the first: a tile's addresses, barriers and
// waits cost as many instructions as its rows.
#include "wgs_layer_norm.cuh"

namespace wgs {

namespace {

// 1 / sqrt(v): the hardware's approximation and one step of Newton's method, which
// would make NaN of an infinite one.
__device__ __forceinline__ float reciprocal_root(float v) {
    const float r = rsqrtf(v), better = fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
    return v > 0.f && r > 0.f ? better : r;
}

// The row's statistics: with m = round(sum x / width) the distances d = x - m are
// small whatever the mean's size, and their own mean, which m's rounding leaves,
// comes off the variance and the result.
template <typename E, int kC, int kTeam, bool kWhole>
__global__ void __launch_bounds__(forward_warps(kC, kBytes<E>) * 32, forward_blocks_per_sm(kC)) layer_norm_forward(const LayerNormArgs a) {
    extern __shared__ __align__(16) char shared[];
    __shared__ __align__(16) float2 exchange[2][kMeet];
    __shared__ __align__(16) char edge_bytes[kWhole ? 16 : kEdgeBytes];
    using P = Place<E, kC, kTeam, kWhole>;
    constexpr int kPairs = P::kPairs, kHalf = P::kHalf;
    P p(a, exchange, shared_address(shared + a.kept_bytes));
    const int all = p.capacity() * P::kV;
    float *weight = reinterpret_cast<float *>(shared), *bias = weight + all;
    __shared__ __align__(16) char ends[kWhole ? 16 : P::kKeptEdges];
    const uint32_t masks = shared_address(ends);
    const uint32_t edges = shared_address(edge_bytes);
    p.look_ahead();
    p.clear_slots();
    pdl_prologue();
    for (int s = 0; s < a.stages; ++s) p.fetch();
    p.keep_param(weight, a.weight, 1.f);
    p.keep_param(bias, a.bias, 0.f);
    if constexpr (!kWhole) p.keep_edges(ends);
    __syncthreads();

    for (; p.pass < p.passes; p.advance()) {
        p.arrived();
        float2 x[kPairs];
        p.template load<false>(0, masks, x);
        if (a.tensors == 2) {
            float2 add[kPairs];
            p.template load<false>(1, masks, add);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) x[i] = add2(x[i], add[i]);
            if constexpr (!std::is_same<E, F32>::value) {   // as the residual stream holds them
#pragma unroll
                for (int i = 0; i < kPairs; ++i) x[i] = E::to_f2(E::from_f2(x[i].x, x[i].y));
            }
            p.store(a.total, edges, x);
        }
        p.fetch();
        // a chain of additions a chunk
        float2 s = both(0.f);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            float2 t = x[c * kHalf];
#pragma unroll
            for (int i = 1; i < kHalf; ++i) t = add2(t, x[c * kHalf + i]);
            s = c ? add2(s, t) : t;
        }
        const float m = p.sum(s.x + s.y) * a.inv;
        float2 d = both(0.f), q = both(0.f);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            // outside the row the distance is 0
            if (kWhole || p.full(c)) {
                const float2 less = both(kWhole && !p.held(c) ? 0.f : -m);
#pragma unroll
                for (int j = 0; j < kHalf; ++j) x[c * kHalf + j] = add2(x[c * kHalf + j], less);
            } else {
                float2 in[kHalf];
                p.inside(ends, c, in);
#pragma unroll
                for (int j = 0; j < kHalf; ++j) x[c * kHalf + j] = fma2(in[j], both(-m), x[c * kHalf + j]);
            }
            float2 dc = both(0.f), qc = both(0.f);
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const float2 v = x[c * kHalf + j];
                dc = j ? add2(dc, v) : v, qc = j ? fma2(v, v, qc) : mul2(v, v);
            }
            d = c ? add2(d, dc) : dc, q = c ? add2(q, qc) : qc;
        }
        const float2 t = p.sum(make_float2(d.x + d.y, q.x + q.y));
        const float m1 = t.x * a.inv;
        float var = fmaf(t.y, a.inv, -m1 * m1);
        if (var < 0.f) var = 0.f;   // (NaN stays)
        const float rstd = reciprocal_root(var + a.eps), less = -m1 * rstd;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            float2 w[kHalf], b[kHalf];
            p.kept(weight, c, w);
            p.kept(bias, c, b);
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                float2 &v = x[c * kHalf + i];
                v = fma2(fma2(v, both(rstd), both(less)), w[i], b[i]);
            }
        }
        p.store(a.out, edges, x);
        if (a.mean && p.there() && p.column_thread() == 0) {
            a.mean[p.row] = m + m1;
            a.rstd[p.row] = rstd;
        }
    }
}

template <typename E, int kC, int kTeam, bool kWhole>
wgs_status run_unit(LayerNormArgs a, cudaStream_t stream) {
    DeviceInfo dev;
    const wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    const ForwardCut f = forward_cut({kC, kTeam}, a.chunks, a.tensors, kBytes<E>, kWhole, a.rows, a.period, dev.sm_count);
    a.team_warps = f.team_warps, a.kept_bytes = f.kept_bytes, a.stages = f.stages;
    auto kernel = layer_norm_forward<E, kC, kTeam, kWhole>;
    // Above 48 KB, its static memory included, a kernel needs the runtime's leave,
    // which belongs to the context; asking for the same amount on every call needs
    // no record of it.  (At most 67 KB beside a stage, and 72 KB of that.)
    if (f.smem > 40 << 10 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostOfSm) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    return launch(kernel, dim3(f.cut.blocks), dim3(f.cut.threads), static_cast<size_t>(f.smem), stream, a);
}

template <typename E, int kC, bool kWhole>
wgs_status run_warps(const LayerNormArgs &a, cudaStream_t stream) {
    if constexpr (forward_has_warps(kC, kBytes<E>, kWhole)) return run_unit<E, kC, 0, kWhole>(a, stream);
    return WGS_ERR_WIDTH;
}

template <typename E, bool kWhole>
wgs_status run_width(const LayerNormArgs &a, cudaStream_t stream) {
    const Unit u = forward_unit(a.chunks, kBytes<E>, kWhole);
    if (u.team == 4) return run_unit<E, 1, 4, kWhole>(a, stream);
    if (u.team == 8 && u.each == 1) return run_unit<E, 1, 8, kWhole>(a, stream);
    if (u.team == 8 && u.each == 2) return run_unit<E, 2, 8, kWhole>(a, stream);
    if (u.team == 8) return run_unit<E, 3, 8, kWhole>(a, stream);
    if (u.team == 16 && u.each == 2) return run_unit<E, 2, 16, kWhole>(a, stream);
    if (u.team == 16) return run_unit<E, 3, 16, kWhole>(a, stream);
    if (u.team == 32 && u.each == 2) return run_unit<E, 2, 32, kWhole>(a, stream);
    if (u.team == 32 && u.each == 3) return run_unit<E, 3, 32, kWhole>(a, stream);
    if (u.team == 32) return run_unit<E, 4, 32, kWhole>(a, stream);
    if (u.each == 2) return run_warps<E, 2, kWhole>(a, stream);
    if (u.each == 3) return run_warps<E, 3, kWhole>(a, stream);
    if (u.each == 4) return run_warps<E, 4, kWhole>(a, stream);
    return run_warps<E, 6, kWhole>(a, stream);
}

template <typename E>
wgs_status run_format(LayerNormArgs a, cudaStream_t stream) {
    return place_rows<E>(&a) ? run_width<E, true>(a, stream) : run_width<E, false>(a, stream);
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
    if (dtype == WGS_F32) return run_format<F32>(a, stream);
    if (dtype == WGS_F16) return run_format<Fp16>(a, stream);
    return run_format<Bf16>(a, stream);
}

}  // namespace

}  // namespace wgs

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
