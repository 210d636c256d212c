// Gradients of layer norm with weight and bias (sm_103a).
//
// With h = (x - mean) rstd, g = grad_y w and M the mean over the row
//     grad_x = rstd (g - M(g) - h M(g h))  (+ the residual stream's gradient)
//     grad_w = sum grad_y h,   grad_b = sum grad_y   (all rows).
//
// Design.  One pass over the rows, bound by their bytes: a thread's columns are the
// same in all its rows, so their sums stay in registers while rows stream past; a
// block's units add theirs up in shared memory, and a second launch the blocks', all
// in a fixed order.  One block an SM, which walks the rows with all others.
//
// Measured, us a call in a row of calls, and of the copy rate: [131040, 192] fp16 29.7
// (75 %), FP32 49.6 (90 %); [32760, 1536] bf16 with the residual stream's gradient 66
// (90 %); [32761, 771] bf16 55 (40 %).  A thread's 24 columns take 48 registers of sums
// beside 48 of values, so twelve warps an SM: they issue in half of their cycles and
// wait for their own results (shuffles, shared memory) in most others.  Units of fewer
// columns a thread need fewer registers and have the same twelve warps.  The second launch
// shows 2 to 3 us at the end of a call.
#include "wgs_layer_norm.cuh"

namespace wgs {

namespace {

constexpr int kMostBlocks = 152;   // of a launch, and of the workspace's sums
constexpr int kRing = 168 << 10;   // shared memory of a block's slots, at most but for wide rows

template <typename E, int kC, int kTeam, bool kWhole>
__global__ void __launch_bounds__(kThreads, 1) layer_norm_backward(const LayerNormArgs a) {
    extern __shared__ __align__(16) char shared[];
    __shared__ __align__(16) float2 exchange[2][kMeet];
    __shared__ __align__(16) char edge_bytes[kWhole ? 16 : kEdgeBytes];
    using P = Place<E, kC, kTeam, kWhole>;
    constexpr int kPairs = P::kPairs, kHalf = P::kHalf;
    P p(a, exchange, shared_address(shared + a.kept_bytes));
    float *weight = reinterpret_cast<float *>(shared);
    char *mask_words = reinterpret_cast<char *>(weight + p.capacity() * P::kV);
    const uint32_t masks = shared_address(mask_words);
    const uint32_t edges = shared_address(edge_bytes);
    p.look_ahead();
    p.clear_slots();
    pdl_prologue();
    for (int s = 0; s < a.stages; ++s) p.fetch();
    // the statistics of two passes ahead
    auto stats = [&](int64_t row) {
        return row < a.rows ? make_float2(__ldg(a.mean + row), __ldg(a.rstd + row)) : both(0.f);
    };
    float2 now = stats(p.row), next = stats(p.row + p.row_step);
    p.keep_param(weight, a.weight, 1.f);
    if constexpr (!kWhole) p.keep_masks(mask_words);
    __syncthreads();
    float2 gw[kPairs], gb[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) gw[i] = gb[i] = both(0.f);

    for (; p.pass < p.passes; p.advance()) {
        const float2 later = stats(p.row + 2 * p.row_step);
        const float2 rstd = both(now.y);
        p.arrived();
        float2 h[kPairs], g[kPairs];
        // Outside the row h is not -mean rstd, which may pass FP32's range, and then 0 h is no
        // number, as in rows of one large value.  In ragged rows the mean stands there, as near
        // as the format holds it: that is the value itself in rows of one value, and in all others
        // mean rstd is no more than 2^24 sqrt(2 width).
        p.template load<true>(0, masks, h, P::filled(now.x));
        p.template load<true>(1, masks, g);
        float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            float2 w[kHalf], a1, a2;      // a chain of additions a chunk
            p.kept(weight, c, w);
            const float2 less = both(kWhole && !p.held(c) ? 0.f : -now.x);
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const int i = c * kHalf + j;
                h[i] = mul2(add2(h[i], less), rstd);
                gb[i] = add2(gb[i], g[i]);
                gw[i] = fma2(g[i], h[i], gw[i]);
                g[i] = mul2(g[i], w[j]);
                a1 = j ? add2(a1, g[i]) : g[i];
                a2 = j ? fma2(g[i], h[i], a2) : mul2(g[i], h[i]);
            }
            s1 = c ? add2(s1, a1) : a1, s2 = c ? add2(s2, a2) : a2;
        }
        const float2 t = p.sum(make_float2(s1.x + s1.y, s2.x + s2.y));
        const float2 c1 = both(-t.x * a.inv), c2 = both(-t.y * a.inv);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) g[i] = mul2(fma2(h[i], c2, add2(g[i], c1)), rstd);
        if (a.tensors == 3) {
            p.template load<true>(2, masks, h);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) g[i] = add2(g[i], h[i]);
        }
        p.fetch();
        p.store(a.out, edges, g);
        now = next, next = later;
    }
    if (!a.part) return;

    // The block's sums: a warp's rows, then the units, in their order.
    cp_async_wait<0>();
    __syncthreads();
    if constexpr (!P::kMulti) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
#pragma unroll
            for (int o = 16; o >= kTeam; o >>= 1) {
                gw[i].x += __shfl_xor_sync(0xffffffffu, gw[i].x, o);
                gw[i].y += __shfl_xor_sync(0xffffffffu, gw[i].y, o);
                gb[i].x += __shfl_xor_sync(0xffffffffu, gb[i].x, o);
                gb[i].y += __shfl_xor_sync(0xffffffffu, gb[i].y, o);
            }
    }
    float *all = reinterpret_cast<float *>(shared), *mine = all + static_cast<size_t>(p.index) * 2 * a.width;
    if (P::kMulti || p.thread < kTeam) {
#pragma unroll
        for (int i = 0; i < kC * P::kV; ++i) {
            const int col = p.column(i / P::kV) + i % P::kV;
            if (col < 0 || col >= a.width) continue;
            mine[col] = i & 1 ? gw[i / 2].y : gw[i / 2].x;
            mine[a.width + col] = i & 1 ? gb[i / 2].y : gb[i / 2].x;
        }
    }
    __syncthreads();
    const int units = blockDim.x / (p.warps * 32);
    float *part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.width;
    for (int i = threadIdx.x; i < 2 * a.width; i += blockDim.x) {
        float s = all[i];
        for (int u = 1; u < units; ++u) s += all[static_cast<size_t>(u) * 2 * a.width + i];
        part[i] = s;
    }
}

// grad_weight (blockIdx.y 0) and grad_bias (1): the blocks' sums, eight columns a
// block, 16 threads a column.  So few threads find room beside the first launch's
// blocks of up to 160 registers a thread and are there when those end; beside the others
// (some of three chunks a thread, those of six) they start behind them.
constexpr int kParamCols = 8, kParamGroups = 16;

template <typename E>
__global__ void __launch_bounds__(kParamCols * kParamGroups) layer_norm_params(const float *part, int blocks, int width,
                                                                               void *grad_weight, void *grad_bias,
                                                                               bool p32) {
    __shared__ float sums[kParamGroups / 4][kParamCols];
    pdl_prologue();
    const int group = threadIdx.x / kParamCols, lane = threadIdx.x & 31, col = blockIdx.x * kParamCols + (threadIdx.x & 7);
    const float *p = part + static_cast<int64_t>(blockIdx.y) * width + col;
    float s = 0.f;
    if (col < width) {
#pragma unroll
        for (int b = group; b < kMostBlocks; b += kParamGroups)
            if (b < blocks) s += __ldcg(p + b * 2ll * width);
    }
    // the four groups of a warp, then the warps
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (lane < kParamCols) sums[threadIdx.x >> 5][lane] = s;
    __syncthreads();
    void *out = blockIdx.y ? grad_bias : grad_weight;
    if (threadIdx.x >= kParamCols || col >= width || !out) return;
    const float t = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
    if (p32)
        static_cast<float *>(out)[col] = t;
    else if constexpr (!std::is_same<E, F32>::value)
        static_cast<uint16_t *>(out)[col] = static_cast<uint16_t>(E::from_f2(t, 0.f));
}

template <typename E, int kC, int kTeam, bool kWhole>
wgs_status run_unit(LayerNormArgs a, cudaStream_t stream, int *blocks) {
    DeviceInfo dev;
    const wgs_status st = current_device(&dev);
    if (st != WGS_OK) return st;
    using P = Place<E, kC, kTeam, kWhole>;
    a.team_warps = kTeam == 0 ? static_cast<int>(ceil_div(a.chunks, 32 * kC)) : 1;
    const Cut cut = cut_rows(a.rows, a.period, a.team_warps, P::kRowsPerPass, kWarps, dev.sm_count < kMostBlocks ? dev.sm_count : kMostBlocks);
    *blocks = cut.blocks;
    const int stage = cut.threads * a.tensors * kC * 16;
    a.stages = kRing / stage < 1 ? 1 : kRing / stage < kMaxStages ? kRing / stage : kMaxStages;
    // the weight, and what of a ragged row's chunks is its own
    a.kept_bytes = kC * (kTeam == 0 ? 32 * a.team_warps : kTeam) * (kWhole ? 4 * P::kV : 4 * P::kV + 16);
    int smem = a.kept_bytes + a.stages * stage;
    const int sums = 8 * a.width * cut.units;
    if (smem < sums) smem = sums;
    auto kernel = layer_norm_backward<E, kC, kTeam, kWhole>;
    // As the forward's.  (At most 68 KB beside a stage of six chunks from three
    // tensors, 99 KB, and 51 KB beside 168 KB of others.)
    if (smem > 40 << 10 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 << 10) != cudaSuccess) {
        cudaGetLastError();
        return WGS_ERR_LAUNCH;
    }
    return launch(kernel, dim3(cut.blocks), dim3(cut.threads), static_cast<size_t>(smem), stream, a);
}

// As the forward's.
template <typename E, bool kWhole>
wgs_status run_width(const LayerNormArgs &a, cudaStream_t stream, int *blocks) {
    const int n = a.chunks;
    if (n <= 4) return run_unit<E, 1, 4, kWhole>(a, stream, blocks);
    if (n <= 8) return run_unit<E, 1, 8, kWhole>(a, stream, blocks);
    if (n <= 16) return run_unit<E, 2, 8, kWhole>(a, stream, blocks);
    if (n <= 24) return run_unit<E, 3, 8, kWhole>(a, stream, blocks);
    if (n <= 32) return run_unit<E, 2, 16, kWhole>(a, stream, blocks);
    if (n <= 48) return run_unit<E, 3, 16, kWhole>(a, stream, blocks);
    if (n <= 64) return run_unit<E, 2, 32, kWhole>(a, stream, blocks);
    if (n <= 96) return run_unit<E, 3, 32, kWhole>(a, stream, blocks);
    const int each = chunks_of_units(n, std::is_same<E, F32>::value);
    if (each == 2) return run_unit<E, 2, 0, kWhole>(a, stream, blocks);
    if (each == 3) return run_unit<E, 3, 0, kWhole>(a, stream, blocks);
    if constexpr (std::is_same<E, F32>::value) return run_unit<E, 6, 0, kWhole>(a, stream, blocks);
    return WGS_ERR_WIDTH;
}

template <typename E>
wgs_status run_format(LayerNormArgs a, cudaStream_t stream, int *blocks) {
    return place_rows<E>(&a) ? run_width<E, true>(a, stream, blocks) : run_width<E, false>(a, stream, blocks);
}

}  // namespace

}  // namespace wgs

using namespace wgs;

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
    int blocks = 0;   // no rows: the launch that ends the (empty) sums alone
    DeviceInfo dev;
    wgs_status st = current_device(&dev);
    if (st == WGS_OK && rows > 0)
        st = dtype == WGS_F32   ? run_format<F32>(a, stream, &blocks)
             : dtype == WGS_F16 ? run_format<Fp16>(a, stream, &blocks)
                                : run_format<Bf16>(a, stream, &blocks);
    if (st != WGS_OK || !params) return st;
    auto kernel = dtype == WGS_F16    ? layer_norm_params<Fp16>
                  : dtype == WGS_BF16 ? layer_norm_params<Bf16>
                                      : layer_norm_params<F32>;
    return launch(kernel, dim3(static_cast<unsigned>(ceil_div(width, kParamCols)), 2), dim3(kParamCols * kParamGroups), 0, stream,
                  static_cast<const float *>(a.part), blocks, width, grad_weight, grad_bias, a.p32);
}
