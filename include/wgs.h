/*
 * wgs.h -- C ABI of the GB300 (sm_103a) block-glue kernels of a
 * shifted-window (Swin / Pangu-Weather style) transformer block.
 *
 * Sources (page title, section):
 *   [P1] "BW1000 gfx936 Pangu-Weather inference profiling"
 *        (l189.com news 2144533)
 *        s1  the profile: LayerNorm, index_select (two per block), GELU
 *        s3  fixed-width LayerNorm, affine folded into the next Linear
 *        s4  fused residual add + norm, keeping the FP16 rounding point
 *        s5  window gather with a precomputed INT32 index protocol, and the
 *            fused norm-then-gather
 *        s6, s7  the ops kept in the final combination (bias-mask, restore
 *            path) and the fusions rejected
 *   [P3] "PyTorch + HIP fused bias + GELU on Hygon DCU"
 *        (forum.sourcefind.cn)
 *        s3  math semantics: tanh-approximate GELU of input + bias (backward
 *            left out there; added here)
 *        s6  interface checks: clear errors for bad inputs, empty input
 *            launches nothing, work goes on the caller's stream, launch
 *            status is checked
 *        s10, s12  other dtypes as hardening (bfloat16 here)
 *
 * Conventions shared by every device entry point
 *   - All tensor pointers are DEVICE pointers on the current CUDA device,
 *     row-major and dense (row r starts at r * width elements).
 *   - The caller owns every buffer.  The library allocates no device
 *     memory, never synchronises the stream and never touches the default
 *     stream unless the caller passes it (stream 0).
 *   - Work is enqueued on `stream`; the call returns once it is enqueued.
 *     Kernels are launched with programmatic dependent launch: one may be
 *     scheduled while the previous kernel on the stream drains, and before
 *     waiting for it may ask L2 to fetch the lines of its first input rows
 *     (an index-driven kernel also reads its first index entries, L2 only,
 *     to steer those fetches).  No value read before the previous kernel
 *     has completed reaches a result: indices and rows are read again after
 *     the wait, so the usual stream order holds for every buffer.  (A call of
 *     several kernels, position_bias_bwd or group_norm_act and its backward,
 *     may have its second one read the call's inputs while its first one
 *     runs, never before that one has waited; embedding_bwd's last one reads the
 *     workspace so.)
 *   - Arguments are checked before anything is launched; a failed check
 *     returns a status and launches nothing.  A launch failure reported by
 *     the runtime returns WGS_ERR_LAUNCH.
 *   - A call with zero rows (or zero indices) returns WGS_OK and launches
 *     nothing; its pointers may then be NULL.
 *   - fp16 is IEEE binary16; "fp16(v)" below is round-to-nearest-even.
 *   - The kernels run only on compute capability 10.3 (sm_103a); on any
 *     other device the entry points return WGS_ERR_ARCH.
 *   - Calls are thread-safe; the shared state is the per-device index
 *     error words read by wgs_check_error() (and the scratch array of
 *     bias_gelu_tanh_bwd_noalloc).  Kernels name the error words
 *     directly, so no device address is kept between calls.
 *   - The first call of an entry point on a device (per dtype) caches what it
 *     needs from the runtime (SM count, resident CTAs per SM); make those
 *     calls outside stream capture.  Other calls, captured or not, make no
 *     such query.  Both depend on the device only, not on its context.  The
 *     16-bit GELU backward also raises its first pass's shared-memory limit,
 *     which belongs to the context: the first call on a device does it, and
 *     in a later context (after cudaDeviceReset, say) the first launch there
 *     is rejected by the runtime, the limit raised and the launch retried;
 *     make that call outside stream capture too.  (position_bias_bwd, the
 *     group and layer norms and embedding_bwd raise theirs on every call, which
 *     captures as well.)
 */
#ifndef WGS_H
#define WGS_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* 1: the LayerNorm family, gathers and bias + GELU in fp16 / fp32.
 * 2: adds the bfloat16 forms, the GELU backward (with and without a
 *    workspace), the attention bias-mask add and the region-label builder;
 *    the backward's workspace query covers zero rows.
 * Entry points added since (position bias by buckets, group norm, layer norm
 * with weights, embedding) change no call of version 2, so the number stays. */
#define WGS_ABI_VERSION 2

typedef enum {
    WGS_OK = 0,
    WGS_ERR_NULL = 1,    /* a required pointer is NULL                      */
    WGS_ERR_SHAPE = 2,   /* negative size, or sizes inconsistent            */
    WGS_ERR_WIDTH = 3,   /* width not supported by this entry point         */
    WGS_ERR_ALIGN = 4,   /* a pointer is not aligned as required            */
    WGS_ERR_DTYPE = 5,   /* unknown dtype code                              */
    WGS_ERR_ARCH = 6,    /* current device is not compute capability 10.3   */
    WGS_ERR_LAUNCH = 7,  /* the CUDA runtime rejected the launch            */
    WGS_ERR_INDEX = 8,   /* a gather index was outside [-1, n_src)          */
    WGS_ERR_ALIAS = 9,   /* buffers overlap in a way the operation forbids  */
    WGS_ERR_CUDA = 10,   /* another CUDA runtime call failed                */
    WGS_ERR_TOO_LARGE = 11 /* larger than the library's fixed scratch       */
} wgs_status;

typedef enum { WGS_F32 = 0, WGS_F16 = 1, WGS_BF16 = 2 } wgs_dtype;

/* Activations of group_norm_act. */
typedef enum { WGS_ACT_NONE = 0, WGS_ACT_SILU = 1, WGS_ACT_GELU_TANH = 2 } wgs_act;

/* Index-map construction order (wgs_build_window_index). */
#define WGS_SHIFT_THEN_PAD 0
#define WGS_PAD_THEN_SHIFT 1

/* Human-readable name of a status; never NULL. */
const char *wgs_status_string(wgs_status s);

/* WGS_ABI_VERSION of the built library. */
int32_t wgs_abi_version(void);

/* ------------------------------------------------------------------ */
/* ln_fwd -- LayerNorm without affine                          [P1 s3] */
/* ------------------------------------------------------------------ */
/* For each of `rows` rows of `width` fp16 values:
 *     mean = sum(x) / width,  var = sum((x - mean)^2) / width   (FP32)
 *     y    = fp16((x - mean) / sqrt(var + eps))
 * The affine scale and shift are not applied: the model folds them into
 * the following Linear at load time.
 *   x, y   fp16 [rows, width], 16-byte aligned.  y == x (in place) is
 *          allowed; any other overlap returns WGS_ERR_ALIAS.
 *   width  192 or 384 only (else WGS_ERR_WIDTH): the model's two hidden
 *          widths; there is no generic fallback.
 *   eps    added to the variance inside the square root (1e-5 in the model). */
wgs_status ln_fwd(const void *x, void *y, int64_t rows, int32_t width, float eps,
                  cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* residual_add_ln_fwd -- fused residual add + LayerNorm       [P1 s4] */
/* ------------------------------------------------------------------ */
/*     residual_out = fp16(fp32(residual) + fp32(branch))   (written out)
 *     y            = LN(residual_out)                       (as ln_fwd)
 * The normalisation starts from the ROUNDED fp16 residual_out, the same
 * rounding point as a separate add followed by a separate LayerNorm.
 *   residual, branch, residual_out, y  fp16 [rows, width], 16-byte aligned.
 *   residual_out may equal residual or branch; y may equal residual or
 *   branch; residual_out and y must be distinct; partial overlaps return
 *   WGS_ERR_ALIAS.
 *   width  192 or 384 only. */
wgs_status residual_add_ln_fwd(const void *residual, const void *branch, void *residual_out,
                               void *y, int64_t rows, int32_t width, float eps,
                               cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* window_gather -- shifted-window token gather               [P1 s5] */
/* ------------------------------------------------------------------ */
/* For d in [0, n_idx):
 *     dst[d] = src[idx[d]]   if 0 <= idx[d] < n_src   (bit-exact row copy)
 *     dst[d] = 0             if idx[d] == -1           (all-zero pad row)
 * so padding needs no zero-filled tensor.  An index outside [-1, n_src) is
 * a caller error: its row is written as zeros and the device error word is
 * set (see wgs_check_error); nothing faults.
 *   src  fp16 [n_src, width], dst fp16 [n_idx, width], both 16-byte
 *        aligned; they must not overlap (WGS_ERR_ALIAS).
 *   idx  int32 [n_idx], 4-byte aligned, device memory.  Usually built once
 *        per window shape with wgs_build_window_index and copied to the
 *        device.
 *   width  any multiple of 8 (rows are whole 16-byte chunks); 192 and 384
 *          take a specialised path. */
wgs_status window_gather(const void *src, const int32_t *idx, void *dst, int64_t n_src,
                         int64_t n_idx, int32_t width, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* norm_gather -- fused LayerNorm then window gather          [P1 s5] */
/* ------------------------------------------------------------------ */
/*     dst[d] = LN(src[idx[d]])  for a valid index, 0 for idx[d] == -1
 * The normalised tensor is never materialised: each gathered row is
 * normalised in registers on its way to dst.  Results equal ln_fwd
 * followed by window_gather bit for bit.  Buffers, index rules and errors
 * as window_gather; width 192 or 384 only. */
wgs_status norm_gather(const void *src, const int32_t *idx, void *dst, int64_t n_src,
                       int64_t n_idx, int32_t width, float eps, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* window_reverse_add_ln_fwd -- window reverse + residual add + LN     */
/*                                          [P1 s5 inverse, s4, s7]    */
/* ------------------------------------------------------------------ */
/* After window attention the windowed rows return to token order (the
 * inverse of window_gather: crop pads, undo the window order and the
 * cyclic shift), join the residual stream and feed norm2, in one pass.
 * P1 s7 keeps such a "restore path" op; s4 fixes the rounding point:
 *     residual_out[t] = fp16(fp32(residual[t]) + fp32(windows[inv_idx[t]]))
 *     y[t]            = LN(residual_out[t])                   (as ln_fwd)
 *   residual, residual_out, y  fp16 [rows, width], 16-byte aligned;
 *          residual_out and y may each equal residual, must differ from
 *          each other; other overlaps return WGS_ERR_ALIAS.
 *   windows  fp16 [n_windowed, width], 16-byte aligned, read at the rows
 *          inv_idx names; must not overlap the outputs.
 *   inv_idx  int32 [rows]: the windowed row of each token, usually from
 *          wgs_build_window_inverse.  A value outside [0, n_windowed) sets
 *          the device error word and that token takes no branch
 *          (residual_out = residual, bit for bit).
 *   width  192 or 384 only. */
wgs_status window_reverse_add_ln_fwd(const void *residual, const void *windows,
                                     const int32_t *inv_idx, void *residual_out, void *y,
                                     int64_t rows, int64_t n_windowed, int32_t width, float eps,
                                     cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* residual_add_norm_gather -- residual add + norm1 + window gather    */
/*                                                  [P1 s4, s5]        */
/* ------------------------------------------------------------------ */
/* At a block boundary the residual stream is updated and written out (s4)
 * and the next block's norm1 output is consumed only by its window gather
 * (s5); one pass does all three:
 *     residual_out[s] = fp16(fp32(residual[s]) + fp32(branch[s]))
 *     dst[d]          = LN(residual_out[idx[d]])   (zero row for -1)
 * Equal, bit for bit, to residual_add_ln_fwd followed by window_gather of
 * its y.  Each source row s is processed by the destination row that names
 * it: rows of residual_out that idx never names are NOT written (a map from
 * wgs_build_window_index names every token exactly once).
 *   residual, branch, residual_out  fp16 [n_src, width], 16-byte aligned;
 *          residual_out may equal residual or branch (in place is exact
 *          only when idx names each row at most once).
 *   dst    fp16 [n_idx, width], must not overlap anything else.
 *   idx    int32 [n_idx], as for window_gather (bad values: zero row and
 *          the device error word).
 *   width  192 or 384 only. */
wgs_status residual_add_norm_gather(const void *residual, const void *branch, const int32_t *idx,
                                    void *residual_out, void *dst, int64_t n_src, int64_t n_idx,
                                    int32_t width, float eps, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* bfloat16 forms of the LayerNorm family                               */
/*      [P3 s3 and s12 list BF16 among the formats a hardened op covers] */
/* ------------------------------------------------------------------ */
/* Same arguments, rules and errors as the fp16 entry points above, with
 * every 16-bit tensor in bfloat16: elements widen exactly to FP32, the
 * statistics are FP32, and results round to nearest-even bfloat16.  The
 * residual sum is round_bf16(fp32 a + fp32 b), which equals rounding the
 * exact sum once (binary32 has at least 2 * 8 + 2 significand bits).
 * window_gather copies rows bit for bit and serves both formats. */
wgs_status ln_fwd_bf16(const void *x, void *y, int64_t rows, int32_t width, float eps,
                       cudaStream_t stream);
wgs_status residual_add_ln_fwd_bf16(const void *residual, const void *branch, void *residual_out,
                                    void *y, int64_t rows, int32_t width, float eps,
                                    cudaStream_t stream);
wgs_status norm_gather_bf16(const void *src, const int32_t *idx, void *dst, int64_t n_src,
                            int64_t n_idx, int32_t width, float eps, cudaStream_t stream);
wgs_status window_reverse_add_ln_fwd_bf16(const void *residual, const void *windows,
                                          const int32_t *inv_idx, void *residual_out, void *y,
                                          int64_t rows, int64_t n_windowed, int32_t width,
                                          float eps, cudaStream_t stream);
wgs_status residual_add_norm_gather_bf16(const void *residual, const void *branch,
                                         const int32_t *idx, void *residual_out, void *dst,
                                         int64_t n_src, int64_t n_idx, int32_t width, float eps,
                                         cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* bias_gelu_tanh -- fused bias + tanh-approximate GELU       [P3 s3] */
/* ------------------------------------------------------------------ */
/*     t = x + bias[col]   (rounded once to the tensor dtype)
 *     y = 0.5 t (1 + tanh(sqrt(2/pi) (t + 0.044715 t^3)))
 * evaluated in FP32 and rounded to the tensor dtype.
 *   x, y   [rows, width] of `dtype` (WGS_F32, WGS_F16 or WGS_BF16); y == x allowed,
 *          other overlaps return WGS_ERR_ALIAS.
 *   bias   [width] of `dtype`; must not overlap y.
 *   width  any value >= 1.  A 16-byte vector path runs when width is a
 *          multiple of 4 (f32) or 8 (16-bit types) and all pointers are 16-byte
 *          aligned; otherwise a scalar path runs (same results). */
wgs_status bias_gelu_tanh(const void *x, const void *bias, void *y, int64_t rows, int32_t width,
                          wgs_dtype dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* bias_gelu_tanh_bwd -- backward of bias + tanh-GELU                   */
/*          [P3 s3: the tutorial op leaves backward out; this adds it]  */
/* ------------------------------------------------------------------ */
/* Gradient of y = gelu_tanh(x + bias) with an eager backward's rounding
 * points:
 *     t         = round(x + bias[c])                         (as forward)
 *     grad_x    = round(grad_y * gelu'(t))   (gelu' evaluated in FP32)
 *     grad_bias = round(sum over rows of grad_x[., c])       (FP32 sum)
 * The column sum is deterministic: per-slab FP32 partial sums go to
 * `workspace`, then one pass adds them in a fixed order; the summation
 * order depends only on rows, width and dtype, so results do not depend on
 * the device.
 *   grad_y, x, grad_x  [rows, width] of `dtype`; grad_x may equal grad_y,
 *          other overlaps return WGS_ERR_ALIAS.
 *   bias, grad_bias    [width] of `dtype`, disjoint from everything else.
 *   workspace  device memory of at least
 *          wgs_bias_gelu_bwd_workspace_bytes(rows, width) bytes (one slab of
 *          width floats when rows == 0), 16-byte aligned, owned by the
 *          caller, disjoint from the tensors; its contents on entry do not
 *          matter.
 *   rows == 0 writes grad_bias = 0 (two small launches); width == 0 returns
 *   WGS_OK and launches nothing.  The 16-byte vector path needs width a
 *   multiple of 4 (f32) or 8 (16-bit types) and aligned tensors; otherwise
 *   a scalar path runs (same results). */
size_t wgs_bias_gelu_bwd_workspace_bytes(int64_t rows, int32_t width);
wgs_status bias_gelu_tanh_bwd(const void *grad_y, const void *x, const void *bias, void *grad_x,
                              void *grad_bias, void *workspace, size_t workspace_bytes,
                              int64_t rows, int32_t width, wgs_dtype dtype, cudaStream_t stream);

/* bias_gelu_tanh_bwd_noalloc -- the same backward without a workspace.
 * The reference pages have no counterpart; it exists for callers that
 * cannot give this library device memory: an op inside a host runtime that
 * owns every allocation and passes its plugins no allocator or workspace,
 * or a hot path that must not call cudaMalloc because that call can
 * synchronise the device.  The partial column sums then live in one array
 * of 1,310,720 floats (5 MiB) built into the library, which every GPU that
 * loads the library keeps until the process exits.
 *   Arguments, results and errors as bias_gelu_tanh_bwd, without
 *   `workspace`.  Sizes whose partial sums would not fit (more than
 *   1,310,720 floats: min(608, ceil(rows / 216)) slabs x width, so any row
 *   count up to width 2048) return WGS_ERR_TOO_LARGE and launch nothing.
 *   Allocates nothing.  Every call looks up the array's device address in
 *   the calling thread's current context (cudaGetSymbolAddress, a host-side
 *   lookup), so a device reset or a second context on the device is safe.
 *   The first call in a context also loads the library's device code there:
 *   make that first call before any stream capture.
 *   All calls on a device share the array, which keeps whatever the last
 *   call left there; nothing in it needs to start at zero, because every
 *   partial sum is written before it is read.  Calls whose work overlaps on
 *   the GPU (other streams, other host threads) race on the array: run one
 *   at a time per device. */
wgs_status bias_gelu_tanh_bwd_noalloc(const void *grad_y, const void *x, const void *bias,
                                      void *grad_x, void *grad_bias, int64_t rows, int32_t width,
                                      wgs_dtype dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* window_bias_mask_add -- position bias + shift mask before softmax    */
/*                                                          [P1 s6, s7] */
/* ------------------------------------------------------------------ */
/* P1 s7 keeps a "bias-mask" op in the final combination and s6 rejects
 * fusing it with softmax; the pages give no arithmetic.  This library's
 * reading is the shifted-window transformer's general one: the attention
 * logits of every window and head receive a position bias and, in shifted
 * blocks, a mask between rows that the cyclic roll brought together:
 *     t[w,h,i,j]   = fp(scores[w,h,i,j] + bias[type[w],h,i,j])
 *     out[w,h,i,j] = fp(t + (region[w*n+i] == region[w*n+j] ? 0 : m))
 * where fp() rounds to nearest-even in `dtype` and m = fp(mask_value); the
 * mask term is added to every element (so -0 becomes +0 where it is 0).
 * With region == NULL (an unshifted block) out = t.
 *   scores, out  [n_win, heads, n, n] of dtype (WGS_F16 or WGS_BF16);
 *                out may equal scores, other overlaps return WGS_ERR_ALIAS.
 *   bias         [n_types, heads, n, n] of dtype: the position bias already
 *                expanded from its table, one slab per window type.
 *   win_type     int32 [n_win] in [0, n_types), or NULL for type 0 (then
 *                n_types may be 1).  A type outside the range writes that
 *                window's outputs as zeros and sets the device error word
 *                (wgs_check_error); nothing faults.
 *   region       int32 [n_win * n] labels (wgs_build_shift_regions), or NULL.
 * n_win * heads * n must be below 2^31 (else WGS_ERR_SHAPE).  The 16-byte
 * path needs n a multiple of 8 (n <= 2048), scores / bias / out 16-byte
 * aligned and region 16-byte aligned; otherwise a scalar path runs (same
 * results). */
wgs_status window_bias_mask_add(const void *scores, const void *bias, const int32_t *win_type,
                                const int32_t *region, void *out, int64_t n_win, int32_t heads,
                                int32_t n, int32_t n_types, float mask_value, wgs_dtype dtype,
                                cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* position_bias -- a learned position bias by buckets                  */
/* ------------------------------------------------------------------ */
/* What window_bias_mask_add reads as its `bias` is, in training, expanded
 * from a table of learned values: a bucket map sends every (query, key)
 * pair p = i * n_k + j of a window to a row of the table.
 *     bias[t,h,p] = fp(table[t, bucket[p], h])   for 0 <= bucket[p] < n_buckets
 *     bias[t,h,p] = 0                             for bucket[p] == -1
 * fp() rounds once, to nearest even, to `dtype`.  A bucket outside
 * [-1, n_buckets) gives 0 and sets the device error word (wgs_check_error);
 * nothing faults.
 *   table   [n_types, n_buckets, heads] of table_dtype: WGS_F32, or `dtype`.
 *   bucket  int32 [n_pairs], device memory; usually from
 *           wgs_build_window_buckets or wgs_build_distance_buckets.
 *   bias    [n_types, heads, n_pairs] of dtype (any wgs_dtype); must not
 *           overlap the inputs (WGS_ERR_ALIAS).
 * n_pairs must be below 2^31 - 4096 and heads * n_buckets below 2^26 (else
 * WGS_ERR_SHAPE).  Pointers need their element's alignment; with n_pairs a multiple of 8 and bucket and
 * bias 16-byte aligned the heads of a bucket are read together (same
 * results). */
wgs_status position_bias(const void *table, const int32_t *bucket, void *bias, int32_t n_types,
                         int32_t heads, int64_t n_pairs, int32_t n_buckets, wgs_dtype table_dtype,
                         wgs_dtype dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* position_bias_bwd -- the table's gradient                            */
/* ------------------------------------------------------------------ */
/* The bias addition passes the gradient of its output to the logits and to
 * the bias unchanged, so with grad the gradient of the logits
 *     grad_table[t,b,h] = fp(sum of grad[w,h,p] over the windows w with
 *                            win_type[w] == t and pairs p with bucket[p] == b)
 * summed in FP32 in an order that depends on the sizes and the map alone: windows
 * of a type in runs of at most 128, the runs, a bucket's pairs in 32s, and those
 * sums, so that rounding errors grow with the longest of these, not with all.
 *   grad      [n_win, heads, n_pairs] of dtype (any wgs_dtype).
 *   plan      device copy of the bucket map's plan (wgs_build_bucket_plan),
 *             16-byte aligned, with its n_slots.  A plan of other sizes than
 *             the call's gives a zero gradient and sets the device error word.
 *   win_type  int32 [n_win] in [0, n_types), or NULL for type 0.  A window
 *             of another type adds to no gradient and sets the error word.
 *   grad_table  [n_types, n_buckets, heads] of table_dtype (WGS_F32, or
 *             `dtype`); every entry is written, 0 where nothing is added.
 * n_pairs must be below 2^31 - 4096, n_win at most 2^31 - 65537, heads * n_buckets
 * below 2^26 and the tiles of 4096 pairs of all heads and types below 2^31 (else
 * WGS_ERR_SHAPE).  A block looks at the types of all windows of its share:
 * n_types is meant to be a few hundred at most.
 *   workspace at least wgs_position_bias_bwd_workspace_bytes(...) bytes,
 *             16-byte aligned, disjoint from the tensors; its contents on
 *             entry do not matter.  Calls that overlap on the GPU need
 *             workspaces of their own.  (0 bytes for sizes that the call refuses.) */
size_t wgs_position_bias_bwd_workspace_bytes(int64_t n_win, int32_t heads, int32_t n_types,
                                             int64_t n_pairs, int64_t n_slots);
wgs_status position_bias_bwd(const void *grad, const int32_t *plan, const int32_t *win_type,
                             void *grad_table, void *workspace, size_t workspace_bytes,
                             int64_t n_win, int32_t heads, int64_t n_pairs, int32_t n_buckets,
                             int64_t n_slots, int32_t n_types, wgs_dtype dtype,
                             wgs_dtype table_dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* Host-side bucket maps and plans                                      */
/* ------------------------------------------------------------------ */
/* Buckets of a window's cell pairs, cells numbered row-major as the window
 * index map lays them out.  Axis k contributes q_k * window[k] + k_k of
 * window[k]^2 values when bit k of absolute_axes is set (a bias that knows
 * where in the window the axis stands), else q_k - k_k + window[k] - 1 of
 * 2 window[k] - 1 values; the axes combine row-major.  The count is -1, and
 * the builder returns WGS_ERR_SHAPE, for extents below 1, an axis bit above
 * 7, more than 46340 cells or a count above INT32_MAX.  out_len must be at
 * least the square of the cell count.  Host memory only. */
int64_t wgs_window_bucket_count(const int32_t window[3], int32_t absolute_axes);
wgs_status wgs_build_window_buckets(const int32_t window[3], int32_t absolute_axes,
                                    int32_t *out_host, int64_t out_len);

/* Buckets of the signed distance d = j - (i + q_start) between key j and
 * query i of a sequence (q_start: the first query's position; n_q = 1 for
 * one new token).  Of the buckets of one direction (n_buckets / 2 with
 * bidirectional = 1, else n_buckets) the first half, E, hold the distances
 * 0 ... E - 1 themselves; a larger |d| goes to
 *     E + floor((buckets - E) log(|d| / E) / log(max_distance / E)),
 * at most the last (a distance within 1e-9 of a border counts as on it).
 * With bidirectional = 1 keys behind the query use the first half of the
 * buckets and keys ahead (d > 0) the second; with 0 keys ahead have no
 * bucket (-1).  WGS_ERR_SHAPE for negative sizes, fewer than two buckets a
 * direction, an odd n_buckets with bidirectional = 1, max_distance <= E, or
 * out_len < n_q * n_k.  Host memory only. */
wgs_status wgs_build_distance_buckets(int64_t n_q, int64_t n_k, int64_t q_start,
                                      int32_t n_buckets, int32_t max_distance,
                                      int32_t bidirectional, int32_t *out_host, int64_t out_len);

/* The plan of a bucket map (host int32 [n_pairs], values in [-1,
 * n_buckets)): for tiles of 4096 pairs, the pairs of each bucket.  Built once
 * per map, on one host thread (about 13 ms for 1024 x 1024 pairs and 50 ms for
 * 2047 x 2047: a map that changes with a sequence's length costs that each
 * time), and copied to the device, which a captured graph cannot do anew.  wgs_bucket_plan_words returns its size
 * in int32 words and its slot count (a bucket's pairs in a tile make a slot or
 * more), or -1 for invalid sizes or a value outside [-1, n_buckets), for
 * which the builder returns WGS_ERR_SHAPE or WGS_ERR_INDEX.  Host memory
 * only. */
int64_t wgs_bucket_plan_words(const int32_t *bucket_host, int64_t n_pairs, int32_t n_buckets,
                              int64_t *n_slots);
wgs_status wgs_build_bucket_plan(const int32_t *bucket_host, int64_t n_pairs, int32_t n_buckets,
                                 int32_t *plan_host, int64_t plan_words);

/* ------------------------------------------------------------------ */
/* group_norm_act -- group norm with an activation, channels last       */
/* ------------------------------------------------------------------ */
/* x holds n samples of `spatial` rows of `channels` values; a group is
 * channels / groups neighbouring channels over all rows of a sample:
 *     mean, var   over the spatial * channels / groups values (biased, FP32)
 *     rstd = 1 / sqrt(var + eps)
 *     y    = fp(act((x - mean) * rstd * weight[c] + bias[c]))
 * in FP32, rounded once to `dtype`.  The statistics are sums of distances from
 * references near the mean, so neither the mean's size nor rows far from all
 * others cost accuracy; distances whose squares pass FP32's range (beyond about
 * 1e18) are not covered.  act: WGS_ACT_NONE, WGS_ACT_SILU
 * (z / (1 + exp(-z))) or WGS_ACT_GELU_TANH (as bias_gelu_tanh's); any other
 * value returns WGS_ERR_DTYPE.
 *   x, y    [n, spatial, channels] of dtype (any wgs_dtype); y == x allowed,
 *           other overlaps return WGS_ERR_ALIAS.
 *   weight, bias  [channels] of param_dtype (WGS_F32, or `dtype`), both or
 *           neither (NULL: 1 and 0).
 *   mean, rstd  float [n, groups], written for the backward; both or neither.
 *   workspace  at least wgs_group_norm_act_workspace_bytes(...) bytes,
 *           16-byte aligned, disjoint from the tensors; its contents on entry
 *           do not matter.  Calls that overlap on the GPU need their own.
 * channels: a multiple of groups, at most 4096, with groups at most 2048 (else
 * WGS_ERR_WIDTH).  n at most 65535, spatial below 2^31 (else WGS_ERR_SHAPE);
 * n == 0 or spatial == 0 launches nothing.  Rows are moved in 16-byte chunks
 * when channels is a multiple of 4 (f32) or 8 (16-bit types) and x and y are
 * 16-byte aligned, else in pairs of elements or single ones.  Sums run in an
 * order that depends on the sizes and on which of these it is. */
size_t wgs_group_norm_act_workspace_bytes(int64_t n, int64_t spatial, int32_t channels,
                                          int32_t groups);
wgs_status group_norm_act(const void *x, const void *weight, const void *bias, void *y, float *mean,
                          float *rstd, void *workspace, size_t workspace_bytes, int64_t n,
                          int64_t spatial, int32_t channels, int32_t groups, float eps, wgs_act act,
                          wgs_dtype dtype, wgs_dtype param_dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* group_norm_act_bwd -- its gradients                                  */
/* ------------------------------------------------------------------ */
/* With h = (x - mean) rstd, z = h weight + bias, dz = grad_y act'(z) and M()
 * the mean over a group:
 *     grad_x      = fp(rstd (dz weight - M(dz weight) - h M(dz weight h)))
 *     grad_weight = fp(sum of dz h),   grad_bias = fp(sum of dz)  (all rows)
 * in FP32, each rounded once.  A thread adds its rows one after another, of which
 * there are about rows / 152 over its block's row groups: terms of one sign leave
 * the sums off by a few 1e-7 at 131040 rows of 192 FP32 values, by 5e-5 at 11
 * million.
 *   grad_y, x, grad_x  as x above; grad_x may equal grad_y or x.
 *   mean, rstd  as the forward wrote them.
 *   grad_weight, grad_bias  [channels] of param_dtype; NULL skips either
 *           (both must be NULL where weight and bias are).
 *   n == 0 or spatial == 0 writes zeros to grad_weight and grad_bias. */
size_t wgs_group_norm_act_bwd_workspace_bytes(int64_t n, int64_t spatial, int32_t channels,
                                              int32_t groups);
wgs_status group_norm_act_bwd(const void *grad_y, const void *x, const void *weight,
                              const void *bias, const float *mean, const float *rstd, void *grad_x,
                              void *grad_weight, void *grad_bias, void *workspace,
                              size_t workspace_bytes, int64_t n, int64_t spatial, int32_t channels,
                              int32_t groups, wgs_act act, wgs_dtype dtype, wgs_dtype param_dtype,
                              cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* layer_norm -- layer norm with weight and bias, any width             */
/* ------------------------------------------------------------------ */
/* ln_fwd folds the affine part into the following Linear; a block in training
 * keeps it, and reads the statistics again on its way back.  For each row:
 *     mean = sum(x) / width,  var = sum((x - mean)^2) / width
 *     rstd = 1 / sqrt(var + eps)
 *     y    = fp((x - mean) * rstd * weight[c] + bias[c])
 * in FP32, rounded once to `dtype`.  The variance and y are formed from the
 * distances to the row's rounded mean and corrected for its rounding, so the
 * mean's size costs no accuracy; sums of values, or of their distances'
 * squares, that pass FP32's range are not covered.
 *   x, y    [rows, width] of dtype (any wgs_dtype); y == x allowed, other
 *           overlaps return WGS_ERR_ALIAS.
 *   weight, bias  [width] of param_dtype (WGS_F32, or `dtype`); NULL: 1 and 0
 *           (a bias needs a weight).
 *   mean, rstd  float [rows], written for the backward; both or neither.
 * width: 1 to 8192 (else WGS_ERR_WIDTH).  Pointers need their element's
 * alignment.  Rows are moved in 16-byte chunks whatever the width, so the first
 * one's 16 bytes in memory may be read from their start where x does not begin on
 * 16; tensors whose rows start at different places in a chunk are moved element by
 * element.  Sums run in an order that depends on the sizes, the format and where
 * rows start. */
wgs_status layer_norm(const void *x, const void *weight, const void *bias, void *y, float *mean,
                      float *rstd, int64_t rows, int32_t width, float eps, wgs_dtype dtype,
                      wgs_dtype param_dtype, cudaStream_t stream);

/* residual_add_layer_norm -- the residual add and the norm in one pass:
 *     residual_out = fp(residual + branch)   (written out)
 *     y            = layer_norm(residual_out)
 * with the rounding point of residual_add_ln_fwd.  residual_out and y may each
 * equal residual or branch, must differ from each other; other overlaps return
 * WGS_ERR_ALIAS. */
wgs_status residual_add_layer_norm(const void *residual, const void *branch, const void *weight,
                                   const void *bias, void *residual_out, void *y, float *mean,
                                   float *rstd, int64_t rows, int32_t width, float eps,
                                   wgs_dtype dtype, wgs_dtype param_dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* layer_norm_bwd -- the gradients of both                              */
/* ------------------------------------------------------------------ */
/* With h = (x - mean) rstd, g = grad_y weight and M() the mean over a row:
 *     grad_x      = fp(rstd (g - M(g) - h M(g h)) + grad_residual)
 *     grad_weight = fp(sum of grad_y h),  grad_bias = fp(sum of grad_y)  (all rows)
 * in FP32, each rounded once.  x is the forward's x, or residual_out;
 * grad_residual is the gradient that reaches residual_out past the norm (NULL:
 * none), and grad_x then is the gradient of residual and of branch.  A thread
 * adds its rows one after another, of which there are about rows / 152 over its
 * block's units; the sums' order depends on what the forward's does.
 *   grad_y, x, grad_residual, grad_x  as x above; grad_x may equal any of
 *           the others.
 *   mean, rstd  as the forward wrote them.
 *   grad_weight, grad_bias  [width] of param_dtype; NULL skips either.
 *   workspace  at least wgs_layer_norm_bwd_workspace_bytes(...) bytes, 16-byte
 *           aligned, disjoint from the tensors; its contents on entry do not
 *           matter, and it may be NULL where both gradients are.  Calls that
 *           overlap on the GPU need their own.
 *   rows == 0 writes zeros to grad_weight and grad_bias. */
size_t wgs_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t width);
wgs_status layer_norm_bwd(const void *grad_y, const void *x, const float *mean, const float *rstd,
                          const void *weight, const void *grad_residual, void *grad_x,
                          void *grad_weight, void *grad_bias, void *workspace,
                          size_t workspace_bytes, int64_t rows, int32_t width, wgs_dtype dtype,
                          wgs_dtype param_dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* embedding -- rows of a table by index, scaled                        */
/* ------------------------------------------------------------------ */
/*     out[i] = fp(scale * table[idx[i]])   for 0 <= idx[i] < n_rows
 *     out[i] = 0                            for idx[i] == -1 (a pad)
 * The product is one in FP32, which fp() rounds to nearest even in `dtype`.
 * window_gather's rule for indices: one outside [-1, n_rows) gives a zero row
 * and sets the device error word (wgs_check_error); nothing faults.
 *   table   [n_rows, width] of table_dtype: WGS_F32, or `dtype`.
 *   idx     int32 [n_idx].
 *   out     [n_idx, width] of dtype (any wgs_dtype); must not overlap the
 *           inputs (WGS_ERR_ALIAS).
 * width: 1 to 32768 (else WGS_ERR_WIDTH).  n_idx and n_rows below 2^31 - 1
 * (else WGS_ERR_SHAPE).  Pointers need their element's alignment; 16 bytes of the
 * table are moved at a time where all rows start on as many (same results). */
wgs_status embedding(const void *table, const int32_t *idx, void *out, int64_t n_idx,
                     int64_t n_rows, int32_t width, float scale, wgs_dtype table_dtype,
                     wgs_dtype dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* embedding_bwd -- the table's gradient                                */
/* ------------------------------------------------------------------ */
/*     grad_table[r] = fp(scale * sum of grad[i] over the i with idx[i] == r)
 * summed in FP32 over the indices sorted by row, positions in order, cut into pieces
 * of equal size: an order that depends on idx, the sizes and the format alone.
 * With scale 1 it is also the gradient of window_gather through a map that may
 * name a row more than once.  scale is finite (else rows that no index names may be
 * no numbers).  An index of -1 adds to no row, one outside [-1,
 * n_rows) to none and sets the device error word.
 *   grad        [n_idx, width] of dtype (any wgs_dtype).  Where 16-bit rows are no
 *               whole 16-byte chunks they are read by words of 4 bytes, and so the 2
 *               bytes before the first row where it does not begin on 4.
 *   grad_table  [n_rows, width] of table_dtype (WGS_F32, or `dtype`); every
 *               row is written, zeros where no index names it (all of them with
 *               n_idx == 0).
 *   workspace at least wgs_embedding_bwd_workspace_bytes(...) bytes, 16-byte
 *             aligned, disjoint from the tensors; its contents on entry do not
 *             matter.  Calls that overlap on the GPU need their own.  (0 bytes
 *             for sizes that the call refuses.)
 * Sizes as above. */
size_t wgs_embedding_bwd_workspace_bytes(int64_t n_idx, int64_t n_rows, int32_t width);
wgs_status embedding_bwd(const void *grad, const int32_t *idx, void *grad_table, void *workspace,
                         size_t workspace_bytes, int64_t n_idx, int64_t n_rows, int32_t width,
                         float scale, wgs_dtype dtype, wgs_dtype table_dtype, cudaStream_t stream);

/* ------------------------------------------------------------------ */
/* Host-side window index map                                 [P1 s5] */
/* ------------------------------------------------------------------ */
/* The page fixes the protocol (INT32 per destination row, >= 0 source
 * token, -1 zero row, precomputed once per window shape); the
 * construction below is this library's reading of it:
 *   - tokens are the row-major flattening of a grid[0] x grid[1] x grid[2]
 *     (Z, H, W) grid;
 *   - the padded grid has extents padded[k] >= grid[k]; padded == NULL
 *     rounds each extent up to a multiple of window[k];
 *   - windows tile the padded grid from the origin, the last one on an axis
 *     cut short when the padded extent is not a window multiple;
 *   - destination rows run window by window (row-major over the window
 *     grid), then row-major over the cells of each window;
 *   - WGS_SHIFT_THEN_PAD: a cell (z,h,w) inside the grid reads token
 *     ((z+s0) mod Z, (h+s1) mod H, (w+s2) mod W) -- a cyclic roll by
 *     -shift -- and every other cell is -1;
 *     WGS_PAD_THEN_SHIFT: the roll runs over the padded grid, and a rolled
 *     position outside the grid is -1.
 * A block feeds one map to its gather, its attention (window_bias_mask_add)
 * and its window reverse, and a batched attention needs equal windows: pass
 * padded extents that are window multiples (padded == NULL does this), e.g.
 * 4 x 96 x 96 for the 4 x 91 x 90 grid at window (2, 6, 12).  A map with a
 * cut last window (4 x 96 x 90 there) is valid for the gathers alone.
 * Host memory only; no CUDA call is made. */

/* Number of destination rows (product of the padded extents), or -1 for
 * invalid extents: grid or window < 1, padded < grid, a rounded-up extent
 * above INT32_MAX, or a product (of the padded extents or of the grid)
 * that does not fit in int64.  The builders below return WGS_ERR_SHAPE for
 * the same extents. */
int64_t wgs_window_index_count(const int32_t grid[3], const int32_t window[3],
                               const int32_t *padded);

/* Fill out_host[0 .. count) with the map.  out_len must be at least the
 * count (else WGS_ERR_SHAPE); the token count must fit in int32. */
wgs_status wgs_build_window_index(const int32_t grid[3], const int32_t window[3],
                                  const int32_t shift[3], const int32_t *padded, int32_t flags,
                                  int32_t *out_host, int64_t out_len);

/* Fill inv_host[0 .. grid[0]*grid[1]*grid[2]) with the inverse map: the
 * windowed row that holds each token (same arguments as
 * wgs_build_window_index; out_len must be at least the token count, else
 * WGS_ERR_SHAPE).  Host memory only; no CUDA call is made. */
wgs_status wgs_build_window_inverse(const int32_t grid[3], const int32_t window[3],
                                    const int32_t shift[3], const int32_t *padded, int32_t flags,
                                    int32_t *inv_host, int64_t out_len);

/* Fill out_host[0 .. count) with the shift-mask region label of every
 * windowed row, in the map's destination order (same arguments as
 * wgs_build_window_index, plus axes_mask).  Along axis k (bit k of
 * axes_mask set) a row's cell c holds the token rolled in from c + s_k of
 * the roll's period (the grid for WGS_SHIFT_THEN_PAD, the padded grid for
 * WGS_PAD_THEN_SHIFT, s_k the shift taken modulo that period); when s_k is
 * not 0 the cell lies past the roll's seam if c + s_k >= period_k.  The
 * label is the sum over masked axes of 2^k * [past the seam along k]; pad
 * cells follow the same rule.  Two rows of a window share a label exactly
 * when the roll put no seam between them along a masked axis, the regions
 * of the classic shifted-window attention mask.  axes_mask = 7 masks every
 * axis; a periodic axis (longitude) can be left out.  Host memory only;
 * out_len must be at least the count, else WGS_ERR_SHAPE. */
wgs_status wgs_build_shift_regions(const int32_t grid[3], const int32_t window[3],
                                   const int32_t shift[3], const int32_t *padded, int32_t flags,
                                   int32_t axes_mask, int32_t *out_host, int64_t out_len);

/* Read and clear the current device's index error words after the work
 * already queued on `stream` has finished.  This call synchronises
 * `stream`.  Returns WGS_ERR_INDEX if any gather since the last check met
 * an index outside [-1, n_src), any window reverse an inverse index outside
 * [0, n_windowed), or any window_bias_mask_add a window type outside
 * [0, n_types), or a position-bias call a bucket, window type or plan out of
 * its range, or an embedding call an index outside [-1, n_rows);
 * WGS_ERR_LAUNCH if a kernel since then gave up waiting for its own
 * copies to arrive (its outputs are not to be used), and then WGS_ERR_INDEX from
 * the next check if there was a bad index too; WGS_OK otherwise.  The words are
 * shared by every stream of the device. */
wgs_status wgs_check_error(cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WGS_H */
