/*
 * ctr.h -- C ABI of the GB300 (sm_103a) transposed-convolution library.
 *
 * The operation is dense (groups = 1) 1-D or 2-D ConvTranspose, in the scatter form
 *
 *     y[b, oc, i*s - p + t] += x[b, ic, i] * w[ic, oc, t]      (per spatial dimension)
 *     y[b, oc, o]           += bias[oc]
 *
 * with L_out = (L_in - 1)*s - 2p + k + op per spatial dimension and the weight in the
 * un-flipped torch layout [C_in][C_out][k...].  Sources:
 *   - "[ExecuTorch][WebGPU] Add optimized conv2d op" (PR #20849), Implementation and
 *     Constraints: the gather condition, the un-flipped [IC, OC, KH, KW] weight, the optional
 *     bias, output_padding < stride;
 *   - "[XNNPACK] Lower dense transposed convs as one polyphase conv + depth to space"
 *     (PR #25037), Summary: the polyphase lowering for k = m*s (one stride-1 conv with m
 *     taps, phase-major, then the phase interleave and the padding slice), which is the
 *     library's main path;
 *   - "[WebGPU] optimizations for audio models" (PR #33978), ConvTranspose commits: the
 *     X[M, C_in] x W[C_in, k*C_out] GEMM plus col2im path, the prepacked constant weight,
 *     f32 intermediates, the bias added once, the empty-input case.
 *
 * Call sequence:
 *     ctr_plan_create -> (ctr_plan_set_*) -> ctr_packed_weight_bytes / ctr_workspace_bytes
 *     -> ctr_prepack_weight (once per weight) -> ctr_plan_bind_workspace
 *     -> ctr_forward (any number of times) -> ctr_plan_check -> ctr_plan_destroy
 *
 * Conventions for every call:
 *   - Every call returns a ctr_status (or a size / string); nothing throws or aborts.
 *   - Device pointers are plain CUDA device addresses in the current device's context.
 *     Streams are cudaStream_t values passed as void* (NULL = the legacy default stream).
 *   - The caller owns every device buffer: x, w, w_packed, bias, y and the workspace.  The
 *     library never frees, keeps or aliases them beyond the call (and, for the workspace,
 *     the binding).  The plan owns its host metadata and a 4-byte device status word.
 *   - ctr_forward and ctr_prepack_weight are asynchronous on the given stream and never
 *     allocate, free or synchronise.
 *   - Tensors are contiguous, row-major, in the plan's I/O dtype:
 *         x    [N][C_in][L_in]            or [N][C_in][H][W]
 *         w    [C_in][C_out/G][k]         or [C_in][C_out/G][kH][kW]   (G groups, default 1)
 *         bias [C_out]                    (may be NULL)
 *         y    [N][C_out][L_out]          or [N][C_out][H_out][W_out]
 *     (x and y channels last with ctr_plan_set_layout(plan, CTR_LAYOUT_NHWC))
 *     and each must start on a 16-byte boundary (CTR_ERR_MISALIGNED otherwise).
 *   - A plan is not thread-safe: calls on one plan must not overlap on the host.  Two
 *     ctr_forward calls on one plan that run concurrently on the GPU (different streams)
 *     share its workspace and race; serialise them or use one plan per stream.
 */
#ifndef CTR_H
#define CTR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ctr_plan_s *ctr_plan_t;

typedef enum {
    CTR_OK = 0,
    CTR_ERR_INVALID_ARG = 1,     /* a size, geometry or handle is invalid */
    CTR_ERR_UNSUPPORTED = 2,     /* valid ConvTranspose this library does not implement */
    CTR_ERR_MISALIGNED = 3,      /* a pointer is not 16-byte aligned */
    CTR_ERR_NO_WORKSPACE = 4,    /* workspace needed but unbound or too small */
    CTR_ERR_CUDA = 5,            /* a CUDA runtime or launch error */
    CTR_ERR_DEVICE_TIMEOUT = 6,  /* a bounded device-side wait gave up (see ctr_plan_check) */
    CTR_ERR_NOT_PREPARED = 7     /* ctr_forward before ctr_prepack_weight on this plan */
} ctr_status;

typedef enum {
    CTR_F32 = 0,   /* fp32 I/O; each operand split as hi = tf32(v), lo = v - hi: hi*hi as a tf32
                      tensor-core product, hi*lo + lo*hi as bf16 products, fp32 accumulate
                      (rel_l2 within 1e-5 of fp32 arithmetic) */
    CTR_BF16 = 1,  /* bf16 I/O; bf16 tensor-core products, fp32 accumulate, one final rounding */
    CTR_F16 = 2    /* fp16 I/O; fp16 tensor-core products, fp32 accumulate and intermediates,
                      one final rounding ("[WebGPU] optimizations for audio models", review
                      commits: for float16 the packed weight and the K-padded input stay in the
                      I/O type while sums and column buffers are f32).  Not on the depthwise
                      kernel (grouped fp16 plans run the gather kernel) nor the iSTFT plan. */
} ctr_dtype;

typedef enum {
    CTR_ACT_NONE = 0,
    CTR_ACT_LEAKY_RELU = 1       /* y = y >= 0 ? y : slope * y, after the bias, before rounding */
} ctr_act;

typedef enum {
    CTR_PATH_AUTO = 0,
    CTR_PATH_POLYPHASE = 1,      /* polyphase implicit GEMM on tcgen05 (taps zero-padded to m*s) */
    CTR_PATH_COL2IM = 2,         /* tcgen05 GEMM into an fp32 column buffer, then col2im */
    CTR_PATH_GATHER = 3,         /* direct gather on CUDA cores (any groups) */
    CTR_PATH_DEPTHWISE = 4       /* one input channel per group (groups = C_in), CUDA cores */
} ctr_path;

/*
 * Create a plan.  Host only: validates the geometry, picks the path and the tiling.  The
 * only CUDA call reads the current device's SM count; without a GPU it assumes 152 SMs, so
 * plans can be created and inspected on a machine without one.
 *   out            receives the plan (set to NULL on failure)
 *   ndim           1 or 2 spatial dimensions
 *   N, C_in, C_out batch and channels: N >= 0, C_in >= 1, C_out >= 1
 *   in_spatial     ndim input sizes, each >= 0 (0 = empty input: y = bias or zeros)
 *   kernel         ndim kernel sizes >= 1
 *   stride         ndim strides >= 1
 *   padding        ndim paddings >= 0 (front and back; ctr_plan_set_pads separates them)
 *   output_padding ndim values with 0 <= op < stride (may be NULL = zeros)
 *   dtype          ctr_dtype (CTR_F32, CTR_BF16 or CTR_F16)
 * Every output size must be >= 1.  Groups, dilation and separate front/back pads are set
 * afterwards (ctr_plan_set_groups, ctr_plan_set_dilation, ctr_plan_set_pads; defaults: one
 * group, dilation 1, the back pad equal to `padding`).  Returns CTR_ERR_INVALID_ARG on any
 * violation.  A layer whose pads are only valid once separated or dilated (a front pad that,
 * taken on both sides, would leave no output) is created with zero padding and given its
 * pads by ctr_plan_set_pads, after ctr_plan_set_dilation.
 */
ctr_status ctr_plan_create(ctr_plan_t *out, int ndim, int64_t N, int64_t C_in, int64_t C_out,
                           const int64_t *in_spatial, const int64_t *kernel,
                           const int64_t *stride, const int64_t *padding,
                           const int64_t *output_padding, int dtype);

/*
 * Grouped transposed convolution (default 1 group): groups must divide C_in and C_out; the
 * weight is then [C_in][C_out/groups][k...] and output channel oc sums only the input
 * channels of its group ("[ExecuTorch][WebGPU] Add optimized conv2d op", Implementation:
 * the [IC, OC/groups, KH, KW] weight).  groups = C_in (C_out = M * C_in; M = 1 is the
 * depthwise upsampler of "[XNNPACK] Lower dense transposed convs as one polyphase conv +
 * depth to space", DecomposeDepthwiseConvTransposePass commit) runs on the depthwise path
 * (CTR_PATH_DEPTHWISE) for 1-D kernels with k/s in {2/2, 3/2, 4/2, 4/4, 8/4, 8/8, 16/8} and
 * square 2-D kernels 2x2/2, 3x3/2, 4x4/2, 4x4/4; other grouped plans run on the gather path.
 * The tensor-core paths need one group: forcing one on a grouped plan, or grouping a plan
 * forced onto one, returns CTR_ERR_UNSUPPORTED and leaves the plan unchanged.  Host only,
 * same ordering rule as ctr_plan_set_path; CTR_ERR_INVALID_ARG when groups does not divide
 * both channel counts, after ctr_prepack_weight, or on a chained plan.
 */
ctr_status ctr_plan_set_groups(ctr_plan_t plan, int64_t groups);

/*
 * Dilation (default 1 per dimension): taps are dil samples apart, so tap t of input i lands
 * at o = i*s - p_front + t*dil and L_out = (L_in - 1)*s + (k - 1)*dil + 1 + op - p_front -
 * p_back ("[ExecuTorch][WebGPU] Add optimized conv2d op", Implementation: the gather
 * condition (oh + pH - kh*dH) divisible by the stride; "[WebGPU] optimizations for audio
 * models": the ConvTranspose tests with pads, dilations or output_padding).
 *   dilation  ndim values >= 1
 * A dilated plan runs the col2im GEMM over its k real taps (C_in >= 16 and k*C_out >= 64)
 * or the gather kernel; a forced polyphase path packs the zero-inserted kernel of
 * (k - 1)*dil + 1 taps.  The depthwise path is undilated: forcing it on a dilated plan, or
 * dilating a plan forced onto it, returns CTR_ERR_UNSUPPORTED and leaves the plan unchanged.
 * Host only, with the same ordering rule as ctr_plan_set_path; CTR_ERR_INVALID_ARG for a
 * value < 1, an output size < 1, after ctr_prepack_weight, or on a chained plan (the plan is
 * then unchanged).
 */
ctr_status ctr_plan_set_dilation(ctr_plan_t plan, const int64_t *dilation);

/*
 * Separate front and back pads per dimension (the ONNX ConvTranspose `pads` attribute:
 * begin values, then end values), replacing the symmetric `padding` of ctr_plan_create.
 * The output is the unpadded result with p_front positions cut at the front and p_back at
 * the back (output_padding positions are added at the back first): L_out = (L_in - 1)*s +
 * (k - 1)*dil + 1 + op - p_front - p_back.  ("[XNNPACK] Lower dense transposed convs as one
 * polyphase conv + depth to space", Summary: the padding slice; "[WebGPU] optimizations for
 * audio models": the ConvTranspose tests with pads.)
 *   pads_begin, pads_end  ndim values >= 0 each
 * Every path takes any pads.  Host only, with the same ordering rule as ctr_plan_set_path;
 * CTR_ERR_INVALID_ARG for a negative pad, an output size < 1, after ctr_prepack_weight, or on
 * a chained plan (the plan is then unchanged).
 */
ctr_status ctr_plan_set_pads(ctr_plan_t plan, const int64_t *pads_begin, const int64_t *pads_end);

typedef enum {
    CTR_LAYOUT_NCHW = 0,   /* x [N][C_in][spatial...], y [N][C_out][out spatial...] (default) */
    CTR_LAYOUT_NHWC = 1    /* channels last: x [N][spatial...][C_in], y [N][out spatial...][C_out] */
} ctr_layout;

/*
 * Memory layout of x and y (default CTR_LAYOUT_NCHW); the weight keeps its torch layout.
 * Channels-last tensors are what image and audio pipelines often hold ("[XNNPACK] Lower dense
 * transposed convs as one polyphase conv + depth to space": the inpainting network's profile
 * spends a quarter of its time in NCHW <-> NHWC transposes around the deconvolutions).  The
 * tensor-core paths stage an NHWC input with a row copy (their staged operand is channels-last
 * already) and write an NHWC output from the same output stage that feeds a chained plan; the
 * gather kernel indexes NHWC directly.  The depthwise kernel is NCHW only (a grouped NHWC plan
 * runs the gather kernel) and so are streaming plans.  Host only, with the same ordering rule
 * as ctr_plan_set_path; CTR_ERR_INVALID_ARG for another value or after ctr_prepack_weight;
 * CTR_ERR_UNSUPPORTED on a streaming plan or one forced onto the depthwise path (the plan is
 * then unchanged).
 */
ctr_status ctr_plan_set_layout(ctr_plan_t plan, int layout);

typedef enum {
    CTR_AUTO_PAD_NOTSET = 0,      /* explicit pads (ctr_plan_create / ctr_plan_set_pads) */
    CTR_AUTO_PAD_SAME_UPPER = 1,  /* output = input * stride, odd total padding: extra at the end */
    CTR_AUTO_PAD_SAME_LOWER = 2,  /* output = input * stride, odd total padding: extra in front */
    CTR_AUTO_PAD_VALID = 3        /* no padding */
} ctr_auto_pad;

/*
 * The ONNX ConvTranspose `auto_pad` and `output_shape` attributes ("[WebGPU] optimizations
 * for audio models": the ConvTranspose tests run the ONNX operator's attributes), resolved
 * into the front and back pads of ctr_plan_set_pads.  Per dimension, with the plan's stride
 * s, kernel k, dilation d and output_padding op, the unpadded output has
 * full = (L_in - 1)*s + (k - 1)*d + 1 + op samples, and
 *   - output_shape given (any auto_pad): total = full - output_shape;
 *   - else SAME_UPPER / SAME_LOWER: total = full - L_in*s;
 *   - else VALID: no padding (total = 0);  NOTSET: the plan keeps its pads.
 * SAME_UPPER puts total/2 (rounded down) in front and the rest at the end; every other
 * setting puts the rest in front and total/2 at the end.  So the output is the unpadded
 * result's samples front .. full - back - 1, of length output_shape (or L_in*s).
 *   auto_pad      a ctr_auto_pad value
 *   output_shape  ndim output sizes, or NULL
 * A negative total (an output longer than the unpadded result) would need negative pads:
 * CTR_ERR_UNSUPPORTED.  Set dilation first (ctr_plan_set_dilation): the pads depend on it.
 * Host only, with the same ordering rule as ctr_plan_set_path; CTR_ERR_INVALID_ARG for an
 * unknown auto_pad, an output size < 1, after ctr_prepack_weight, or on a chained or
 * streaming plan (the plan is then unchanged).
 */
ctr_status ctr_plan_set_auto_pad(ctr_plan_t plan, int auto_pad, const int64_t *output_shape);

/*
 * Streaming 1-D ConvTranspose (default off): the input arrives as consecutive chunks of
 * L_in frames (a streaming audio decoder's upsampler), and each ctr_forward emits the
 * s*L_in output samples that its frames complete.  Concatenated, the outputs of a stream are
 * the unpadded ConvTranspose of the concatenated input, (L - 1)*s + k samples, without its
 * last k - s ("[XNNPACK] Lower dense transposed convs as one polyphase conv + depth to
 * space", Test plan and the Phonon fix: the overlap-add of a streaming decoder).  Those last
 * samples come out with the following chunk; zero frames flush them at the end of a stream.
 *
 * The polyphase form makes the state an input state. Output phase position q reads frames
 * q - (m - 1) .. q (m = ceil(k/s)). So the plan carries each batch item's last m - 1
 * input frames in its workspace and puts them in front of the next chunk. The
 * not-yet-complete output samples are not held back. Any chunk length works, including
 * chunks shorter than m - 1 frames.
 *
 * Requires: 1-D, padding = output_padding = 0, k >= s, one group, no dilation,
 * m - 1 <= 16, and the polyphase path.  The path is forced; a plan that cannot take it returns
 * CTR_ERR_UNSUPPORTED and stays unchanged.  Afterwards ctr_plan_output_shape reports
 * s*L_in. ctr_workspace_bytes includes the carried frames, B*(m - 1) staged rows.
 * ctr_plan_stream_reset must zero them before the first ctr_forward, after every
 * ctr_plan_bind_workspace, and to start a new stream (CTR_ERR_NOT_PREPARED otherwise).
 * Calls of one stream must run in stream order, one at a time: each reads the frames the
 * previous one carried.  ctr_forward_noalloc refuses streaming plans
 * (CTR_ERR_UNSUPPORTED).
 *
 * Host only, with the same ordering rule as ctr_plan_set_path.  CTR_ERR_INVALID_ARG for
 * enable not 0 or 1, after ctr_prepack_weight, or on a chained plan.  Once streaming, a
 * plan refuses ctr_plan_set_groups, _set_dilation, _set_pads and ctr_plan_chain
 * (CTR_ERR_INVALID_ARG), and ctr_plan_set_path with any path but the polyphase one
 * (CTR_ERR_UNSUPPORTED).  enable = 0 restores the plain plan, with the path it had before
 * streaming was turned on (the automatic path, or the one ctr_plan_set_path forced).
 */
ctr_status ctr_plan_set_streaming(ctr_plan_t plan, int enable);

/* Zero a streaming plan's carried input frames (asynchronous on `stream`): the next
 * ctr_forward starts a new stream.  CTR_ERR_INVALID_ARG when the plan is not streaming,
 * CTR_ERR_NO_WORKSPACE when its workspace is unbound or too small. */
ctr_status ctr_plan_stream_reset(ctr_plan_t plan, void *stream);

/* Fuse an activation into the output stage (default CTR_ACT_NONE).  Host only. */
ctr_status ctr_plan_set_activation(ctr_plan_t plan, int act, float negative_slope);

/*
 * Force a path (default CTR_PATH_AUTO) and optionally the split-K factor of the tensor-core
 * paths (0 = automatic, else 1..16).  Host only.  Must come before ctr_packed_weight_bytes,
 * ctr_workspace_bytes and ctr_prepack_weight, because the packed layout and the workspace
 * depend on the path; calling it after ctr_prepack_weight returns CTR_ERR_INVALID_ARG.
 * The tensor-core paths index tiles, staged input positions and packed weight rows in 32
 * bits: a plan that exceeds 2^31 of any of them runs the gather path when chosen
 * automatically, and forcing a tensor-core path on it returns CTR_ERR_UNSUPPORTED.
 * CTR_PATH_DEPTHWISE needs groups = C_in and a compiled geometry (ctr_plan_set_groups),
 * and the tensor-core paths one group; a path the plan cannot take returns
 * CTR_ERR_UNSUPPORTED and leaves the plan unchanged.
 */
ctr_status ctr_plan_set_path(ctr_plan_t plan, int path, int split_k);

typedef enum {
    CTR_PHASE_AUTO = 0,      /* the library chooses (below) */
    CTR_PHASE_UNPADDED = 1,  /* phases of the unpadded output, the padding sliced at the store */
    CTR_PHASE_OUTPUT = 2     /* phases of the output itself, the padding folded into the taps */
} ctr_phase_origin;

/*
 * Where the polyphase path's phase positions start.  "[XNNPACK] Lower dense transposed convs
 * as one polyphase conv + depth to space" (Summary) computes the phases of the unpadded
 * output and slices the padding off afterwards (CTR_PHASE_UNPADDED): output o = s*q + j - p,
 * so with p mod s != 0 every run of s phases starts at an odd offset and the output stage
 * writes elements one by one.  CTR_PHASE_OUTPUT re-indexes the phases by the output itself,
 * o = s*Q + J: with p = s*pq + pm, phase J takes the taps s*(m-1-v) + J + pm of the kernel
 * (zero where that is outside it), which needs one more tap per phase when pm > 0, and reads
 * input Q + pq - (m-1) + v.  Both compute the same sums of the same products; only zero
 * products are added or removed.  CTR_PHASE_AUTO takes the output phases when p mod s = 0
 * (no extra tap) and otherwise when the layer is bound by its output stores rather than by
 * its products (estimated from the tile model), for a plan whose output is not chained.
 * Streaming plans keep the unpadded phases.  A tuning and test override: host only, with the
 * same ordering rule as ctr_plan_set_path; CTR_ERR_INVALID_ARG for another value or after
 * ctr_prepack_weight.  Ignored by the paths other than polyphase.
 */
ctr_status ctr_plan_set_phase_origin(ctr_plan_t plan, int origin);

/*
 * Force the phase-row tile of the tensor-core paths: the number of packed weight rows one
 * output tile covers, i.e. the MMA N extent (0 = automatic, else 64, 128 or 256).  A tuning
 * and test override with no counterpart on the pages; every value gives the same result
 * bit for bit.  Host only, with the same ordering rule as ctr_plan_set_path; returns
 * CTR_ERR_INVALID_ARG for another value or after ctr_prepack_weight.
 */
ctr_status ctr_plan_set_tile(ctr_plan_t plan, int block_n);

/*
 * Chain two plans so that `plan`'s output feeds `next`'s input without a staging pass, as
 * in a decoder's stack of upsampling layers (two ConvTransposes with an activation between:
 * "[XNNPACK] Lower dense transposed convs as one polyphase conv + depth to space", Test
 * plan).  Afterwards:
 *   - ctr_forward(plan, x, w, bias, y = NULL, stream) writes its output, with bias and
 *     activation applied and rounded to the I/O type, straight into the channels-last
 *     staged-input layout inside next's workspace (fp32: as its tf32 and bf16-pair planes, exactly
 *     what next's staging would have made of the torch-layout output), and no y;
 *   - ctr_forward(next, x = NULL, ...) reads it from there instead of staging an x.
 * Results are bit-identical to the unchained calls.  Requirements (CTR_ERR_INVALID_ARG
 * otherwise): both plans on a tensor-core path (polyphase or col2im), the same dtype and
 * batch, next's C_in equal to plan's C_out and next's input spatial size equal to plan's
 * output size.  At each forward, next's workspace must be bound (CTR_ERR_NO_WORKSPACE)
 * and must not overlap plan's (CTR_ERR_INVALID_ARG); the first forward after binding
 * zeroes next's staged buffer once (its halos stay zero).  Run plan, then next, on the
 * same stream.  A chained plan packs its weight rows for this output (phase-major within
 * each tile), so ctr_plan_chain(plan, ...) must come before ctr_prepack_weight(plan)
 * (CTR_ERR_INVALID_ARG after it), and a plan packed for a chain whose other end was
 * destroyed refuses to run.  ctr_plan_chain(plan, NULL) unchains; destroying either plan
 * unchains both.  Host only; no counterpart of the call itself on the pages.
 */
ctr_status ctr_plan_chain(ctr_plan_t plan, ctr_plan_t next);

/*
 * Run a chained pair of layers -- plan and the plan it is chained to (ctr_plan_chain) -- as
 * one kernel that keeps the first layer's output in shared memory as the second layer's
 * operand, instead of writing it to the second plan's staged input and reading it back
 * (the two-layer stack of "[XNNPACK] Lower dense transposed convs as one polyphase conv +
 * depth to space", Test plan).  The result is bit-identical to ctr_forward(plan, x, ...)
 * followed by ctr_forward(next, NULL, ...).
 *   x            plan's input as for ctr_forward (NULL when a chained previous plan staged it)
 *   w_packed, bias        plan's packed weight and bias
 *   next_w_packed, next_bias   the next plan's
 *   y            the next plan's output
 * Needs (CTR_ERR_UNSUPPORTED otherwise, see ctr_plan_fusable): 1-D, bf16 or fp16, both on
 * the polyphase path without split-K; plan with stride >= 2 and exactly 64 output channels
 * in one tile of 128 phase rows; next with 64 input channels, one row tile of 64 or 128
 * rows, an NCHW output and no further chain.  Both plans prepacked (CTR_ERR_NOT_PREPARED)
 * and plan's workspace bound (CTR_ERR_NO_WORKSPACE); the next plan's workspace is not used.
 * Asynchronous on stream; device-side timeouts are reported by ctr_plan_check(plan, ...).
 * No counterpart of the call itself on the pages.
 */
ctr_status ctr_forward_fused(ctr_plan_t plan, const void *x, const void *w_packed,
                             const void *bias, const void *next_w_packed,
                             const void *next_bias, void *y, void *stream);

/* 1 when ctr_forward_fused can run plan and the plan it is chained to, else 0. */
int ctr_plan_fusable(ctr_plan_t plan);

/* The path the plan will run (a ctr_path other than AUTO), or -1 for a NULL plan. */
int ctr_plan_get_path(ctr_plan_t plan);

/* Write the ndim output sizes into out_spatial. */
ctr_status ctr_plan_output_shape(ctr_plan_t plan, int64_t *out_spatial);

/* Bytes of the packed weight buffer ctr_prepack_weight writes (0 for a NULL plan). */
size_t ctr_packed_weight_bytes(ctr_plan_t plan);

/* Bytes of device workspace ctr_forward needs (may be 0; 0 for a NULL plan). */
size_t ctr_workspace_bytes(ctr_plan_t plan);

/*
 * Bind a caller-owned device workspace of at least ctr_workspace_bytes(plan) bytes,
 * 256-byte aligned.  The binding lasts until the next bind or ctr_plan_destroy; the
 * workspace must stay allocated meanwhile.  Binding NULL with 0 bytes is allowed when the
 * plan needs no workspace.
 */
ctr_status ctr_plan_bind_workspace(ctr_plan_t plan, void *dev_ptr, size_t bytes);

/*
 * Pack a weight for this plan (once per weight; asynchronous on stream).
 *   w         device, [C_in][C_out/groups][k...] in the plan's dtype
 *   w_packed  device, ctr_packed_weight_bytes(plan) bytes, written in full
 * The packed weight is valid only for plans with the same geometry, dtype and path.  The
 * first call on a plan also allocates the plan's 4-byte device status word on the current
 * device (the only allocation the library makes).
 */
ctr_status ctr_prepack_weight(ctr_plan_t plan, const void *w, void *w_packed, void *stream);

/*
 * y = ConvTranspose(x, w) + bias, then the plan's activation, rounded once to the I/O dtype.
 *   x         device input, [N][C_in][spatial...]
 *   w_packed  device, written by ctr_prepack_weight for this plan's geometry
 *   bias      device [C_out] or NULL
 *   y         device output, [N][C_out][out spatial...], written in full
 *   stream    cudaStream_t as void*
 * Asynchronous; launch failures return CTR_ERR_CUDA.  Device-side errors (a bounded wait
 * that gave up) are reported by ctr_plan_check.  x and y must not overlap.  For a chained
 * plan (ctr_plan_chain) y must be NULL; for the plan it feeds, x may be NULL.
 */
ctr_status ctr_forward(ctr_plan_t plan, const void *x, const void *w_packed, const void *bias,
                       void *y, void *stream);

/*
 * ctr_forward for callers that cannot allocate device memory (a host framework whose
 * allocator owns all device memory, code running while a CUDA graph is captured, real-time
 * audio callbacks).  The source pages have no counterpart of this call.
 *   plan      a plan from ctr_plan_create; no ctr_prepack_weight, workspace binding or other
 *             device allocation is needed for it
 *   x, bias   device inputs as for ctr_forward (bias may be NULL)
 *   w         device weight in its torch layout [C_in][C_out][k...] (not packed: every call
 *             packs it into the library's scratch)
 *   y         device output as for ctr_forward
 *   stream    cudaStream_t as void*
 * Scratch (packed weight, staged input, split-K partials, a status word) lives in one
 * static 32 MiB device array that the CUDA driver reserves on each device that loads the
 * library and keeps until the process exits.  Plans needing more than that (the packed
 * weight plus ctr_workspace_bytes plus 256 bytes) get CTR_ERR_NO_WORKSPACE before anything
 * runs.  This call performs no cudaMalloc, cudaFree or other allocation.  Its first call on
 * a device looks up the array's device address (cudaGetSymbolAddress) with that device
 * current; make that first call before any stream capture.  Every call shares the one
 * array: calls whose GPU work overlaps (different streams, or several host threads) race on
 * it and must be serialised by the caller.  Bounded-wait timeouts are recorded in the
 * array's status word, which every call clears at its start (this call does not
 * synchronise); ctr_plan_check of any plan, on the same device, reads and clears it, so a
 * check right after a call reports that call's timeout.  Returns as ctr_forward otherwise.
 */
ctr_status ctr_forward_noalloc(ctr_plan_t plan, const void *x, const void *w, const void *bias,
                               void *y, void *stream);

/*
 * Synchronise stream, then read and clear the plan's device status word, and the status word
 * of ctr_forward_noalloc's scratch on the current device once an allocation-free call has
 * run there.  Returns CTR_OK, CTR_ERR_DEVICE_TIMEOUT when a kernel's bounded wait gave up
 * since the last check (its output is then incomplete), or CTR_ERR_CUDA.
 */
ctr_status ctr_plan_check(ctr_plan_t plan, void *stream);

/*
 * Limit, in nanoseconds, of every bounded device-side wait of the tensor-core kernels
 * (default 4e9).  A test hook: a tiny limit makes the waits give up on a healthy run, so
 * the timeout path can be exercised without a fault.  Host only.
 */
ctr_status ctr_plan_set_wait_limit_ns(ctr_plan_t plan, uint64_t limit_ns);

/*
 * Measurement hook: when both are non-NULL, every later ctr_forward records the
 * caller-owned CUDA events `before` and `after` (cudaEvent_t as void*) on its stream
 * immediately before and after the plan's main kernel (the tensor-core GEMM on the polyphase
 * and col2im paths, the gather kernel otherwise), so cudaEventElapsedTime gives that
 * kernel's own duration.  Pass NULL, NULL to stop.  Host only; the events must outlive
 * the calls that record them.  A ctr_forward captured into a CUDA graph records them as
 * external event nodes, so they time every replay.
 */
ctr_status ctr_plan_set_timing_events(ctr_plan_t plan, void *before, void *after);

/* Human-readable summary of the plan's path and tiling into buf (NUL-terminated). */
ctr_status ctr_plan_describe(ctr_plan_t plan, char *buf, size_t len);

/* Free the plan's host metadata and status word.  NULL is ignored.  Does not synchronise:
 * call it only after the plan's work on the GPU has finished. */
void ctr_plan_destroy(ctr_plan_t plan);

/* Static description of a status code. */
const char *ctr_status_string(ctr_status status);

/* Number of GPU kernels this library has launched in this process (a monotonic counter
 * for benchmarks and tests). */
uint64_t ctr_launch_count(void);

/* ------------------------------------------------------------------------------------
 * Inverse STFT through an inverse real FFT.
 *
 * The same result as ctr_forward on a 1-D plan with C_in = n_fft + 2, C_out = 1, kernel
 * n_fft, stride hop and the windowed inverse real-DFT basis as weight: channel f of the
 * input holds the real part of bin f (0 <= f <= n_fft/2), channel n_fft/2 + 1 + f its
 * imaginary part, and the weight rows are c_f win[t] cos(2 pi f t/N) / N and
 * -c_f win[t] sin(2 pi f t/N) / N (c_0 = c_{N/2} = 1, else 2).  "[WebGPU] optimizations for
 * audio models" computes the source-separation model's inverse STFT as that ConvTranspose1d;
 * here each frame is an inverse real FFT (O(n_fft log n_fft) instead of O(n_fft^2)), times
 * the window, and the frames are overlap-added at stride hop, sliced by the padding, plus
 * an optional scalar bias.
 *
 *   spec  device, [N][n_fft + 2][frames], fp32 (16-byte aligned)
 *   y     device, [N][1][L_out], fp32, L_out = (frames - 1)*hop - 2*padding + n_fft
 *         + output_padding (16-byte aligned)
 *   window  device, [n_fft] fp32 synthesis window (16-byte aligned)
 *   bias  device, [1] fp32 or NULL
 *
 * n_fft is a power of two in [4, 8192]; hop >= 1; 0 <= output_padding < hop; padding >= 0.
 * fp32 only: CTR_BF16 returns CTR_ERR_UNSUPPORTED.  The plan owns no device memory: the
 * caller binds a workspace of ctr_istft_workspace_bytes (twiddles, the scaled window, the
 * windowed frames, fp32 [N][frames][n_fft], and the spectra as frame-major complex rows,
 * [N][frames][n_fft/2 + 2] pairs) and sets the window once (a kernel on `stream`);
 * ctr_istft_forward then launches three kernels (the spectra to frame-major rows, the
 * per-frame FFT, then the overlap-add as a gather, summing frames in ascending order:
 * deterministic) and never allocates or synchronises.  Errors as for the ConvTranspose plan; CTR_ERR_NOT_PREPARED before
 * ctr_istft_set_window (rebinding the workspace clears it).
 * ------------------------------------------------------------------------------------ */
typedef struct ctr_istft_s *ctr_istft_t;

ctr_status ctr_istft_create(ctr_istft_t *out, int64_t N, int64_t n_fft, int64_t hop,
                            int64_t frames, int64_t padding, int64_t output_padding, int dtype);
ctr_status ctr_istft_output_length(ctr_istft_t plan, int64_t *L_out);
size_t ctr_istft_workspace_bytes(ctr_istft_t plan);
ctr_status ctr_istft_bind_workspace(ctr_istft_t plan, void *workspace, size_t bytes);
ctr_status ctr_istft_set_window(ctr_istft_t plan, const void *window, void *stream);
ctr_status ctr_istft_forward(ctr_istft_t plan, const void *spec, const void *bias, void *y,
                             void *stream);
ctr_status ctr_istft_describe(ctr_istft_t plan, char *buf, size_t len);
/* As ctr_plan_set_timing_events, around the kernels of ctr_istft_forward. */
ctr_status ctr_istft_set_timing_events(ctr_istft_t plan, void *before, void *after);
void ctr_istft_destroy(ctr_istft_t plan);

/* ------------------------------------------------------------------------------------
 * Attention of one new token over a paged key-value cache.
 *
 * The decode step of an autoregressive model that feeds the streaming upsamplers above with
 * frames: for each of B sequences, one query per head reads the keys and values of all
 * tokens so far, which lie in fixed-size pages that a table lists:
 *
 *     n    = lens[b] + (k_new ? 1 : 0)            tokens, slots 0 .. n - 1
 *     lo   = window > 0 ? max(0, n - window) : 0   first slot that is attended to
 *     p[j] = softmax over lo <= j < n of  scale * (q[b, h] . K[j, h / (H_q / H_kv)])
 *     out[b, h] = sum over j of p[j] * V[j, h / (H_q / H_kv)]          (0 when n = 0)
 *
 * Slot j of sequence b is row j % page_size of page tables[b][j / page_size].  With k_new and
 * v_new the call first puts them at slot lens[b] (in the same launch); the caller advances
 * lens afterwards.  lens[b] < 0 marks an idle row: nothing is written to the cache, out = 0.
 * With weights enabled the call also accumulates the attention weight of every slot,
 *
 *     weights_out[b, hk, j] = (j < lens[b] ? weights_in[b, hk, j] : 0)
 *                             + sum over the heads h of hk's group of p[j]      (0 <= j < n)
 *
 * which ctr_attn_evict uses to choose what a full cache gives up.
 *
 * Buffers (device, contiguous unless a stride is given; q, k_new, v_new, the pages, out and
 * their strides in bytes on 16-byte boundaries, the int32 and fp32 arrays on their elements'):
 *   q             [B][H_q][D] in the plan's dtype, q_stride elements from row b to b + 1
 *   k_new, v_new  [B][H_kv][D], kv_stride elements between rows; both or neither NULL
 *   k_pages, v_pages  [num_pages][H_kv][page_size][D] (CTR_CACHE_HEAD_MAJOR) or
 *                 [num_pages][page_size][H_kv][D] (CTR_CACHE_TOKEN_MAJOR), bound to the plan
 *   tables        [B][max_pages] int32 page numbers; entries past a sequence's last page are
 *                 not read
 *   lens          [B] int32
 *   weights_in, weights_out  [B][H_kv][max_pages * page_size] fp32; may be the same buffer;
 *                 weights_in NULL reads as zeros; slots >= n are left alone
 *   out           [B][H_q][D]
 * Rows of stale pages past a sequence's end may hold anything, NaN included.
 *
 * Sums, softmax statistics and weights are fp32; out is rounded once to the dtype.  The
 * probabilities of 16-bit caches keep 15 bits or more in the product with V (fp16: down to 2^-22 of
 * the largest; their last bit is at least 2^-37 of it).  The result does not depend on timing:
 * partial results join in a fixed order.  A NaN or infinite score makes its head's outputs and weights
 * NaN; a head whose scores are all -inf gives 0.
 * A page number outside [0, num_pages) hides its slots, and a length past the table's capacity
 * is cut to it (without room for the new row, which is then not put); ctr_attn_check reports
 * either as CTR_ERR_INVALID_ARG.  Two sequences may share pages that neither appends to.
 * ------------------------------------------------------------------------------------ */
typedef struct ctr_attn_s *ctr_attn_t;

typedef enum {
    CTR_CACHE_HEAD_MAJOR = 0,   /* pages [H_kv][page_size][D] (default) */
    CTR_CACHE_TOKEN_MAJOR = 1   /* pages [page_size][H_kv][D] */
} ctr_cache_layout;

/*
 * Create an attention plan (host only).  1 <= B <= 1024; 1 <= H_kv, H_q a multiple of it,
 * H_q / H_kv <= 128; D a multiple of 16 up to 256; page_size >= 1; max_pages >= 1;
 * B * H_kv <= 2^20, max_pages * page_size <= 2^28, and the product of all four (times H_q /
 * H_kv / 8, rounded up) <= 2^36.  dtype: CTR_F32, CTR_BF16 or CTR_F16.
 * CTR_ERR_INVALID_ARG for sizes < 1 or H_q no multiple of H_kv, CTR_ERR_UNSUPPORTED
 * beyond the limits.
 */
ctr_status ctr_attn_create(ctr_attn_t *out, int64_t B, int64_t H_q, int64_t H_kv, int64_t D,
                           int64_t page_size, int64_t max_pages, int dtype);
/* Page layout (default CTR_CACHE_HEAD_MAJOR).  Host only, as the next three calls. */
ctr_status ctr_attn_set_layout(ctr_attn_t plan, int layout);
/* Score scale (default 1 / sqrt(D)); must be finite. */
ctr_status ctr_attn_set_scale(ctr_attn_t plan, float scale);
/* Attend to the last `window` slots only (default 0 = all). */
ctr_status ctr_attn_set_window(ctr_attn_t plan, int64_t window);
/* Accumulate weights (default 0): the workspace then also holds one fp32 score per query head
 * and slot.  Unbinds the workspace. */
ctr_status ctr_attn_set_weights(ctr_attn_t plan, int enable);
/* Allow ctr_attn_forward_chunk (default 0): the workspace then also holds its partial results.
 * Unbinds the workspace. */
ctr_status ctr_attn_set_chunks(ctr_attn_t plan, int enable);
/* Limit, in nanoseconds, of the waits of a 16-bit chunk's kernel for its own copies and products (default
 * 1e10).  A test hook, as ctr_plan_set_wait_limit_ns: any other limit runs a kernel that polls, and is slower. */
ctr_status ctr_attn_set_wait_limit_ns(ctr_attn_t plan, uint64_t limit_ns);
size_t ctr_attn_workspace_bytes(ctr_attn_t plan);
/* Bind a caller-owned workspace (256-byte aligned), as ctr_plan_bind_workspace. */
ctr_status ctr_attn_bind_workspace(ctr_attn_t plan, void *dev_ptr, size_t bytes);
/* Clear the workspace's status word (asynchronous on stream): once after each
 * ctr_attn_bind_workspace, before the first ctr_attn_forward or ctr_attn_evict
 * (CTR_ERR_NOT_PREPARED otherwise).  What a call reports there stays until ctr_attn_check or the
 * next reset. */
ctr_status ctr_attn_reset(ctr_attn_t plan, void *stream);
/* Bind the caller-owned cache pages; they must stay allocated while bound.  At most 2^36 elements
 * each (CTR_ERR_UNSUPPORTED beyond). */
ctr_status ctr_attn_bind_cache(ctr_attn_t plan, void *k_pages, void *v_pages, int64_t num_pages);
/* One decode step.  Asynchronous on stream; never allocates or synchronises.  weights_out is
 * required when weights are enabled and must be NULL (as weights_in) otherwise. */
ctr_status ctr_attn_forward(ctr_attn_t plan, const void *q, int64_t q_stride, const void *k_new,
                            const void *v_new, int64_t kv_stride, const int32_t *tables,
                            const int32_t *lens, const float *weights_in, float *weights_out,
                            void *out, void *stream);
/*
 * Attention of a chunk of new tokens -- a prompt, a piece of one, drafted tokens -- whose K and V rows
 * are in the cache already (ctr_attn_put).  Sequence b has the rows starts[b] .. starts[b + 1] - 1 of q;
 * its token i, at slot lens[b] + i, attends to the slots up to its own:
 *
 *     end  = lens[b] + i + 1;   lo = window > 0 ? max(0, end - window) : 0
 *     p[j] = softmax over lo <= j < end of  scale * (q[t, h] . K[j, h / (H_q / H_kv)])
 *     out[t, h] = sum over j of p[j] * V[j, h / (H_q / H_kv)]
 *
 *   q       [T][H_q][D] in the plan's dtype, q_stride elements between rows (q, out and the stride
 *           in bytes on 16-byte boundaries)
 *   tables  [B][max_pages] int32; only the entries of slots that some row attends to are read
 *   lens    [B] int32: tokens before the chunk; lens[b] < 0 marks an idle sequence, whose rows give 0
 *   starts  [B + 1] int32, ascending, 0 <= starts[0], starts[B] <= T; rows of out outside
 *           [starts[0], starts[B]) are left alone
 *   out     [T][H_q][D]
 * Needs ctr_attn_set_chunks(plan, 1) (CTR_ERR_NOT_PREPARED), T * H_q / H_kv <= 2^30 and T <= 2^24.  A plan
 * with weights accumulates none here.
 *
 * Scores, softmax statistics and sums are fp32; the probabilities of 16-bit caches are rounded once to the
 * dtype for the product with V (8 bits in bf16, 11 in fp16, where ctr_attn_forward keeps 15; fp16: to multiples of
 * 2^-37 of the largest, and to one at least where all rows of a tile attend to the slot); out is rounded
 * once.  The result does not depend on timing.  What a row does not attend to never reaches it, infinities and
 * NaN in V and stale rows included; an infinite V that a row attends to makes that output infinite (a weight below
 * 2^-126 of the row's largest counts as 0 and gives NaN), a NaN or +inf score makes the head's outputs NaN, and
 * a row without slots or whose scores are all -inf gives 0.  Page numbers out of range hide their slots.
 * starts out of order or range make their sequence empty, and tokens past the table's capacity
 * attend to the slots below it; ctr_attn_check reports all three as CTR_ERR_INVALID_ARG.
 */
ctr_status ctr_attn_forward_chunk(ctr_attn_t plan, const void *q, int64_t q_stride, int64_t T,
                                  const int32_t *tables, const int32_t *lens, const int32_t *starts,
                                  void *out, void *stream);
/*
 * Evict from the cache by accumulated attention weight: of the lens[b] slots of every
 * (sequence, KV head) keep n = min(lens[b], budget) -- the first `sinks`, the last `recent`,
 * and of the others those with the largest weight (ties: the lowest slot; NaN counts as
 * lowest) -- and copy their K and V rows, in slot order, to slots 0 .. n - 1 of the pages in
 * dst_tables.  Each head keeps slots of its own.  The source pages are not changed, so pages
 * shared with other sequences stay valid; no destination page may be a source page or occur
 * twice.
 *   weights      [B][H_kv][max_pages * page_size] fp32
 *   dst_tables   [B][dst_pitch] int32, dst_pitch >= ceil(budget / page_size)
 *   slots        [B][H_kv][budget] int32: the kept slots, ascending, then -1
 *   lens_out     [B] int32: n (lens[b] itself for an idle row); may not be lens
 *   weights_out  [B][H_kv][weights_pitch] fp32, weights_pitch >= budget: the kept weights,
 *                entries from n on left alone; NULL or != weights
 * Requires budget >= 1 and sinks + recent <= budget (CTR_ERR_INVALID_ARG).  Page numbers out
 * of range are skipped and reported by ctr_attn_check, as above.  Needs the bound cache and,
 * for the status word, the workspace.
 */
ctr_status ctr_attn_evict(ctr_attn_t plan, const int32_t *tables, const int32_t *lens,
                          const float *weights, const int32_t *dst_tables, int64_t dst_pitch,
                          int64_t budget, int64_t sinks, int64_t recent, int32_t *slots,
                          int32_t *lens_out, float *weights_out, int64_t weights_pitch,
                          void *stream);
/* Synchronise stream, then read and clear the status word: CTR_OK, CTR_ERR_INVALID_ARG when a
 * call since the last check met a page number, slot, length or start out of range,
 * CTR_ERR_DEVICE_TIMEOUT when a kernel gave up waiting for its own copies or products (a defect;
 * its outputs are not valid), or CTR_ERR_CUDA. */
ctr_status ctr_attn_check(ctr_attn_t plan, void *stream);
ctr_status ctr_attn_describe(ctr_attn_t plan, char *buf, size_t len);
void ctr_attn_destroy(ctr_attn_t plan);

/* ------------------------------------------------------------------------------------
 * Rotary positions, alone or on the way into the cache.
 *
 * Pair i of the first R columns of a head's D -- columns (i, i + R/2) with CTR_ROPE_HALF (default), (2i,
 * 2i + 1) with CTR_ROPE_INTERLEAVED -- is turned by the token's position; the other columns are copied:
 *
 *     x' = m (x cos a - y sin a),   y' = m (x sin a + y cos a),   a = position * f_i
 *     f_i = base^(-2i/R)                                    (base 10000, m = magnitude = 1 by default)
 *     CTR_ROPE_SCALE_LINEAR   f_i / factor
 *     CTR_ROPE_SCALE_PARTS    (1 - g) f_i / factor + g f_i,  g = (original f_i / 2 pi - low) / (high - low),
 *                             at least 0 and at most 1: pairs that turn fewer than `low` times over
 *                             `original` positions are scaled, those of more than `high` turns are not
 *
 * or frequencies of the caller's own (a ramp over the pair's number instead of its turns, for one).  Angles are
 * reduced to at most half a turn, to 2^-32 turn plus the position times the 53-bit rounding of f_i, and then rounded to
 * fp32, which is 2^-26 turn at most; the products are fp32, rounded once to the dtype.  Positions are int32; a
 * negative one turns backwards, so that a call with the negated positions is the transpose
 * (the gradient of a call with respect to its input, from the gradient of its output).
 * ------------------------------------------------------------------------------------ */
typedef struct ctr_rope_s *ctr_rope_t;

typedef enum {
    CTR_ROPE_HALF = 0,
    CTR_ROPE_INTERLEAVED = 1
} ctr_rope_layout;

typedef enum {
    CTR_ROPE_SCALE_NONE = 0,
    CTR_ROPE_SCALE_LINEAR = 1,
    CTR_ROPE_SCALE_PARTS = 2
} ctr_rope_scaling;

/* 2 <= R <= D, R even (CTR_ERR_INVALID_ARG); D <= 512 (CTR_ERR_UNSUPPORTED).  Host only, as the calls
 * down to ctr_rope_frequencies. */
ctr_status ctr_rope_create(ctr_rope_t *out, int64_t D, int64_t R, int dtype);
ctr_status ctr_rope_set_layout(ctr_rope_t plan, int layout);
/* base >= 1, finite.  Drops the caller's own frequencies, as ctr_rope_set_scaling does. */
ctr_status ctr_rope_set_base(ctr_rope_t plan, double base);
/* factor > 0 (LINEAR, PARTS); original > 0 and 0 <= low < high (PARTS); all finite. */
ctr_status ctr_rope_set_scaling(ctr_rope_t plan, int scaling, double factor, double original, double low,
                                double high);
ctr_status ctr_rope_set_magnitude(ctr_rope_t plan, float magnitude);
/* The R/2 frequencies, in radians a position: set to the caller's (finite), or read. */
ctr_status ctr_rope_set_frequencies(ctr_rope_t plan, const double *frequencies, int64_t n);
ctr_status ctr_rope_frequencies(ctr_rope_t plan, double *frequencies, int64_t n);
/*
 * q [T][H_q][D] and k [T][H_k][D] (either may have no heads) to q_out and k_out, each in place or
 * apart from every other buffer, any row strides (in elements, at least a row), aligned to their elements.
 * positions [T] int32.  T <= 2^24, H_q, H_k <= 2^14.  Asynchronous on stream.
 */
ctr_status ctr_rope_forward(ctr_rope_t plan, const void *q, int64_t q_stride, int64_t H_q, const void *k,
                            int64_t k_stride, int64_t H_k, const int32_t *positions, int64_t T, void *q_out,
                            int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream);
/*
 * Put T tokens' K and V rows into the cache of an attention plan, at slots[t] (row slots[t] %
 * page_size of page slots[t] / page_size; < 0: nowhere), K turned by `rope` if one is given; with q (which
 * needs rope) also turn q [T][H_q][D] to q_out (which may be q).  rope has the plan's D and dtype.
 *   k, v   [T][H_kv][D], kv_stride elements between rows; slots [T] int64, no slot twice; positions [T]
 *          int32, needed with rope
 * q, k, v, q_out and the strides in bytes on 16-byte boundaries.  Slots past the cache are skipped and
 * reported by ctr_attn_check.  Needs the bound cache and the workspace, as ctr_attn_forward.
 */
ctr_status ctr_attn_put(ctr_attn_t plan, ctr_rope_t rope, const void *q, int64_t q_stride, const void *k,
                        const void *v, int64_t kv_stride, const int32_t *positions, const int64_t *slots,
                        int64_t T, void *q_out, int64_t q_out_stride, void *stream);
ctr_status ctr_rope_describe(ctr_rope_t plan, char *buf, size_t len);
void ctr_rope_destroy(ctr_rope_t plan);

/* ------------------------------------------------------------------------------------
 * Pages of the cache for new tokens, and their slots and positions, on the GPU.
 *
 * The free list is two buffers of the caller's: free_pages [num_pages] int32, of which the first *count
 * are free.  Sequence b has lens[b] tokens in the first ceil(lens[b] / page_size) pages of its row of
 * tables [B][max_pages]; lens[b] < 0 marks an idle one.
 *
 * ctr_pages_reserve makes room for counts[b] more tokens in each sequence: pages from the end of the
 * list into the table where the last page does not hold them, and for every new token, sequence by
 * sequence, its slot page * page_size + row and its position.  Requests are served in order: one is
 * granted, as a whole, if the rows of all requests up to it are at most `rows`, and if it needs no page
 * or the pages that all requests up to it need are on the list.
 *     granted [B]      counts[b], or 0
 *     starts [B + 1]   first row of each sequence: sums of the granted counts
 *     slots [rows] int64, positions [rows] int32; rows from starts[B] on get -1 and 0
 *     lens_out [B]     lens[b] + granted[b]
 * ctr_pages_release gives back the pages behind the first keep[b] tokens of each sequence (keep[b] <
 * 0: all of them, and the sequence becomes idle), the last sequence's last page first, so that they come
 * out again in the order they had, and sets their table entries to -1.
 *     lens_out [B]     min(lens[b], keep[b]), -1 for keep[b] < 0; idle sequences stay as they are
 * Neither changes lens.  A page is given back by one sequence only: pages that sequences share are the
 * caller's to keep apart.
 *
 * A count < 0, a length out of range and a request past the table's capacity are refused (granted 0);
 * they, page numbers out of range (their slots are -1) and a list that would hold more than num_pages pages
 * are reported by ctr_pages_check as CTR_ERR_INVALID_ARG.
 * ------------------------------------------------------------------------------------ */
typedef struct ctr_pages_s *ctr_pages_t;

/* 1 <= B <= 1024, page_size >= 1, max_pages >= 1, max_pages * page_size <= 2^28.  Host only. */
ctr_status ctr_pages_create(ctr_pages_t *out, int64_t B, int64_t page_size, int64_t max_pages);
/* Bind the caller's free list, 1 <= num_pages < 2^31. */
ctr_status ctr_pages_bind_list(ctr_pages_t plan, int32_t *free_pages, int32_t *count, int64_t num_pages);
size_t ctr_pages_workspace_bytes(ctr_pages_t plan);
/* Bind a caller-owned workspace (256-byte aligned). */
ctr_status ctr_pages_bind_workspace(ctr_pages_t plan, void *dev_ptr, size_t bytes);
/* Clear the workspace (asynchronous on stream): once after each ctr_pages_bind_workspace.  refill = 1
 * also puts all pages on the list, page 0 last. */
ctr_status ctr_pages_reset(ctr_pages_t plan, int refill, void *stream);
/* Asynchronous on stream; rows <= 2^30.  No output may be an input or another output. */
ctr_status ctr_pages_reserve(ctr_pages_t plan, int32_t *tables, const int32_t *lens, const int32_t *counts,
                             int64_t rows, int32_t *granted, int32_t *starts, int64_t *slots,
                             int32_t *positions, int32_t *lens_out, void *stream);
ctr_status ctr_pages_release(ctr_pages_t plan, int32_t *tables, const int32_t *lens, const int32_t *keep,
                             int32_t *lens_out, void *stream);
/* As ctr_attn_check. */
ctr_status ctr_pages_check(ctr_pages_t plan, void *stream);
ctr_status ctr_pages_describe(ctr_pages_t plan, char *buf, size_t len);
void ctr_pages_destroy(ctr_pages_t plan);

/* ------------------------------------------------------------------------------------
 * Sampling the next token (a code of the codec) from logits and given random numbers.
 *
 * Per row, with l the logits as fp32 (NaN reads as -inf), m their maximum, the order (l
 * descending, index ascending) and w_i = exp((l_i - m) / T), 1 where l_i = m, kept is the
 * shortest of these prefixes of the order, but at least its first token:
 *     T <= 0        the first token (greedy)
 *     top_k > 0     the first top_k tokens
 *     top_p < 1     the tokens with (mass of the tokens before them) < top_p * (mass of the
 *                   top_k tokens)
 *     min_p > 0     the tokens with w_i >= min_p
 * (a NaN top_p or min_p filters nothing, a NaN T is greedy)
 * and the token is the kept one with the largest w_i / max(noise_i, FLT_MIN) (ties: the lowest
 * index).  With independent Exp(1) numbers as noise this is a draw from the kept tokens in
 * proportion to w (the exponential race).  A token with l_i = -inf is never drawn; a row
 * of nothing else gives -1.  Masses are added in a fixed order in fp32 within a thread and as
 * 64-bit integers (units of 2^-35) beyond it, so the kept set does not depend on timing.
 *
 *   logits   [rows][vocab] in the plan's dtype, row stride in elements (any, >= vocab)
 *   noise    [rows][vocab] fp32, row stride in elements
 *   temperature, top_p, min_p  [rows] fp32 or NULL (1, 1 and 0);  top_k  [rows] int32 or NULL
 *   tokens   [rows] int64
 * Every buffer is aligned to its elements (CTR_ERR_MISALIGNED otherwise), so a slice of a
 * larger tensor will do.  1 <= vocab <= 2^20, 0 <= rows <= 2^20.  No workspace;
 * ctr_sampler_forward is asynchronous on stream and never allocates or synchronises.
 * ------------------------------------------------------------------------------------ */
typedef struct ctr_sampler_s *ctr_sampler_t;

ctr_status ctr_sampler_create(ctr_sampler_t *out, int64_t rows, int64_t vocab, int dtype);
ctr_status ctr_sampler_forward(ctr_sampler_t plan, const void *logits, int64_t logits_stride,
                               const float *noise, int64_t noise_stride,
                               const float *temperature, const int32_t *top_k,
                               const float *top_p, const float *min_p, int64_t *tokens,
                               void *stream);
ctr_status ctr_sampler_describe(ctr_sampler_t plan, char *buf, size_t len);
void ctr_sampler_destroy(ctr_sampler_t plan);

#ifdef __cplusplus
}
#endif

#endif /* CTR_H */
