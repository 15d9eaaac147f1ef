/*
 * hdq.h -- C ABI of libhdq, the MI355X (gfx950) library for the hot path of
 * 6Bit-Diffusion's dynamic mixed-precision quantization (DMPQ) of video
 * diffusion transformer linear layers.
 *
 * What the method computes, per linear layer and per denoising step
 * (sources: "6Bit-Diffusion" summary of arXiv:2603.18742 on vetunion.cn,
 * sections one, three and four; the gist.science explainer "6Bit-Diffusion:
 * Inference-Time Mixed-Precision Quantization for Video Diffusion Models",
 * sections 2 and 4):
 *   1. choose the activation precision from the relative difference of the
 *      module's input and output at the previous step (large: INT8, small:
 *      NVFP4), INT8 when there is no previous step, and full precision when
 *      the input's outlier ratio max|x| / mean|x| is too large;
 *   2. rotate the activations with a block Hadamard transform and quantize
 *      them in the same pass;
 *   3. run the quantized linear layer against weights prepared the same way.
 * hdq_select_precision is step 1, hdq_quantize is step 2 (and the offline
 * weight preparation), hdq_linear is steps 2 + 3.
 *
 * Conventions, for every entry point:
 *  - All tensors are row-major with the reduction dimension K contiguous:
 *    activations X [M, K], weights W [N, K], outputs Y [M, N] = X W^T.
 *  - bf16 tensors are raw 16-bit patterns (the upper half of an IEEE float).
 *  - Every pointer marked "device" is device memory the caller owns and keeps
 *    alive until the enqueued work has finished.  The library allocates no
 *    memory, never synchronises, and enqueues all work on `stream` (a
 *    hipStream_t passed as void*; NULL is the default stream).
 *  - Arguments are validated before anything is enqueued; on error nothing
 *    is enqueued and a negative HDQ_ERR_* code is returned.  A kernel fault
 *    surfaces at the caller's next synchronisation.
 *  - Calls are thread-safe; calls that share output or workspace buffers on
 *    overlapping streams race, as any stream work would.
 *  - Rotation: every aligned block of `had_block` consecutive elements along
 *    K is multiplied by H_b / sqrt(b), H_b the Sylvester Hadamard matrix, in
 *    float32 by the fast Walsh-Hadamard butterfly (strides 1, 2, 4, ... in
 *    that order) and one multiply by fl32(1/sqrt(b)).  Weights and
 *    activations are rotated alike, so (XQ)(WQ)^T = XW^T.  had_block 1
 *    rotates nothing.
 *  - Quantized codes use round-half-to-even.  Non-finite inputs are outside
 *    the quantizers' contract; hdq_select_precision routes them to BF16.
 */
#ifndef HDQ_H
#define HDQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---- */
#define HDQ_OK 0
#define HDQ_ERR_INVALID (-1)     /* NULL pointer, bad enum or bad struct field  */
#define HDQ_ERR_SHAPE (-2)       /* size <= 0, K not a multiple of had_block or */
                                 /* of the format's block, had_block not a      */
                                 /* power of two in [1, 128], shapes disagree   */
#define HDQ_ERR_UNSUPPORTED (-3) /* precision/format/output-dtype combination   */
#define HDQ_ERR_HIP (-4)         /* a kernel launch failed                      */
#define HDQ_ERR_WORKSPACE (-5)   /* ws NULL or ws_bytes below what is required  */

/* ---- quantized formats (hdq_qtensor.fmt) ---- */
/* INT8, one fp32 scale per row: s = max|y| / 127, q = rne(y * (127 / max|y|)).
 * codes: int8 [rows, cols]; row_scale: fp32 [rows].  (The "INT8" activation
 * format of the summary's section one, per token.) */
#define HDQ_FMT_INT8_ROW 0
/* INT4, one fp32 scale per row (per output channel of a weight): same as
 * INT8 with 7 for 127.  codes: uint8 [rows, cols/2], element 2j in the low
 * nibble of byte j, two's complement; row_scale: fp32 [rows].  (The 4-bit
 * weights of the summary's W4A6 configuration, section four.) */
#define HDQ_FMT_INT4_ROW 1
/* NVFP4: FP4 E2M1 codes with one E4M3 scale per aligned 16 elements and one
 * fp32 tensor scale s_t = amax / 2688 (amax of the rotated tensor):
 * value = e2m1(code) * e4m3(blk_scale) * s_t.  codes: uint8 [rows, cols/2]
 * (even element in the low nibble); blk_scale: uint8 [rows, cols/16];
 * tensor_scale: fp32 [1].  (The "NVFP4" format of section one; the pages do
 * not define it, the encodings are those of the OCP MX v1.0 formats.) */
#define HDQ_FMT_NVFP4 2
/* NVFP4 bytes restricted so that every aligned pair of 16-blocks shares one
 * power-of-two scale (s_t = amax / 1536, scale = smallest power of two that
 * fits the pair): a valid NVFP4 tensor that is also MXFP4-shaped, so the
 * GEMM runs on gfx950's block-scaled FP4 matrix instructions. */
#define HDQ_FMT_NVFP4_MX 3
/* NVFP4 bytes restricted so that every aligned 16-block's scale is a power
 * of two (its own: s_t = amax / 1536, scale = smallest power of two that
 * fits the block): valid NVFP4, computed exactly on the block-scaled FP4
 * matrix instructions in two passes per 32 elements (one per 16-block half),
 * so at up to half the MX recipe's rate. */
#define HDQ_FMT_NVFP4_P2 4

/* ---- precisions (decisions) ---- */
#define HDQ_PREC_NVFP4 0
#define HDQ_PREC_INT8 1
#define HDQ_PREC_BF16 2 /* full precision: unrotated bf16 x bf16 GEMM */

/* ---- output dtypes of hdq_linear ---- */
#define HDQ_DTYPE_F32 0
#define HDQ_DTYPE_BF16 1
#define HDQ_DTYPE_I32 2 /* INT8 path only: the raw int32 accumulators */

/* ---- workspace queries (hdq_workspace_bytes op) ---- */
#define HDQ_OP_SELECT 0
#define HDQ_OP_QUANTIZE 1
#define HDQ_OP_LINEAR 2
#define HDQ_OP_SELECT_Q8 3
#define HDQ_OP_DQ_QUANTIZE 4
#define HDQ_OP_DQ_LINEAR 5

/* A quantized tensor.  The caller allocates every buffer (device memory)
 * and fills the pointers; hdq_quantize fills fmt, had_block, rows, cols. */
typedef struct hdq_qtensor {
    int32_t fmt;          /* HDQ_FMT_*                                       */
    int32_t had_block;    /* Hadamard block the rows were rotated with       */
    int64_t rows;         /* logical shape of the unquantized tensor         */
    int64_t cols;
    void *codes;          /* device, layout per format (see above)           */
    float *row_scale;     /* device, INT8/INT4 only (may be NULL otherwise)  */
    uint8_t *blk_scale;   /* device, NVFP4 formats only                      */
    float *tensor_scale;  /* device fp32[1], NVFP4 formats only              */
    void *dec;            /* NULL, or (NVFP4 formats) device bf16 [rows,
                           * cols]: each element's E2M1 value times its E4M3
                           * block scale, without the tensor scale -- exact in
                           * bf16.  hdq_quantize fills it when given; with
                           * plain NVFP4 on both operands of a GEMM the exact
                           * NVFP4 product reads its operands from it.
                           * Ignored for the INT formats.                    */
} hdq_qtensor;

/* A linear layer's weights in every form a precision may need.  Members a
 * call does not use may be NULL / zeroed. */
typedef struct hdq_weights {
    int64_t N;            /* output features                                 */
    int64_t K;            /* input features                                  */
    const void *w_bf16;   /* device bf16 [N, K], unrotated: HDQ_PREC_BF16    */
    hdq_qtensor w_int4;   /* HDQ_FMT_INT4_ROW [N, K]: HDQ_PREC_INT8          */
    hdq_qtensor w_fp4;    /* HDQ_FMT_NVFP4 or _MX [N, K]: HDQ_PREC_NVFP4     */
} hdq_weights;

/*
 * hdq_select_precision -- step 1 (summary section one: the previous step's
 * input/output difference picks INT8 or NVFP4; section three: the outlier
 * ratio max/mean forces full precision, and INT8 is used when there is no
 * previous-step difference; explainer sections 2 and 4).
 *
 *   prev_in, prev_out : device bf16 [prev_numel] each, the module's input and
 *                       output at the previous step; both NULL = no history.
 *   cur_in            : device bf16 [rows, cols], the current input.
 *   had_block         : 0, or the Hadamard block (power of two in [2, 128],
 *                       dividing cols) used to also report the rotated amax.
 *   delta_thresh, ratio_thresh : thresholds (e.g. 0.1 and 50).
 *   decision_dev      : device int32[1] <- HDQ_PREC_*.
 *   stats_dev         : device fp32[5] <- {delta, ratio, max|x|, mean|x|,
 *                       rotated amax (0 when had_block == 0)}.
 *   ws, ws_bytes      : device scratch, >= hdq_workspace_bytes(HDQ_OP_SELECT,
 *                       rows, cols, prev_numel, 0) bytes.
 * delta = sum|prev_out - prev_in| / sum|prev_in| (0 if both sums are 0, +inf
 * if only the denominator is, NaN without history); ratio = max|x| / mean|x|
 * over cur_in (0 for all zeros, NaN if cur_in holds a NaN or an infinity).
 * Decision: ratio not <= ratio_thresh -> BF16; else no history -> INT8; else
 * delta not < delta_thresh -> INT8; else NVFP4.  Sums are float32 partials
 * reduced in double in a fixed order, so results are deterministic.
 */
int hdq_select_precision(const void *prev_in, const void *prev_out, int64_t prev_numel,
                         const void *cur_in, int64_t rows, int64_t cols, int32_t had_block,
                         float delta_thresh, float ratio_thresh, int32_t *decision_dev,
                         float *stats_dev, void *ws, size_t ws_bytes, void *stream);

/*
 * hdq_delta_sums and hdq_select_precision_sums -- step 1 in two parts (same
 * sources as hdq_select_precision).  The difference statistic depends only
 * on the previous step's tensors, so it can be computed off the critical
 * path (e.g. on a second stream while earlier layers' GEMMs run), leaving
 * only the current input for the selection proper.
 *
 * hdq_delta_sums:
 *   prev_in, prev_out : device bf16 [numel] each (the module's previous-step
 *                       input and output).
 *   sums_dev          : device double[2] <- {sum|prev_out - prev_in|,
 *                       sum|prev_in|}.
 *   ws, ws_bytes      : device scratch, >= hdq_workspace_bytes(HDQ_OP_SELECT,
 *                       1, numel, numel, 0) bytes.
 * hdq_select_precision_sums:
 *   delta_sums_dev    : device double[2 * delta_parts]: delta_parts pairs
 *                       {sum|prev_out - prev_in|, sum|prev_in|} over parts
 *                       of the tensors, summed in order (delta_parts = 1:
 *                       the double[2] of hdq_delta_sums; more: the chunk
 *                       partials of hdq_linear_dispatch_delta).  Complete
 *                       before this call's kernels run (same stream or an
 *                       event), or NULL for no history.
 *   delta_parts       : >= 1 when delta_sums_dev is given (HDQ_ERR_SHAPE
 *                       otherwise); ignored for NULL.
 *   the other arguments are those of hdq_select_precision.
 * The two calls together write what hdq_select_precision writes for the
 * same tensors, bit for bit when numel == rows * cols (the statistics'
 * per-workgroup partials and their fixed-order reduction are the same); for
 * other sizes, equal up to the rounding of the double sums.
 */
int hdq_delta_sums(const void *prev_in, const void *prev_out, int64_t numel, double *sums_dev,
                   void *ws, size_t ws_bytes, void *stream);
int hdq_select_precision_sums(const double *delta_sums_dev, int64_t delta_parts, const void *cur_in,
                              int64_t rows, int64_t cols, int32_t had_block, float delta_thresh,
                              float ratio_thresh, int32_t *decision_dev, float *stats_dev,
                              void *ws, size_t ws_bytes, void *stream);

/*
 * hdq_select_quantize_int8 -- hdq_select_precision_sums fused with the INT8
 * per-token quantization of the same input (steps 1 and 2 for the INT8
 * path): x is read once, the INT8 codes are written whatever the decision
 * turns out to be (a caller then runs the INT8 GEMM gated on the decision).
 *   delta_sums_dev, delta_parts, cur_in, rows, cols, thresholds,
 *   decision_dev, stats_dev:
 *                 as for hdq_select_precision_sums; had_block must be > 0.
 *   xq8         : caller-allocated INT8_ROW buffers (codes int8 [rows, cols],
 *                 row_scale fp32 [rows]); fmt, had_block, rows, cols are
 *                 written.
 *   ws, ws_bytes: >= hdq_workspace_bytes(HDQ_OP_SELECT_Q8, rows, cols, 0, 0)
 *                 bytes (one partial per row).
 * The codes equal hdq_quantize's INT8_ROW codes bit for bit; the decision,
 * delta, max|x| and rotated amax equal hdq_select_precision_sums'; mean |x|
 * and the ratio agree up to the order of the double sum of |x| (per row
 * here, per chunk range there).  Rows over 16384 columns run the two passes
 * one after the other.
 */
int hdq_select_quantize_int8(const double *delta_sums_dev, int64_t delta_parts, const void *cur_in,
                             int64_t rows, int64_t cols, int32_t had_block, float delta_thresh,
                             float ratio_thresh, int32_t *decision_dev, float *stats_dev,
                             hdq_qtensor *xq8, void *ws, size_t ws_bytes, void *stream);

/*
 * hdq_select_quantize_int8_noalloc -- hdq_select_quantize_int8 with no
 * workspace argument, for callers that cannot allocate device memory: code
 * recorded under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.  Same arguments and results as hdq_select_quantize_int8
 * (bit for bit), without ws / ws_bytes.
 *   Scratch: the per-row statistics partials live in a static device array
 *   of HDQ_NOALLOC_SCRATCH_BYTES bytes, one per GPU the library runs on,
 *   held until the process ends.  Its address is looked up once per device
 *   (hipGetSymbolAddress, with that device current) on the first call there;
 *   the call allocates nothing.
 *   Limit: hdq_workspace_bytes(HDQ_OP_SELECT_Q8, rows, cols, 0, 0) (48 bytes
 *   per row, at least 48 KiB) must not exceed HDQ_NOALLOC_SCRATCH_BYTES, i.e.
 *   rows <= 43690; larger inputs return HDQ_ERR_TOO_LARGE before anything is
 *   enqueued.
 *   Sharing: every call on one GPU uses that GPU's one array and overwrites
 *   it (nothing in it needs to start at zero).  Calls that overlap on one GPU
 *   (other streams or threads, with the earlier call's kernels not yet done)
 *   race on it: order them on one stream or with events.
 */
#define HDQ_NOALLOC_SCRATCH_BYTES (2u << 20)
#define HDQ_ERR_TOO_LARGE (-6)   /* input beyond an allocation-free call's fixed scratch */
int hdq_select_quantize_int8_noalloc(const double *delta_sums_dev, int64_t delta_parts,
                                     const void *cur_in, int64_t rows, int64_t cols,
                                     int32_t had_block, float delta_thresh, float ratio_thresh,
                                     int32_t *decision_dev, float *stats_dev, hdq_qtensor *xq8,
                                     void *stream);

/*
 * hdq_quantize -- step 2: block-Hadamard rotation fused with quantization
 * (summary sections one and four).  Also prepares weights offline.
 *
 *   x           : device bf16 [rows, cols].
 *   had_block   : power of two in [2, 128] dividing cols.
 *   fmt         : HDQ_FMT_*; cols must be a multiple of 2 (INT4), 16 (NVFP4)
 *                 or 32 (NVFP4_MX).
 *   tensor_amax : NVFP4 formats: device fp32[1] holding the amax of the
 *                 rotated tensor (e.g. stats_dev + 4 from
 *                 hdq_select_precision), or NULL to compute it in a pre-pass
 *                 (then ws must hold hdq_workspace_bytes(HDQ_OP_QUANTIZE,
 *                 rows, cols, 0, fmt) bytes).  Ignored for INT formats.
 *   decision_dev: NULL, or device int32[1]: the kernels then do their work
 *                 only when it holds the precision that consumes `fmt`
 *                 (HDQ_PREC_INT8 for INT8_ROW, HDQ_PREC_NVFP4 for the NVFP4
 *                 formats; not allowed with INT4_ROW), so one enqueued call
 *                 serves a device-side decision without a host round trip.
 *   out         : host struct with caller-allocated device buffers sized for
 *                 the format; fmt, had_block, rows, cols are written.  For
 *                 the NVFP4 formats a non-NULL out->dec also receives the
 *                 codes' exact bf16 values (gated like the codes).
 * Rows whose max |rotated value| is below 2^-100 get zero codes and a zero
 * scale; an NVFP4 tensor whose amax is below 2^-100 gets s_t = 0 and zero
 * codes and scale bytes.
 */
int hdq_quantize(const void *x, int64_t rows, int64_t cols, int32_t had_block, int32_t fmt,
                 const float *tensor_amax, const int32_t *decision_dev, hdq_qtensor *out,
                 void *ws, size_t ws_bytes, void *stream);

/*
 * hdq_linear -- steps 2 + 3: Y[M, N] = quantized X[M, K] times the weights'
 * matching form (summary section one: NVFP4 or INT8 activations against
 * 4-bit weights; section three: full-precision fallback).
 *
 *   precision   : HDQ_PREC_* to run, or -1 to read it from decision_dev on
 *                 the device (every candidate kernel is enqueued and the ones
 *                 not selected exit at once; no host synchronisation).
 *   decision_dev: NULL, or device int32[1].  With precision -1 it selects
 *                 the path; with a fixed precision P the work is done only
 *                 when it holds P (so a caller can enqueue each path's
 *                 pieces, e.g. one quantization shared by several GEMMs).
 *   x           : device bf16 [M, K] (the unrotated activations).
 *   xq          : NULL, or already-quantized activations to use instead of
 *                 quantizing x (fixed precision INT8 or NVFP4 only; its format
 *                 must match the weights': INT8_ROW for INT8, the w_fp4
 *                 format for NVFP4).
 *   x_amax      : NVFP4 only: device fp32[1] rotated amax of x, or NULL to
 *                 compute it in a pre-pass.
 *   w           : weights; w->K == K and had_block of both quantized forms
 *                 must be equal; the needed forms must be present.
 *   y, y_dtype  : device output [M, N]: HDQ_DTYPE_F32 or _BF16 (all
 *                 precisions), _I32 (INT8 only: raw accumulators).
 *   ws, ws_bytes: device scratch >= hdq_workspace_bytes(HDQ_OP_LINEAR, M, K,
 *                 N, w_fp4.fmt) (0 when xq is given for INT8).
 * INT8:  acc = sum_k qx*qw (exact int32); y = fl32(fl32(acc * sx[m]) * sw[n]).
 * NVFP4: y = s_tx * s_tw * sum over 16-blocks of E_x E_w sum_k e2m1 e2m1,
 *        float32 accumulation.  Plain NVFP4 (HDQ_FMT_NVFP4) runs on bf16
 *        MFMAs: when xq->dec (and w->w_fp4.dec) are given the GEMM reads
 *        those exact bf16 values, otherwise it decodes the codes as it
 *        stages them -- the same products in the same order, so the same
 *        output bits.  Both copies given is the fastest form.
 * BF16:  y = x w^T with the unrotated bf16 operands, float32 accumulation.
 */
int hdq_linear(int32_t precision, const int32_t *decision_dev, const void *x,
               const hdq_qtensor *xq, const float *x_amax, int64_t M, int64_t K,
               const hdq_weights *w, void *y, int32_t y_dtype, void *ws, size_t ws_bytes,
               void *stream);

/*
 * hdq_linear_dispatch -- step 3 for a device-side decision in one launch:
 * the GEMM of the precision decision_dev names (summary section one: INT8
 * or NVFP4 activations against 4-bit weights; section three: full
 * precision), with every path's operands already prepared -- xq8 (INT8_ROW
 * from hdq_quantize or hdq_select_quantize_int8), xq4 (the weights' FP4
 * format), x (bf16, unrotated) and all three weight forms.  Results equal
 * hdq_linear(P, decision_dev, x or xq, ...) of the decided P, bit for bit.
 * One kernel reads the decision and runs that GEMM (K a multiple of 256 and
 * 2 * K * max(M, N) < 2^31); other shapes enqueue the three gated GEMMs.
 * Plain NVFP4 with xq4->dec (and w->w_fp4.dec) given reads the decoded
 * operands, as hdq_linear does.
 * y_dtype F32 or BF16.  No workspace.
 */
int hdq_linear_dispatch(const int32_t *decision_dev, const void *x, const hdq_qtensor *xq8,
                        const hdq_qtensor *xq4, int64_t M, int64_t K, const hdq_weights *w,
                        void *y, int32_t y_dtype, void *stream);

/*
 * hdq_linear_dispatch_delta -- hdq_linear_dispatch that also computes part
 * of step 1's difference statistic (summary section one: the previous
 * step's input/output difference) for later layer calls, inside the same
 * launch.  The difference depends only on earlier tensors, so it can run
 * beside this call's compute-bound GEMM: on workgroups appended after the
 * GEMM's persistent ones, which hold the CUs the GEMM leaves free and,
 * once its workgroups retire, every CU, claiming chunks from a queue until
 * none is left.  The launch ends when both are done, so the difference
 * never shares the GPU with the memory-bound passes of the next call.
 *
 * The tensors of one module are split into chunks of HDQ_DELTA_CHUNK
 * elements; chunk c's {sum|prev_out - prev_in|, sum|prev_in|} (float over
 * each 8 elements, double beyond, in a fixed order: the same whichever
 * workgroup runs it) go to partials[2c], partials[2c + 1].  A module's
 * chunks may be spread over several calls; once all of them have run,
 * partials is the delta_sums_dev input of hdq_select_quantize_int8 or
 * hdq_select_precision_sums with delta_parts = ceil(numel / HDQ_DELTA_CHUNK).
 *
 *   decision_dev ... stream: as for hdq_linear_dispatch, except that only
 *              the one-launch kernel's shapes are taken (K a multiple of 256,
 *              2 * K * max(M, N) < 2^31; HDQ_ERR_SHAPE otherwise).
 *   slices   : nslices (0..HDQ_DELTA_MAX_SLICES) chunk ranges:
 *     prev_in, prev_out : device bf16 [numel] each, 16-byte aligned.
 *     numel             : elements per tensor, a positive multiple of 8.
 *     chunk_begin/end   : the chunks [chunk_begin, chunk_end) to run here,
 *                         within [0, ceil(numel / HDQ_DELTA_CHUNK)].
 *     partials          : device double [2 * ceil(numel / HDQ_DELTA_CHUNK)].
 *   queue_dev: device uint32[2], zero before the first call; every call
 *              with work leaves it zero again.  Calls that may overlap
 *              (other streams) need their own queue.
 * With nslices = 0 (or empty ranges) this is hdq_linear_dispatch's GEMM
 * alone.  The GEMM output equals hdq_linear_dispatch's bit for bit.
 */
#define HDQ_DELTA_CHUNK 65536
#define HDQ_DELTA_MAX_SLICES 4
typedef struct hdq_delta_slice {
  const void *prev_in;
  const void *prev_out;
  int64_t numel;
  int64_t chunk_begin;
  int64_t chunk_end;
  double *partials;
} hdq_delta_slice;

int hdq_linear_dispatch_delta(const int32_t *decision_dev, const void *x, const hdq_qtensor *xq8,
                              const hdq_qtensor *xq4, int64_t M, int64_t K, const hdq_weights *w,
                              void *y, int32_t y_dtype, const hdq_delta_slice *slices,
                              int32_t nslices, uint32_t *queue_dev, void *stream);

/*
 * hdq_tdc_decide -- the temporal delta cache's skip rule (summary on
 * vetunion.cn, section two; gist.science explainer, section three), for n
 * modules at once, once per diffusion step.  A module whose output changed
 * little between its last two computed steps reuses its cached output at
 * the next step; an accumulator adds the predicted change of every skipped
 * step and forces a computation once it would pass its budget.
 *   sums_dev : device double [n][2]; for a module computed at this step
 *              with an earlier output, {sum|new - earlier|, sum|earlier|}
 *              (hdq_delta_sums(earlier, new, ...) writes exactly this);
 *              ignored otherwise.  With parts_offsets_dev: pairs of partial
 *              sums, module i's being pairs [off[i], off[i + 1]), summed in a
 *              fixed order (e.g. the chunk partials hdq_linear_dispatch_delta
 *              writes for the two outputs while later modules' GEMMs run).
 *   parts_offsets_dev: NULL, or device int64 [n + 1], nondecreasing.
 *   state_dev: device int32 [n]: 0 skipped at this step, 1 computed with no
 *              earlier output, 2 computed with one (sums valid).
 *   c_dev    : device float [n], in/out: relative change between the last
 *              two computed outputs (NaN: none yet); rewritten when state
 *              is 1 (NaN) or 2 (diff / base in double, then float; base 0
 *              gives 0 if diff is 0, else +inf).
 *   acc_dev  : device float [n], in/out: reset to 0 when state != 0.
 *   skip_dev : device int32 [n] <- 1 when the next step reuses the cache:
 *              c < tau_skip and fl32(acc + c) <= tau_acc (NaN is false);
 *              acc then becomes fl32(acc + c).
 * Errors: HDQ_ERR_INVALID for a null pointer, HDQ_ERR_SHAPE for n <= 0 or
 * n >= 2^31.  The state arrays are the caller's; one call per step.
 */
int hdq_tdc_decide(const double *sums_dev, const int64_t *parts_offsets_dev, const int32_t *state_dev,
                   float *c_dev, float *acc_dev, int32_t *skip_dev, int64_t n, float tau_skip,
                   float tau_acc, void *stream);

/* ---- DeltaQuant cube-delta quantization (a second workload) ---------------
 * DeltaQuant (paper-radar CVPR 2026 listing, abstract): video activations are
 * grouped in local 3D spatiotemporal cubes; each cube's mean token (the core)
 * is kept in FP8 and only each token's difference from it is quantized to 4
 * bits.  Here: the tokens of a frames x height x width grid are the rows of
 * x, frame outermost ((f * height + h) * width + w); cubes are cube_f x
 * cube_h x cube_w blocks, ragged at the far edges, numbered the same way over
 * the cube grid.  The core is the float32 sum of its tokens in that order
 * divided by their count; it is stored as E4M3 with one fp32 scale per cube,
 * max|core| / 448 (0 below 2^-100), each code the nearest E4M3 of |c| / s
 * (ties to even) with the sign in bit 7 and a zero magnitude stored as +0.  A
 * token's difference fl32(x - fl32(E * s)) is quantized to NVFP4 (fmt) with
 * no rotation (had_block 1) and the tensor scale of the largest |difference|.
 */
typedef struct hdq_dq_grid {
  int64_t frames, height, width;
  int32_t cube_f, cube_h, cube_w;
} hdq_dq_grid;

/* Cubes of the grid, -1 for a bad grid (a size <= 0, over 2^31 - 1 tokens, or
 * more than 256 tokens per cube). */
int64_t hdq_dq_cubes(const hdq_dq_grid *g);

/*
 * hdq_dq_quantize -- the activation side.
 *   x          : device bf16 [tokens, K], K a multiple of 32, at most 32768.
 *   fmt        : HDQ_FMT_NVFP4, _NVFP4_MX or _NVFP4_P2 for the differences.
 *   core_codes : device uint8 [cubes, K] (signed E4M3); core_scale: fp32 [cubes].
 *   core_bf16  : NULL, or device bf16 [cubes, K]: the signed E4M3 code values
 *                (exact), the bf16 core GEMM's operand (plain NVFP4, or K not
 *                a multiple of 128).
 *   delta      : fmt, had_block 1, rows = tokens, cols = K, with codes,
 *                blk_scale and tensor_scale set (written).
 *   ws, ws_bytes: device scratch >= hdq_workspace_bytes(HDQ_OP_DQ_QUANTIZE, ...)
 *                (256 bytes).
 * Non-finite values (not covered by the method's description): when any
 * difference is not finite -- which a NaN or infinite element of x, or a
 * cube sum or a difference beyond the float32 range, always causes -- the
 * tensor scale *delta->tensor_scale is written as NaN, a flag on the device;
 * the codes and scales are then unspecified (a linear layer on them yields
 * NaN outputs).  Finite inputs never raise it.
 */
int hdq_dq_quantize(const void *x, int64_t K, const hdq_dq_grid *g, int32_t fmt, uint8_t *core_codes,
                    float *core_scale, void *core_bf16, hdq_qtensor *delta, void *ws, size_t ws_bytes,
                    void *stream);

/* NVFP4 weights (any of the three formats, [N, K]) to device bf16 [N, K]
 * holding E2M1 x block scale per element (exact), the tensor scale left out:
 * the core GEMM's weight operand, made once per layer. */
int hdq_dq_decode_weights(const hdq_qtensor *w_fp4, void *w_dec, void *stream);

/* Scratch bytes hdq_dq_linear needs for this grid, reduction size K, N
 * outputs and difference format fmt: the core GEMM's fp32 [cubes, N], plus an
 * fp32 [tokens, N] only when the difference GEMM cannot add the core term in
 * its own epilogue (plain NVFP4, K not a multiple of 256, N not a multiple of
 * 4 or operands past 32-bit offsets).  0 on bad arguments. */
size_t hdq_dq_linear_workspace_bytes(const hdq_dq_grid *g, int64_t K, int64_t N, int32_t fmt);

/*
 * hdq_dq_linear -- y = (differences) x W^T + (the token's cube core) x W^T.
 *   delta       : from hdq_dq_quantize; w_fp4: the layer's NVFP4 weights in
 *                 the same format with had_block 1 (hdq_quantize with
 *                 had_block 1 rotates nothing), N a multiple of 4.
 *   core_codes, core_scale: from hdq_dq_quantize.
 *   core_bf16, w_dec: the bf16 core values (hdq_dq_quantize) and decoded
 *                 weights (hdq_dq_decode_weights); needed only when the
 *                 weights' block scales are not powers of two or K is not a
 *                 multiple of 128 (plain NVFP4), may be NULL otherwise.
 *   y, y_dtype  : device [tokens, N], HDQ_DTYPE_F32 or _BF16.
 *   ws, ws_bytes: >= hdq_dq_linear_workspace_bytes(g, K, N, delta->fmt)
 *                 (hdq_workspace_bytes(HDQ_OP_DQ_LINEAR, tokens, cubes, N, 0)
 *                 is an upper bound for every route).
 * The core GEMM yc = sum_k core * w (exact products, float32 accumulation)
 * runs on the FP8 x FP4 scaled matrix instructions straight from the core's
 * E4M3 codes and the weights' E2M1 codes with their power-of-two block
 * scales (MX and per-16 power-of-two formats, K % 128 == 0), else on the
 * bf16 ones from core_bf16 and w_dec; the difference GEMM is the NVFP4 GEMM
 * of the format, which adds the core term in its epilogue (MX and per-16
 * formats, K % 256 == 0) or writes fp32 into ws for a combine pass; either
 * way y = fl(yd + fl32(fl32(yc * s_core) * s_w)).  Errors: HDQ_ERR_INVALID
 * for a NULL pointer the route needs.
 */
int hdq_dq_linear(const hdq_dq_grid *g, const uint8_t *core_codes, const void *core_bf16, const float *core_scale,
                  const hdq_qtensor *delta, const hdq_qtensor *w_fp4, const void *w_dec, void *y, int32_t y_dtype,
                  void *ws, size_t ws_bytes, void *stream);

/* ---- FP8 block-128 linear layers -------------------------------------------
 * y = x W^T with both operands in FP8 (OCP E4M3) and one fp32 scale for each
 * block of 128: of a row for activations (HDQ_FP8_ROWS), of 128 x 128 elements
 * for weights (HDQ_FP8_BLOCKS, the layout of FP8 checkpoints with block
 * scales).  Neither the summary nor the explainer has this format; it stands
 * between the INT8 x INT4 layer and the bf16 fallback.
 *
 * A tensor [rows, cols], kb = ceil(cols / 128) blocks per row:
 *   codes : device uint8 [rows, 128 * kb], 16-byte aligned; E4M3, columns
 *           past cols hold zeros.
 *   scale : device fp32, ROWS: [kb, rows] (a block column's scales are
 *           contiguous over the rows); BLOCKS: [ceil(rows / 128), kb].
 * With y the (rotated) values and a = max|y| over a block:
 *   s = fl32(a / 448), code = E4M3 nearest to fl32(y * fl32(448 / a)), ties
 *   to even, so value = code * s.  A block with a < 2^-100 gets s = 0 and
 *   zero codes; a block holding a NaN or an infinity gets s = NaN and zero
 *   codes, so that the outputs that read it are NaN.
 * No output may overlap an input or the scratch. */
#define HDQ_FP8_ROWS 0
#define HDQ_FP8_BLOCKS 1
#define HDQ_FP8_MAX_COLS (1 << 22)
#define HDQ_FP8_MAX_ROWS 0x7ffffc00
typedef struct hdq_fp8_tensor {
  int32_t layout;    /* HDQ_FP8_*                                     */
  int32_t had_block; /* Hadamard block the rows were rotated with     */
  int64_t rows;      /* logical shape of the unquantized tensor       */
  int64_t cols;
  uint8_t *codes;    /* device, see above                             */
  float *scale;      /* device, see above                             */
} hdq_fp8_tensor;

/*
 * hdq_fp8_quantize -- rotation fused with FP8 quantization.
 *   x        : device bf16 [rows, cols], 16-byte aligned; cols a multiple of
 *              8 and of had_block, at most HDQ_FP8_MAX_COLS; rows at most
 *              HDQ_FP8_MAX_ROWS.
 *   had_block: power of two in [1, 128]; 1 rotates nothing.  Sums are taken in
 *              float32 and scaled last: one past its range makes the block NaN.
 *   out      : host struct with caller-allocated codes and scale; layout,
 *              had_block, rows, cols are written.
 */
int hdq_fp8_quantize(const void *x, int64_t rows, int64_t cols, int32_t had_block, int32_t layout,
                     hdq_fp8_tensor *out, void *stream);

/* Scratch bytes hdq_fp8_linear needs when xq is NULL (the quantized
 * activations; 0 when the layer quantizes them in its own kernel); with xq
 * given it needs none.  0 on bad arguments. */
size_t hdq_fp8_linear_workspace_bytes(int64_t M, int64_t K, int64_t N, int32_t y_dtype);

/*
 * hdq_fp8_linear -- Y[M, N] = X[M, K] W[N, K]^T.
 *   x       : device bf16 [M, K] (unrotated), quantized as hdq_fp8_quantize
 *             does with the weights' had_block; ignored when xq is given.
 *   xq      : NULL, or the activations as HDQ_FP8_ROWS [M, K] with the
 *             weights' had_block.
 *   w       : HDQ_FP8_BLOCKS [N, K].  K as hdq_fp8_quantize's cols; M and N
 *             any size up to HDQ_FP8_MAX_ROWS.
 *   y       : device [M, N], HDQ_DTYPE_BF16 or HDQ_DTYPE_F32, 16-byte aligned
 *             (as x is).
 *   ws      : device scratch, 256-byte aligned, ws_bytes >=
 *             hdq_fp8_linear_workspace_bytes(M, K, N, y_dtype) unless xq is
 *             given.  Nothing in it needs a value before the call; calls that
 *             may overlap need their own.
 * y = sum over 128-blocks b of sx[b, m] sw[n / 128, b] sum_{k in b} cx cw, each
 * scale pair and block sum combined in float32 (scale pairs whose product is
 * outside its range are outside the layer's).  With a bf16 output the block
 * sums run on the FP8 matrix instructions, whose products are aligned to the
 * largest one of an instruction (at least 14 fraction bits: about 1.3e-5 of
 * the result in the 2-norm, where rounding to bf16 costs 1.7e-3); with an fp32
 * output on the bf16 ones (codes are exact in bf16), with float32 sums (up to
 * 1e-7 of the result): the one to take, and round, where a bf16 result from
 * float32 sums is wanted.
 */
int hdq_fp8_linear(const void *x, const hdq_fp8_tensor *xq, int64_t M, int64_t K, const hdq_fp8_tensor *w,
                   void *y, int32_t y_dtype, void *ws, size_t ws_bytes, void *stream);

/* ---- group norm, channels last -----------------------------------------------
 * x [n, length, channels], a group being channels / groups adjacent channels
 * of one sample (the norm of video decoders' residual and attention blocks,
 * whose projections are the linear layers above):
 *   t = (x - mean) / sqrt(var + eps) * weight + bias,
 * mean and (biased) variance over the group's length x channels / groups
 * elements; y = t (HDQ_ACT_NONE) or t / (1 + e^-t) (HDQ_ACT_SILU).  A thread
 * sums at most 16 rows of a channel at a time in float32, about their first
 * one; these means and squared deviations are joined in float64.  Finite x of
 * any size are normalized, where weight / sqrt(var + eps) is in float32's normal
 * range and, without an eps to hide them, deviations are at least 2^-100; a NaN
 * or an infinity makes its group's outputs NaN.  The SiLU takes the hardware's
 * exponential and reciprocal: off by at most (2 |t| / (1 + e^t) + 6) 2^-24 of
 * itself, and 0 where it is below 2^-119.  Apart from y = x, no output may
 * overlap an input or the scratch. */
#define HDQ_ACT_NONE 0
#define HDQ_ACT_SILU 1
#define HDQ_GROUP_NORM_MAX_CHANNELS 8192

/* Scratch bytes of hdq_group_norm (fp8 0; 0 for sizes that run in one launch)
 * or hdq_group_norm_fp8 (fp8 1); 0 on bad arguments. */
size_t hdq_group_norm_workspace_bytes(int64_t n, int64_t length, int64_t channels, int32_t groups, int32_t fp8);

/*
 * hdq_group_norm
 *   x, y        : device [n, length, channels], 16-byte aligned, each
 *                 HDQ_DTYPE_BF16 or HDQ_DTYPE_F32; y may be x (same type).
 *   groups      : divides channels (at most HDQ_GROUP_NORM_MAX_CHANNELS);
 *                 n * length at most HDQ_FP8_MAX_ROWS.
 *   weight, bias: device fp32 [channels], or NULL for 1 and 0.
 *   eps         : 0 to 1e30.
 *   ws, ws_bytes: device scratch, 256-byte aligned, >=
 *                 hdq_group_norm_workspace_bytes(n, length, channels, groups,
 *                 0) (NULL where that is 0).  Nothing in it needs a value
 *                 before the call; calls that may overlap need their own.
 */
int hdq_group_norm(const void *x, int32_t x_dtype, int64_t n, int64_t length, int64_t channels, int32_t groups,
                   const float *weight, const float *bias, float eps, int32_t act, void *y, int32_t y_dtype,
                   void *ws, size_t ws_bytes, void *stream);

/*
 * hdq_group_norm_fp8 -- the same norm with its float32 result rotated and
 * quantized in registers, as hdq_fp8_quantize does with a bf16 tensor: the
 * activations of an hdq_fp8_linear without a round trip through memory.
 *   channels    : also a multiple of 8 and of had_block.
 *   out         : codes and scale for HDQ_FP8_ROWS [n * length, channels];
 *                 layout, had_block, rows, cols are written.
 *   ws, ws_bytes: as hdq_group_norm's, with the size for fp8 1.
 *   the other arguments are hdq_group_norm's.
 */
int hdq_group_norm_fp8(const void *x, int32_t x_dtype, int64_t n, int64_t length, int64_t channels, int32_t groups,
                       const float *weight, const float *bias, float eps, int32_t act, int32_t had_block,
                       hdq_fp8_tensor *out, void *ws, size_t ws_bytes, void *stream);

/* ---- linear layers of few tokens with 4-bit weights in groups ----------------
 * y[m, n] = sum over groups g of s[n, g] sum_{k in g} (u[n, k] - z[n, g]) x[m, k]:
 * activations stay bf16, weights are codes u of 0 to 15 with one bf16 scale s
 * and, optionally, a zero point z (0 to 255; 8 without) for each group of 32,
 * 64 or 128 columns of a row.  For one to a few dozen tokens (conditioning
 * vectors, single-token serving), where reading the weights is what takes the
 * time; any number of tokens is taken.
 *
 * A tensor [N, K] is kept packed in tiles of 16 rows x 128 columns, both
 * rounded up (hdq_w4_pack and hdq_w4_quantize write it, padding included):
 *   codes : device, hdq_w4_bytes(..., HDQ_W4_CODES) bytes, 16-byte aligned;
 *   scale : device bf16, hdq_w4_bytes(..., HDQ_W4_SCALE) bytes, 16-byte aligned;
 *   zero  : NULL, or device, hdq_w4_bytes(..., HDQ_W4_ZERO) bytes, 16-byte aligned.
 * N at most HDQ_W4_MAX_ROWS, K a multiple of 32 and of the group, at most
 * HDQ_FP8_MAX_COLS. */
#define HDQ_W4_CODES 0
#define HDQ_W4_SCALE 1
#define HDQ_W4_ZERO 2
#define HDQ_W4_MAX_ROWS (1 << 27)
#define HDQ_W4_MAX_TOKENS (1 << 20)
typedef struct hdq_w4_tensor {
  int64_t N;
  int64_t K;
  int32_t group;
  uint8_t *codes;
  uint16_t *scale;
  uint8_t *zero;
} hdq_w4_tensor;

/* Bytes of one of a packed tensor's buffers; 0 on bad arguments. */
size_t hdq_w4_bytes(int64_t N, int64_t K, int32_t group, int32_t buffer);

/*
 * hdq_w4_pack -- weights whose codes lie in rows, two a byte, into tiles.
 *   codes : device uint8 [N, K / 2], the even column in the low nibble.
 *   scale : device bf16 [N, K / group] (scales of other types are rounded to it first).
 *   zero  : device uint8 [N, K / group]; given exactly when out->zero is.
 *   out   : N, K, group and the buffers set by the caller.
 */
int hdq_w4_pack(const uint8_t *codes, const void *scale, const uint8_t *zero, const hdq_w4_tensor *out, void *stream);

/*
 * hdq_w4_quantize -- bf16 weights [N, K] (16-byte aligned), rounded to nearest.
 * Without out->zero s = bf16(max|w| / 7), u = clamp(rne(w / s) + 8, 0, 15); with it
 * s = bf16((max - min) / 15), z = rne(-min / s), u = clamp(rne(w / s) + z, 0, 15),
 * 0 counted among the values.  A group whose scale would be below 2^-100 gets
 * s = 0; one with a NaN or an infinity s = NaN.
 */
int hdq_w4_quantize(const void *w, const hdq_w4_tensor *out, void *stream);

/*
 * hdq_w4_linear
 *   x : device bf16 [M, K], 16-byte aligned; M 0 (nothing is done) to
 *       HDQ_W4_MAX_TOKENS.
 *   y : device [M, N], HDQ_DTYPE_BF16 or HDQ_DTYPE_F32, aligned to an element.
 * A group's sum is taken in float32 on the matrix instructions, as
 * sum (16 + u) x - (16 + z) sum x with exact products, and scaled and added in
 * float32; the error is that of a float32 sum over terms (32 + u + z) |s x| in
 * place of |u - z| |s x|.  A token with a NaN or an infinity, or with such a sum past float32's
 * range, gets NaN or infinities; the others' outputs are not touched by it.
 *   ws, ws_bytes : device scratch, 256-byte aligned, >=
 *       hdq_w4_linear_workspace_bytes(M, N, K) (NULL where that is 0, as for one
 *       token of up to 32640 columns).  Nothing in it needs a value before the call; calls that
 *       may overlap need their own.
 */
int hdq_w4_linear(const void *x, int64_t M, const hdq_w4_tensor *w, void *y, int32_t y_dtype, void *ws,
                  size_t ws_bytes, void *stream);

/* Scratch bytes hdq_w4_linear needs; 0 on bad arguments. */
size_t hdq_w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* ---- heads: norms, rotary positions, a quantized key-value cache ---------------
 * What lies between a QKV projection and the attention.  A tensor of heads is
 * a view [batch, length, heads, dim] of bf16 or fp32 elements, dim (1 to
 * HDQ_HEAD_MAX_DIM) contiguous and the other strides free, in elements: the
 * slice of a projection's output that holds the queries, say.  Bases and
 * strides of whole 16 bytes, and dim a multiple of 8, are the fast ones.
 * batch * length is 0 (nothing is done) to HDQ_FP8_MAX_ROWS, heads of a call
 * together at most HDQ_HEAD_MAX_HEADS.  An output may be its own input (same
 * type and strides); otherwise nothing written may overlap anything read or
 * written.  An output's heads lie apart: of its dimensions longer than 1, each
 * stride is at least what the smaller ones span.  Views that break this by
 * their own strides or begin at one address are refused. */
#define HDQ_HEAD_MAX_DIM 512
#define HDQ_HEAD_MAX_HEADS (1 << 20)
typedef struct hdq_heads {
  void *data;           /* device                                          */
  int32_t dtype;        /* HDQ_DTYPE_BF16 or HDQ_DTYPE_F32                 */
  int32_t heads;
  int64_t batch_stride; /* in elements, >= 0                               */
  int64_t token_stride;
  int64_t head_stride;
} hdq_heads;

/* Norm over each head's dim elements, in float32, then weight and bias:
 *   LAYER: (x - mean) / sqrt(var + eps) w + b;  RMS: x / sqrt(mean(x^2) + eps) w + b.
 * weight, bias: device fp32 [dim], or NULL for 1 and 0.  eps 0 to 1e30; a
 * head of zeros stays zero at eps 0.  Finite heads of any size are normed
 * (sums that leave float32's range are taken again, scaled); a NaN or an
 * infinity makes its head NaN.  A layer norm's mean is within a few float32
 * roundings of the head's deviations, however far from 0 its elements are: a head
 * further off than its deviation is taken again, about one of its elements, and
 * a constant one gives the biases. */
#define HDQ_HEAD_NORM_NONE 0
#define HDQ_HEAD_NORM_LAYER 1
#define HDQ_HEAD_NORM_RMS 2
typedef struct hdq_head_norm {
  int32_t kind;
  float eps;
  const float *q_weight;
  const float *q_bias;
  const float *k_weight;
  const float *k_bias;
} hdq_head_norm;

/* Rotary positions: of a head's first `dim` elements (even), pair j -- elements
 * 2j and 2j + 1 (INTERLEAVED) or j and j + dim / 2 (HALF) -- is turned by
 * t = 2 pi frac(p turns[j]): (a, b) <- scale (a cos t - b sin t, b cos t + a sin t).
 * p is the token's position on the pair's axis: the first axis_dim[0] / 2 pairs
 * belong to axis 0, the next axis_dim[1] / 2 to axis 1, and so on (axis_dim of
 * the `axes` axes add up to dim).  A token with a negative position on any
 * axis is not rotated (text tokens in front of a video's).  p turns[j] is taken
 * in float64 in two parts, so its fraction is off by the rounding of turns[j]
 * alone, p 2^-53 turns[j] (p up to 2^53; larger ones are rounded to float64);
 * cosine and sine are float32. */
#define HDQ_ROPE_INTERLEAVED 0
#define HDQ_ROPE_HALF 1
#define HDQ_ROPE_MAX_AXES 3
typedef struct hdq_rope {
  int32_t layout;
  int32_t dim;             /* rotated elements, 0: none (the rest is ignored) */
  int32_t axes;            /* 1 to HDQ_ROPE_MAX_AXES                          */
  int32_t axis_dim[3];
  float scale;
  const double *turns;     /* device [dim / 2], turns per position            */
  const int64_t *positions; /* device, element (axis, batch, token) at        */
  int64_t pos_axis_stride; /* axis pos_axis_stride + ...                      */
  int64_t pos_batch_stride;
  int64_t pos_token_stride;
} hdq_rope;

/* Frequencies on the host: turns[j] = base^(-2 j / dim) / (2 pi), j < dim / 2, with
 * one axis' dim, and a long context's scaling:
 *   NONE;
 *   LINEAR: all divided by factor;
 *   BASE  : base times factor^(dim / (dim - 2)), so that the slowest pair is
 *           divided by factor and the fastest kept (dim > 2);
 *   RAMP  : turns[j] / factor where a pair makes at most `slow` turns over
 *           `length` positions (the context trained on), turns[j] from `fast`
 *           turns on, and the blend linear in the turns between.
 * factor >= 1; length, slow, fast (0 <= slow < fast) count for RAMP alone.
 * Writes float64 [dim / 2] to host memory. */
#define HDQ_ROPE_SCALE_NONE 0
#define HDQ_ROPE_SCALE_LINEAR 1
#define HDQ_ROPE_SCALE_BASE 2
#define HDQ_ROPE_SCALE_RAMP 3
int hdq_rope_turns(int32_t dim, double base, int32_t scaling, double factor, double length, double slow, double fast,
                   double *turns_host);

/*
 * hdq_qk_norm_rope -- queries and keys normed and rotated in one pass.
 *   q, k         : inputs of the same dtype, batch, length and dim; k (and
 *                  k_out) may be NULL for one tensor alone.
 *   norm         : NULL or kind NONE: not normed.
 *   rope         : NULL or dim 0: not rotated.
 *   q_out, k_out : of the same dtype as each other, heads as q's and k's.
 */
int hdq_qk_norm_rope(const hdq_heads *q, const hdq_heads *k, int64_t batch, int64_t length, int32_t dim,
                     const hdq_head_norm *norm, const hdq_rope *rope, const hdq_heads *q_out,
                     const hdq_heads *k_out, void *stream);

/* A cache of keys and values, `slots` tokens of heads x dim elements each, in
 * 8 or 4 bits.  dim is a multiple of 8, at most HDQ_HEAD_MAX_DIM; a group of
 * elements (dim itself, or a power of two from 8 on that divides it) shares an
 * fp32 scale; had_block (a power of two to 128 that divides dim, 1: none) is
 * the block Hadamard rotation the elements are stored with.
 *   codes : device uint8 [slots, heads, dim] (INT8, FP8: E4M3) or
 *           [slots, heads, dim / 2] (INT4, even element in the low nibble, two's
 *           complement), 8-byte aligned.
 *   scale : device fp32 [slots, heads, dim / group].
 * With y the rotated values and a = max|y| of a group: scale = fl32(a / top), code =
 * rne(y * fl32(top / a)), top 127, 448 (E4M3 nearest, ties to even) or 7.  A group
 * with a < 2^-100 gets scale 0 and zero codes, one with a NaN or an infinity
 * scale NaN and zero codes.  y comes from float32 butterflies and one product with
 * 1 / sqrt(had_block): a sum of theirs past float32's range counts as an infinity.
 * slots may be 0; the buffers are never NULL. */
#define HDQ_CACHE_INT8 0
#define HDQ_CACHE_FP8 1
#define HDQ_CACHE_INT4 2
typedef struct hdq_kv_cache {
  int32_t fmt;
  int32_t group;
  int32_t had_block;
  int32_t heads;
  int32_t dim;
  int64_t slots;
  uint8_t *k_codes;
  float *k_scale;
  uint8_t *v_codes;
  float *v_scale;
} hdq_kv_cache;

/*
 * hdq_qkv_to_cache -- the same pass with the keys, normed and rotated, and the
 * values, as they are, quantized into the cache.
 *   q, q_out : NULL for keys and values alone.
 *   k, v     : [batch, length, cache heads, dim] of q's dtype.
 *   slots    : device int64 [batch * length], each token's slot; tokens with a
 *              slot below 0 or past the cache's are left out (their queries are
 *              still written).  Slots of one call are distinct: of two tokens
 *              with one slot the outcome is a mix.
 * Slots not named keep their codes and scales.
 */
int hdq_qkv_to_cache(const hdq_heads *q, const hdq_heads *k, const hdq_heads *v, int64_t batch, int64_t length,
                     const hdq_head_norm *norm, const hdq_rope *rope, const hdq_heads *q_out,
                     const int64_t *slots, const hdq_kv_cache *cache, void *stream);

/*
 * hdq_cache_read -- slots' keys and values, rotated back.
 *   slots        : device int64 [tokens] (0 to HDQ_FP8_MAX_ROWS of them); a
 *                  slot may come more than once, one below 0 or past the
 *                  cache's reads zeros.
 *   k_out, v_out : device [tokens, heads, dim], HDQ_DTYPE_BF16 or HDQ_DTYPE_F32,
 *                  16-byte aligned.
 */
int hdq_cache_read(const hdq_kv_cache *cache, const int64_t *slots, int64_t tokens, void *k_out, void *v_out,
                   int32_t y_dtype, void *stream);

/* Scratch bytes an entry point needs.  op = HDQ_OP_SELECT: (M = rows,
 * K = cols, N = prev_numel); HDQ_OP_SELECT_Q8: (M = rows, K = cols);
 * HDQ_OP_QUANTIZE: (M = rows, K = cols, fmt);
 * HDQ_OP_LINEAR: (M, K, N, fmt = the weights' FP4 format, or -1 when only
 * INT8/BF16 will run); HDQ_OP_DQ_QUANTIZE: 256; HDQ_OP_DQ_LINEAR: (M = tokens,
 * K = cubes, N).  Returns 0 on bad arguments. */
size_t hdq_workspace_bytes(int32_t op, int64_t M, int64_t K, int64_t N, int32_t fmt);

/* Static text for a status code. */
const char *hdq_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int hdq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HDQ_H */
