/*
 * segquant.h -- C ABI of libsegquant: the DualScale x SegLinear W8A8 linear
 * layer on AMD Instinct MI355X (gfx950).
 *
 * Sources (cited by page title and section):
 *   [P1] "SegQuant: A Semantics-Aware and Generalizable Quantization
 *        Framework for Diffusion Models", paper notes (papernotes.org,
 *        CVPR 2026): "SegLinear" (output- and input-segmented patterns and
 *        their equations), "DualScale" (split, scales, reconstruction,
 *        hardware-native execution), framework table (AMax calibrator).
 *   [P2] "SegQuant", project page (hliangzhao.me/works/segquant.html):
 *        section 2 (SegLinear equations), section 3 (polarity-aware
 *        quantisation Q_dual, s+ and s-, reconstruction, one batched launch
 *        with a fused epilogue).
 *
 * What the layer computes (Y = X W, X in R^{M x K}, W in R^{K x N}):
 *   split      X+ = max(X,0), X- = min(X,0)                     [P1 DualScale]
 *   scales     s+ = max(X)/127, s- = |min(X)|/128, per K-segment  [P2 s.3]
 *   quantise   q+ = clamp(rne(fp32(x+ * inv+)), 0, 127)
 *              q- = clamp(rne(fp32(x- * inv-)), -128, 0)          [P2 s.3 Q_dual]
 *   products   A+_i = q+_i W_q,i and A-_i = q-_i W_q,i (int32, exact) over
 *              the K-range of segment i, both halves against one W tile
 *   epilogue   y = sum_i w_scale[i][n] (s+_i A+_i + s-_i A-_i), fp32,
 *              stored bf16 (round to nearest even)      [P1/P2 reconstruction]
 * Output-segmented layers [P1 SegLinear pattern one] differ only in their
 * weight-scale groups, which w_scale expresses per column; input-segmented
 * layers [P1 SegLinear pattern two] carry one (s+, s-) pair and one weight
 * scale group per K-segment.
 *
 * Conventions for every entry point
 *   - Tensor pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates or frees device memory and keeps no pointer after the
 *     call returns.  The only scratch memory is the optional, caller-owned
 *     workspace of segquant_gemm_w8a8_seg (its size from
 *     segquant_gemm_workspace_bytes) and the caller-owned workspaces of
 *     segquant_groupnorm_quantize, segquant_adapter_add and
 *     segquant_gemm_mxfp4.
 *   - Segment lists are HOST arrays (offset[n], width[n]), read only during
 *     the call: offsets start at 0, are contiguous, widths are positive and
 *     sum to the segmented dimension.  Every K-segment boundary except the
 *     end of K is a multiple of 64 (one MFMA K-step); n <= SEGQ_MAX_KSEG.
 *   - Activation scale table: DEVICE fp32 [4][n_kseg], rows
 *     s_pos, s_neg, inv_pos, inv_neg (segquant_calibrate_amax writes it).
 *   - bf16 tensors are passed as uint16_t bit patterns, row-major with a
 *     leading dimension (elements) >= the row length.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Work is enqueued
 *     asynchronously; no call synchronises the host.
 *   - Every call returns SEGQ_OK or a negative status.  All argument checks
 *     run before any HIP call, so an invalid call enqueues nothing and
 *     changes no buffer.  segquant_last_error() gives the thread's detail
 *     text for its last failing call.  Nothing is thrown, printed or aborted.
 *   - The library is thread-safe; its only state is that thread-local text.
 *   - Inputs must not hold NaN (MXFP4 carries it: see there).  +-Inf saturates to the end of its half's
 *     code range when that half's inverse scale is nonzero; an infinite
 *     value in a half whose scale is zero is outside the contract.
 */
#ifndef SEGQUANT_H
#define SEGQUANT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define SEGQ_OK 0
#define SEGQ_ERR_NULL (-1)        /* a required pointer is NULL */
#define SEGQ_ERR_SHAPE (-2)       /* a size or leading dimension is invalid */
#define SEGQ_ERR_SEGMENTS (-3)    /* a segment list is malformed */
#define SEGQ_ERR_ALIGN (-4)       /* a size, boundary or pointer is misaligned */
#define SEGQ_ERR_UNSUPPORTED (-5) /* valid but beyond this library's limits */
#define SEGQ_ERR_HIP (-6)         /* a HIP launch or runtime call failed */

/* Limits. */
#define SEGQ_MAX_KSEG 128
/* Widest K-segment whose int32 products cannot overflow:
 * floor((2^31 - 1) / (128 * 127)). */
#define SEGQ_MAX_KSEG_WIDTH 132104

/* Layouts of a quantised activation. */
#define SEGQ_Q_SIGNED 0 /* one int8 plane [M][ld_q] holding q+ + q- (the
                           halves have disjoint support, so this is lossless:
                           q+ = max(Q,0), q- = min(Q,0)) */
#define SEGQ_Q_PLANES 1 /* two int8 planes [2][M][ld_q]: q+ then q- */

/* Flags for segquant_gemm_w8a8_seg. */
#define SEGQ_GEMM_AUTO 0u        /* pick the kernel from the shape */
#define SEGQ_GEMM_FORCE_TILE 1u  /* the MFMA tile kernel, any M */
#define SEGQ_GEMM_FORCE_SMALLM 2u /* the weight-streaming kernel (M <= 16) */
#define SEGQ_GEMM_FUSED_QUANT 4u  /* quantise bf16 input inside the GEMM kernel
                                     even when a workspace is given */
#define SEGQ_GEMM_SINGLE_SCALE 8u /* single-scale W8A8: see segquant_gemm_w8a8_seg */
#define SEGQ_GEMM_W4 16u          /* w_packed holds 4-bit weights (segquant_quantize_weight_w4) */

/* Kernel choices reported by segquant_gemm_kernel_for. */
#define SEGQ_KERNEL_TILE 1
#define SEGQ_KERNEL_SMALLM 2

/*
 * segquant_calibrate_amax -- AMax calibration of the static activation
 * scales [P1 framework table, AMax; P1 DualScale scale equation; P2 s.3].
 * For each K-segment i, over X[:, segment i]:
 *   mx = max(0, max x), mn = min(0, min x)
 *   s_pos = mx/127, s_neg = |mn|/128, inv_pos = 127/mx, inv_neg = 128/|mn|
 * each quotient formed in fp64 and rounded once to fp32; an inverse whose
 * range is zero is 0 (that half then quantises to all zeros).
 *   x_bf16      device bf16 [M][ld_x]
 *   act_scales  device fp32 [4][n_kseg] (output; also used as the reduction
 *               buffer while the call runs)
 * Three short launches on `stream`.  M may be 0 (all scales become 0).
 */
int segquant_calibrate_amax(const uint16_t *x_bf16, int64_t M, int64_t K, int64_t ld_x,
                            int32_t n_kseg, const int32_t *kseg_offset,
                            const int32_t *kseg_width, float *act_scales, void *stream);

/*
 * segquant_calibrate_amax_single -- the single-scale baseline's calibration
 * [P2 deployment-cost table, INT8 baseline row; P1 limitations section:
 * DualScale doubles the products, so it may be enabled only for layers whose
 * activations are polarity-asymmetric].  Per K-segment i, one symmetric
 * range a = max(max x, -min x) over X[:, segment i]:
 *   s = a/127, inv = 127/a (fp64 quotients rounded once to fp32; 0 when a = 0)
 * written into BOTH halves of the table (s_pos = s_neg = s, inv_pos =
 * inv_neg = inv).  With such a table the DualScale quantiser yields the
 * plain symmetric codes clamp(rne(fp32(x * inv)), -127, 127), and the layer
 * equals textbook per-segment W8A8; SEGQ_GEMM_SINGLE_SCALE then computes it
 * with one product instead of two.  Arguments and launches as
 * segquant_calibrate_amax.
 */
int segquant_calibrate_amax_single(const uint16_t *x_bf16, int64_t M, int64_t K, int64_t ld_x,
                                   int32_t n_kseg, const int32_t *kseg_offset,
                                   const int32_t *kseg_width, float *act_scales, void *stream);

/*
 * segquant_quantize_dualscale -- polarity split and dual-scale quantisation
 * [P1 DualScale split and quantisation scheme; P2 s.3 Q_dual] of a bf16
 * activation, HBM to HBM, for the pre-quantised GEMM path.
 *   x_bf16      device bf16 [M][ld_x]
 *   act_scales  device fp32 [4][n_kseg] (reads the inv rows)
 *   q_out       device int8: SEGQ_Q_SIGNED -> [M][ld_q];
 *               SEGQ_Q_PLANES -> [2][M][ld_q] (q+ plane, then q- plane)
 * One launch.  M may be 0.
 */
int segquant_quantize_dualscale(const uint16_t *x_bf16, int64_t M, int64_t K, int64_t ld_x,
                                int32_t n_kseg, const int32_t *kseg_offset,
                                const int32_t *kseg_width, const float *act_scales,
                                int8_t *q_out, int64_t ld_q, int32_t q_layout, void *stream);

/* Activations for segquant_activate_quantize and (with SEGQ_ACT_NONE)
 * segquant_groupnorm_quantize. */
#define SEGQ_ACT_NONE 0 /* z itself (group norm only) */
#define SEGQ_ACT_SILU 1 /* z / (1 + exp(-z)) */
#define SEGQ_ACT_GELU 2 /* z/2 * (1 + erf(z / sqrt(2))), the exact form */

/*
 * segquant_activate_quantize -- the producer fused with the quantisation:
 * the SiLU or GELU whose outputs carry the polarity asymmetry DualScale is
 * for [P1 DualScale motivation; P2 section 3], applied to a bf16
 * pre-activation and quantised in the same pass, so the activated bf16 X
 * never round-trips through HBM.  Per element:
 *   x = bf16_rne(act(z))   with act evaluated in fp32 (library expf;
 *                          GELU as z/2 erfc(-z/sqrt 2), which is accurate
 *                          for negative z)
 *   codes of x exactly as segquant_quantize_dualscale
 *   z_bf16      device bf16 [M][ld_z]
 *   act_kind    SEGQ_ACT_SILU or SEGQ_ACT_GELU
 *   act_scales  device fp32 [4][n_kseg], calibrated on x (may be NULL when
 *               q_out is NULL)
 *   q_out       optional device int8, layout and ld_q as for
 *               segquant_quantize_dualscale
 *   x_out       optional device bf16 [M][ld_xo]: x itself (for the offline
 *               calibration, or for another consumer of the bf16 values)
 * At least one of q_out and x_out.  One launch; M may be 0.
 */
int segquant_activate_quantize(const uint16_t *z_bf16, int64_t M, int64_t K, int64_t ld_z,
                               int32_t act_kind, int32_t n_kseg, const int32_t *kseg_offset,
                               const int32_t *kseg_width, const float *act_scales,
                               int8_t *q_out, int64_t ld_q, int32_t q_layout, uint16_t *x_out,
                               int64_t ld_xo, void *stream);

/*
 * segquant_groupnorm_quantize -- group norm of a channels-last image fused
 * with the modulation, the activation and the quantisation: what an image
 * UNet's layers read.  B samples of P pixels (rows) of C channels, row
 * b * P + p; group g holds the D = C / groups neighbouring channels
 * g*D .. g*D + D-1 of every row.  Per sample and group, over its P * D values:
 *   mu = mean z, v = mean (z - mu)^2                                  (fp32)
 *   t  = (z - mu) / sqrt(v + eps) * gamma[c] + beta[c]
 *   t  = t * (1 + scale[b][c]) + shift[b][c]
 *   x  = bf16_rne(act(t)); codes of x exactly as segquant_quantize_dualscale
 *   z_bf16      device bf16 [B * P][ld_z]
 *   groups      1 .. C, a divisor of C (groups = C: instance norm)
 *   eps         at least 2^-126
 *   gamma, beta device fp32 [C], each optional (NULL: 1 and 0)
 *   scale, shift  device bf16 [B][ld_mod], each optional (NULL: 0): two chunks
 *               of a conditioning layer's output as they are, ld_mod its
 *               leading dimension (ignored when both are NULL)
 *   act_kind    SEGQ_ACT_NONE, SEGQ_ACT_SILU or SEGQ_ACT_GELU.  act(t) is
 *               within 2^-17 of its true value, relative, down to 2^-125
 *               (segquant_activate_quantize: 2^-19), so the two calls may
 *               round to neighbouring bf16 values
 *   act_scales, q_out, ld_q, q_layout, x_out, ld_xo
 *               the outputs of segquant_activate_quantize, K-segments over
 *               the C channels.  x_out may be z_bf16 when ld_xo = ld_z
 *               (outputs and workspace must not overlap each other or an
 *               input otherwise: SEGQ_ERR_SHAPE).
 *   workspace   device scratch, 16-byte aligned, of at least
 *               segquant_groupnorm_workspace_bytes() bytes (SEGQ_ERR_UNSUPPORTED
 *               with fewer), contents undefined afterwards; calls that share
 *               one must be ordered.  NULL where that size is 0.
 * One launch where a group of a sample fits a workgroup's registers, else
 * two.  The order of every sum is fixed: the same call gives the same bits.
 * Tensor pointers 16-byte aligned, ld_z, ld_xo and ld_mod multiples of 8,
 * ld_q of 16; C needs no alignment.  C <= 2^20, B <= 65535.  B or P may be 0.
 * A group whose values or squared deviations add up to 2^128 or more overflows
 * fp32.
 */
int segquant_groupnorm_quantize(const uint16_t *z_bf16, int64_t B, int64_t P, int64_t C,
                                int64_t ld_z, int32_t groups, float eps, const float *gamma,
                                const float *beta, const uint16_t *scale, const uint16_t *shift,
                                int64_t ld_mod, int32_t act_kind, int32_t n_kseg,
                                const int32_t *kseg_offset, const int32_t *kseg_width,
                                const float *act_scales, int8_t *q_out, int64_t ld_q,
                                int32_t q_layout, uint16_t *x_out, int64_t ld_xo, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Workspace of segquant_groupnorm_quantize for these sizes (0: none).  On
 * invalid sizes returns 0 and sets segquant_last_error(). */
size_t segquant_groupnorm_workspace_bytes(int64_t B, int64_t P, int64_t C, int32_t groups);

/*
 * segquant_adanorm_quantize -- the AdaNorm block in front of a quantised
 * layer: the gated residual update, layer norm, and the modulation by the
 * shift and scale that the request's conditioning layer emits [P2 section 1;
 * P1 SegLinear, the AdaNorm chunking], fused with the quantisation.  For row m
 * of request r, over its K values:
 *   h' = bf16_rne(h + gate[r] * branch)           (where branch is given)
 *   mu = mean h', v = mean (h' - mu)^2                                (fp32)
 *   t  = (h' - mu) / sqrt(v + eps) * gamma[k] + beta[k]
 *   x  = bf16_rne(t * (1 + scale[r][k]) + shift[r][k])
 *   codes of x exactly as segquant_quantize_dualscale
 *   h_bf16      device bf16 [M][ld_h], the residual stream
 *   branch      optional device bf16 [M][ld_b]: the last block's output
 *   gate        optional, only with branch: device bf16 [n_req][ld_mod]
 *               (NULL: 1)
 *   h_out       optional, only with branch: device bf16 [M][ld_ho], h';
 *               may be h_bf16 when ld_ho = ld_h, or branch when ld_ho = ld_b
 *   gamma, beta device fp32 [K], each optional (NULL: 1 and 0)
 *   scale, shift  device bf16 [n_req][ld_mod], each optional (NULL: 0); scale,
 *               shift and gate share ld_mod: chunks of one layer's output
 *   n_req       >= 1
 *   row_offset  device int32 [n_req + 1]: request r holds rows row_offset[r]
 *               .. row_offset[r+1] - 1 (none where they are equal).  Rows
 *               before the first or behind the last request are left as they
 *               are in every output.  The offsets must not decrease; if they
 *               do, which request's parameters a row gets is unspecified (no
 *               access leaves the arrays).  NULL: n_req requests of M / n_req
 *               rows each, n_req a divisor of M.
 *   act_scales, q_out, ld_q, q_layout, x_out, ld_xo
 *               the outputs of segquant_activate_quantize; here neither need
 *               be given if h_out is
 * One launch, no workspace.  Tensor pointers 16-byte aligned (row_offset 4),
 * ld_h, ld_b, ld_ho, ld_xo and ld_mod multiples of 8, ld_q of 16; K needs no
 * alignment; K-segment boundaries up to 4194240.  M may be 0.  Outputs must
 * not overlap each other or, but for h_out as above, inputs: SEGQ_ERR_SHAPE.
 * A row whose values or squared deviations add up to 2^128 or more overflows fp32.
 */
int segquant_adanorm_quantize(const uint16_t *h_bf16, int64_t M, int64_t K, int64_t ld_h,
                              const uint16_t *branch, int64_t ld_b, const uint16_t *gate,
                              uint16_t *h_out, int64_t ld_ho, float eps, const float *gamma,
                              const float *beta, const uint16_t *scale, const uint16_t *shift,
                              int64_t ld_mod, int32_t n_req, const int32_t *row_offset,
                              int32_t n_kseg, const int32_t *kseg_offset,
                              const int32_t *kseg_width, const float *act_scales, int8_t *q_out,
                              int64_t ld_q, int32_t q_layout, uint16_t *x_out, int64_t ld_xo,
                              void *stream);

/*
 * Microscaled 4-bit floating point (MXFP4, of the OCP Microscaling Formats
 * specification, version 1.0).  Along K, blocks of 32 neighbours share a power
 * of two 2^(s - 127), s one byte; an element is a 4-bit float c times it, c =
 * 0, 0.5, 1, 1.5, 2, 3, 4 or 6 (codes 0 .. 7; bit 3 the sign).  Quantising:
 *   s = max(0, 127 + floor(log2 max |x|) - 2)        (0 for a block of zeros)
 *   c = x / 2^(s - 127) rounded to nearest, ties to the even code, magnitudes
 *       above 6 to 6
 * A block that holds an infinity or a NaN gets s = 255, which is NaN: so are
 * its values and every product with it.
 *
 * An MXFP4 matrix of R rows and K columns (K % 64 == 0) is two byte arrays in
 * the operand order of the matrix cores, rows padded to a multiple of 16:
 *   codes   KT = ceil(K / 128).  The codes of row r, columns k and k + 1 (k
 *           even) in the low and high half of byte
 *           ((r/16 * KT + k/128) * 64 + k%128/32 * 16 + r%16) * 16 + k%32/2
 *   scales  KS = ceil(K / 512).  s of row r, block k/32 in byte
 *           ((r/16 * KS + k/512) * 64 + k%128/32 * 16 + r%16) * 4 + k%512/128
 * Columns K .. 128 KT - 1 hold codes and scales 0, the rest of the padding
 * anything.  Rows of an activation are tokens, of a weight output columns.
 */

/* Bytes of the two arrays (0 for sizes that have no such matrix; R may be 0). */
size_t segquant_mxfp4_code_bytes(int64_t R, int64_t K);
size_t segquant_mxfp4_scale_bytes(int64_t R, int64_t K);

/*
 * segquant_quantize_mxfp4 -- x = bf16_rne(act(z)), or z itself
 * (SEGQ_ACT_NONE), as MXFP4.  act(z) is within 2^-17 of its true value, relative,
 * down to 2^-125 (the bound of segquant_groupnorm_quantize, not its bits).  SiLU
 * and GELU of an infinity of either sign make their block NaN, as z = NaN does: at
 * one end the formulas are an infinity, at the other an infinity times 0.
 *   z_bf16      device bf16 [M][ld_z]
 *   codes, scales  device, the arrays of M rows and K columns, 16- and 4-byte
 *               aligned; they must not overlap each other or z_bf16
 * One launch per 1048544 rows.  Requires K % 64 == 0, z_bf16 16-byte aligned, ld_z a
 * multiple of 8, M <= 2^27, K <= 2^22.  M may be 0.
 */
int segquant_quantize_mxfp4(const uint16_t *z_bf16, int64_t M, int64_t K, int64_t ld_z,
                            int32_t act_kind, uint8_t *codes, uint8_t *scales, void *stream);

/*
 * segquant_quantize_weight_mxfp4 -- a weight W [K][N] (Y = X W) as an MXFP4
 * matrix of N rows and K columns.
 *   w           device fp32 [K][ld_w]
 * Requires K % 64 == 0, N % 16 == 0, K <= 2^22, N <= 2^27.  Offline; one launch.
 */
int segquant_quantize_weight_mxfp4(const float *w, int64_t K, int64_t N, int64_t ld_w,
                                   uint8_t *codes, uint8_t *scales, void *stream);

/* segquant_unpack_mxfp4 -- the fp32 values [R][ld_x] of an MXFP4 matrix.  For
 * inspection and tests.  One launch. */
int segquant_unpack_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K,
                          float *x, int64_t ld_x, void *stream);

/*
 * segquant_gemm_mxfp4 -- the linear layer on MXFP4 weights and activations:
 *   y[m][n] = bf16_rne( sum_k x[m][k] w[n][k] )
 * in fp32, by the matrix cores' scaled products of 128 columns.  The
 * activation is either
 *   z_bf16 != NULL: bf16 [M][ld_z], quantised by the call as by
 *                   segquant_quantize_mxfp4 with act_kind, or
 *   x_codes, x_scales != NULL: an MXFP4 matrix of M rows (act_kind
 *                   SEGQ_ACT_NONE).
 *   w_codes, w_scales  an MXFP4 matrix of N rows
 *   y_bf16      device bf16 [M][ld_y]
 *   workspace   device scratch, 16-byte aligned, of at least
 *               segquant_gemm_mxfp4_workspace_bytes() bytes where z_bf16 is
 *               given (SEGQ_ERR_UNSUPPORTED with fewer), contents undefined
 *               afterwards; calls that share one must be ordered.  NULL where
 *               that size is 0.
 * One launch, or quantisation and product where a workspace is asked for (some of
 * those calls leave it unused).  The order of every sum is fixed.  y_bf16 and the workspace must not overlap each
 * other or an input: SEGQ_ERR_SHAPE.  Requires K % 64 == 0, N % 16 == 0, 16-byte
 * aligned pointers (scales 4), ld_z and ld_y multiples of 8, M and N <= 2^27,
 * K <= 2^22, M * N <= 2^37.  M may be 0.
 */
int segquant_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint16_t *z_bf16, int64_t ld_z,
                        int32_t act_kind, const uint8_t *x_codes, const uint8_t *x_scales,
                        const uint8_t *w_codes, const uint8_t *w_scales, uint16_t *y_bf16,
                        int64_t ld_y, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace of segquant_gemm_mxfp4 on bf16 input of these sizes (0: none).  On
 * invalid sizes returns 0 and sets segquant_last_error(). */
size_t segquant_gemm_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * segquant_rmsnorm_quantize -- the residual update and root-mean-square norm in
 * front of a quantised layer, fused with its quantisation.  Over the K values
 * of each row:
 *   h' = bf16_rne(h + branch)                    (where branch is given)
 *   x  = bf16_rne(h' / sqrt(mean h'^2 + eps) * gamma[k])             (fp32)
 *   codes of x exactly as segquant_quantize_dualscale; its MXFP4 form exactly as
 *   segquant_quantize_mxfp4
 *   h_bf16, branch, h_out  as segquant_adanorm_quantize
 *   eps         at least 2^-126
 *   gamma       device fp32 [K], optional (NULL: 1)
 *   n_kseg .. ld_xo  the outputs of segquant_activate_quantize
 *   mx_codes, mx_scales  device, both or neither: x as an MXFP4 matrix of M rows
 *               (then K % 64 == 0 and K <= 2^22)
 * At least one of h_out, q_out, x_out and mx_codes.  One launch, no workspace;
 * the order of every sum is fixed.  Alignment as segquant_adanorm_quantize
 * (mx_codes 16, mx_scales 4).  M may be 0.  Outputs must not overlap each other
 * or, but for h_out as there, inputs: SEGQ_ERR_SHAPE.  Any finite h' will do: where
 * its squares overflow fp32, the row is summed once more with smaller values.
 */
int segquant_rmsnorm_quantize(const uint16_t *h_bf16, int64_t M, int64_t K, int64_t ld_h,
                              const uint16_t *branch, int64_t ld_b, uint16_t *h_out, int64_t ld_ho,
                              float eps, const float *gamma, int32_t n_kseg,
                              const int32_t *kseg_offset, const int32_t *kseg_width,
                              const float *act_scales, int8_t *q_out, int64_t ld_q,
                              int32_t q_layout, uint16_t *x_out, int64_t ld_xo, uint8_t *mx_codes,
                              uint8_t *mx_scales, void *stream);

/* Which elements of a head turn together, of its first R: 2i and 2i + 1, or
 * i and i + R/2. */
#define SEGQ_ROTARY_PAIRS 0
#define SEGQ_ROTARY_HALVES 1
#define SEGQ_ROTARY_MAX_AXES 8
#define SEGQ_ROTARY_MAX_HEAD 512

/*
 * segquant_qk_rotary -- what stands between the QKV layer and attention: the
 * root-mean-square norm of each head of q and k, then rotary positions of one
 * or several axes (text; height and width; time, height and width).  For every
 * sample b, token l and head, over its D elements:
 *   t   = x / sqrt(mean x^2 + eps) * gamma[d]      (where norm; else t = x)
 *   a'  = a cos u - b sin u,  b' = b cos u + a sin u   for pair i = (a, b) of
 *         the first R elements of t, u = positions[l][axis of i] * freq[i]
 *   out = bf16_rne(t'); elements from R on are not turned
 * R is the sum of the axis widths: the first axis has the first
 * axis_width[0] / 2 pairs, and so on.  Angles are formed in fp64 and reduced
 * before they are rounded: any int32 position is as good as a small one, at
 * frequencies up to 2^48 in magnitude.
 * The norm takes any finite head, as segquant_rmsnorm_quantize.
 *   q, k        device bf16 [B][L][heads][D], any strides, which are HOST
 *               arrays of three: elements between samples, tokens and heads,
 *               multiples of 8, not negative.  k may be NULL: q alone.
 *   q_out, k_out  the same; each may be its input with the same strides
 *   norm        0: no norm (gammas NULL)
 *   eps         at least 2^-126 (unused without norm)
 *   q_gamma, k_gamma  device fp32 [D], each optional (NULL: 1)
 *   positions   device int32 [L][n_axes], or one such table per sample,
 *               pos_batch_stride elements apart (0: one for all)
 *   axis_width  HOST array, n_axes of them: even, not negative, R a multiple of
 *               16 up to D
 *   freq        device fp64 [R / 2], radians per position
 *               (segquant_rotary_frequencies gives the usual ones)
 * One launch; nothing is summed out of order.  Requires D a multiple of 8 up to
 * SEGQ_ROTARY_MAX_HEAD, 16-byte aligned q, k, outputs and gammas, 8-byte aligned
 * freq, B * L * heads <= 2^30 for q and k together.  B or L may be 0.  An output
 * must not overlap itself, the other or, but for its own as above, an input:
 * SEGQ_ERR_SHAPE.  Beside another tensor of the same sample and token strides,
 * and heads side by side in both or of one stride (q and k inside one QKV
 * matrix), the overlap is exact; else a tensor's whole extent counts where its
 * rows are not evenly spaced.
 */
int segquant_qk_rotary(int64_t B, int64_t L, int32_t D, const uint16_t *q, int32_t q_heads,
                       const int64_t *q_stride, uint16_t *q_out, const int64_t *q_out_stride,
                       const uint16_t *k, int32_t k_heads, const int64_t *k_stride,
                       uint16_t *k_out, const int64_t *k_out_stride, int32_t norm, float eps,
                       const float *q_gamma, const float *k_gamma, const int32_t *positions,
                       int64_t pos_batch_stride, int32_t n_axes, const int32_t *axis_width,
                       const double *freq, int32_t style, void *stream);

/* The usual frequencies, theta^(-2j / width) for pair j of an axis, into the HOST
 * array freq [R / 2].  Host-only: no GPU work. */
int segquant_rotary_frequencies(int32_t n_axes, const int32_t *axis_width, double theta,
                                double *freq);

/* Storage granularity and limit of adapter ranks. */
#define SEGQ_ADAPTER_RANK_STEP 16
#define SEGQ_ADAPTER_RANK_MAX 256

/*
 * segquant_adapter_add -- low-rank adapters of many requests beside a shared
 * layer.  For row m of request r with adapter i = adapter[r], and column n in
 * N-segment j:
 *   t[q]    = alpha[i] * sum_k x[m][k] * a[i][j * rank + q][k]
 *   y[m][n] = bf16_rne( base[m][n] + sum_{q < rank_of[i]} t[q] * b[i][n][q] )
 * The products of bf16 values are summed in fp32 and t is an fp32 value (where
 * it is below 2^-110 in magnitude it loses bits, as in bf16).  An output-segmented layer [P1 SegLinear, pattern one]
 * has one pair of factors per N-segment; a single segment is the usual
 * low-rank adapter.
 *   x_bf16      device bf16 [M][ld_x]: the layer's input before quantisation
 *   n_req, row_offset  as segquant_adanorm_quantize, row_offset required; rows
 *               of no request are left as they are in y.  Where offsets
 *               decrease, rows that are not in one request alone may hold
 *               anything
 *   adapter     device int32 [n_req]; an index outside [0, n_adapters) (-1,
 *               say) means no adapter: y = base for that request's rows
 *   rank        stored rank, a multiple of SEGQ_ADAPTER_RANK_STEP up to
 *               SEGQ_ADAPTER_RANK_MAX
 *   rank_of     optional device int32 [n_adapters]: true ranks, clamped to
 *               [0, rank]; what a and b hold past them is never used (NULL:
 *               every adapter has the stored rank)
 *   a           device bf16 [n_adapters][n_nseg * rank][K]
 *   b           device bf16 [n_adapters][N][rank]
 *   alpha       optional device fp32 [n_adapters] (NULL: 1)
 *   n_nseg, nseg_offset, nseg_width
 *               N-segments (host), boundaries multiples of 16
 *   base_bf16   optional device bf16 [M][ld_base]: the layer's output (NULL:
 *               0); may be y_bf16 when ld_base = ld_y
 *   y_bf16      device bf16 [M][ld_y]; y_bf16 and the workspace must not
 *               overlap each other or, but for base_bf16 as above, an input:
 *               SEGQ_ERR_SHAPE
 *   workspace   device scratch, 16-byte aligned, of at least
 *               segquant_adapter_workspace_bytes() bytes (SEGQ_ERR_UNSUPPORTED
 *               with fewer), contents undefined afterwards; calls that share
 *               one must be ordered.  NULL where that size is 0.
 * One launch, or two through the workspace.  The order of every sum is fixed.
 * Requires K % 64 == 0,
 * N % 16 == 0, 16-byte aligned tensor pointers (int32 arrays and alpha 4),
 * ld_x, ld_base and ld_y multiples of 8, M <= 2^27, N <= 1048560,
 * n_req <= 2^22.  M may be 0.
 */
int segquant_adapter_add(int64_t M, int64_t N, int64_t K, const uint16_t *x_bf16, int64_t ld_x,
                         int32_t n_req, const int32_t *row_offset, const int32_t *adapter,
                         int32_t n_adapters, int32_t rank, const int32_t *rank_of,
                         const uint16_t *a, const uint16_t *b, const float *alpha, int32_t n_nseg,
                         const int32_t *nseg_offset, const int32_t *nseg_width,
                         const uint16_t *base_bf16, int64_t ld_base, uint16_t *y_bf16,
                         int64_t ld_y, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace of segquant_adapter_add for these sizes (0: none).  On invalid
 * sizes returns 0 and sets segquant_last_error(). */
size_t segquant_adapter_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t n_req,
                                        int32_t rank, int32_t n_nseg, const int32_t *nseg_offset,
                                        const int32_t *nseg_width);

/*
 * segquant_weight_packed_bytes -- size of the packed int8 weight for a
 * K x N layer: K*N bytes when K % 64 == 0 and N % 16 == 0, else 0.
 * The packed layout is tiles of 64 (k) x 16 (n) bytes, 1 KiB each, stored
 * n-tile major: tile (nt, kt) at byte (nt * (K/64) + kt) * 1024; inside a
 * tile, byte (g*16 + j)*16 + b holds W_q[kt*64 + g*16 + b][nt*16 + j]
 * (g in 0..3, j in 0..15, b in 0..15): the operand order of the int8
 * 16x16x64 matrix-core instruction, one 16-byte row per lane.
 */
size_t segquant_weight_packed_bytes(int64_t K, int64_t N);

/*
 * segquant_quantize_weight -- symmetric int8 weight quantisation per group
 * [P1 SegLinear, both patterns: each segment quantised on its own; P2 s.2],
 * packed for the kernels.  The group of (k, n) is (K-segment of k) x
 * (N-segment of n), or (K-segment of k) x {n} when per_column != 0 (then
 * the N-segment list is ignored and may be NULL).  Per group:
 *   a = max |w|, s_w = a/127 and inv_w = 127/a (fp64 quotients rounded
 *   once to fp32; inv_w = 0 when a = 0),
 *   w_q = clamp(rne(fp32(w * inv_w)), -127, 127)
 *   w          device fp32 [K][ld_w] (Y = X W)
 *   w_packed   device int8, segquant_weight_packed_bytes(K, N) bytes
 *   w_scale    device fp32 [n_kseg][N]: the s_w of the group holding
 *              (K-segment i, column n) -- the epilogue's per-column scale
 * Requires K % 64 == 0, N % 16 == 0.  Offline; four short launches.
 */
int segquant_quantize_weight(const float *w, int64_t K, int64_t N, int64_t ld_w,
                             int32_t n_kseg, const int32_t *kseg_offset,
                             const int32_t *kseg_width, int32_t n_nseg,
                             const int32_t *nseg_offset, const int32_t *nseg_width,
                             int32_t per_column, int8_t *w_packed, float *w_scale,
                             void *stream);

/*
 * segquant_quantize_weight_w4 -- the 4-bit weights of W4A8, the pages'
 * second precision [P2 deployment-cost table, SegQuant-4 row; P1
 * experiments, W4A8], with the same groups as segquant_quantize_weight:
 *   s_w = a/7, inv_w = 7/a, w_q = clamp(rne(fp32(w * inv_w)), -7, 7)
 * Packed in 512-byte tiles that mirror the int8 ones (tile (nt, kt) at byte
 * (nt * K/64 + kt) * 512; lane l = g*16 + j of a tile owns bytes l*8 .. l*8+7
 * holding W_q[kt*64 + g*16 + b][nt*16 + j], b = 0..15, as codes + 8 in
 * nibbles: byte i (i = 0..3) of the first dword holds b = i in its low and
 * b = i + 4 in its high nibble, byte i of the second dword b = 8 + i and
 * b = 12 + i).  segquant_weight_packed_bytes_w4(K, N) = K*N/2 bytes.
 * Arguments, w_scale and launches as segquant_quantize_weight.
 */
int segquant_quantize_weight_w4(const float *w, int64_t K, int64_t N, int64_t ld_w,
                                int32_t n_kseg, const int32_t *kseg_offset,
                                const int32_t *kseg_width, int32_t n_nseg,
                                const int32_t *nseg_offset, const int32_t *nseg_width,
                                int32_t per_column, int8_t *w_packed, float *w_scale,
                                void *stream);

size_t segquant_weight_packed_bytes_w4(int64_t K, int64_t N);

/* segquant_unpack_weight_w4 -- 4-bit packed weights -> int8 codes
 * [K][ld_w] row-major (values in [-7, 7]).  For inspection and tests. */
int segquant_unpack_weight_w4(const int8_t *w_packed, int64_t K, int64_t N, int8_t *w_kn,
                              int64_t ld_w, void *stream);

/*
 * segquant_unpack_weight -- inverse of the packing: w_packed -> device int8
 * W_q [K][ld_w] row-major.  For inspection and tests.  One launch.
 */
int segquant_unpack_weight(const int8_t *w_packed, int64_t K, int64_t N, int8_t *w_kn,
                           int64_t ld_w, void *stream);

/*
 * segquant_gemm_w8a8_seg -- the DualScale x SegLinear W8A8 linear layer in
 * ONE launch [P1 DualScale hardware-native execution; P2 s.3: both polarity
 * products in one batched launch, combined in a fused epilogue]:
 *   y[m][n] = bf16( sum_i w_scale[i][n] * (s_pos[i]*A+_i[m][n]
 *                                          + s_neg[i]*A-_i[m][n]) )
 * with A+-_i the exact int32 products of the quantised halves over K-segment
 * i against W_q (both halves read one W tile).  The activation is either
 *   x_bf16 != NULL: bf16 [M][ld_x], quantised inside the kernel with the inv
 *                   rows of act_scales (xq must be NULL), or
 *   xq != NULL:     the output of segquant_quantize_dualscale with the same
 *                   act_scales, layout q_layout, leading dimension ld_q.
 *   w_packed   from segquant_quantize_weight (K x N)
 *   w_scale    device fp32 [n_kseg][N]
 *   act_scales device fp32 [4][n_kseg]
 *   y_bf16     device bf16 [M][ld_y] (output)
 *   acc_debug  optional device int32 [2][n_kseg][M][N]: when not NULL the
 *              kernel also stores every per-segment accumulator A+_i
 *              (plane 0) and A-_i (plane 1); NULL in production.
 *   workspace  optional device scratch of workspace_bytes bytes, 16-byte
 *              aligned, owned by the caller.  With bf16 input and at least
 *              segquant_gemm_workspace_bytes() bytes, the call may quantise
 *              X into it first (the segquant_quantize_dualscale kernel,
 *              signed codes, ld_q = K) and run the GEMM from the codes: two
 *              launches, the same results.  Its contents are undefined
 *              afterwards; calls that share one workspace must be ordered
 *              (same stream).  NULL, or fewer bytes than asked for: one
 *              fused launch.
 *   flags      SEGQ_GEMM_AUTO, or force one kernel for testing
 *              (SEGQ_GEMM_FUSED_QUANT: never use the workspace), or'ed with
 *              SEGQ_GEMM_SINGLE_SCALE: single-scale W8A8.  Only the + half
 *              of act_scales is read: each element is quantised with inv_pos
 *              of its segment (code in [-128, 127]) and
 *                y[m][n] = bf16( sum_i w_scale[i][n] * s_pos[i] * A_i[m][n] )
 *              with A_i the exact int32 product of the signed codes: one
 *              product per element instead of two.  With a table from
 *              segquant_calibrate_amax_single this is the DualScale formula
 *              of that table.  acc_debug then receives A_i in plane 0 and
 *              plane 1 is not written.  Takes bf16 or SEGQ_Q_SIGNED input
 *              (SEGQ_Q_PLANES: SEGQ_ERR_UNSUPPORTED).
 *              SEGQ_GEMM_W4: w_packed is from segquant_quantize_weight_w4
 *              (W4A8; same formula with the 4-bit codes).  The small-M
 *              streaming kernel reads the 4-bit tiles directly (half the
 *              weight bytes); every other shape first widens them to int8
 *              tiles in the workspace, which must then hold K*N bytes (plus
 *              the quantise-first bytes; segquant_gemm_workspace_bytes with
 *              the same flags gives the total), else SEGQ_ERR_UNSUPPORTED.
 * Requires K % 64 == 0, N % 16 == 0, every K-segment width <=
 * SEGQ_MAX_KSEG_WIDTH (each segment's int32 sums stay below 2^31; K itself
 * has no further bound), 16-byte aligned tensor pointers, ld_x and ld_q
 * multiples of 8 and 16 elements, ld_y a multiple of 2.  M may be 0 (no
 * launch).  SEGQ_GEMM_FORCE_SMALLM requires M <= 16.
 */
int segquant_gemm_w8a8_seg(int64_t M, int64_t N, int64_t K,
                           const uint16_t *x_bf16, int64_t ld_x,
                           const int8_t *xq, int64_t ld_q, int32_t q_layout,
                           const int8_t *w_packed, const float *w_scale,
                           int32_t n_kseg, const int32_t *kseg_offset,
                           const int32_t *kseg_width, const float *act_scales,
                           uint16_t *y_bf16, int64_t ld_y, int32_t *acc_debug,
                           void *workspace, size_t workspace_bytes,
                           uint32_t flags, void *stream);

/*
 * segquant_gemm_w8a8_seg_noalloc -- segquant_gemm_w8a8_seg without a
 * workspace and without any device allocation, for callers that cannot
 * allocate: code under stream capture, tight serving loops, harnesses that
 * forbid hipMalloc.  Arguments, validation, results and errors are those of
 * segquant_gemm_w8a8_seg (same kernels, bit-identical outputs), less the
 * workspace.
 *
 * What the ordinary call would use a workspace for (the quantise-first int8
 * codes, M*K bytes; the int8 widening of 4-bit weights, K*N bytes) comes from
 * a device array of SEGQ_NOALLOC_SCRATCH_BYTES that the library holds on
 * every GPU it runs on until the process ends (its address is looked up on
 * the first call on each device).  Quantise-first codes that would not fit
 * are replaced by the fused launch (same codes and products); a required
 * widening that does not fit is refused with SEGQ_ERR_UNSUPPORTED before any
 * HIP call.  All calls on one GPU share its array: calls that overlap on one
 * GPU race, so order them (one stream).  The call makes no hipMalloc or
 * hipFree and calls no allocating library routine.
 */
#define SEGQ_NOALLOC_SCRATCH_BYTES (64u << 20)
int segquant_gemm_w8a8_seg_noalloc(int64_t M, int64_t N, int64_t K,
                                   const uint16_t *x_bf16, int64_t ld_x,
                                   const int8_t *xq, int64_t ld_q, int32_t q_layout,
                                   const int8_t *w_packed, const float *w_scale,
                                   int32_t n_kseg, const int32_t *kseg_offset,
                                   const int32_t *kseg_width, const float *act_scales,
                                   uint16_t *y_bf16, int64_t ld_y, int32_t *acc_debug,
                                   uint32_t flags, void *stream);

/*
 * segquant_gemm_workspace_bytes -- the workspace with which
 * segquant_gemm_w8a8_seg, given bf16 input of this shape and these
 * K-segments, quantises first (M * K bytes), or 0 when it quantises inside
 * the GEMM kernel anyway.  The large-M kernel re-quantises each activation
 * tile once per output column tile; from six column tiles on, one separate
 * quantisation pass costs less.  On invalid arguments returns 0 and sets
 * segquant_last_error().
 */
size_t segquant_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t n_kseg,
                                     const int32_t *kseg_offset, const int32_t *kseg_width,
                                     uint32_t flags);

/*
 * segquant_gemm_halves -- which halves a layer needs, from its static scales
 * ([P1] "SegQuant" notes, DualScale section, and its limitations: the
 * negative half exists for polarity-asymmetric activations; with no negative
 * values its term of the reconstruction vanishes).  Host-only: no GPU work.
 *   act_scales_host  HOST fp32 [4][n_kseg], a copy of the table written by
 *                    segquant_calibrate_amax (the scales are static, so the
 *                    copy is taken once, after calibration)
 * Returns SEGQ_GEMM_SINGLE_SCALE when s_neg and inv_neg are 0 in every
 * K-segment (the calibration data held no negative value), else 0.  Or'ed
 * into the flags of segquant_gemm_w8a8_seg with this same table, the layer
 * then runs one product per element instead of two and, for an input with
 * no negative elements, gives exactly the DualScale result (the + half's
 * codes and products are the same; the - half's are all zero).  A negative
 * element, which DualScale with s_neg = 0 quantises to 0, is instead
 * quantised with the + half's scale.  On a NULL table or n_kseg outside
 * [1, SEGQ_MAX_KSEG] returns SEGQ_ERR_NULL or SEGQ_ERR_SEGMENTS and sets
 * segquant_last_error().
 */
int segquant_gemm_halves(const float *act_scales_host, int32_t n_kseg);

/* Which kernel family segquant_gemm_w8a8_seg runs for this shape under
 * `flags` (SEGQ_KERNEL_*), or a negative status when the shape is invalid.
 * SEGQ_KERNEL_TILE is the large-M family: the tile kernel, or, for several
 * K-segments on int8 codes (the quantise-first path included) and for any
 * call whose K exceeds the tile kernel's running int32 sums
 * (K * 128 * 127 >= 2^31), the kernel that stages both operands in LDS and
 * folds each segment's own sums; which of the two depends on the segment
 * list and the activation format, not on the shape alone. */
int segquant_gemm_kernel_for(int64_t M, int64_t N, int64_t K, uint32_t flags);

/* Text for a status code (static storage). */
const char *segquant_status_string(int status);

/* Detail of this thread's last failing call ("" if none); valid until the
 * thread's next call into the library. */
const char *segquant_last_error(void);

/* Library version, major*10000 + minor*100 + patch. */
int segquant_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SEGQUANT_H */
