/*
 * hsq.h -- C ABI of libhsq: the inference-time W4A4 linear layer with a
 * rank-r high-precision branch, for AMD Instinct MI355X (gfx950).
 *
 * The layer (Deflating the Hessian, abstract; thelatestinai.com paper page,
 * Figure 1 caption): every weight is split into a high-precision low-rank
 * component and a low-bit residual, W ~ L1*L2 + Q(R).  Weights and
 * activations are 4-bit with one scale per 64-wide group of the input
 * dimension (same page, Table 1 and Table 8 captions: W4A4, group-64).  A
 * diagonal smoothing moves range from the activations to the weights
 * without changing the full-precision product (H-SVDQuant explainer,
 * rit.work, section on Hessian deflation, last paragraph).  As in the
 * two-branch inference form of DiRotQ (papernotes.org, key design 2), the
 * high-precision branch runs on the unquantized (smoothed) activations:
 *
 *   xh[m,k]  = X[m,k] * fl32(1 / lambda[k])                    smoothing
 *   sx[m,g]  = fp16_rne(fl32(absmax_{k in g} |xh[m,k]| / 7))   (0 if absmax = 0; saturates at 65504)
 *   qx[m,k]  = clamp(rint(xh[m,k] * fl32(1 / sx[m,g])), -8, 7) (all 0 if sx = 0)
 *   U[m,j]   = sum_k xh[m,k] * L1[k,j]                         rank-r down projection
 *   P[m,n,g] = sum_{k in g} qx[m,k] * qw[k,n]                  int32, exact
 *   Y[m,n]   = sum_g P[m,n,g] * sx[m,g] * sw[g,n] + sum_j U[m,j] * L2[j,n] + bias[n]
 *
 * Group g covers input channels [64g, 64g + 64).  The entry points whose
 * names end in _g take the group width as an argument, 64 or 128 (group g
 * then covers [group*g, group*g + group)); the Qwen3-8B experiments of the
 * same page use group-128 (Table 3, 4, 6 and 7 captions).  Rounding is
 * IEEE-754 round-to-nearest-even throughout; rint rounds ties to even.
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers (HIP global memory), owned and
 *     allocated by the caller, 16-byte aligned, row-major and densely packed.
 *     The library never allocates or frees memory.
 *   - bf16 and fp16 values travel as uint16_t bit patterns.
 *   - `stream` is a hipStream_t passed as void* (NULL: the null stream).
 *     Work is enqueued asynchronously on it; the call returns once enqueued.
 *   - Arguments are validated before anything is enqueued; on an error the
 *     call returns a negative HSQ_E_* code and enqueues nothing.  Faults that
 *     happen while kernels run surface at the caller's next synchronisation.
 *   - Debugging: with HSQ_DEBUG set in the environment (any value but "0"),
 *     every call that enqueues work waits for its stream before returning
 *     and reports a failure of its own kernels as HSQ_E_HIP, with
 *     hsq_last_hip_error() naming it.  While the stream is being captured
 *     into a graph the call does not wait (waiting is not allowed there).
 *   - The library keeps no state between calls (except the per-device
 *     scratch of hsq_w4a4_lowrank_linear_noalloc) and is thread-safe; no
 *     C++ exception crosses this interface.
 *   - Limits: K % 64 == 0 and K >= 64; M, N >= 1; 0 <= r <= 32;
 *     1 <= batch <= 16; M * K, M * N, K * N < 2^31; and, for the linear,
 *     16*ceil(M/16) * Kp < 2^32 and 16*ceil(N/16) * Kp < 2^32 with
 *     Kp = K rounded up to 128 (the padded int8 activation codes and the
 *     int8 part of the packed residual are addressed through 32-bit buffer
 *     resources).
 */
#ifndef HSQ_H
#define HSQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---- */
#define HSQ_OK            0
#define HSQ_E_INVAL      -1  /* null pointer, size out of range, bad dtype or kernel choice; the
                              * 16-bit linear, the norm, the layer with 16-bit activations and
                              * the 4-bit cache: an output over another operand */
#define HSQ_E_SHAPE      -2  /* K not a positive multiple of 64, a window outside the matrix, sizes
                              * that do not divide or that no kernel has (the 4-bit cache) */
#define HSQ_E_ALIGN      -3  /* a pointer is not 16-byte aligned */
#define HSQ_E_WORKSPACE  -4  /* workspace missing or smaller than the size function returns */
#define HSQ_E_HIP        -5  /* the HIP runtime refused a launch */
#define HSQ_E_SCRATCH    -6  /* hsq_w4a4_lowrank_linear_noalloc: the sizes need more
                                workspace than its static scratch holds */

/* ---- output dtypes ---- */
#define HSQ_F32   0
#define HSQ_BF16  1
#define HSQ_F16   2  /* the 16-bit linear, the layer normalisation, the layer with 16-bit
                      * activations and the 4-bit cache only */

/* ---- kernel choice for the residual contraction ---- */
#define HSQ_KERNEL_AUTO    0  /* SKINNY for M <= 64, TILED otherwise */
#define HSQ_KERNEL_TILED   1  /* LDS-tiled int8-MFMA kernel, one workgroup per output tile */
#define HSQ_GROUP_64     64
#define HSQ_GROUP_128   128

#define HSQ_KERNEL_SKINNY  2  /* weight-streaming kernel for M <= 64: the waves of a
                                 workgroup split K and reduce in a fixed order */

/* Version of the packed-weight layout written by hsq_pack_weights (2:
 * nibbles, then int8 operands; see hsq_packed_weight_bytes). */
int hsq_layout_version(void);

/* Static text for a status code (never NULL). */
const char *hsq_status_string(int status);

/* The HIP runtime's text for the error behind the last HSQ_E_HIP returned
 * on the calling host thread ("no HIP error" if there was none).  Static
 * storage, never NULL. */
const char *hsq_last_hip_error(void);

/* Bytes of one packed residual (K x N int4 codes) as hsq_pack_weights
 * writes it (layout version 2): Np * Kp / 2 bytes of nibbles followed by
 * Np * Kp bytes of the same codes as int8 operands, Np = N rounded up to
 * 16, Kp = K rounded up to 128; 3/2 * Np * Kp in all.  The weight-streaming
 * contraction for few tokens reads the nibbles (half a byte per weight);
 * the tiled contraction for many tokens moves the int8 operands into LDS
 * unchanged, which saves its vector ALU -- the unit that bounds it -- the
 * nibble unpacking.  Returns 0 if K or N is invalid. */
size_t hsq_packed_weight_bytes(int K, int N);

/* Pack residual codes into the layout the contraction kernels read.
 * Operation: the 4-bit residual Q(R) of W ~ L1*L2 + Q(R) (Deflating the
 * Hessian, abstract), group-64 (Table 1 caption).
 *   codes   in : K x N int8 (input channel x output channel), values in [-8, 7]
 *   packed  out: hsq_packed_weight_bytes(K, N) bytes; padding is zero codes
 *   d_status out: one device int; set to 0 (by a kernel: the call enqueues
 *                 kernels only, so it can be captured in a HIP graph),
 *                 then to 1 if any code lies outside [-8, 7] (that code's
 *                 low nibble is stored).  The caller reads it after
 *                 synchronising.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_HIP. */
int hsq_pack_weights(const int8_t *codes, int K, int N, uint8_t *packed, int *d_status,
                     void *stream);

/* Inverse of hsq_pack_weights (testing and inspection).
 *   packed in : hsq_packed_weight_bytes(K, N) bytes
 *   codes  out: K x N int8 in [-8, 7]
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_HIP. */
int hsq_unpack_weights(const uint8_t *packed, int K, int N, int8_t *codes, void *stream);

/* Smooth and quantize activations per token in 64-wide groups, and form the
 * rank-r down projection of the smoothed, unquantized activations (the
 * xh, sx, qx and U lines of the formula block above).
 *   X      in : M x K bf16
 *   lambda in : K fp16 smoothing factors (X is divided by them)
 *   L1     in : K x r bf16 (may be NULL when r == 0)
 *   qx     out: M x K/2 bytes; byte j of a row holds code 2j in its low
 *               nibble and code 2j+1 in its high nibble, two's complement
 *   sx     out: M x K/64 fp16 scales
 *   U      out: M x r fp32 (may be NULL when r == 0)
 * K <= 12288 for this entry point (HSQ_E_INVAL beyond).
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_HIP. */
int hsq_quantize_act(const uint16_t *X, int M, int K, const uint16_t *lambda,
                     const uint16_t *L1, int r, uint8_t *qx, uint16_t *sx, float *U,
                     void *stream);

/* Workspace bytes hsq_w4a4_lowrank_linear and hsq_w4a4_group_partials need
 * for these sizes (any kernel choice).  Returns 0 if a size is invalid. */
size_t hsq_workspace_bytes(int M, int K, int N, int r, int batch);

/* The fused W4A4 + rank-r linear layer, for `batch` projections that share
 * the input X and the smoothing factors (e.g. Q, K and V).  Computes Y of the
 * formula block above: one pass over X quantizes it and forms U, then the
 * int4 x int4 contraction keeps an int32 partial sum per 64-wide group,
 * rescales it by sx * sw in fp32, and adds U * L2 and the bias.
 *   X        in : M x K bf16
 *   lambda   in : K fp16
 *   packed_w in : batch blobs of hsq_packed_weight_bytes(K, N) bytes, back to back
 *   sw       in : batch x K/64 x N fp16 weight scales
 *   L1       in : batch x K x r bf16   (NULL when r == 0)
 *   L2       in : batch x r x N bf16   (NULL when r == 0)
 *   bias     in : batch x N bf16, or NULL for no bias
 *   Y        out: batch x M x N, fp32 (y_dtype HSQ_F32) or bf16 (HSQ_BF16, RNE)
 *   workspace   : ws_bytes >= hsq_workspace_bytes(M, K, N, r, batch) device
 *                 bytes, scratch owned by the caller; its contents on entry
 *                 do not matter and are clobbered.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_WORKSPACE, HSQ_E_HIP. */
int hsq_w4a4_lowrank_linear(const uint16_t *X, int M, int K, int N, int batch,
                            const uint16_t *lambda, const uint8_t *packed_w,
                            const uint16_t *sw, const uint16_t *L1, const uint16_t *L2, int r,
                            const uint16_t *bias, void *Y, int y_dtype, void *workspace,
                            size_t ws_bytes, void *stream);

/* As hsq_w4a4_lowrank_linear, with the contraction kernel chosen by
 * `kernel` (HSQ_KERNEL_*; SKINNY with M > 64 is HSQ_E_INVAL). */
int hsq_w4a4_lowrank_linear_ex(const uint16_t *X, int M, int K, int N, int batch,
                               const uint16_t *lambda, const uint8_t *packed_w,
                               const uint16_t *sw, const uint16_t *L1, const uint16_t *L2,
                               int r, const uint16_t *bias, void *Y, int y_dtype,
                               void *workspace, size_t ws_bytes, int kernel, void *stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * layer as hsq_w4a4_lowrank_linear (group 64, contraction kernel chosen
 * as for HSQ_KERNEL_AUTO), with its workspace in a static device array of
 * HSQ_NOALLOC_SCRATCH_BYTES (64 MiB) inside the library instead of a caller
 * buffer.  Every GPU the library runs on holds its own array until the
 * process ends; the first call on a device looks up that device's address
 * of it (no allocation).  The call uses the array of the CURRENT device
 * (hipGetDevice); `stream` must belong to that device.  The call allocates
 * and frees nothing.  All calls on one GPU share its array: calls that may
 * overlap in time on one GPU (two streams, two host threads without
 * ordering) race on it and must be serialised by the caller; calls in order
 * on one stream are safe.  No part of the array needs to start zeroed (the
 * quantization pass rewrites everything the contraction reads).
 * Sizes whose workspace (hsq_workspace_bytes(M, K, N, r, batch)) exceeds
 * the array return HSQ_E_SCRATCH before anything is enqueued; every
 * configuration of the diffusion and LLM layers here fits (the largest,
 * 4608 tokens x 12288 channels, needs about 64 MB).
 * Other arguments and errors as for hsq_w4a4_lowrank_linear. */
#define HSQ_NOALLOC_SCRATCH_BYTES (64u << 20)
int hsq_w4a4_lowrank_linear_noalloc(const uint16_t *X, int M, int K, int N, int batch,
                                    const uint16_t *lambda, const uint8_t *packed_w,
                                    const uint16_t *sw, const uint16_t *L1, const uint16_t *L2,
                                    int r, const uint16_t *bias, void *Y, int y_dtype,
                                    void *stream);

/* The same layer in two stages on one stream, for callers that time or
 * schedule them separately, or reuse one quantized input for several
 * contractions with the same (M, K, batch, r).
 *   hsq_w4a4_quantize_stage: the smoothing / quantization / U pass over X
 *     (X, lambda, L1 as for the linear) into `workspace`.
 *   hsq_w4a4_contract_stage: the residual contraction, rescale and U*L2 +
 *     bias epilogue (packed_w, sw, L2, bias, Y as for the linear), reading
 *     the workspace the quantize stage wrote for the same M, K, r and batch.
 * Running both equals hsq_w4a4_lowrank_linear_ex.  The workspace must not
 * be reused by another quantize stage until the contract stages that read it
 * have run (stream order guarantees this on one stream).
 * Errors: as hsq_w4a4_lowrank_linear_ex. */
int hsq_w4a4_quantize_stage(const uint16_t *X, int M, int K, int N, int batch,
                            const uint16_t *lambda, const uint16_t *L1, int r, void *workspace,
                            size_t ws_bytes, void *stream);
int hsq_w4a4_contract_stage(int M, int K, int N, int batch, const uint8_t *packed_w,
                            const uint16_t *sw, const uint16_t *L2, int r, const uint16_t *bias,
                            void *Y, int y_dtype, void *workspace, size_t ws_bytes, int kernel,
                            void *stream);

/* Test export: the per-group int32 partial sums P[m,n,g] (formula block
 * above) of one projection, produced by the same quantization pass and the
 * same contraction loop as hsq_w4a4_lowrank_linear_ex with this `kernel`,
 * with the rescaling epilogue replaced by a store of P.  Only the window
 * m in [m0, m0+mc), n in [n0, n0+nc) is written.
 *   X, lambda, packed_w : as for the linear (one projection)
 *   P        out: mc x nc x K/64 int32
 *   workspace   : as for the linear with batch = 1, r = 0
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE (window outside M x N), HSQ_E_ALIGN,
 *         HSQ_E_WORKSPACE, HSQ_E_HIP. */
int hsq_w4a4_group_partials(const uint16_t *X, int M, int K, int N, const uint16_t *lambda,
                            const uint8_t *packed_w, int m0, int mc, int n0, int nc,
                            int32_t *P, void *workspace, size_t ws_bytes, int kernel,
                            void *stream);

/* ---- the same layer with the group width as an argument ----
 * group is HSQ_GROUP_64 or HSQ_GROUP_128 (anything else: HSQ_E_INVAL) and
 * must divide K (HSQ_E_SHAPE otherwise).  Every scale array then has K/group
 * groups: sw is batch x K/group x N fp16, P is mc x nc x K/group int32.
 * The packed weights are the same for both widths (hsq_pack_weights).  With
 * group = 64 each function equals its counterpart above.  A group-128
 * scale covers two 64-channel blocks: the contraction accumulates their two
 * int32 block sums before the one rescale by sx * sw. */
size_t hsq_workspace_bytes_g(int M, int K, int N, int r, int batch, int group);
int hsq_w4a4_lowrank_linear_g(const uint16_t *X, int M, int K, int N, int batch, int group,
                              const uint16_t *lambda, const uint8_t *packed_w,
                              const uint16_t *sw, const uint16_t *L1, const uint16_t *L2,
                              int r, const uint16_t *bias, void *Y, int y_dtype,
                              void *workspace, size_t ws_bytes, int kernel, void *stream);
int hsq_w4a4_quantize_stage_g(const uint16_t *X, int M, int K, int N, int batch, int group,
                              const uint16_t *lambda, const uint16_t *L1, int r, void *workspace,
                              size_t ws_bytes, void *stream);
int hsq_w4a4_contract_stage_g(int M, int K, int N, int batch, int group, const uint8_t *packed_w,
                              const uint16_t *sw, const uint16_t *L2, int r, const uint16_t *bias,
                              void *Y, int y_dtype, void *workspace, size_t ws_bytes, int kernel,
                              void *stream);
int hsq_w4a4_group_partials_g(const uint16_t *X, int M, int K, int N, int group,
                              const uint16_t *lambda, const uint8_t *packed_w, int m0, int mc,
                              int n0, int nc, int32_t *P, void *workspace, size_t ws_bytes,
                              int kernel, void *stream);

/* ---- asymmetric activations ----
 * The activation format of the INT W4A4 setting in the DiRotQ notes
 * (papernotes.org, experimental setup): activations quantized per token and
 * group asymmetrically, weights symmetrically as above.  The notes print no
 * formula; this library reads it as the min-max quantizer with 16 levels
 * whose range is widened to contain 0 (so that 0 is a level):
 *   lo[m,g]  = min(0, min_{k in g} xh[m,k]),  hi[m,g] = max(0, max_{k in g} xh[m,k])
 *   sx[m,g]  = fp16_rne(fl32(fl32(hi - lo) / 15))   (0 if hi == lo; saturates at 65504)
 *   z[m,g]   = clamp(rint(fl32(-lo * fl32(1 / sx))), 0, 15)      zero point
 *   q[m,k]   = clamp(rint(fl32(xh * fl32(1 / sx))) + z, 0, 15)  (all 0 if sx = 0)
 *   qx[m,k]  = q[m,k] - z[m,g]                      in [-15, 15]
 * and P, U, Y as in the formula block (with this qx).  qx fits the int8
 * operand of the contraction, so both contraction kernels run unchanged.
 * act_quant is HSQ_AQ_SYMMETRIC (the formula block; each function then
 * equals its _g counterpart) or HSQ_AQ_ASYMMETRIC; anything else is
 * HSQ_E_INVAL.  Arguments, workspace and errors otherwise as for the _g
 * functions. */
#define HSQ_AQ_SYMMETRIC   0
#define HSQ_AQ_ASYMMETRIC  1
int hsq_w4a4_lowrank_linear_aq(const uint16_t *X, int M, int K, int N, int batch, int group,
                               int act_quant, const uint16_t *lambda, const uint8_t *packed_w,
                               const uint16_t *sw, const uint16_t *L1, const uint16_t *L2, int r,
                               const uint16_t *bias, void *Y, int y_dtype, void *workspace,
                               size_t ws_bytes, int kernel, void *stream);
int hsq_w4a4_quantize_stage_aq(const uint16_t *X, int M, int K, int N, int batch, int group,
                               int act_quant, const uint16_t *lambda, const uint16_t *L1, int r,
                               void *workspace, size_t ws_bytes, void *stream);
int hsq_w4a4_group_partials_aq(const uint16_t *X, int M, int K, int N, int group, int act_quant,
                               const uint16_t *lambda, const uint8_t *packed_w, int m0, int mc,
                               int n0, int nc, int32_t *P, void *workspace, size_t ws_bytes,
                               int kernel, void *stream);

/* ---- MX-fp4 format variant of the layer ----
 * The same layer (smoothing, rank-r branch on the smoothed activations,
 * bias) with both 4-bit operands of the residual product in MX-fp4 (OCP
 * Microscaling Formats v1.0) instead of int4 with fp16 group-64 scales: per
 * 32 consecutive values along K one e8m0 scale 2^X, X = floor(log2 amax) - 2
 * (stored as X + 127, clamped to [0, 254]; a zero block stores 127), and
 * e2m1 elements {0, 0.5, 1, 1.5, 2, 3, 4, 6} rounded to nearest (ties to the
 * even mantissa), magnitudes above 6 saturating; the code keeps the value's
 * sign bit, also where the magnitude rounds to 0 (-0, code 8).  The activations are
 * blocked per token, the residual per output column.  The product runs on
 * gfx950's scaled fp4 MFMA, which applies both scales.
 * hsq_mx_pack_weights: R (K x N fp32, the residual, row-major) -> packed
 *   (hsq_mx_packed_weight_bytes(K, N) bytes: codes in MFMA operand order,
 *   then the scales).
 * hsq_mx_lowrank_linear: Y (M x N, HSQ_F32 or HSQ_BF16) = Q(Xh) Q(R) +
 *   (Xh L1) L2 + bias; X, lambda, L1 (K x r), L2 (r x N), bias (N) as for
 *   hsq_w4a4_lowrank_linear with batch 1; workspace of
 *   hsq_mx_workspace_bytes(M, K, r) bytes.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE (K not a multiple of 64), HSQ_E_ALIGN,
 * HSQ_E_WORKSPACE, HSQ_E_HIP. */
size_t hsq_mx_packed_weight_bytes(int K, int N);
int hsq_mx_pack_weights(const float *R, int K, int N, uint8_t *packed, void *stream);
size_t hsq_mx_workspace_bytes(int M, int K, int r);
int hsq_mx_lowrank_linear(const uint16_t *X, int M, int K, int N, const uint16_t *lambda,
                          const uint8_t *packed_mx, const uint16_t *L1, const uint16_t *L2, int r,
                          const uint16_t *bias, void *Y, int y_dtype, void *workspace, size_t ws_bytes,
                          void *stream);

/* ---- fused two-layer chain: Y = down(act(up(X))) ----
 * Two linears of the kind above (group 64, one projection each, ranks r_up
 * and r_down) with an elementwise activation between them, as in the MLP
 * of a diffusion transformer block (FLUX.1: an up-projection of width H,
 * GELU, a down-projection; 3072 -> 12288 -> 3072 at its model width).  The
 * up layer's contraction does not write its output:
 * its epilogue applies the activation in fp32 and forms, from that fp32
 * value, the down layer's smoothed input, its group-64 scales and int4
 * codes (the quantizer of the formula block above, applied to
 * a[m,k] = act(Y_up[m,k]) instead of a bf16 X) and the partial sums of the
 * down layer's rank branch U_down = (a * fl32(1/lambda_down)) L1_down.
 * The down layer then runs its contraction on them: the hidden activation
 * never travels through HBM as a bf16 tensor and the down layer has no
 * quantization pass.
 *   act   HSQ_ACT_IDENTITY, or HSQ_ACT_GELU_TANH: the tanh form of GELU,
 *         0.5 y (1 + tanh(z)), z = 0.7978845608 (y + 0.044715 y^3), computed
 *         in fp32 as y / (1 + e(-2z)) with e(x) = p(r) * 2^n, n = rint(x *
 *         1.44269504), r = (x - n * 0.693145751953125) - n *
 *         1.428606765330187e-6, p the degree-6 Taylor polynomial of exp
 *         in Horner form, x clamped to [-87, 88], every operation rounded
 *         once (no fused multiply-add)
 *   Y          out: M x N, HSQ_F32 or HSQ_BF16
 *   Y_hidden   optional out (NULL: not written): M x H fp32, the up
 *              layer's output before the activation (a test export)
 *   r_down     0 .. 8; the up layer runs the tiled contraction unsplit
 * All other arguments as for hsq_w4a4_lowrank_linear, per layer.
 * Performance: on an MI355X this call is SLOWER than the two layers run
 * as separate hsq_w4a4_lowrank_linear calls (FLUX.1 MLP, 4608 tokens:
 * 0.70-0.71 ms fused vs 0.60-0.61 ms separate, the separate path without
 * any activation pass).  The up contraction is bound by its per-group VALU
 * rescale, and the fused epilogue adds about 50 VALU instructions per
 * output element (GELU, smoothing, absmax, codes, rank-r dot product) to
 * it, more than the bf16 round trip and quantization pass it removes.  Use
 * it where the hidden activation must not be materialised, not for speed.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE (K or H not a multiple of 64),
 * HSQ_E_ALIGN, HSQ_E_WORKSPACE, HSQ_E_HIP. */
#define HSQ_ACT_IDENTITY   0
#define HSQ_ACT_GELU_TANH  1
size_t hsq_mlp_workspace_bytes(int M, int K, int H, int N, int r_up, int r_down);
int hsq_w4a4_lowrank_mlp(const uint16_t *X, int M, int K, int H, int N, const uint16_t *lambda_up,
                         const uint8_t *packed_up, const uint16_t *sw_up, const uint16_t *L1_up,
                         const uint16_t *L2_up, int r_up, const uint16_t *bias_up, int act,
                         const uint16_t *lambda_down, const uint8_t *packed_down,
                         const uint16_t *sw_down, const uint16_t *L1_down, const uint16_t *L2_down,
                         int r_down, const uint16_t *bias_down, void *Y, int y_dtype, float *Y_hidden,
                         void *workspace, size_t ws_bytes, void *stream);

/* ---- calibration: the Hessian, its deflation, the closed-form L2 ----
 * The steps that produce a layer's factors (Deflating the Hessian, paper
 * page: abstract and Figure 1 caption; H-SVDQuant explainer, rit.work,
 * section on Hessian deflation).  The pages give no formulas; these follow
 * the plainest reading (the activation-noise surrogate term is left out):
 *
 *   H      = Xh^T Xh                     Xh[m,k] = X[m,k] * fl32(1/lambda[k]) (as above)
 *   C      = L1^T H L1                   r x r
 *   Hperp  = H - (H L1) C^-1 (H L1)^T     deflated Hessian: Hperp L1 = 0
 *   E      = W - deq(Q(R))               deq(Q(R))[k,n] = code[k,n] * sw[k/group, n]
 *   L2*    = C^-1 (H L1)^T E             the output-side factor minimising
 *                                        || Xh E - Xh L1 L2 ||_F
 *
 * Sizes: K a multiple of 64 with 64 <= K <= 16384 (HSQ_E_SHAPE / _INVAL),
 * 1 <= r <= 32.  H, Hperp are K x K fp32 row-major.  Pointers are device
 * pointers, 16-byte aligned; buffers are the caller's.  All arithmetic is
 * fp32 except C and its inverse (fp64); results are deterministic. */

/* Workspace of hsq_hessian_accumulate (0: none needed; also 0 for invalid
 * sizes).  Few 128 x 128 blocks of H (small K) split the tokens across
 * workgroups, whose fp32 partial blocks live here. */
size_t hsq_hessian_workspace_bytes(int M, int K);

/* H = Xh^T Xh (accumulate = 0) or H += Xh^T Xh (accumulate = 1), over the
 * M calibration tokens of X (M x K bf16, row-major) with the layer's
 * smoothing lambda (K fp16).  Both triangles of H are written.  Stream the
 * calibration set through several calls with accumulate = 1.
 * M * K < 2^30.  Errors: HSQ_E_INVAL (null pointer, sizes, accumulate not
 * 0/1), HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_WORKSPACE, HSQ_E_HIP. */
int hsq_hessian_accumulate(const uint16_t *X, int M, int K, const uint16_t *lambda, float *H,
                           int accumulate, void *workspace, size_t ws_bytes, void *stream);

/* Workspace of hsq_deflate_hessian (0 for invalid sizes). */
size_t hsq_deflate_workspace_bytes(int K, int r);

/* Deflates H by span(L1) (L1: K x r bf16, the layer's input-side factor):
 *   HL1   out: K x r fp32, H L1
 *   Cinv  out: r x r fp64, (L1^T H L1)^-1 (Gauss-Jordan, partial pivoting;
 *         a singular C gives NaN)
 *   Hperp out: K x K fp32; may be H itself (in place), must not otherwise
 *         overlap it.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_WORKSPACE,
 * HSQ_E_HIP. */
int hsq_deflate_hessian(const float *H, int K, const uint16_t *L1, int r, float *Hperp, float *HL1,
                        double *Cinv, void *workspace, size_t ws_bytes, void *stream);

/* Workspace of hsq_closed_form_l2 (0 for invalid sizes). */
size_t hsq_closed_form_l2_workspace_bytes(int K, int N, int r);

/* The closed-form output-side factor L2* = Cinv (HL1)^T E (r x N fp32 out)
 * from the outputs of hsq_deflate_hessian and one projection's weight:
 *   W        K x N bf16, the full-precision (smoothed) weight
 *   packed_w the packed residual codes of its quantized residual
 *            (hsq_pack_weights layout), sw its (K/group) x N fp16 scales
 *   group    HSQ_GROUP_64 or HSQ_GROUP_128 (must divide K)
 * E is decoded on the fly and never stored.  K * N < 2^31.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_WORKSPACE,
 * HSQ_E_HIP. */
int hsq_closed_form_l2(const float *HL1, const double *Cinv, int K, int N, int r, int group,
                       const uint16_t *W, const uint8_t *packed_w, const uint16_t *sw, float *L2,
                       void *workspace, size_t ws_bytes, void *stream);

/* ---- 16-bit linear layer with bias, activation and residual ----
 * The unquantized form of the layer, for the projections a W4A4 model keeps
 * in 16 bits and, with the gradients below, for training those and the norms
 * (the W4A4 layer itself has no gradient: a backward pass ends there unless the
 * caller gives the layer's dequantized weight to hsq_linear_backward):
 *
 *   Z[m,n] = sum_k X[m,k] W[k,n] + bias[n]
 *   Y[m,n] = act(Z[m,n]) + residual[m,n]
 *
 * with 16-bit operands, fp32 sums and an fp32 epilogue, rounded once at each
 * store.  Any M, K, N >= 1 with M * K, K * N, M * N < 2^30 (K and N
 * rounded up to 8 where they are row lengths) and K, N <= 2^24.
 *   X         in : M x K of `dtype` (HSQ_BF16 or HSQ_F16)
 *   W         in : K x N of `dtype` (input channel x output channel)
 *   bias      in : N of `dtype`, or NULL
 *   act          : HSQ_ACT_IDENTITY, HSQ_ACT_GELU_TANH, HSQ_ACT_GELU (0.5 z
 *                  (1 + erf(z / sqrt 2))) or HSQ_ACT_SILU (z / (1 + exp(-z)))
 *   residual  in : M x N of `y_dtype`, or NULL; may be Y itself
 *   Y         out: M x N of `y_dtype`, which is HSQ_F32 or `dtype`
 *   Z         out: M x N of `dtype`, or NULL: the values before the
 *                  activation, as hsq_linear_backward takes them
 *   workspace    : ws_bytes >= hsq_linear_workspace_bytes(M, K, N) device
 *                  bytes (NULL is fine where that is 0); its contents on
 *                  entry do not matter and are clobbered, here as in the
 *                  three functions below: calls in order may share one,
 *                  calls that overlap in time need one each
 * No output (the workspace among them) may overlap another operand, except Y
 * the residual, all of it: HSQ_E_INVAL.  Results do not
 * depend on earlier calls or on timing: sums run in a fixed order.
 * Errors: HSQ_E_INVAL, HSQ_E_ALIGN, HSQ_E_WORKSPACE, HSQ_E_HIP. */
#define HSQ_ACT_GELU       2  /* the 16-bit linear only */
#define HSQ_ACT_SILU       3  /* the 16-bit linear only */
size_t hsq_linear_workspace_bytes(int M, int K, int N);
int hsq_linear(const uint16_t *X, int M, int K, int N, int dtype, const uint16_t *W,
               const uint16_t *bias, int act, const void *residual, void *Y, int y_dtype,
               uint16_t *Z, void *workspace, size_t ws_bytes, void *stream);

/* Its backward pass, from dY = dL/dY:
 *
 *   dZ = dY * act'(Z)      dX = dZ W^T      dW = X^T dZ      dbias[n] = sum_m dZ[m,n]
 *
 * (dL/dresidual is dY itself.)  dZ is rounded to `dtype` as the operand of
 * the two products, an fp32 dY too; dbias sums the unrounded dZ.  In HSQ_F16
 * a dZ of 2^-25 and less counts as 0 in dX and dW, one below 2^-14 keeps fewer
 * bits, and one of 65520 and more is infinite: scale the loss by a power of two,
 * which changes nothing else, to keep it in between.
 *   dY      in : M x N of `y_dtype` (HSQ_F32 or `dtype`)
 *   X, W    in : as for hsq_linear
 *   Z       in : M x N of `dtype`, from hsq_linear (ignored and may be NULL
 *                for HSQ_ACT_IDENTITY)
 *   dX      out: M x K of `dtype`, or NULL: not wanted
 *   dW      out: K x N of `dtype`, or NULL: not wanted
 *   dbias   out: N of `dtype`, or NULL: not wanted
 *   workspace  : ws_bytes >= hsq_linear_backward_workspace_bytes(M, K, N)
 * W may be NULL where dX is, X where dW is; one output at least is wanted.
 * No output (the workspace among them) may overlap another operand that the
 * call reads or writes: HSQ_E_INVAL.
 * Errors: HSQ_E_INVAL, HSQ_E_ALIGN, HSQ_E_WORKSPACE, HSQ_E_HIP. */
size_t hsq_linear_backward_workspace_bytes(int M, int K, int N);
int hsq_linear_backward(const void *dY, int y_dtype, const uint16_t *X, int M, int K, int N,
                        int dtype, const uint16_t *W, const uint16_t *Z, int act, uint16_t *dX,
                        uint16_t *dW, uint16_t *dbias, void *workspace, size_t ws_bytes,
                        void *stream);

/* ---- layer normalisation ----
 * The norm before the layer, per row of X over its C channels:
 *
 *   mean = (1/C) sum_c x[c]     rstd = ((1/C) sum_c (x[c] - mean)^2 + eps)^(-1/2)
 *   y[c] = (x[c] - mean) * rstd * weight[c] + bias[c]
 *
 * weight and bias are given per group of M / groups consecutive rows: groups =
 * 1 is the usual affine norm, one group per image the modulated norm of a
 * diffusion transformer (weight = 1 + scale, bias = shift).
 *   X        in : M x C of x_dtype (HSQ_F32, HSQ_BF16, HSQ_F16)
 *   weight   in : groups x C of p_dtype, or NULL (1)
 *   bias     in : groups x C of p_dtype, or NULL (0)
 *   Y        out: M x C of y_dtype; may be X itself where the types are equal
 *   mean,
 *   rstd     out: M fp32 each, or NULL: as the backward pass takes them
 * y_dtype is x_dtype, or any of the three where x_dtype is HSQ_F32; p_dtype
 * is HSQ_F32 or y_dtype.  1 <= C <= 16384, groups divides M (HSQ_E_SHAPE)
 * and is at most 65535, M <= 2^25, M * C < 2^31; eps is finite and not
 * negative.
 * No other output may overlap another operand: HSQ_E_INVAL.
 * Arithmetic is fp32, the variance taken around the finished mean: a row whose
 * squared differences do not sum within fp32 has rstd 0.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_HIP. */
int hsq_layer_norm(const void *X, int x_dtype, int M, int C, int groups, const void *weight,
                   const void *bias, int p_dtype, float eps, void *Y, int y_dtype, float *mean,
                   float *rstd, void *stream);

/* Its backward pass, from dY = dL/dY, with xh = (x - mean) * rstd and
 * g = dy * weight:
 *
 *   dx = rstd (g - mean_c(g) - xh mean_c(g xh))
 *   dweight[c] = sum over the group's rows of dy xh,   dbias[c] = sum of dy
 *
 *   dY       in : M x C of y_dtype       X, weight, mean, rstd in: as above
 *   dX       out: M x C of x_dtype, or NULL: not wanted
 *   dweight,
 *   dbias    out: groups x C of p_dtype, or NULL: not wanted
 *   workspace   : ws_bytes >= hsq_layer_norm_backward_workspace_bytes(M, C,
 *                 groups) (NULL is fine where neither dweight nor dbias is wanted)
 * One output at least is wanted; no output (the workspace among them) may
 * overlap another operand: HSQ_E_INVAL.  Sums run in a fixed order.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_WORKSPACE, HSQ_E_HIP. */
size_t hsq_layer_norm_backward_workspace_bytes(int M, int C, int groups);
int hsq_layer_norm_backward(const void *dY, int y_dtype, const void *X, int x_dtype, int M, int C,
                            int groups, const float *mean, const float *rstd, const void *weight,
                            int p_dtype, void *dX, void *dweight, void *dbias, void *workspace,
                            size_t ws_bytes, void *stream);

/* ---- the layer with its activations left in 16 bits, for few tokens ----
 * The same weights (packed residual, scales, lambda, L1, L2, bias) under
 * activations that are not quantized: the weight-only form, for decoding,
 * where the read of the weights is all that counts.
 *
 *   xh[m,k] = X[m,k] / lambda[k]
 *   Y[m,n]  = sum_g sw[g,n] sum_{k in g} xh[m,k] qw[k,n]
 *             + sum_j (sum_k xh[m,k] L1[k,j]) L2[j,n] + bias[n] + residual[m,n]
 *
 *   X         in : M x K of `dtype` (HSQ_BF16 or HSQ_F16), 1 <= M <= 64
 *   group        : 64 or 128, divides K
 *   lambda    in : K fp16, or NULL: 1
 *   packed_w  in : batch blobs of hsq_pack_weights, back to back
 *   sw        in : batch x K/group x N fp16
 *   L1, L2    in : batch x K x r and batch x r x N of `dtype` (NULL where r = 0)
 *   bias      in : batch x N of `dtype`, or NULL
 *   residual  in : batch x M x N of `y_dtype`, or NULL; may be Y itself
 *   Y         out: batch x M x N of `y_dtype`, which is HSQ_F32 or `dtype`
 *   workspace    : ws_bytes >= hsq_w4a16_workspace_bytes(M, K, N, r, batch,
 *                  group, lambda != NULL, y_dtype) device bytes (NULL is fine
 *                  where that is 0); its contents on entry do not matter, and
 *                  calls that overlap in time need one each
 * Products and sums are fp32, rounded once at the store.  With lambda, xh enters
 * them as fp16 numbers under a power of two per row and group: 11 bits where Y is
 * bf16, 22 bits where it is fp16 or fp32; and the terms of their sums are cut at
 * 2^-14, or 2^-20, of the row's largest |xh| in the group.  A row of xh that
 * holds an infinity or a NaN gives NaN; one whose 31 |xh| do not sum within
 * fp32 over a group may.  Sizes as for the linear (K % 64, r, batch), with
 * M * K, M * N, K * N < 2^31.  No output (the workspace among them) may overlap
 * another operand, except Y the residual, all of it: HSQ_E_INVAL.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE, HSQ_E_ALIGN, HSQ_E_WORKSPACE, HSQ_E_HIP. */
#define HSQ_W4A16_MAX_M 64
size_t hsq_w4a16_workspace_bytes(int M, int K, int N, int r, int batch, int group, int smooth, int y_dtype);
int hsq_w4a16_lowrank_linear(const uint16_t *X, int M, int K, int N, int batch, int group, int dtype,
                             const uint16_t *lambda, const uint8_t *packed_w, const uint16_t *sw,
                             const uint16_t *L1, const uint16_t *L2, int r, const uint16_t *bias,
                             const void *residual, void *Y, int y_dtype, void *workspace,
                             size_t ws_bytes, void *stream);

/* ---- key / value cache in 4 bits ----
 * Keys and values of a decoder's attention, quantized as they are written.  Per
 * token, head and group of 64 channels x:
 *
 *   HSQ_AQ_ASYMMETRIC  lo = min(0, min x), hi = max(0, max x)
 *                      s = fp16_rne((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15)
 *                      n = clamp(rint(x / s) + z, 0, 15)
 *   HSQ_AQ_SYMMETRIC   s = fp16_rne(max |x| / 7), z = 8
 *                      n = clamp(rint(x / s), -8, 7) + 8
 *
 * and the value held is s (n - z).  The quotients are those of the real numbers,
 * ties to even; s saturates at 65504, and s = 0 holds zeros; a group with an
 * infinity or a NaN holds NaN.
 *
 * The cache is a device buffer of num_pages pages of hsq_kv_page_bytes(
 * page_size, kv_heads, head_dim) bytes, 16-byte aligned, in a layout of the
 * library's own (it can be copied page by page).  head_dim is 64, 128 or 256;
 * page_size, in tokens, a power of two from 32 to 2^20.  Every call says where the
 * sequences lie by
 *   block_table in : batch x table_width int32, position t of sequence b is on
 *                    page block_table[b][t / page_size]
 *   kv_lens     in : batch int32, tokens of each sequence, the call's own included
 *   cu_tokens   in : batch + 1 int32, sequence b's rows of the call are
 *                    [cu_tokens[b], cu_tokens[b+1]) of T; or NULL: T / batch rows
 *                    each.  Its n rows are positions kv_lens[b] - n and on.
 *   max_tokens     : no sequence has more rows (a bound, which may be above T;
 *                    ignored where cu_tokens is NULL);
 *                    rows beyond it are left alone
 * (these three arrays are 4-byte aligned).  They are read on the device only, and
 * whatever they hold, no access leaves the operands: a position that is
 * negative, at or past table_width * page_size, or on a page that is not in [0,
 * num_pages), is not there: it is not written, reads back as 0, and takes no part
 * in the attention.  Rows of no sequence are left as they were.  Two rows of one
 * call must not be written to the same place (a page named twice).
 * Limits: batch <= 65535, heads <= 4096, T <= 2^24, table_width * page_size <=
 * 2^30, batch * max_tokens < 2^36, and launches of fewer than 2^23 workgroups (which
 * follow T, not batch * max_tokens, where that is a loose bound): HSQ_E_INVAL.
 * Strides are in elements from row to row, multiples of 8 and no less than a dense
 * row; the heads of a row are dense. */
size_t hsq_kv_page_bytes(int page_size, int kv_heads, int head_dim);

/* Writes T rows of keys and values (T x kv_heads x head_dim, HSQ_BF16 or HSQ_F16,
 * row strides k_stride and v_stride) into the cache.  quant is HSQ_AQ_SYMMETRIC or
 * HSQ_AQ_ASYMMETRIC; a cache may hold both.  The cache may not overlap K or V.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE (head_dim, page_size, T not a multiple of
 * batch where cu_tokens is NULL, a stride), HSQ_E_ALIGN, HSQ_E_HIP. */
int hsq_kv_cache_write(const uint16_t *K, int k_stride, const uint16_t *V, int v_stride, int T, int dtype,
                       int kv_heads, int head_dim, int quant, uint8_t *cache, int num_pages, int page_size,
                       const int32_t *block_table, int table_width, const int32_t *kv_lens,
                       const int32_t *cu_tokens, int batch, int max_tokens, void *stream);

/* Reads back the values held of the rows that a write with the same arguments
 * writes (any stretch of a sequence: kv_lens is where it ends): K and V, T x
 * kv_heads x head_dim dense, of dtype HSQ_F32, HSQ_BF16 or HSQ_F16, one rounding.
 * Neither may overlap the other or the cache.  Errors as hsq_kv_cache_write. */
int hsq_kv_cache_read(const uint8_t *cache, int num_pages, int page_size, int kv_heads, int head_dim,
                      const int32_t *block_table, int table_width, const int32_t *kv_lens,
                      const int32_t *cu_tokens, int batch, int T, int max_tokens, void *K, void *V,
                      int dtype, void *stream);

/* Attention of T query rows over the cache:
 *
 *   e[i,t] = scale q_i . k_t        y_i = sum_t exp(e[i,t]) v_t / sum_t exp(e[i,t])
 *   lse[i] = log sum_t exp(e[i,t])
 *
 * per query head h, over head h / (q_heads / kv_heads) of the cache.  Row i of a
 * sequence's n is at position kv_lens[b] - n + i and sees, with causal = 1, the
 * tokens that are not after it and, where window > 0, less than window before it;
 * with causal = 0 (window 0) all kv_lens[b] tokens.  A row that sees nothing is 0
 * with lse = -infinity; what it does not see has no part in it, NaN either.
 *   Q       in : T x q_heads x head_dim of `dtype` (HSQ_BF16 or HSQ_F16), row
 *                stride q_stride
 *   scale      : positive, 1e30 at most; where it takes a row's largest |q| to 2^122
 *                or beyond, that row's lse is cut (Y, of finite scores, is not affected)
 *   Y       out: T x q_heads x head_dim dense of y_dtype (HSQ_F32 or `dtype`)
 *   lse     out: T x q_heads fp32, or NULL
 *   workspace  : ws_bytes >= hsq_kv_attention_workspace_bytes(T, q_heads,
 *                kv_heads, head_dim, batch, max_tokens, table_width * page_size)
 *                device bytes (NULL is fine where that is 0); contents do not
 *                matter; calls that overlap in time need one each
 * (max_tokens is T / batch where cu_tokens is NULL.)  The scores are fp32 sums,
 * whose terms q n of a group of 64 channels are cut at 2^-20 of the row's largest |q|;
 * exp(e) times a value's scale is rounded to 11 bits for a bf16 Y, to 22 for fp16 and fp32,
 * neither finer than 2^-32 of the row's largest over all groups of 64 channels (so a group
 * whose scales are 2^-10 of another's loses bits of an fp32 Y, 2^-21 of a 16-bit one, and
 * is 0 below 2^-33);
 * and the terms of the sums of values are cut at 2^-14, or 2^-20, of the group's largest.
 * Results do not depend on timing: sums run in a fixed order.  No output (the
 * workspace among them) may overlap another operand: HSQ_E_INVAL.
 * Errors: HSQ_E_INVAL, HSQ_E_SHAPE (as above, or kv_heads does not divide
 * q_heads), HSQ_E_ALIGN, HSQ_E_WORKSPACE, HSQ_E_HIP. */
size_t hsq_kv_attention_workspace_bytes(int T, int q_heads, int kv_heads, int head_dim, int batch,
                                        int max_tokens, int capacity);
int hsq_kv_attention(const uint16_t *Q, int q_stride, int T, int dtype, int q_heads, const uint8_t *cache,
                     int num_pages, int page_size, int kv_heads, int head_dim, const int32_t *block_table,
                     int table_width, const int32_t *kv_lens, const int32_t *cu_tokens, int batch,
                     int max_tokens, float scale, int causal, int window, void *Y, int y_dtype, float *lse,
                     void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* HSQ_H */
