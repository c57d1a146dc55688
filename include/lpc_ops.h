/*
 * lpc_ops.h -- the training and serving operators of liblpc.so that stand next
 * to the low-precision collectives: what a rank computes with the E4M3 rows an
 * all-to-all delivers (the FP8 block-scaled product, for one weight or for one
 * weight per expert, and its backward pass), what decides where rows go (the
 * expert router), what follows the gradient allreduce (AdamW, and Muon for
 * matrices), and the same experts' layers in bf16 (products and their backward
 * pass) and with weights in microscaled 4-bit floating point.
 *
 * Formats are those of lpc.h: E4M3FN codes, one FP32 scale s = absmax/448 per
 * 128 elements, code = E4M3(fl32(x / s)), a block whose scale is zero has all
 * codes 0x00.  A weight has one scale per 128 x 128 tile.
 *
 * Conventions are those of lpc.h: device pointers unless said otherwise, the
 * caller owns every buffer, nothing is allocated and no state is kept, work is
 * enqueued on `stream`, arguments are checked on the host before anything is
 * enqueued (dtype LPC_ERR_DTYPE, then nothing to do LPC_OK, null pointers
 * LPC_ERR_NULL, alignment LPC_ERR_ALIGN, shape LPC_ERR_SHAPE; 16-byte alignment
 * of every pointer but a mask's, any, and those to row counts and to single
 * numbers (loss, dloss, grad_scale), 4 bytes), a refused launch, one of 2^32
 * lanes or more among them, is LPC_ERR_HIP.  Values that a call reads from
 * device memory (row counts, expert indices) are checked by the kernels:
 * one out of range reads and writes nothing out of bounds.  Outputs must not
 * overlap inputs unless a call says otherwise.  Every result is the same from
 * call to call: no sum depends on the order in which workgroups run.
 *
 * Inputs must be finite (router logits may also be -infinity), and so must the
 * sums; otherwise the affected results are unspecified.  The FP8 products
 * multiply a block's two scales first, rounded to FP32: that must be finite too,
 * also where the block's sum is small or zero, and where it is below 2^-126 it
 * has a denormal's precision, which changes a result by at most 2^-125 a block.
 */
#ifndef LPC_OPS_H
#define LPC_OPS_H

#include "lpc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LPC_MAX_GROUPS 1024    /* weights of one grouped product */
#define LPC_MAX_EXPERTS 1024   /* experts of one router */
#define LPC_MAX_TOPK 16        /* experts a row is sent to */
#define LPC_MAX_ROW ((size_t)1 << 28)      /* n and k of bf16 and MXFP4 products are below this */
#define LPC_MAX_MATRIX ((size_t)1 << 40)   /* elements of one matrix operand */

/* ---------------------------------------------------------------------- */
/* FP8 block-scaled product                                                 */
/* ---------------------------------------------------------------------- */

/* out[r, j] = sum over blocks b of 128 of
 *   xs[r, b] * ws[g, j/128, b] * (sum over i in b of x[r, i] * w[g, j, i])
 * for the group g that row r belongs to, rounded once to out_t.
 *   FP32 out: products and sums are held in FP32; off by at most
 *      (128 + k/128 + 4) 2^-23 of the sum of the terms' magnitudes.
 *   BF16 out: the FP8 matrix instruction, twice as fast, holds less.  Of each 8
 *      neighbouring elements (0..7, 8..15, ...) it cuts every product of two
 *      codes towards zero to a multiple of 2^(E-13) before it adds them, E
 *      being the largest sum of two codes' exponents among the 8 (products of
 *      zero left out, codes below 2^-6 counted as 2^-6); all other sums are
 *      FP32.  Eight products are thus off by less than 7 * 2^(E-13) together,
 *      which is below 2^-10 of the largest of them where no code is below 2^-6.
 *      On normally distributed data that is 1.3e-5 of a block's sum (2-norm),
 *      1/100 of what rounding to BF16 adds; where large products cancel it can
 *      be all that is left (448*448 - 448*448 + 6*(1*1) gives 0).  A caller who
 *      needs such sums asks for FP32 out.
 *   x  [rows, k] codes, xs [rows, k/128]: rows quantized by lpc_quantize_fp8,
 *      lpc_quantize_fp8_rows or received through an all-to-all
 *   w  [groups, n, k] codes, ws [groups, ceil(n/128), k/128]
 *   counts [groups] rows of each group; group g's rows follow group g-1's.  May
 *      be NULL when groups == 1 (all rows).  A negative count is taken as 0,
 *      and groups end at `rows`; rows past the last group give zeros.
 *   out [rows, n] of type out_t
 *   k a positive multiple of 128; any n; rows, k, n < 2^31, groups in
 *   1..LPC_MAX_GROUPS, each matrix at most LPC_MAX_MATRIX elements (else
 *   LPC_ERR_SHAPE).  rows == 0 or n == 0: LPC_OK, no work.
 * The gradient of the rows is the same call on the incoming gradient's row
 * codes and the weight's codes with rows and columns exchanged.              */
lpc_status lpc_gemm_fp8(const uint8_t *x, const float *xs, size_t rows, size_t k,
                        const uint8_t *w, const float *ws, size_t n,
                        int groups, const int32_t *counts,
                        void *out, lpc_dtype out_t, hipStream_t stream);

/* Rows of the padded layout that the two calls below write and
 * lpc_gemm_fp8_wgrad reads: each group starts at a multiple of 128, after the
 * groups before it rounded up to 128.  The result depends on the sizes alone
 * and is enough for any counts: 128 * (ceil(rows/128) + groups - 1), or 0 when
 * rows == 0, rows >= 2^31 (which every call refuses) or groups < 1.  No HIP
 * call.                                                                      */
size_t lpc_padded_rows(size_t rows, int groups);

/* Quantize a matrix along its columns, and in the same pass along its rows:
 * the two forms of an incoming gradient that the backward pass of
 * lpc_gemm_fp8 multiplies.
 *   y [rows, n] of type `in`; n a multiple of 128
 *   codes_t [n, P] with P = lpc_padded_rows(rows, groups): column j of y as
 *      codes, one scale per 128 rows of a group; a group's last block is filled
 *      up with zeros.  scales_t [P/128, n].  Blocks past the last group's are
 *      not written.
 *   codes [rows, n], scales [rows, n/128]: lpc_quantize_fp8's result for the
 *      rows that belong to a group (others are not written).  Both NULL: not
 *      computed; only one NULL: LPC_ERR_NULL.
 *   groups, counts as for lpc_gemm_fp8                                       */
lpc_status lpc_quantize_fp8_cols(const void *y, lpc_dtype in, size_t rows, size_t n,
                                 int groups, const int32_t *counts,
                                 uint8_t *codes_t, float *scales_t,
                                 uint8_t *codes, float *scales, hipStream_t stream);

/* The same for rows that are held as codes already: column j of the values
 * fl32(E4M3(x[r, j]) * xs[r, j/128]), quantized along the column.            */
lpc_status lpc_requantize_fp8_cols(const uint8_t *x, const float *xs, size_t rows, size_t k,
                                   int groups, const int32_t *counts,
                                   uint8_t *codes_t, float *scales_t, hipStream_t stream);

/* Gradient of the weights: dw[g, j, i] = sum over the blocks b of group g's
 * padded rows of ys[b, j] * xs[b, i] * (sum over r in b of yt[j, r] * xt[i, r]).
 *   yt [n, P], ys [P/128, n]; xt [k, P], xs [P/128, k]: the column forms of the
 *      incoming gradient and of the rows, P = lpc_padded_rows(rows, groups)
 *   dw [groups, n, k] FP32, products and sums held as for an FP32 out of
 *      lpc_gemm_fp8; zeros for a group without rows
 *   any n and k; rows == 0 writes zeros (yt, ys, xt and xs may then be NULL). */
lpc_status lpc_gemm_fp8_wgrad(const uint8_t *yt, const float *ys, size_t n,
                              const uint8_t *xt, const float *xs, size_t k,
                              size_t rows, int groups, const int32_t *counts,
                              float *dw, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Expert router                                                            */
/* ---------------------------------------------------------------------- */

/* Device workspace of lpc_router_forward, in bytes, for these sizes (0 where
 * none is needed or the sizes are refused).  No HIP call.                    */
size_t lpc_router_workspace_bytes(size_t rows, int experts);

/* For each row: p = softmax of the logits, the topk experts of the largest
 * logits (ties to the lowest index, in descending order) and their gates, p or,
 * with normalize != 0, p over the sum of the chosen p.  Over the rows:
 *   valid     rows that mask keeps and that have a logit above -infinity
 *   counts[e] rows that chose e
 *   load[e]   sum of p[., e] over max(valid, 1)
 *   slope[e]  coef * E * counts[e] / (max(valid, 1) * topk) / max(valid, 1), the
 *             derivative of loss by each p[., e], the counts held fixed
 *   loss[0]   sum over e of coef * E * load[e] * counts[e] / (max(valid, 1) * topk)
 * A logit of -infinity (or NaN) is an expert the row may not use: p = 0, never
 * chosen.  A row that is not valid chooses nothing and counts nowhere.  Slots
 * left without an expert have index -1 and gate 0.  exp is good to 2 units in
 * the last place; a p below 2^-125 is zero or denormal.
 *   logits [rows, experts] of type `in`; mask [rows] uint8 or NULL (keep all)
 *   out_experts [rows, topk] int32, gates [rows, topk]
 *   counts [experts] int32, load [experts], slope [experts], loss [1]
 *   workspace  at least lpc_router_workspace_bytes, no initial contents needed;
 *      NULL where that is 0
 *   experts in 1..LPC_MAX_EXPERTS, topk in 1..min(experts, LPC_MAX_TOPK),
 *   rows < 2^31 (else LPC_ERR_SHAPE).  rows == 0: counts, load, slope and loss
 *   are zero (logits, out_experts and gates may be NULL).                    */
lpc_status lpc_router_forward(const void *logits, lpc_dtype in, size_t rows, int experts, int topk,
                              int normalize, float coef, const uint8_t *mask,
                              int32_t *out_experts, float *gates, int32_t *counts,
                              float *load, float *slope, float *loss,
                              void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Gradient of the logits: of the gates by dgates, and of the loss by dloss
 * through slope.  Recomputes p; takes experts, slope and the arguments of the
 * forward call.  A slot whose index is outside [0, experts), or whose logit is
 * not allowed, is an empty slot.  A row's indices must differ.
 *   out_experts [rows, topk], dgates [rows, topk], slope [experts], dloss [1]
 *   dlogits [rows, experts] of type `in`; zero where a logit is -infinity and
 *   in rows that are not valid.  rows == 0: LPC_OK, no work.                 */
lpc_status lpc_router_backward(const void *logits, lpc_dtype in, size_t rows, int experts, int topk,
                               int normalize, const uint8_t *mask,
                               const int32_t *out_experts, const float *slope,
                               const float *dgates, const float *dloss,
                               void *dlogits, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* AdamW over many tensors                                                  */
/* ---------------------------------------------------------------------- */

/* One tensor of a step: n elements, any count.  Device pointers, 16-byte
 * aligned.
 *   param  FP32, updated in place;  grad  of the plan's type, read
 *   state_bits 32: m and v are FP32, the scale pointers are not used
 *   state_bits 8:  m and v are E4M3 codes [n] with one scale per 128 elements
 *                  [ceil(n/128)]; v holds the SQUARE ROOT of the second moment,
 *                  and a positive root keeps a code above zero
 *   copy   bf16 copy of the updated param, or NULL in every tensor           */
typedef struct {
    float *param;
    const void *grad;
    void *m;
    void *v;
    float *m_scales;
    float *v_scales;
    uint16_t *copy;
    size_t n;
} lpc_adamw_tensor;

/* Bytes of the plan of these tensors.  tensors: host array; 0 for no work, for
 * sizes that are refused and for NULL.  No HIP call.                         */
size_t lpc_adamw_plan_bytes(const lpc_adamw_tensor *tensors, int count);

/* Check the tensors and write the plan to HOST memory (`plan`, of
 * lpc_adamw_plan_bytes bytes); the caller copies it to a 16-byte aligned device
 * buffer and keeps it as long as the tensors stay where they are.
 *   *chunks  workgroups of a step, given to lpc_adamw_step
 *   state_bits 8 or 32 (else LPC_ERR_DTYPE).  Tensors with n == 0 are left out.
 *   Tensors must not overlap.                                                */
lpc_status lpc_adamw_plan(const lpc_adamw_tensor *tensors, int count, lpc_dtype grad_t, int state_bits,
                          void *plan, size_t plan_bytes, size_t *chunks);

/* One step over every tensor of a plan, one launch:
 *   g = grad * grad_scale[0] (grad_scale NULL: 1)
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - lr weight_decay)
 *           - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in FP32, every operation rounded on its own; the scalars in front are
 * computed in double and rounded once.
 *   plan      DEVICE copy of the plan;  chunks, grad_t, state_bits as planned
 *   step >= 1, beta1 and beta2 in [0, 1) (else LPC_ERR_SHAPE)                */
lpc_status lpc_adamw_step(const void *plan, size_t chunks, lpc_dtype grad_t, int state_bits,
                          int64_t step, double lr, double beta1, double beta2, double eps,
                          double weight_decay, const float *grad_scale, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* bf16 products                                                            */
/* ---------------------------------------------------------------------- */

/* out[r, j] = sum over i of x[r, i] * w[g, j, i] for the group g that row r
 * belongs to, rounded once to out_t.  Products are exact and sums are held in
 * FP32: off by at most 2 k 2^-24 of the sum of the terms' magnitudes, and by
 * 2 k 2^-149 where these are below FP32's normal numbers.
 *   x [rows, k], w [groups, n, k] bf16; out [rows, n] of type out_t
 *   counts as for lpc_gemm_fp8: group g's rows follow group g-1's, a negative
 *      count is taken as 0, groups end at `rows`, rows past the last group give
 *      zeros; may be NULL when groups == 1
 *   k a positive multiple of 8; any n; k, n < LPC_MAX_ROW, rows < 2^31,
 *   groups in 1..LPC_MAX_GROUPS, each matrix at most LPC_MAX_MATRIX elements,
 *   and of the result at most 2^23 - 512 tiles of 256 x 256, where each group's rows
 *   count as whole tiles (else LPC_ERR_SHAPE).  rows == 0 or n == 0: LPC_OK, no
 *   work.                                                                    */
lpc_status lpc_gemm_bf16(const uint16_t *x, size_t rows, size_t k,
                         const uint16_t *w, size_t n, int groups, const int32_t *counts,
                         void *out, lpc_dtype out_t, hipStream_t stream);

/* Gradient of the rows: dx[r, i] = sum over j of dy[r, j] * w[g, j, i], of the
 * weight as it lies; rows past the last group give zeros.
 *   dy [rows, n], w [groups, n, k] bf16; dx [rows, k] of type out_t
 *   n and k positive multiples of 8 (else LPC_ERR_SHAPE), the rest as above.
 *   rows == 0 or k == 0: LPC_OK, no work.                                    */
lpc_status lpc_gemm_bf16_dgrad(const uint16_t *dy, size_t rows, size_t n,
                               const uint16_t *w, size_t k, int groups, const int32_t *counts,
                               void *dx, lpc_dtype out_t, hipStream_t stream);

/* Gradient of the weights: dw[g, j, i] = sum over the rows r of group g of
 * dy[r, j] * x[r, i]; zeros for a group without rows.
 *   dy [rows, n], x [rows, k] bf16; dw [groups, n, k] of type out_t
 *   n and k multiples of 8 (else LPC_ERR_SHAPE), the rest as above, with the
 *   tiles of each dw[g] by itself.  n == 0 or k == 0: LPC_OK, no work; rows == 0
 *   writes zeros (dy and x may then be NULL).                                */
lpc_status lpc_gemm_bf16_wgrad(const uint16_t *dy, size_t n, const uint16_t *x, size_t k,
                               size_t rows, int groups, const int32_t *counts,
                               void *dw, lpc_dtype out_t, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Microscaled 4-bit floating point (MXFP4)                                 */
/* ---------------------------------------------------------------------- */

/* The OCP format: E2M1 codes (sign, then magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6),
 * two to a byte, the first of the two in the low bits, and per 32 elements an
 * exponent byte e for the scale 2^(e-127).  For n elements: codes [n/2] and
 * scales [n/32].                                                             */

/* scale = 2^(floor(log2(absmax of the 32)) - 2), no less than 2^-127 (which a
 * block of zeros gets); code = E2M1(x / scale), to nearest, ties to even, what
 * is above 5 to 6.
 *   x [n] of type `in`; n a multiple of 32, at most LPC_MAX_MATRIX (else
 *   LPC_ERR_SHAPE).  A matrix's rows are quantized by one call if their length
 *   is a multiple of 32.  n == 0: LPC_OK, no work.                           */
lpc_status lpc_quantize_mxfp4(const void *x, lpc_dtype in, size_t n,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream);

/* out[i] = E2M1 value of code i times its block's scale, rounded to out_t
 * (exact but for what lies below out_t's normal numbers).  Bytes as
 * lpc_quantize_mxfp4 writes them, 0 to 252.                                  */
lpc_status lpc_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, size_t n,
                                void *out, lpc_dtype out_t, hipStream_t stream);

/* out[r, j] = sum over blocks b of 32 of
 *   2^(xs[r, b] - 127) * 2^(ws[g, j, b] - 127) * (sum over i in b of x[r, i] * w[g, j, i])
 * for the group g that row r belongs to, rounded once to out_t.  Sums are held
 * in FP32: off by at most 2 k 2^-24 of the sum of the terms' magnitudes, and by
 * 2 k 2^-149 where these are below FP32's normal numbers.
 *   x  codes [rows, k/2], xs [rows, k/32]; w codes [groups, n, k/2], ws
 *      [groups, n, k/32]: rows as lpc_quantize_mxfp4 writes them; an exponent
 *      byte of 255 makes a NaN of every sum it is part of
 *   counts, rows past the last group and limits as for lpc_gemm_bf16, but k a
 *   positive multiple of 128                                                 */
lpc_status lpc_gemm_mxfp4(const uint8_t *x, const uint8_t *xs, size_t rows, size_t k,
                          const uint8_t *w, const uint8_t *ws, size_t n,
                          int groups, const int32_t *counts,
                          void *out, lpc_dtype out_t, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Muon over many matrices                                                  */
/* ---------------------------------------------------------------------- */

#define LPC_MUON_MAX_SIDE ((size_t)1 << 20)    /* rows or columns of a matrix */
#define LPC_MUON_MAX_ITERATIONS 10

/* `batch` matrices of rows x cols one after the other, as a layer of experts
 * holds them.  Device pointers, 16-byte aligned.
 *   param  FP32, updated in place;  grad  of the plan's type, read
 *   m      FP32 momentum, updated in place
 *   copy   bf16 copy of the updated param, or NULL (for each tensor)
 *   scale  of this tensor's updates                                          */
typedef struct {
    float *param;
    const void *grad;
    float *m;
    uint16_t *copy;
    size_t batch, rows, cols;
    double scale;
} lpc_muon_tensor;

/* What a step of a plan launches; lpc_muon_plan writes it and lpc_muon_step
 * takes it as it is.                                                         */
typedef struct {
    size_t matrices, chunks, squares, updates, smalls;
    size_t workspace_bytes;
} lpc_muon_work;

/* Bytes of the plan of these tensors.  tensors: host array; 0 for no work, for
 * sizes that are refused and for NULL.  No HIP call.                         */
size_t lpc_muon_plan_bytes(const lpc_muon_tensor *tensors, int count);

/* Check the tensors and write the plan to HOST memory (`plan`, of
 * lpc_muon_plan_bytes bytes); the caller copies it to a 16-byte aligned device
 * buffer and keeps it as long as the tensors stay where they are.
 *   Tensors without elements are left out.  rows and cols at most
 *   LPC_MUON_MAX_SIDE; of all matrices together at most 2^23 - 512 tiles of
 *   256 x 256, and fewer than 2^24 matrices and chunks of 4096 elements (else
 *   LPC_ERR_SHAPE).  Tensors must not overlap.                               */
lpc_status lpc_muon_plan(const lpc_muon_tensor *tensors, int count, lpc_dtype grad_t,
                         void *plan, size_t plan_bytes, lpc_muon_work *work);

/* One step over every matrix of a plan:
 *   g = grad * grad_scale[0] (grad_scale NULL: 1)
 *   m = beta m + (1 - beta) g
 *   u = nesterov ? (1 - beta) g + beta m : m
 *   X = u / |u| (Frobenius; zeros if u is), then `iterations` times
 *       A = X X^T,  B = -4.775 A + 2.0315 A A,  X = 3.4445 X + B X
 *   param = param (1 - lr weight_decay) - lr scale X
 * m and the parameters' last line in FP32, every operation rounded on its own;
 * |u| in 64 bits.  X is held in fp16 halves of together 22 bits and the products
 * take its high half, A and B in fp16, sums in FP32.  On the matrices measured,
 * of full and of low rank, X is off by at most 3.2e-3 of itself (2-norm) after
 * five iterations; after ten by 7.2e-3, and by 2.2e-2 where its rank is low, as in
 * FP32 throughout.  Where rows or cols is 32 or less, u is FP32 and all from there
 * to the last line in 64 bits.
 *   plan   DEVICE copy of the plan;  work, grad_t as planned
 *   workspace  device memory of work->workspace_bytes, no initial contents
 *      needed; steps that overlap need one each
 *   beta in [0, 1), iterations in 1..LPC_MUON_MAX_ITERATIONS (else
 *   LPC_ERR_SHAPE)                                                           */
lpc_status lpc_muon_step(const void *plan, const lpc_muon_work *work, lpc_dtype grad_t,
                         double lr, double beta, int nesterov, double weight_decay, int iterations,
                         const float *grad_scale, void *workspace, size_t workspace_bytes,
                         hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LPC_OPS_H */
