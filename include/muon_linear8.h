/*
 * muon_linear8.h - C ABI of libmuon's 8-bit linear layer: the operators that
 * lead from a residual stream to the weight gradient a Muon step takes, with
 * activations and weights kept in 8 bits.
 *
 *   muon_rmsnorm_forward    h = x + residual, y = h * rstd * weight, y as
 *                           rows of the type or as 8-bit rows
 *   muon_rmsnorm_backward   dx (= dresidual) and dweight; h from rows of the
 *                           type or from 8-bit rows
 *   muon_q8_quantize        rows to 8 bits (activation checkpoint, weights)
 *   muon_q8_dequantize      8-bit rows back
 *   muon_q8_matmul          Y  = x w^T from 8-bit rows of x and w
 *   muon_q8_grad_input      dX = dY w  from 8-bit rows of w
 *   muon_q8_grad_weight     dW = dY^T x from 8-bit rows of x (the checkpoint)
 *
 * The 8-bit form of a row v of length n: scale = 2^e with the smallest
 * e >= -126 for which max|v| <= 127 * 2^e, q = v / scale rounded to nearest,
 * ties to even, so |q| <= 127 and |v - q * scale| <= scale / 2.  A row that
 * holds a NaN or an infinity gets scale NaN and q = 0: what is computed from
 * it is NaN.  Products accept any scales and any int8 values; the gradient
 * products round q * scale to bf16, which is exact for powers of two.
 *
 * Conventions:
 *   - Matrices are row-major with unit column stride; ld* is the distance of
 *     rows in elements (ld >= columns; ignored for at most one row).  Rows
 *     need no alignment beyond the element's own.
 *   - x, y, h, dy, dx are fp32 or bf16 (muon_dtype), norm weights, scales,
 *     rstd and dweight fp32; dy of the gradient products is bf16.
 *   - All pointers are device pointers owned by the caller.  A call with no
 *     output elements enqueues nothing and may be given null pointers.
 *   - Calls enqueue on `stream`, do not synchronise and allocate nothing;
 *     they may be captured into a graph.  Where a call takes a workspace, its
 *     size comes from the matching *_workspace call, its address must be
 *     256-byte aligned, and its contents between calls are irrelevant.
 *     Results do not depend on timing: sums have a fixed order.
 *   - Outputs may not overlap inputs, except that h may be x or residual,
 *     y may be x, and dx may be dy or dh (the same address and ld).
 *   - Errors as in muon.h: host validation first, nothing enqueued on any
 *     status other than MUON_OK and MUON_ERR_HIP.  Row widths above 32768
 *     (norm and 8-bit rows), dimensions above 2^24, and matmul's k above
 *     131071 (int32 sums of 8-bit products) give MUON_ERR_UNSUPPORTED.
 */
#ifndef MUON_LINEAR8_H
#define MUON_LINEAR8_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* h = x + residual rounded to the type (h = x and the h argument unused if
 * residual is NULL); rstd = 1 / sqrt(mean(h^2) + eps) per row;
 * y = h * rstd * weight, also where rstd itself is outside fp32's normal
 * numbers (rms of h over 2^126 or under 2^-128).  Exactly one of y and q is given: y takes rows of
 * the type, q and scale the 8-bit form of the unrounded y.  The sum of
 * squares, rstd, the 8-bit scale and rounding are carried in 64 bits, so q
 * does not depend on how a row is split over the hardware.  (A row whose
 * largest |y| passes fp32's range counts as non-finite in 8 bits.)
 * eps >= 0. */
muon_status muon_rmsnorm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                 const float* weight, muon_dtype dtype, int64_t rows, int64_t cols,
                                 float eps, void* h, int64_t ldh, void* y, int64_t ldy, int8_t* q,
                                 int64_t ldq, float* scale, float* rstd, hipStream_t stream);

/* With g = dy * weight and n = h * rstd per row:
 *   dx = rstd * (g - n * mean(g * n)) + dh   (dh nullable: the gradient that
 *        reaches h through the residual stream)
 *   dweight = sum over rows of dy * n
 * h_scale NULL: h holds rows of the type; else int8 rows with that scale. */
muon_status muon_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t* workspace_bytes);
muon_status muon_rmsnorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh,
                                  const float* h_scale, const float* rstd, const float* weight,
                                  const void* dh, int64_t lddh, muon_dtype dtype, int64_t rows,
                                  int64_t cols, void* dx, int64_t lddx, float* dweight, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream);

/* 8-bit form of each row, and back (x = q * scale rounded to the type). */
muon_status muon_q8_quantize(const void* x, int64_t ldx, muon_dtype dtype, int64_t rows, int64_t cols,
                             int8_t* q, int64_t ldq, float* scale, hipStream_t stream);
muon_status muon_q8_dequantize(const int8_t* q, int64_t ldq, const float* scale, int64_t rows,
                               int64_t cols, void* x, int64_t ldx, muon_dtype dtype,
                               hipStream_t stream);

/* The products below, t tokens, weights n x k (out x in):
 *   MUON_Q8_MATMUL       a = xq (t x k), b = wq (n x k)
 *   MUON_Q8_GRAD_INPUT   a = dy (t x n), b = wq (n x k)
 *   MUON_Q8_GRAD_WEIGHT  a = dy (t x n), b = xq (t x k)
 * The workspace depends on the sizes, row distances and 16-byte alignment
 * of the operands a and b (addresses are not read). */
typedef enum { MUON_Q8_MATMUL = 0, MUON_Q8_GRAD_INPUT = 1, MUON_Q8_GRAD_WEIGHT = 2 } muon_q8_product;
muon_status muon_q8_workspace(muon_q8_product product, const void* a, int64_t lda, const void* b,
                              int64_t ldb, int64_t t, int64_t n, int64_t k, size_t* workspace_bytes);

/* y[t][n] = x_scale[t] * w_scale[n] * sum_k xq[t][k] * wq[n][k]; the sum is
 * exact (int32), then scaled in fp32, by x_scale first (past 2^97 that may
 * overflow though w_scale would bring it back), and rounded to the type. */
muon_status muon_q8_matmul(const int8_t* xq, int64_t ldx, const float* x_scale, const int8_t* wq,
                           int64_t ldw, const float* w_scale, int64_t t, int64_t n, int64_t k, void* y,
                           int64_t ldy, muon_dtype dtype, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* dx[t][k] = sum_n dy[t][n] * (w_scale[n] * wq[n][k]), dy bf16, fp32 sums. */
muon_status muon_q8_grad_input(const void* dy, int64_t lddy, const int8_t* wq, int64_t ldw,
                               const float* w_scale, int64_t t, int64_t n, int64_t k, void* dx,
                               int64_t lddx, muon_dtype dtype, void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* dw[n][k] = sum_t dy[t][n] * (x_scale[t] * xq[t][k]), dy bf16, fp32 sums;
 * accumulate != 0 adds to what dw holds (in fp32, rounded to the type).  dw
 * contiguous in fp32 or bf16 is the G that muon_step_batched takes. */
muon_status muon_q8_grad_weight(const void* dy, int64_t lddy, const int8_t* xq, int64_t ldx,
                                const float* x_scale, int64_t t, int64_t n, int64_t k, void* dw,
                                int64_t lddw, muon_dtype dtype, int accumulate, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_LINEAR8_H */
