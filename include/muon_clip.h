/*
 * muon_clip.h - C ABI of libmuon's gradient clipping: the global norm over
 * many tensors, and their scaling to a largest norm, ahead of a Muon step.
 *
 *   norm = sqrt(sum of the squares of all elements of all tensors)
 *   out  = g * (max_norm / norm) where norm > max_norm, else g
 *
 * The sum is held in 64 bits, so that no square overflows or vanishes, in a
 * fixed order: the same bits on every run.  The norm is rounded to fp32 once
 * (to infinity past its range); the factor follows from the 64-bit norm and is
 * rounded once to fp32's 24 bits, also where it is smaller than fp32's normal
 * numbers; a product with it is rounded to fp32, and from there to the output's
 * type.  An infinite gradient gives the factor 0 (finite gradients become 0,
 * infinite ones NaN), a NaN one NaN.
 *
 * Conventions:
 *   - Tensors are flat runs of elements, fp32 or bf16 each (dtypes), aligned to
 *     their elements; the arrays of pointers and sizes are host arrays that
 *     are read before the call returns.
 *   - All tensors and the norm are device memory owned by the caller.  Calls
 *     enqueue on `stream`, do not synchronise and allocate nothing; they may be
 *     captured into a graph (which keeps the pointers).  The workspace holds
 *     at least muon_clip_workspace bytes, 256-byte aligned; its contents
 *     between calls are irrelevant.
 *   - Errors as in muon.h: host validation first, nothing enqueued on any
 *     status other than MUON_OK and MUON_ERR_HIP.
 */
#ifndef MUON_CLIP_H
#define MUON_CLIP_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

muon_status muon_clip_workspace(int num, const int64_t* numel, const muon_dtype* dtypes, size_t* workspace_bytes);

/* norm[0] = the global norm, in fp32 (0 for no elements). */
muon_status muon_grad_norm(int num, const void* const* g, const int64_t* numel, const muon_dtype* dtypes, float* norm,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The norm as above, and out[i] = the clipped g[i] in out_dtypes[i]; max_norm
 * >= 0, which may be infinite (never clips).  out[i] may be g[i] itself (with its type): then
 * nothing is written unless the norm is over max_norm.  Apart from that, no
 * out (nor the norm) may overlap a g or another out, nor, where out[i] is g[i],
 * one g another: ranges of addresses that do give MUON_ERR_INVALID_ARGUMENT. */
muon_status muon_clip_grads(int num, const void* const* g, const int64_t* numel, const muon_dtype* dtypes,
                            void* const* out, const muon_dtype* out_dtypes, float max_norm, float* norm,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_CLIP_H */
