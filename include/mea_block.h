/*
 * mea_block.h -- C ABI of the transformer-block operators of libmea.so: the
 * normalisation of rows (layer norm, rms norm).
 *
 * Everything mea.h states for its entry points holds here too: device
 * pointers owned by the caller, asynchronous calls on `stream`, status codes
 * and mea_last_error, no allocation, no synchronisation, dense contiguous
 * tensors (unaligned ones take a scalar path unless an entry says otherwise),
 * an element count of zero is a no-op, results bitwise deterministic.
 * bf16 results are rounded once, to nearest even, from fp32 arithmetic.
 *
 * Entry points: mea_norm_fwd, mea_norm_bwd (+ _workspace_bytes).
 */
#ifndef MEA_BLOCK_H
#define MEA_BLOCK_H

#include "mea.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Normalisation of rows (mea_norm_*). */
typedef enum { MEA_LAYER_NORM = 0, MEA_RMS_NORM = 1 } mea_norm_t;

/* Normalisation of rows, forward.  x is [rows x C], each row one token (or
 * position):
 *   MEA_LAYER_NORM  mean = sum x / C, var = sum (x - mean)^2 / C,
 *                   invstd = 1 / sqrt(var + eps),
 *                   y = gamma (x - mean) invstd + beta;
 *   MEA_RMS_NORM    the same with mean = 0 (var = sum x^2 / C).
 *   dtype        storage of x and y.
 *   param_dtype  storage of gamma and beta (either dtype beside either x).
 *   x            device, [rows x C] row-major, read only; the one tensor kept
 *                for the backward beside the row statistics.  rows and C are
 *                below 2^31 (else MEA_ERR_UNSUPPORTED).
 *   gamma, beta  device, [C], read only; NULL stands for 1 and 0.
 *   eps          >= 0.
 *   y            device, [rows x C], written.
 *   mean, invstd device fp32 [rows], written; either may be NULL; mean is
 *                ignored for MEA_RMS_NORM.
 * Row statistics are fp32 sums (over long rows fp64), the variance a second
 * pass over the row; y is rounded once.  Outputs must not overlap an input
 * or each other.
 * Source: layer normalisation in its standard definition; the save-input-only
 * scheme of the Swish page applied to it (x and two floats per row are kept,
 * y is re-populated by the same call where a backward needs it again). */
MEA_API mea_status_t mea_norm_fwd(mea_norm_t norm, mea_dtype_t dtype, mea_dtype_t param_dtype, int64_t rows,
                                  int64_t C, const void *x, const void *gamma, const void *beta, float eps,
                                  void *y, float *mean, float *invstd, mea_stream_t stream);

/* Bytes of device workspace mea_norm_bwd needs for dgamma or dbeta.  Pure host
 * arithmetic; 0 for an empty or unsupported shape. */
MEA_API size_t mea_norm_bwd_workspace_bytes(int64_t rows, int64_t C);

/* Normalisation of rows, backward, from x, dy and the row statistics:
 *   xhat = (x - mean) invstd, a = dy gamma,
 *   dx = invstd (a - sum(a) / C - xhat sum(a xhat) / C)   (layer norm; rms
 *   norm without the first sum), dgamma = sum over rows of dy xhat,
 *   dbeta = sum over rows of dy.
 *   x, dy        device, [rows x C] of `dtype`, read only.
 *   gamma        device [C] of `param_dtype`, or NULL (1).
 *   mean, invstd device fp32 [rows], as mea_norm_fwd wrote them (mean is
 *                ignored for MEA_RMS_NORM).
 *   dx           device, written; may be x or dy exactly, no partial overlap.
 *   dgamma,
 *   dbeta        device [C] of `param_dtype`, OVERWRITTEN; either may be NULL.
 *                With rows = 0 they are set to zero.
 *   workspace,
 *   ws_bytes     when dgamma or dbeta is given: device scratch of at least
 *                mea_norm_bwd_workspace_bytes(), 16-byte aligned, any
 *                contents (no counter, no zero-fill).  Calls that share it
 *                must not run concurrently on the GPU.
 * Column sums take at most 1024 rows in fp32 and add those sums in fp64, in
 * an order fixed by the shape. */
MEA_API mea_status_t mea_norm_bwd(mea_norm_t norm, mea_dtype_t dtype, mea_dtype_t param_dtype, int64_t rows,
                                  int64_t C, const void *x, const void *dy, const void *gamma, const float *mean,
                                  const float *invstd, void *dx, void *dgamma, void *dbeta, void *workspace,
                                  size_t ws_bytes, mea_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MEA_BLOCK_H */
