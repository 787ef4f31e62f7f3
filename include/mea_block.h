/*
 * mea_block.h -- C ABI of the transformer-block operators of libmea.so: the
 * normalisation of rows (layer norm, rms norm) and the gated feed-forward
 * block (both projections, the activation and the product in one kernel).
 *
 * Everything mea.h states for its entry points holds here too: device
 * pointers owned by the caller, asynchronous calls on `stream`, status codes
 * and mea_last_error, no allocation, no synchronisation, dense contiguous
 * tensors (unaligned ones take a scalar path unless an entry says otherwise),
 * an element count of zero is a no-op, results bitwise deterministic.
 * bf16 results are rounded once, to nearest even, from fp32 arithmetic.  A
 * bounded wait on a shared-memory barrier that expires in one of these kernels
 * (which does not happen in correct operation) is recorded in the word that
 * mea_matmul_error_word reads.
 *
 * Entry points: mea_norm_fwd, mea_norm_bwd (+ _workspace_bytes);
 * mea_matmul_gated_act_fwd, mea_matmul_gated_act_bwd; mea_matmul.
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
 * Row statistics are fp32 sums (over long rows fp64), the variance sums of
 * squared distances from the row's mean, or from the means of its parts and
 * those merged; y is rounded once.  Outputs must not overlap an input
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
 * an order fixed by the shape, the types and which pointers lie on 16-byte
 * boundaries: the same call repeats its bits, the same values at another
 * alignment may give others. */
MEA_API mea_status_t mea_norm_bwd(mea_norm_t norm, mea_dtype_t dtype, mea_dtype_t param_dtype, int64_t rows,
                                  int64_t C, const void *x, const void *dy, const void *gamma, const float *mean,
                                  const float *invstd, void *dx, void *dgamma, void *dbeta, void *workspace,
                                  size_t ws_bytes, mea_stream_t stream);

/* Gated feed-forward block, forward: two projections of the same input, the
 * activation of one of them and their product,
 *   gate = X Wg^T, up = X Wu^T (bf16 inputs, fp32 accumulation on the tensor
 *   cores), h = f(gate) up.
 *   act, param   activation and its parameter, as in mea_act_fwd (MEA_SWISH:
 *                SwiGLU, MEA_GELU_*: GeGLU, MEA_RELU: ReGLU, MEA_SIGMOID: GLU).
 *   M, N, K      X is [M x K], Wg and Wu are [N x K], h is [M x N]; M or N of
 *                0 is a no-op; K must be positive.  K and N must be multiples
 *                of 8, M, N and K below 2^31 - 1024; otherwise
 *                MEA_ERR_UNSUPPORTED.  Any M from one token up.
 *   x, w_gate,
 *   w_up         device, bf16, row-major (K contiguous), read only, 16-byte
 *                aligned (else MEA_ERR_UNSUPPORTED).  The two weights may be
 *                the halves of one [2N x K] matrix, or the same matrix.
 *   z            device, bf16, [M x 2N], written: row i holds gate in its
 *                first N columns and up in its last N, rounded to bf16: the
 *                tensor to keep for the backward.  NULL where none follows.
 *   h            device, bf16, [M x N], written: f(gate) up formed from the
 *                fp32 accumulators and rounded once.  NULL to form z alone; at
 *                least one of z and h is given.  Outputs are 16-byte aligned
 *                and overlap neither an input nor each other.
 * Source: as mea_matmul_act_fwd (the activation in the epilogue of the matmul
 * that feeds it), for the gated form of the block. */
MEA_API mea_status_t mea_matmul_gated_act_fwd(mea_act_t act, int64_t M, int64_t N, int64_t K, const void *x,
                                              const void *w_gate, const void *w_up, float param, void *z,
                                              void *h, mea_stream_t stream);

/* Gated feed-forward block, backward through the down projection out = h
 * Wd^T and the product: with d = G Wd (never stored) and the stored z,
 *   dz = [d up f'(gate) | d f(gate)],   h = f(gate) up.
 * dz is the gradient of [gate | up]: dX = dz [Wg; Wu] and [dWg; dWu] = dz^T X
 * are plain products; h, re-populated here instead of being kept by the
 * forward, gives dWd = G^T h.
 *   M, N, K      G is [M x K], Wd is [K x N], z and dz are [M x 2N], h is
 *                [M x N]; restrictions as in mea_matmul_gated_act_fwd.
 *   g            device, bf16, the gradient of out, read only.
 *   w_down       device, bf16, row-major [K x N] (N contiguous: the weight as
 *                the forward uses it, not transposed), read only.
 *   z            device, bf16, [M x 2N] as the forward wrote it.
 *   dz           device, bf16, written; may be z itself (each element is read
 *                before it is written), no partial overlap.
 *   h            device, bf16, written, or NULL; overlaps nothing else.
 *   All pointers 16-byte aligned.
 * h differs from the forward's where z's rounding moves it: it is f(gate) up
 * of z as stored. */
MEA_API mea_status_t mea_matmul_gated_act_bwd(mea_act_t act, int64_t M, int64_t N, int64_t K, const void *g,
                                              const void *w_down, const void *z, float param, void *dz,
                                              void *h, mea_stream_t stream);

/* Matrix product C = op(A) op(B) in bf16 with fp32 accumulation on the tensor
 * cores, each operand read as it is stored: the products around the gated
 * block (h Wd^T; dz [Wg; Wu]; dz^T X and G^T h) without a transposed copy.
 *   trans_a      zero: A is [M x K]; non-zero: A is [K x M] and op(A) = A^T.
 *   trans_b      zero: B is [K x N]; non-zero: B is [N x K] and op(B) = B^T.
 *                Both non-zero is MEA_ERR_UNSUPPORTED.
 *   M, N, K      each below 2^31 - 1024; M or N of 0 is a no-op, K of 0 sets C
 *                to zero.  The rows of A, B and C as stored must be multiples of
 *                8 elements (else MEA_ERR_UNSUPPORTED).
 *   a, b         device, bf16, row-major, read only, 16-byte aligned.
 *   c            device, bf16, [M x N], written, 16-byte aligned; overlaps
 *                neither operand. */
MEA_API mea_status_t mea_matmul(int trans_a, int trans_b, int64_t M, int64_t N, int64_t K, const void *a,
                                const void *b, void *c, mea_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MEA_BLOCK_H */
