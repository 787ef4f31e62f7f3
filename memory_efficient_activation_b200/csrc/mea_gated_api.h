// mea_gated_api.h -- host-side interface of the gated feed-forward kernels
// (both projections, the activation and the product on the tensor cores).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mea {

// All matrices are row-major bf16.
//   mode 0 (forward):  gate = X Wg^T, up = X Wu^T with X [M x K], Wg, Wu
//                      [N x K]; z [M x 2N] = [gate | up] (nullable), h [M x N]
//                      = f(gate) up (nullable; at least one of the two).
//   mode 1 (backward): d = G Wd with G = x [M x K], Wd = w0 [K x N]; zin the
//                      stored [M x 2N]; z [M x 2N] = [d up f'(gate) | d
//                      f(gate)], h (nullable) = f(gate) up.
struct GatedLaunch {
    int act;
    int mode;
    int64_t M, N, K;
    const void *x;
    const void *w0;
    const void *w1;      // forward only
    const void *zin;     // backward only
    void *z;
    void *h;
    float param;
    cudaStream_t stream;
};

// Plain product C [M x N] = op(A) op(B), bf16, fp32 accumulation: A is [M x K]
// (or [K x M] with trans_a), B is [K x N] (or [N x K] with trans_b); not both
// transposed.
struct MatmulPlain {
    int trans_a, trans_b;
    int64_t M, N, K;
    const void *a;
    const void *b;
    void *c;
    cudaStream_t stream;
};

// Products of few output tiles, K shared out over a cluster: the gated
// forward, its backward, or a plain one (x = A, w0 = B, z = C; NT: B is [N x
// K], NN: [K x N], TN: A is [K x M] and B [K x N]).  Tiles of kFewTokens rows
// at most.
constexpr int kFewTokens = 256;
enum FewKind { kFewGated, kFewBwd, kFewNT, kFewNN, kFewTN };
cudaError_t launch_few(const GatedLaunch &a, FewKind kind);
cudaError_t few_error_word(int clear, unsigned int *word);     // synchronous
cudaError_t launch_matmul(const MatmulPlain &p);
cudaError_t launch_gated(const GatedLaunch &a);
cudaError_t gated_error_word(int clear, unsigned int *word);   // synchronous

}  // namespace mea
