// mea_norm_api.h -- host-side interface of the row normalisation kernels
// (layer norm and rms norm over the last axis, forward and backward).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace mea {

struct NormLaunch {
    int rms;                 // 0: layer norm, 1: rms norm
    int dtype;               // Dtype of x, y, dy, dx
    int pdtype;              // Dtype of gamma, beta, dgamma, dbeta
    int64_t rows;
    int64_t C;
    const void *x;
    const void *dy;          // backward only
    const void *gamma;       // nullable (1)
    const void *beta;        // forward only, nullable (0)
    float eps;               // forward only
    void *out;               // y or dx
    float *mean;             // forward: written (nullable; ignored for rms)
    float *invstd;           // forward: written (nullable)
    const float *mean_in;    // backward (ignored for rms)
    const float *invstd_in;  // backward
    void *dgamma;            // backward, nullable
    void *dbeta;             // backward, nullable
    void *workspace;         // backward with dgamma or dbeta
    cudaStream_t stream;
};

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t C);
cudaError_t norm_error_word(int clear, unsigned int *word);   // synchronous
cudaError_t launch_norm_fwd(const NormLaunch &a);
cudaError_t launch_norm_bwd(const NormLaunch &a);

}  // namespace mea
