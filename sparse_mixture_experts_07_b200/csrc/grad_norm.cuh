// Launch parameters of the gradient norm and clipping kernels (grad_norm.cu).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kGradsPerLaunch = 64;
constexpr int kGradParts = 2048;     // partial sums in the workspace

// Up to 64 tensors of one launch, cut into chunks of `chunk` values that the
// CTAs take in turn; chunk_start is the prefix of the tensors' chunk counts.
struct GradList {
    void* ptr[kGradsPerLaunch];
    int64_t numel[kGradsPerLaunch];
    int64_t chunk_start[kGradsPerLaunch + 1];
    int32_t dtype[kGradsPerLaunch];
    int32_t n;
    int32_t chunk;
};

cudaError_t launch_grad_square_sum(const GradList&, bool add, double* part, int parts,
                                   cudaStream_t);
cudaError_t launch_grad_total(const double* part, int parts, double* total, cudaStream_t);
cudaError_t launch_grad_scale(const GradList&, const double* part, int parts, float max_norm,
                              float* norm, int num_sms, cudaStream_t);

}  // namespace moe
