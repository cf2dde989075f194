// Launch parameters of the norm kernels (norm.cu).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxNormH = 32768;   // a row is held in one CTA's registers

struct NormDev {
    const float* weight;   // [H] or NULL (ones)
    const float* bias;     // [H] or NULL (zeros)
    float eps;
    int kind;              // moe_norm_kind
};

struct CombineNormParams {
    const void* y_slots;
    const int32_t* inv;
    const void* residual;  // NULL: zero
    const float* gate;
    void* y_out;           // NULL: not stored
    void* h_out;           // NULL: not stored
    void* xn_out;          // NULL: no next norm
    NormDev post, next;
    int64_t T;
    int H, k, S, gate_kind;
    float scale;
};

struct NormBackwardParams {
    const void* x;
    const void* dout;
    const void* dadd;      // NULL: none
    const float* gate;
    void* dx;
    float* dweight;
    float* dbias;
    float* dgate;
    float* part;           // [CTAs, 2, H]; NULL when no column gradient is wanted
    NormDev norm;
    int64_t T;
    int H, gate_kind;
    float scale;
};

int norm_backward_parts(int64_t T, int H, int num_sms);
cudaError_t launch_combine_norm(const CombineNormParams&, bool bf16, bool vec16, int num_sms,
                                cudaStream_t);
cudaError_t launch_norm_backward(const NormBackwardParams&, bool bf16, bool vec16, int num_sms,
                                 cudaStream_t);

}  // namespace moe
