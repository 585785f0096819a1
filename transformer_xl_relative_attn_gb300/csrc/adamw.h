// Internal interface of the AdamW step (adamw.cu) for the ABI layer.
#pragma once
#include <cuda_runtime.h>

#include "txl_attn.h"

namespace txl {

constexpr int kAdamwBlock = 256;  // elements of one block of the flat state (and of one 8-bit scale)

struct AdamwArgs {
    const txl_adamw_tensor* tensors;
    int n_tensors;
    int bf16_param, bf16_grad, eight_bit;
    float* master;
    void* exp_avg;
    float* exp_avg_scale;
    void* exp_avg_sq;
    float* exp_avg_sq_scale;
    long long* steps;
    const float* lr;
    double beta1, beta2, eps, max_norm;
    unsigned seed;
    float* grad_norm;
    void* workspace;
};

// Blocks of the flat state of these tensors.
long long adamw_blocks(const txl_adamw_tensor* tensors, int n_tensors);
size_t adamw_workspace_bytes(long long blocks);
cudaError_t launch_adamw(const AdamwArgs& a, cudaStream_t stream);

}  // namespace txl
