// Internal interface of the gradient norms (grad_norm.cu) for the ABI layer.
#pragma once
#include <cuda_runtime.h>

#include "txl_attn.h"

namespace txl {

struct GradNormArgs {
    const txl_grad_tensor* tensors;
    int n_tensors;
    double max_norm;  // 0: no clipping
    float* norm;      // [1]
    float* norms;     // [n_tensors] or null
    void* workspace;
};

// Pieces of these tensors (what a CTA sums at a time).
long long grad_norm_pieces(const txl_grad_tensor* tensors, int n_tensors);
size_t grad_norm_workspace_bytes(long long pieces);
cudaError_t launch_grad_norm(const GradNormArgs& a, cudaStream_t stream);

}  // namespace txl
