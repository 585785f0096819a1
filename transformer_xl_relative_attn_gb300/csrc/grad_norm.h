// Internal interface of the gradient norms (grad_norm.cu) for the ABI layer.
#pragma once
#include <cuda_runtime.h>

#include "txl_attn.h"

namespace txl {

// How the tensors are cut: bytes of a piece (what a CTA sums at a time), and pieces in all.
struct GradNormPlan {
    long long piece_bytes, pieces;
};

struct GradNormArgs {
    const txl_grad_tensor* tensors;
    int n_tensors;
    GradNormPlan plan;
    double max_norm;  // 0: no clipping
    float* norm;      // [1]
    float* norms;     // [n_tensors] or null
    void* workspace;
};

GradNormPlan grad_norm_plan(const txl_grad_tensor* tensors, int n_tensors);
size_t grad_norm_workspace_bytes(const GradNormPlan& plan);
cudaError_t launch_grad_norm(const GradNormArgs& a, cudaStream_t stream);

}  // namespace txl
