// Internal interface of the log probabilities from hidden states (linear_logprobs.cu) for the ABI layer.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace txl {

struct LpParams {
    int rows, V;
    int ksteps, klast;     // 64-element steps of K; MMAs (of 16 elements) of the last one
    int bn;                // columns of a tile, a multiple of 64 up to 256
    int n_rt, n_vt;        // tiles of rows and of columns
    int per, chunks;       // column tiles of an item; items per row tile
    const long long* tokens;
    const __nv_bfloat16* bias;  // [V] or null
    int wide_bias;         // bias is 8-byte aligned
    float4* part;          // [rows][2 chunks]: (m, s, t) of each half of an item's columns
    float* given;          // [rows]: the token's logit
    const char* ws_end;    // of the workspace, both buffers in it
    int* status;
};

struct LpPlan {
    bool pair;
    int grid;
    LpParams p;
};

LpPlan linear_logprobs_plan(int rows, int K, int V, bool bias);
size_t linear_logprobs_workspace_bytes(const LpPlan& plan);
// Of x [rows, K], w [V, K] and bias [V] (may be null), bf16, K a multiple of 8.
// cudaErrorInvalidValue: a tensor map could not be encoded.
cudaError_t launch_linear_logprobs(LpPlan plan, const void* x, const void* w, const void* bias, int K, const long long* tokens,
                                   float* logprob, float* lse, float* entropy, void* workspace, size_t ws_bytes, int* status,
                                   cudaStream_t stream);

}  // namespace txl
