// Internal interface of the token log probabilities (token_logprobs.cu) for the ABI layer.
#pragma once
#include <cuda_runtime.h>

namespace txl {

constexpr int kTopMost = 32;  // alternatives of a row: one per lane of a warp

struct TokenLogprobs {
    const void* logits;       // [rows, V], rows ld elements apart
    long long ld;
    const long long* tokens;  // [rows]
    long long rows;
    int V;
    int top;  // alternatives per row, 0: none
    float* logprob;
    float* lse;
    float* entropy;
    long long* top_index;  // [rows, top]
    float* top_logprob;
};

struct TokenLogprobsBwd {
    const void* logits;
    long long ld;
    const long long* tokens;
    const float* lse;
    const float* entropy;   // null without dentropy
    const float* dlogprob;  // each may be null: zeros
    const float* dlse;
    const float* dentropy;
    long long rows;
    int V;
    void* dlogits;  // [rows, V], rows ldd elements apart
    long long ldd;
};

cudaError_t launch_token_logprobs(const TokenLogprobs& a, bool bf16, cudaStream_t stream);
cudaError_t launch_token_logprobs_bwd(const TokenLogprobsBwd& a, bool bf16, cudaStream_t stream);

}  // namespace txl
