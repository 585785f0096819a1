// Internal interface of the Linear layer's gradients (linear_bwd.cu) for the ABI layer.
#pragma once
#include <cuda_runtime.h>

namespace txl {

// dx = dy W (times [x > 0] if relu), dw = dy^T x, db = column sums of dy.  x and
// dx [B, T, K] (heads = 0) or [B, K / 64, T, 64]; dy [B, T, N]; w [N, K].  dx, or
// dw with db, may be null; db alone may be null.  K and N multiples of 8, of 64 for
// K with heads.  cudaErrorInvalidValue: a tensor map could not be encoded.
cudaError_t launch_linear_bwd(const void* dy, const void* x, int heads, int B, int T, int K, const void* w, int N,
                              int relu, void* dx, float* dw, float* db, void* workspace, int* status,
                              cudaStream_t stream);
size_t linear_bwd_workspace_bytes(int heads, int B, int T, int K, int N, bool want_dx, bool want_dw,
                                  bool want_db);

}  // namespace txl
