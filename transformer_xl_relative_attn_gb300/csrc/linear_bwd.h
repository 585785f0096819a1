// Internal interface of the Linear layer's gradients (linear_bwd.cu) for the ABI layer.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace txl {

struct LbParams {
    int T, B;       // rows per batch row, batch rows (rows layout: all rows, 1)
    int K, N;
    int heads;      // x and dx are [B, K / 64, T, 64]
    int n_kt, n_nt, n_tt;  // tiles along K, N and T (per batch row)
    int t_steps;           // 64-row steps per batch row
    int n_steps;           // 64-column steps of N
    int splits;            // of dw's reduction
    int n_w, n_d;          // dw items (tiles * splits), dx tiles
    int heavy, extra;      // see LbSchedule
    int k64, n64;          // K, N are multiples of 64: boxes of several slices
    int db_rows;           // parts of db (row ranges); 0: no parts
    const __nv_bfloat16* x;
    const __nv_bfloat16* dy;
    __nv_bfloat16* dx;
    float* dw;             // [splits, N, K]
    float* db;             // [db_rows, N], without parts [N] or null
    int* status;
};

// How a call is cut: pairs or single CTAs, splits of dw's reduction, schedule.
struct LbPlan {
    bool pair;
    int grid;
    LbParams p;
};

// dx = dy W (0 unless x > 0 if relu), dw = dy^T x, db = column sums of dy.  x and
// dx [B, T, K] (heads = 0) or [B, K / 64, T, 64]; dy [B, T, N]; w [N, K].  dx, or
// dw with db, may be null; db alone may be null.  K and N multiples of 8, of 64 for
// K with heads.  cudaErrorInvalidValue: a tensor map could not be encoded.
LbPlan linear_bwd_plan(int heads, int B, int T, int K, int N, bool want_dx, bool want_dw);
size_t linear_bwd_workspace_bytes(const LbPlan& plan, bool want_db);
cudaError_t launch_linear_bwd(LbPlan plan, const void* dy, const void* x, const void* w, int relu, void* dx, float* dw,
                              float* db, void* workspace, int* status, cudaStream_t stream);

}  // namespace txl
