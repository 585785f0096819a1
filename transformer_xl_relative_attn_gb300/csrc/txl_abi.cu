// extern "C" entry points of libtxl.so (declared in include/txl_attn.h):
// argument validation on the host, then one asynchronous launch on the
// caller's stream.  Nothing here allocates device memory.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <mutex>
#include <new>
#include <vector>
#include <cuda_runtime.h>

#include "adamw.h"
#include "grad_norm.h"
#include "linear_bwd.h"
#include "linear_logprobs.h"
#include "proj_gemm.h"
#include "token_logprobs.h"
#include "txl_attn.h"
#include "txl_device.cuh"

namespace txl {
__device__ int g_dev_status = 0;

cudaError_t launch_tail_m(void* mem, const void* hid, int B, int L, int L_stride, int M,
                          size_t row_bytes, cudaStream_t stream);
cudaError_t launch_mem_reset(void* mem, const unsigned char* flags, int B, long long per_b_bytes,
                             cudaStream_t stream);
cudaError_t launch_ring_push(void* ring, const void* hid, int B, int L, int M, int start,
                             size_t row_bytes, cudaStream_t stream);
cudaError_t launch_attn_bwd_simt(const void* q, const void* k, const void* v, const void* r,
                                 const void* ub, const void* vb, const void* dout, int bf16, int B,
                                 int H, int L, int M, int dh, float scale, int lo_shift, float* dq,
                                 float* dk, float* dv, float* dr, float* du, float* dvb,
                                 cudaStream_t stream);
cudaError_t launch_layer_norm(const void* x, const void* y, const void* gamma, const void* beta,
                              long long rows, int d, float eps, void* out, cudaStream_t stream);
cudaError_t launch_layer_norm_fwd(const void* x, const void* y, const void* gamma, const void* beta,
                                  long long rows, int d, float eps, void* out, float* mean, float* rstd,
                                  int bf16, cudaStream_t stream);
size_t layer_norm_bwd_workspace_bytes(long long rows, int d, int bf16);
cudaError_t launch_layer_norm_bwd(const void* dout, const void* x, const void* y, const void* gamma,
                                  const float* mean, const float* rstd, const void* dres, long long rows,
                                  int d, void* dx, float* dgamma, float* dbeta, void* workspace, int bf16, int* status,
                                  cudaStream_t stream);
cudaError_t launch_attn_simt_f32(const float* q, const float* k, const float* v, const float* r,
                                 const float* ub, const float* vb, int B, int H, int L, int M,
                                 int dh, float scale, int lo_shift, float* out, cudaStream_t stream);
cudaError_t launch_attn_tc_bf16(const void* q, const void* k, const void* v, const void* r,
                                const void* ub, const void* vb, int B, int H, int L, int M,
                                float scale, int lo_shift, void* out, void* workspace, int inject,
                                int* status, cudaStream_t stream);
size_t attn_tc_bf16_workspace_bytes(int B, int H, int L, int M);
cudaError_t launch_attn_tc_bf16_lse(const void* q, const void* k, const void* v, const void* r, const void* ub,
                                    const void* vb, int B, int H, int L, int M, float scale, int lo_shift,
                                    void* out, float* lse, int* status, cudaStream_t stream);
cudaError_t launch_attn_bwd_tc(const void* q, const void* k, const void* v, const void* r, const void* ub,
                               const void* vb, const void* out, const float* lse, const void* dout, int B, int H,
                               int L, int M, float scale, float* dq, float* dk, float* dv, float* dr, float* du,
                               float* dvb, void* workspace, int* status, cudaStream_t stream);
size_t attn_bwd_tc_workspace_bytes(int B, int H, int L, int M);

// first bounds violation recorded by each translation unit (bounds-checked
// builds; 0 otherwise), read and cleared
unsigned long long bounds_word_attn_simt();
unsigned long long bounds_word_attn_tc();
unsigned long long bounds_word_attn_bwd();
unsigned long long bounds_word_attn_bwd_tc();
unsigned long long bounds_word_mem_update();
unsigned long long bounds_word_layer_norm();
unsigned long long bounds_word_proj_gemm();
unsigned long long bounds_word_layer_norm_train();
unsigned long long bounds_word_adamw();
unsigned long long bounds_word_linear_bwd();
unsigned long long bounds_word_token_logprobs();
unsigned long long bounds_word_grad_norm();
unsigned long long bounds_word_linear_logprobs();

}  // namespace txl

namespace {

// Scratch of txl_attn_fwd_noalloc: one static buffer per device (a module
// global exists once per device context).
__device__ __align__(256) unsigned char g_noalloc_scratch[TXL_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_addr[kMaxDevices] = {};

// Address of the static scratch on the current device.  Outside a stream
// capture it is looked up on every call (cheap), so a context torn down and
// rebuilt (cudaDeviceReset) never leaves a stale address in use; inside a
// capture, where the lookup may not run, the address cached by the last
// lookup on this device is used.
void* noalloc_scratch(cudaStream_t stream) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) return nullptr;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (cap == cudaStreamCaptureStatusNone) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess) return nullptr;
        g_scratch_addr[dev] = p;
    }
    return g_scratch_addr[dev];
}

// Test hook of txl_debug_inject: per host thread, consumed by the next
// bf16 attention launch of the same thread.
thread_local int g_inject = 0;

// Device address of the status word on the current device (looked up per
// call: cheap, and correct when the caller switches devices).
int* dev_status_ptr() {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, txl::g_dev_status) != cudaSuccess) return nullptr;
    return static_cast<int*>(p);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

int elem_size(int dtype) { return dtype == TXL_F32 ? 4 : (dtype == TXL_BF16 ? 2 : 0); }

int check_attn_args(const void* q, const void* k, const void* v, const void* r_k,
                    const void* u_bias, const void* v_bias, int B, int H, int L, int M, int d_h,
                    const void* out, int dtype) {
    const int es = elem_size(dtype);
    if (!es) return TXL_ERR_INVALID_ARG;
    if (!q || !k || !v || !r_k || !u_bias || !v_bias || !out) return TXL_ERR_INVALID_ARG;
    if (B <= 0 || H <= 0 || L <= 0 || M < 0 || d_h <= 0) return TXL_ERR_INVALID_ARG;
    if (dtype == TXL_BF16 && d_h != 64) return TXL_ERR_UNSUPPORTED;
    if (dtype == TXL_F32 && d_h > 256) return TXL_ERR_UNSUPPORTED;
    // index arithmetic in the kernels uses 32-bit row counts per (b, h)
    const long long K = (long long)M + L;
    if (K >= (1ll << 30) || (long long)B * H >= (1ll << 30)) return TXL_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(r_k) || !aligned16(u_bias) ||
        !aligned16(v_bias) || !aligned16(out))
        return TXL_ERR_MISALIGNED;
    const size_t nq = (size_t)B * H * L * d_h * es;
    const size_t nkv = (size_t)B * H * K * d_h * es;
    const size_t nr = (size_t)K * H * d_h * es;
    const size_t nb = (size_t)H * d_h * es;
    if (overlap(out, nq, q, nq) || overlap(out, nq, k, nkv) || overlap(out, nq, v, nkv) ||
        overlap(out, nq, r_k, nr) || overlap(out, nq, u_bias, nb) || overlap(out, nq, v_bias, nb))
        return TXL_ERR_ALIAS;
    return TXL_OK;
}

// Arguments of both backward entry points (gradients fp32, inputs in dtype).
int check_bwd_args(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                   const void* v_bias, const void* dout, int B, int H, int L, int M, int d_h, int same_length,
                   int mem_len, const float* dq, const float* dk, const float* dv, const float* dr,
                   const float* du, const float* dvb, int dtype) {
    const int es = elem_size(dtype);
    if (!es) return TXL_ERR_INVALID_ARG;
    if (!q || !k || !v || !r_k || !u_bias || !v_bias || !dout || !dq || !dk || !dv || !dr || !du || !dvb)
        return TXL_ERR_INVALID_ARG;
    if (B <= 0 || H <= 0 || L <= 0 || M < 0 || d_h <= 0) return TXL_ERR_INVALID_ARG;
    if (same_length && (mem_len < M || mem_len >= (1 << 30))) return TXL_ERR_INVALID_ARG;
    if (d_h > 256) return TXL_ERR_UNSUPPORTED;
    const long long K = (long long)M + L;
    if (K >= (1ll << 30) || (long long)B * H * K * d_h >= (1ll << 40)) return TXL_ERR_UNSUPPORTED;
    const void* ins[7] = {q, k, v, r_k, u_bias, v_bias, dout};
    const void* outs[6] = {dq, dk, dv, dr, du, dvb};
    for (const void* p : ins)
        if (!aligned16(p)) return TXL_ERR_MISALIGNED;
    for (const void* p : outs)
        if (!aligned16(p)) return TXL_ERR_MISALIGNED;
    const size_t nq = (size_t)B * H * L * d_h, nkv = (size_t)B * H * K * d_h, nr = (size_t)K * H * d_h,
                 nb = (size_t)H * d_h;
    const size_t in_n[7] = {nq * es, nkv * es, nkv * es, nr * es, nb * es, nb * es, nq * es};
    const size_t out_n[6] = {nq * 4, nkv * 4, nkv * 4, nr * 4, nb * 4, nb * 4};
    for (int o = 0; o < 6; ++o) {
        for (int i2 = 0; i2 < 7; ++i2)
            if (overlap(outs[o], out_n[o], ins[i2], in_n[i2])) return TXL_ERR_ALIAS;
        for (int o2 = o + 1; o2 < 6; ++o2)
            if (overlap(outs[o], out_n[o], outs[o2], out_n[o2])) return TXL_ERR_ALIAS;
    }
    return TXL_OK;
}

// No lower key bound: the plain causal mask with memory.
constexpr int kNoLowerBound = 1 << 30;

// same_length (source-reading notes, MemTransformerLM._forward): with klen =
// M+L and mask_len = klen - mem_len, query i also ignores keys j <= i -
// mask_shift_len, where mask_shift_len = L - mask_len if mask_len > 0, else L.
int lower_shift(int same_length, int L, int M, int mem_len) {
    if (!same_length) return kNoLowerBound;
    const long long mask_len = (long long)M + L - mem_len;
    return mask_len > 0 ? (int)(L - mask_len) : L;
}

int launch_attn(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                const void* v_bias, int B, int H, int L, int M, int d_h, float scale, void* out,
                int dtype, void* workspace, void* stream, int lo_shift = kNoLowerBound) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == TXL_BF16) {
        int* status = dev_status_ptr();
        if (!status) return TXL_ERR_CUDA;
        const int inject = g_inject;
        g_inject = 0;
        e = txl::launch_attn_tc_bf16(q, k, v, r_k, u_bias, v_bias, B, H, L, M, scale, lo_shift, out,
                                     workspace, inject, status, st);
        if (e == cudaErrorInvalidValue) return TXL_ERR_CUDA;  // tensor-map encoding failed
    } else {
        e = txl::launch_attn_simt_f32(
            static_cast<const float*>(q), static_cast<const float*>(k),
            static_cast<const float*>(v), static_cast<const float*>(r_k),
            static_cast<const float*>(u_bias), static_cast<const float*>(v_bias), B, H, L, M, d_h,
            scale, lo_shift, static_cast<float*>(out), st);
    }
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int txl_attn_fwd(const void* q, const void* k, const void* v, const void* r_k,
                 const void* u_bias, const void* v_bias, int B, int H, int L, int M, int d_h,
                 float scale, void* out, int dtype, void* stream) {
    const int rc = check_attn_args(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, out, dtype);
    if (rc != TXL_OK) return rc;
    return launch_attn(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, scale, out, dtype, nullptr,
                       stream);
}

int txl_attn_fwd_ex(const void* q, const void* k, const void* v, const void* r_k,
                    const void* u_bias, const void* v_bias, int B, int H, int L, int M, int d_h,
                    float scale, int same_length, int mem_len, void* out, int dtype, void* stream) {
    const int rc = check_attn_args(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, out, dtype);
    if (rc != TXL_OK) return rc;
    if (same_length && (mem_len < M || mem_len >= (1 << 30))) return TXL_ERR_INVALID_ARG;
    return launch_attn(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, scale, out, dtype, nullptr,
                       stream, lower_shift(same_length, L, M, mem_len));
}

int txl_attn_bwd(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                 const void* v_bias, const void* dout, int B, int H, int L, int M, int d_h, float scale,
                 int same_length, int mem_len, float* dq, float* dk, float* dv, float* dr, float* du,
                 float* dvb, int dtype, void* stream) {
    const int rc = check_bwd_args(q, k, v, r_k, u_bias, v_bias, dout, B, H, L, M, d_h, same_length, mem_len, dq,
                                  dk, dv, dr, du, dvb, dtype);
    if (rc != TXL_OK) return rc;
    const cudaError_t e = txl::launch_attn_bwd_simt(q, k, v, r_k, u_bias, v_bias, dout, dtype == TXL_BF16, B, H,
                                                    L, M, d_h, scale, lower_shift(same_length, L, M, mem_len),
                                                    dq, dk, dv, dr, du, dvb, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

size_t txl_attn_bwd_workspace_bytes(int B, int H, int L, int M, int d_h, int dtype, int same_length) {
    // the tensor-core backward: bf16, d_h = 64, plain causal mask with memory
    if (dtype != TXL_BF16 || d_h != 64 || same_length || B <= 0 || H <= 0 || L <= 0 || M < 0) return 0;
    if ((long long)M + L >= (1ll << 30) || (long long)B * H >= (1ll << 30)) return 0;
    return txl::attn_bwd_tc_workspace_bytes(B, H, L, M);
}

int txl_attn_bwd_ws(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                    const void* v_bias, const void* dout, int B, int H, int L, int M, int d_h, float scale,
                    int same_length, int mem_len, float* dq, float* dk, float* dv, float* dr, float* du,
                    float* dvb, int dtype, void* workspace, size_t ws_bytes, void* stream) {
    const int rc = check_bwd_args(q, k, v, r_k, u_bias, v_bias, dout, B, H, L, M, d_h, same_length, mem_len, dq,
                                  dk, dv, dr, du, dvb, dtype);
    if (rc != TXL_OK) return rc;
    const size_t need = txl_attn_bwd_workspace_bytes(B, H, L, M, d_h, dtype, same_length);
    if (!need)
        return txl_attn_bwd(q, k, v, r_k, u_bias, v_bias, dout, B, H, L, M, d_h, scale, same_length, mem_len, dq,
                            dk, dv, dr, du, dvb, dtype, stream);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < need) return TXL_ERR_WORKSPACE;
    const long long K = (long long)M + L;
    const size_t nq = (size_t)B * H * L * d_h, nkv = (size_t)B * H * K * d_h, nr = (size_t)K * H * d_h,
                 nb = (size_t)H * d_h;
    const void* others[13] = {q, k, v, r_k, u_bias, v_bias, dout, dq, dk, dv, dr, du, dvb};
    const size_t sizes[13] = {nq * 2, nkv * 2, nkv * 2, nr * 2, nb * 2, nb * 2, nq * 2,
                              nq * 4, nkv * 4, nkv * 4, nr * 4, nb * 4, nb * 4};
    for (int o = 0; o < 13; ++o)
        if (overlap(workspace, need, others[o], sizes[o])) return TXL_ERR_ALIAS;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    const cudaError_t e =
        txl::launch_attn_bwd_tc(q, k, v, r_k, u_bias, v_bias, nullptr, nullptr, dout, B, H, L, M, scale, dq, dk, dv,
                                dr, du, dvb, workspace, status, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidValue) return TXL_ERR_CUDA;  // tensor-map encoding failed
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

int txl_attn_fwd_lse(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                     const void* v_bias, int B, int H, int L, int M, int d_h, float scale, void* out, float* lse,
                     int dtype, void* stream) {
    const int rc = check_attn_args(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, out, dtype);
    if (rc != TXL_OK) return rc;
    if (dtype != TXL_BF16) return TXL_ERR_UNSUPPORTED;
    if (!lse) return TXL_ERR_INVALID_ARG;
    if (!aligned16(lse)) return TXL_ERR_MISALIGNED;
    const size_t nl = (size_t)B * H * L * sizeof(float), nq = (size_t)B * H * L * d_h * 2,
                 nkv = (size_t)B * H * ((size_t)M + L) * d_h * 2, nr = ((size_t)M + L) * H * d_h * 2,
                 nb = (size_t)H * d_h * 2;
    if (overlap(lse, nl, out, nq) || overlap(lse, nl, q, nq) || overlap(lse, nl, k, nkv) ||
        overlap(lse, nl, v, nkv) || overlap(lse, nl, r_k, nr) || overlap(lse, nl, u_bias, nb) ||
        overlap(lse, nl, v_bias, nb))
        return TXL_ERR_ALIAS;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    g_inject = 0;
    const cudaError_t e = txl::launch_attn_tc_bf16_lse(q, k, v, r_k, u_bias, v_bias, B, H, L, M, scale,
                                                       kNoLowerBound, out, lse, status,
                                                       static_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidValue) return TXL_ERR_CUDA;
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

int txl_attn_bwd_saved(const void* q, const void* k, const void* v, const void* r_k, const void* u_bias,
                       const void* v_bias, const void* out, const float* lse, const void* dout, int B, int H, int L,
                       int M, int d_h, float scale, float* dq, float* dk, float* dv, float* dr, float* du,
                       float* dvb, int dtype, void* workspace, size_t ws_bytes, void* stream) {
    const int rc = check_bwd_args(q, k, v, r_k, u_bias, v_bias, dout, B, H, L, M, d_h, 0, M, dq, dk, dv, dr, du,
                                  dvb, dtype);
    if (rc != TXL_OK) return rc;
    if (dtype != TXL_BF16 || d_h != 64) return TXL_ERR_UNSUPPORTED;
    if (!out || !lse) return TXL_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(lse)) return TXL_ERR_MISALIGNED;
    const size_t need = txl_attn_bwd_workspace_bytes(B, H, L, M, d_h, dtype, 0);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < need) return TXL_ERR_WORKSPACE;
    const long long K = (long long)M + L;
    const size_t nq = (size_t)B * H * L * d_h, nkv = (size_t)B * H * K * d_h, nr = (size_t)K * H * d_h,
                 nb = (size_t)H * d_h, nl = (size_t)B * H * L;
    const void* others[15] = {q, k, v, r_k, u_bias, v_bias, dout, out, lse, dq, dk, dv, dr, du, dvb};
    const size_t sizes[15] = {nq * 2, nkv * 2, nkv * 2, nr * 2, nb * 2, nb * 2, nq * 2, nq * 2, nl * 4,
                              nq * 4, nkv * 4, nkv * 4, nr * 4, nb * 4, nb * 4};
    for (int o = 0; o < 15; ++o)
        if (overlap(workspace, need, others[o], sizes[o])) return TXL_ERR_ALIAS;
    // the gradients must not overlap the saved forward state either
    const void* gr[6] = {dq, dk, dv, dr, du, dvb};
    const size_t gn[6] = {nq * 4, nkv * 4, nkv * 4, nr * 4, nb * 4, nb * 4};
    for (int o = 0; o < 6; ++o)
        if (overlap(gr[o], gn[o], out, nq * 2) || overlap(gr[o], gn[o], lse, nl * 4)) return TXL_ERR_ALIAS;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    const cudaError_t e =
        txl::launch_attn_bwd_tc(q, k, v, r_k, u_bias, v_bias, out, lse, dout, B, H, L, M, scale, dq, dk, dv, dr, du,
                                dvb, workspace, status, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidValue) return TXL_ERR_CUDA;
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

size_t txl_attn_workspace_bytes(int B, int H, int L, int M, int d_h, int dtype) {
    // only the bf16 kernel splits; sizes a call would reject need nothing
    if (dtype != TXL_BF16 || d_h != 64 || B <= 0 || H <= 0 || L <= 0 || M < 0) return 0;
    if ((long long)M + L >= (1ll << 30) || (long long)B * H >= (1ll << 30)) return 0;
    return txl::attn_tc_bf16_workspace_bytes(B, H, L, M);
}

int txl_attn_fwd_ws(const void* q, const void* k, const void* v, const void* r_k,
                    const void* u_bias, const void* v_bias, int B, int H, int L, int M, int d_h,
                    float scale, void* out, int dtype, void* workspace, size_t ws_bytes,
                    void* stream) {
    const int rc = check_attn_args(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, out, dtype);
    if (rc != TXL_OK) return rc;
    const size_t need = txl_attn_workspace_bytes(B, H, L, M, d_h, dtype);
    if (need) {
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < need)
            return TXL_ERR_WORKSPACE;
        const int es = elem_size(dtype);
        const size_t nq = (size_t)B * H * L * d_h * es, nkv = (size_t)B * H * ((size_t)M + L) * d_h * es;
        if (overlap(workspace, need, out, nq) || overlap(workspace, need, q, nq) ||
            overlap(workspace, need, k, nkv) || overlap(workspace, need, v, nkv))
            return TXL_ERR_ALIAS;
    }
    return launch_attn(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, scale, out, dtype,
                       need ? workspace : nullptr, stream);
}

int txl_mem_update(void* mems, const void* hids, int B, int L, int M, int d, int dtype,
                   void* stream) {
    return txl_mem_update_ext(mems, hids, B, L, M, d, 0, dtype, stream);
}

int txl_mem_update_ext(void* mems, const void* hids, int B, int L, int M, int d, int ext_len,
                       int dtype, void* stream) {
    const int es = elem_size(dtype);
    if (!es || B <= 0 || L <= 0 || M < 0 || d <= 0 || ext_len < 0) return TXL_ERR_INVALID_ARG;
    if (M == 0) return TXL_OK;
    if (!mems || !hids) return TXL_ERR_INVALID_ARG;
    if ((long long)B * (M > L ? M : L) * d >= (1ll << 40)) return TXL_ERR_UNSUPPORTED;
    const size_t row = (size_t)d * es;
    if (overlap(mems, (size_t)B * M * row, hids, (size_t)B * L * row)) return TXL_ERR_ALIAS;
    const int used = ext_len < L ? L - ext_len : 0;  // rows of h that enter the memory
    const cudaError_t e =
        txl::launch_tail_m(mems, hids, B, used, L, M, row, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

int txl_mem_ring_push(void* ring, const void* hids, int B, int L, int M, int d, int start,
                      int* new_start, int dtype, void* stream) {
    const int es = elem_size(dtype);
    if (!es || B <= 0 || L <= 0 || M < 0 || d <= 0 || !new_start) return TXL_ERR_INVALID_ARG;
    if (start < 0 || (M > 0 && start >= M) || (M == 0 && start != 0)) return TXL_ERR_INVALID_ARG;
    if (M == 0) {
        *new_start = 0;
        return TXL_OK;
    }
    if (!ring || !hids) return TXL_ERR_INVALID_ARG;
    if ((long long)B * (M > L ? M : L) * d >= (1ll << 40)) return TXL_ERR_UNSUPPORTED;
    const size_t row = (size_t)d * es;
    if (overlap(ring, (size_t)B * M * row, hids, (size_t)B * L * row)) return TXL_ERR_ALIAS;
    cudaError_t e;
    if (L >= M) {
        // the whole memory is replaced by the newest M rows: the Tail_M copy
        e = txl::launch_tail_m(ring, hids, B, L, L, M, row, static_cast<cudaStream_t>(stream));
        *new_start = 0;
    } else {
        e = txl::launch_ring_push(ring, hids, B, L, M, start, row, static_cast<cudaStream_t>(stream));
        *new_start = (start + L) % M;
    }
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

int txl_mem_reset(void* mems, const void* flags, int B, int rows, int d, int dtype, void* stream) {
    const int es = elem_size(dtype);
    if (!es || B <= 0 || rows < 0 || d <= 0 || !flags) return TXL_ERR_INVALID_ARG;
    if (rows == 0) return TXL_OK;
    if (!mems) return TXL_ERR_INVALID_ARG;
    const long long per_b = (long long)rows * d * es;
    if ((long long)B * per_b >= (1ll << 40)) return TXL_ERR_UNSUPPORTED;
    if (overlap(mems, (size_t)(B * per_b), flags, (size_t)B)) return TXL_ERR_ALIAS;
    const cudaError_t e = txl::launch_mem_reset(mems, static_cast<const unsigned char*>(flags), B, per_b,
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

int txl_sync_status(void* stream) {
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return TXL_ERR_CUDA;
    int status = 0;
    e = cudaMemcpyFromSymbol(&status, txl::g_dev_status, sizeof(int));
    if (e != cudaSuccess) return TXL_ERR_CUDA;
    if (status != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(txl::g_dev_status, &zero, sizeof(int)) != cudaSuccess)
            return TXL_ERR_CUDA;
        return TXL_ERR_DEVICE_TIMEOUT;
    }
    return TXL_OK;
}

int txl_attn_fwd_noalloc(const void* q, const void* k, const void* v, const void* r_k,
                         const void* u_bias, const void* v_bias, int B, int H, int L, int M,
                         int d_h, float scale, void* out, int dtype, void* stream) {
    const int rc = check_attn_args(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, out, dtype);
    if (rc != TXL_OK) return rc;
    const size_t need = txl_attn_workspace_bytes(B, H, L, M, d_h, dtype);
    if (need > TXL_NOALLOC_SCRATCH_BYTES) return TXL_ERR_SCRATCH_LIMIT;
    void* scratch = nullptr;
    if (need) {
        scratch = noalloc_scratch(static_cast<cudaStream_t>(stream));
        if (!scratch) return TXL_ERR_CUDA;
    }
    return launch_attn(q, k, v, r_k, u_bias, v_bias, B, H, L, M, d_h, scale, out, dtype, scratch,
                       stream);
}

int txl_qkv_proj(const void* h, const void* mem, const void* w_qkv, int B, int L, int M, int H,
                 int d_h, void* q, void* k, void* v, void* stream) {
    return txl_qkv_proj_ex(h, TXL_LAYOUT_ROWS, mem, TXL_LAYOUT_ROWS, w_qkv, B, L, M, H, d_h, q, k, v,
                           stream);
}

int txl_qkv_proj_ex(const void* h, int h_layout, const void* mem, int mem_layout,
                    const void* w_qkv, int B, int L, int M, int H, int d_h, void* q, void* k,
                    void* v, void* stream) {
    return txl_qkv_proj_ring(h, h_layout, mem, mem_layout, 0, w_qkv, B, L, M, H, d_h, q, k, v, stream);
}

}  // extern "C"

namespace {

// Host validation of the q/k/v projections (txl_qkv_proj_ring's contract).
int check_qkv(const void* h, int h_layout, const void* mem, int mem_layout, int mem_start,
              const void* w_qkv, int B, int L, int M, int H, int d_h, void* q, void* k, void* v) {
    if (!h || !w_qkv || !q || !k || !v || (M > 0 && !mem)) return TXL_ERR_INVALID_ARG;
    const auto layout_ok = [](int l) { return l == TXL_LAYOUT_ROWS || l == TXL_LAYOUT_HEADS; };
    if (!layout_ok(h_layout) || !layout_ok(mem_layout)) return TXL_ERR_INVALID_ARG;
    if (mem_start < 0 || (M > 0 && mem_start >= M) || (M == 0 && mem_start != 0))
        return TXL_ERR_INVALID_ARG;
    if (mem_start % 128 != 0) return TXL_ERR_UNSUPPORTED;
    if (B <= 0 || L <= 0 || M < 0 || H <= 0 || d_h <= 0) return TXL_ERR_INVALID_ARG;
    if (d_h != 64 || H % 4 != 0 || L % 128 != 0 || M % 128 != 0) return TXL_ERR_UNSUPPORTED;
    const long long d = (long long)H * d_h;
    if ((long long)B * (M + L) * d >= (1ll << 31) || (long long)(M + L) >= (1ll << 20))
        return TXL_ERR_UNSUPPORTED;
    if (!aligned16(h) || !aligned16(w_qkv) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
        (M > 0 && !aligned16(mem)))
        return TXL_ERR_MISALIGNED;
    const size_t nh = (size_t)B * L * d * 2, nm = (size_t)B * M * d * 2, nw = (size_t)3 * d * d * 2;
    const size_t nq = nh, nkv = (size_t)B * (M + L) * d * 2;
    const void* outs[3] = {q, k, v};
    const size_t nout[3] = {nq, nkv, nkv};
    for (int o = 0; o < 3; ++o) {
        if (overlap(outs[o], nout[o], h, nh) || overlap(outs[o], nout[o], w_qkv, nw) ||
            (M > 0 && overlap(outs[o], nout[o], mem, nm)))
            return TXL_ERR_ALIAS;
        for (int o2 = o + 1; o2 < 3; ++o2)
            if (overlap(outs[o], nout[o], outs[o2], nout[o2])) return TXL_ERR_ALIAS;
    }
    return TXL_OK;
}

// Host validation of the position projection (txl_r_proj's contract).
int check_r(const void* emb, const void* w_r, int K, int H, int d_h, void* r_k) {
    if (!emb || !w_r || !r_k || K <= 0 || H <= 0 || d_h <= 0) return TXL_ERR_INVALID_ARG;
    if (d_h != 64 || H % 4 != 0 || K % 128 != 0) return TXL_ERR_UNSUPPORTED;
    const long long d = (long long)H * d_h;
    if ((long long)K * d >= (1ll << 31)) return TXL_ERR_UNSUPPORTED;
    if (!aligned16(emb) || !aligned16(w_r) || !aligned16(r_k)) return TXL_ERR_MISALIGNED;
    const size_t nr = (size_t)K * d * 2;
    if (overlap(r_k, nr, emb, nr) || overlap(r_k, nr, w_r, (size_t)d * d * 2)) return TXL_ERR_ALIAS;
    return TXL_OK;
}

// The q and k|v problems of one layer's projection launch.
void qkv_problems(txl::ProjGemm* gm, const void* h, int h_layout, const void* mem, int mem_layout,
                  int mem_start, const void* w_qkv, int L, int M, long long d, void* q, void* k, void* v) {
    const unsigned char* w = static_cast<const unsigned char*>(w_qkv);
    const int hh = h_layout == TXL_LAYOUT_HEADS, mh = mem_layout == TXL_LAYOUT_HEADS;
    gm[0] = {nullptr, h, 0, L, 0, hh, w, (int)d, L, {q, nullptr, nullptr}};
    gm[1] = {M > 0 ? mem : nullptr, h, M, L, mh, hh, w + (size_t)d * d * 2, (int)(2 * d), M + L,
             {k, v, nullptr}, mem_start};
}

int launch_status(cudaError_t e) {
    if (e == cudaErrorInvalidValue) return TXL_ERR_CUDA;  // a tensor map could not be encoded
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int txl_qkv_proj_ring(const void* h, int h_layout, const void* mem, int mem_layout, int mem_start,
                      const void* w_qkv, int B, int L, int M, int H, int d_h, void* q, void* k,
                      void* v, void* stream) {
    const int rc = check_qkv(h, h_layout, mem, mem_layout, mem_start, w_qkv, B, L, M, H, d_h, q, k, v);
    if (rc != TXL_OK) return rc;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    // one launch: q from h and W_q; k, v from [mem; h] and the W_k, W_v rows
    txl::ProjGemm gm[2];
    qkv_problems(gm, h, h_layout, mem, mem_layout, mem_start, w_qkv, L, M, (long long)H * d_h, q, k, v);
    return launch_status(txl::launch_proj_gemm(gm, 2, B, H * d_h, H * d_h, H, d_h, 0, status,
                                               static_cast<cudaStream_t>(stream)));
}

int txl_qkvr_proj(const void* h, int h_layout, const void* mem, int mem_layout, int mem_start,
                  const void* w_qkv, const void* emb, const void* w_r, int B, int L, int M, int H,
                  int d_h, void* q, void* k, void* v, void* r_k, void* stream) {
    int rc = check_qkv(h, h_layout, mem, mem_layout, mem_start, w_qkv, B, L, M, H, d_h, q, k, v);
    if (rc != TXL_OK) return rc;
    rc = check_r(emb, w_r, M + L, H, d_h, r_k);
    if (rc != TXL_OK) return rc;
    const long long d = (long long)H * d_h;
    const size_t nr = (size_t)(M + L) * d * 2, nq = (size_t)B * L * d * 2, nkv = (size_t)B * (M + L) * d * 2;
    const size_t nh = nq, nm = (size_t)B * M * d * 2, nw = (size_t)3 * d * d * 2;
    // r_k overlaps no other output and no input of the q/k/v problems
    if (overlap(r_k, nr, q, nq) || overlap(r_k, nr, k, nkv) || overlap(r_k, nr, v, nkv) ||
        overlap(r_k, nr, h, nh) || overlap(r_k, nr, w_qkv, nw) || (M > 0 && overlap(r_k, nr, mem, nm)))
        return TXL_ERR_ALIAS;
    const void* outs[3] = {q, k, v};
    const size_t nout[3] = {nq, nkv, nkv};
    for (int o = 0; o < 3; ++o)
        if (overlap(outs[o], nout[o], emb, nr) || overlap(outs[o], nout[o], w_r, (size_t)d * d * 2))
            return TXL_ERR_ALIAS;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    // one launch: q, k|v as in txl_qkv_proj_ring, and r from the position
    // embedding (one batch row, row-major output)
    txl::ProjGemm gm[3];
    qkv_problems(gm, h, h_layout, mem, mem_layout, mem_start, w_qkv, L, M, d, q, k, v);
    gm[2] = {nullptr, emb, 0, M + L, 0, 0, w_r, (int)d, M + L, {r_k, nullptr, nullptr}, 0, 1, 1};
    return launch_status(txl::launch_proj_gemm(gm, 3, B, (int)d, (int)d, H, d_h, 0, status,
                                               static_cast<cudaStream_t>(stream)));
}

int txl_r_proj(const void* emb, const void* w_r, int K, int H, int d_h, void* r_k, void* stream) {
    const int rc = check_r(emb, w_r, K, H, d_h, r_k);
    if (rc != TXL_OK) return rc;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    const long long d = (long long)H * d_h;
    const txl::ProjGemm gm = {nullptr, emb, 0, K, 0, 0, w_r, (int)d, K, {r_k, nullptr, nullptr}};
    return launch_status(txl::launch_proj_gemm(&gm, 1, 1, (int)d, (int)d, H, d_h, 1, status,
                                               static_cast<cudaStream_t>(stream)));
}

int txl_linear(const void* x, int x_layout, int B, int T, int K, const void* w, int N,
               const void* bias, const void* resid, int relu, void* out, void* stream) {
    if (!x || !w || !out || B <= 0 || T <= 0 || K <= 0 || N <= 0) return TXL_ERR_INVALID_ARG;
    if (x_layout != TXL_LAYOUT_ROWS && x_layout != TXL_LAYOUT_HEADS) return TXL_ERR_INVALID_ARG;
    if (T % 128 != 0 || K % 64 != 0 || N % 256 != 0) return TXL_ERR_UNSUPPORTED;
    if ((long long)B * T * (K > N ? K : N) >= (1ll << 31) || (long long)T >= (1ll << 24))
        return TXL_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(w) || !aligned16(out) || (bias && !aligned16(bias)) ||
        (resid && !aligned16(resid)))
        return TXL_ERR_MISALIGNED;
    const size_t nx = (size_t)B * T * K * 2, nw = (size_t)N * K * 2, no = (size_t)B * T * N * 2;
    if (overlap(out, no, x, nx) || overlap(out, no, w, nw) || (bias && overlap(out, no, bias, (size_t)N * 2)))
        return TXL_ERR_ALIAS;
    if (resid && resid != out && overlap(out, no, resid, no)) return TXL_ERR_ALIAS;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    const cudaError_t e = txl::launch_linear(x, x_layout == TXL_LAYOUT_HEADS, B, T, K, w, N, bias, resid,
                                             relu ? 1 : 0, out, status, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidValue) return TXL_ERR_CUDA;
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

int txl_layer_norm(const void* x, const void* y, const void* gamma, const void* beta, long long rows,
                   int d, float eps, void* out, void* stream) {
    if (!x || !gamma || !beta || !out || rows < 0 || d <= 0 || !(eps >= 0.f)) return TXL_ERR_INVALID_ARG;
    if (d % 256 != 0 || d > 2048 || d == 1280 || d == 1792) return TXL_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(out) || (y && !aligned16(y)))
        return TXL_ERR_MISALIGNED;
    const size_t n = (size_t)rows * d * 2;
    if ((out != x && overlap(out, n, x, n)) || (y && out != y && overlap(out, n, y, n)) ||
        overlap(out, n, gamma, (size_t)d * 2) || overlap(out, n, beta, (size_t)d * 2))
        return TXL_ERR_ALIAS;
    const cudaError_t e =
        txl::launch_layer_norm(x, y, gamma, beta, rows, d, eps, out, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH;
}

}  // extern "C"

namespace {

// A byte range of a call's arguments, for overlap checks over many of them.
struct Range {
    uintptr_t at, end;
    bool written;
};

Range range_of(const void* p, size_t n, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + n, written};
}

// Whether a written range overlaps any other.  Sorts the ranges.
bool any_written_overlap(Range* r, size_t n) {
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.at < b.at; });
    uintptr_t end = 0, written_end = 0;  // how far the ranges before this one reach
    for (size_t i = 0; i < n; ++i) {
        if (!r[i].at || r[i].at == r[i].end) continue;
        if (r[i].at < written_end || (r[i].written && r[i].at < end)) return true;
        end = std::max(end, r[i].end);
        if (r[i].written) written_end = std::max(written_end, r[i].end);
    }
    return false;
}

constexpr int kLayerNormMaxD = 16384;

// At most 2^31 - 1 rows (a CTA takes one or more), rows * d below 2^40.
bool row_data_too_large(long long rows, int d) { return rows > 0x7FFFFFFFll || rows > (1ll << 40) / d; }

bool bad_workspace(const void* workspace, size_t bytes, size_t need) {
    return need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || bytes < need);
}

int linear_bwd_sizes(int x_layout, int B, int T, int K, int N) {
    if (x_layout != TXL_LAYOUT_ROWS && x_layout != TXL_LAYOUT_HEADS) return TXL_ERR_INVALID_ARG;
    if (B <= 0 || T <= 0 || K <= 0 || N <= 0) return TXL_ERR_INVALID_ARG;
    if (K % 8 != 0 || N % 8 != 0 || (x_layout == TXL_LAYOUT_HEADS && K % 64 != 0)) return TXL_ERR_UNSUPPORTED;
    const long long rows = (long long)B * T;
    if (rows > (1ll << 28) || K > (1 << 20) || N > (1 << 20)) return TXL_ERR_UNSUPPORTED;
    const long long row_tiles = (x_layout == TXL_LAYOUT_HEADS ? B * ((T + 127ll) / 128) : (rows + 127) / 128) +
                                (N + 127ll) / 128 * 32;  // dw's tiles, over at most 32 splits
    if (row_tiles * ((K + 127ll) / 128) > (1ll << 30)) return TXL_ERR_UNSUPPORTED;
    return TXL_OK;
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Logits: 2^31 - 1 rows, 2^24 columns (a thread's chains of additions stay below 2^11) and 2^40
// elements at most.
constexpr int kMostColumns = 1 << 24;
bool logit_rows_too_large(long long rows, int V, long long ld) {
    return V > kMostColumns || rows > 0x7FFFFFFFll || ld > (1ll << 40) || rows > (1ll << 40) / ld;
}

// Bytes from the first row's begin to the last one's end.
size_t row_span(long long rows, int V, long long ld, int es) { return ((size_t)(rows - 1) * ld + V) * es; }

int linear_logprobs_sizes(long long rows, int K, int V) {
    if (rows < 0 || K <= 0 || V <= 0) return TXL_ERR_INVALID_ARG;
    if (K % 8 != 0 || K > (1 << 20) || V > kMostColumns || rows > (1ll << 28) || rows > (1ll << 40) / V) return TXL_ERR_UNSUPPORTED;
    return TXL_OK;
}

int grad_tensors_status(const txl_grad_tensor* tensors, int n_tensors) {
    if (!tensors || n_tensors <= 0) return TXL_ERR_INVALID_ARG;
    long long total = 0;
    for (int i = 0; i < n_tensors; ++i) {
        if (tensors[i].n < 0 || !elem_size(tensors[i].dtype)) return TXL_ERR_INVALID_ARG;
        if (tensors[i].n > (1ll << 38) || total > (1ll << 40) - tensors[i].n) return TXL_ERR_UNSUPPORTED;
        total += tensors[i].n;
    }
    return TXL_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? TXL_OK : TXL_ERR_LAUNCH; }

}  // namespace

extern "C" {

int txl_layer_norm_fwd(const void* x, const void* y, const void* gamma, const void* beta, long long rows,
                       int d, float eps, void* out, float* mean, float* rstd, int dtype, void* stream) {
    const int es = elem_size(dtype);
    if (!es || rows < 0 || d <= 0 || !(eps >= 0.f)) return TXL_ERR_INVALID_ARG;
    if (d > kLayerNormMaxD || row_data_too_large(rows, d)) return TXL_ERR_UNSUPPORTED;
    if (rows == 0) return TXL_OK;
    if (!x || !gamma || !beta || !out || !mean || !rstd) return TXL_ERR_INVALID_ARG;
    for (const void* p : {x, y, gamma, beta, (const void*)out, (const void*)mean, (const void*)rstd})
        if (!aligned16(p)) return TXL_ERR_MISALIGNED;
    const size_t n = (size_t)rows * d * es, nd = (size_t)d * es, nr = (size_t)rows * sizeof(float);
    Range r[] = {range_of(x, n, false),    range_of(y, n, false),  range_of(gamma, nd, false),
                 range_of(beta, nd, false), range_of(out, n, true), range_of(mean, nr, true),
                 range_of(rstd, nr, true)};
    if (any_written_overlap(r, sizeof(r) / sizeof(r[0]))) return TXL_ERR_ALIAS;
    return cuda_status(txl::launch_layer_norm_fwd(x, y, gamma, beta, rows, d, eps, out, mean, rstd,
                                                  dtype == TXL_BF16, static_cast<cudaStream_t>(stream)));
}

size_t txl_layer_norm_bwd_workspace_bytes(long long rows, int d, int dtype) {
    if (!elem_size(dtype) || rows < 0 || d <= 0 || d > kLayerNormMaxD || row_data_too_large(rows, d)) return 0;
    return txl::layer_norm_bwd_workspace_bytes(rows, d, dtype == TXL_BF16);
}

int txl_layer_norm_bwd(const void* dout, const void* x, const void* y, const void* gamma, const float* mean,
                       const float* rstd, const void* dres, long long rows, int d, void* dx, float* dgamma,
                       float* dbeta, int dtype, void* workspace, size_t ws_bytes, void* stream) {
    const int es = elem_size(dtype);
    if (!es || rows < 0 || d <= 0 || !dgamma || !dbeta) return TXL_ERR_INVALID_ARG;
    if (rows > 0 && (!dout || !x || !gamma || !mean || !rstd || !dx)) return TXL_ERR_INVALID_ARG;
    if (d > kLayerNormMaxD || row_data_too_large(rows, d)) return TXL_ERR_UNSUPPORTED;
    if (!aligned16(dgamma) || !aligned16(dbeta)) return TXL_ERR_MISALIGNED;
    if (rows > 0)
        for (const void* p : {dout, x, y, gamma, (const void*)mean, (const void*)rstd, dres, (const void*)dx})
            if (!aligned16(p)) return TXL_ERR_MISALIGNED;
    const size_t need = txl_layer_norm_bwd_workspace_bytes(rows, d, dtype);
    if (bad_workspace(workspace, ws_bytes, need)) return TXL_ERR_WORKSPACE;
    const size_t n = (size_t)rows * d * es, nd = (size_t)d * sizeof(float), nr = (size_t)rows * sizeof(float);
    Range r[] = {range_of(dout, n, false),  range_of(x, n, false),      range_of(y, n, false),
                 range_of(gamma, rows > 0 ? (size_t)d * es : 0, false), range_of(mean, nr, false),
                 range_of(rstd, nr, false), range_of(dres, n, false),   range_of(dx, n, true),
                 range_of(dgamma, nd, true), range_of(dbeta, nd, true), range_of(workspace, need, true)};
    if (any_written_overlap(r, sizeof(r) / sizeof(r[0]))) return TXL_ERR_ALIAS;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    return cuda_status(txl::launch_layer_norm_bwd(dout, x, y, gamma, mean, rstd, dres, rows, d, dx, dgamma, dbeta,
                                                  workspace, dtype == TXL_BF16, status,
                                                  static_cast<cudaStream_t>(stream)));
}

size_t txl_linear_bwd_workspace_bytes(int x_layout, int B, int T, int K, int N, int want_dx, int want_dw,
                                      int want_db) {
    if (linear_bwd_sizes(x_layout, B, T, K, N) != TXL_OK || (!want_dx && !want_dw)) return 0;
    return txl::linear_bwd_workspace_bytes(
        txl::linear_bwd_plan(x_layout == TXL_LAYOUT_HEADS, B, T, K, N, want_dx != 0, want_dw != 0), want_dw && want_db);
}

int txl_linear_bwd(const void* dy, const void* x, int x_layout, int B, int T, int K, const void* w, int N,
                   int relu_in, void* dx, float* dw, float* db, void* workspace, size_t ws_bytes, void* stream) {
    if (!dy || !x || !w || (!dx && !dw) || (db && !dw)) return TXL_ERR_INVALID_ARG;
    const int rc = linear_bwd_sizes(x_layout, B, T, K, N);
    if (rc != TXL_OK) return rc;
    for (const void* p : {dy, x, w, (const void*)dx, (const void*)dw, (const void*)db})
        if (!aligned16(p)) return TXL_ERR_MISALIGNED;
    const txl::LbPlan plan =
        txl::linear_bwd_plan(x_layout == TXL_LAYOUT_HEADS, B, T, K, N, dx != nullptr, dw != nullptr);
    const size_t need = txl::linear_bwd_workspace_bytes(plan, db != nullptr);
    if (bad_workspace(workspace, ws_bytes, need)) return TXL_ERR_WORKSPACE;
    const size_t rows = (size_t)B * T, nx = rows * K * 2, nw = (size_t)N * K;
    Range r[] = {range_of(dy, rows * N * 2, false),     range_of(x, nx, false),
                 range_of(w, nw * 2, false),            range_of(dx, nx, true),
                 range_of(dw, nw * 4, true),            range_of(db, (size_t)N * 4, true),
                 range_of(need ? workspace : nullptr, need, true)};
    if (any_written_overlap(r, sizeof(r) / sizeof(r[0]))) return TXL_ERR_ALIAS;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    return launch_status(txl::launch_linear_bwd(plan, dy, x, w, relu_in != 0, dx, dw, db, workspace, status,
                                                static_cast<cudaStream_t>(stream)));
}

int txl_token_logprobs(const void* logits, long long ld, const long long* tokens, long long rows, int V, int top,
                       float* logprob, float* lse, float* entropy, long long* top_index, float* top_logprob,
                       int dtype, void* stream) {
    const int es = elem_size(dtype);
    if (!es || rows < 0 || V <= 0 || ld < V || top < 0 || top > V) return TXL_ERR_INVALID_ARG;
    if (logit_rows_too_large(rows, V, ld) || top > txl::kTopMost) return TXL_ERR_UNSUPPORTED;
    if (rows == 0) return TXL_OK;
    if (!logits || !tokens || !logprob || !lse || !entropy || (top != 0) != (top_index != nullptr) ||
        (top != 0) != (top_logprob != nullptr))
        return TXL_ERR_INVALID_ARG;
    if (!aligned_to(logits, es) || !aligned_to(tokens, 8) || !aligned_to(logprob, 4) || !aligned_to(lse, 4) ||
        !aligned_to(entropy, 4) || !aligned_to(top_index, 8) || !aligned_to(top_logprob, 4))
        return TXL_ERR_MISALIGNED;
    const size_t nr = (size_t)rows * sizeof(float);
    Range r[] = {range_of(logits, row_span(rows, V, ld, es), false), range_of(tokens, 2 * nr, false),
                 range_of(logprob, nr, true), range_of(lse, nr, true), range_of(entropy, nr, true),
                 range_of(top_index, 2 * nr * top, true), range_of(top_logprob, nr * top, true)};
    if (any_written_overlap(r, sizeof(r) / sizeof(r[0]))) return TXL_ERR_ALIAS;
    const txl::TokenLogprobs a = {logits, ld, tokens, rows, V, top, logprob, lse, entropy, top_index, top_logprob};
    return cuda_status(txl::launch_token_logprobs(a, dtype == TXL_BF16, static_cast<cudaStream_t>(stream)));
}

int txl_token_logprobs_bwd(const void* logits, long long ld, const long long* tokens, const float* lse,
                           const float* entropy, const float* dlogprob, const float* dlse, const float* dentropy,
                           long long rows, int V, void* dlogits, long long ldd, int dtype, void* stream) {
    const int es = elem_size(dtype);
    if (!es || rows < 0 || V <= 0 || ld < V || ldd < V) return TXL_ERR_INVALID_ARG;
    if ((!dlogprob && !dlse && !dentropy && rows > 0) || (entropy && !dentropy)) return TXL_ERR_INVALID_ARG;
    if (logit_rows_too_large(rows, V, std::max(ld, ldd))) return TXL_ERR_UNSUPPORTED;
    if (rows == 0) return TXL_OK;
    if (!logits || !tokens || !lse || !dlogits || (dentropy && !entropy)) return TXL_ERR_INVALID_ARG;
    if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(tokens, 8)) return TXL_ERR_MISALIGNED;
    for (const float* p : {lse, entropy, dlogprob, dlse, dentropy})
        if (!aligned_to(p, 4)) return TXL_ERR_MISALIGNED;
    const size_t nr = (size_t)rows * sizeof(float);
    const bool in_place = dlogits == logits && (ldd == ld || rows == 1);
    Range r[] = {range_of(in_place ? nullptr : logits, row_span(rows, V, ld, es), false),
                 range_of(dlogits, row_span(rows, V, ldd, es), true),
                 range_of(tokens, 2 * nr, false),
                 range_of(lse, nr, false),
                 range_of(entropy, nr, false),
                 range_of(dlogprob, nr, false),
                 range_of(dlse, nr, false),
                 range_of(dentropy, nr, false)};
    if (any_written_overlap(r, sizeof(r) / sizeof(r[0]))) return TXL_ERR_ALIAS;
    const txl::TokenLogprobsBwd a = {logits, ld, tokens, lse, entropy, dlogprob, dlse, dentropy, rows, V, dlogits, ldd};
    return cuda_status(txl::launch_token_logprobs_bwd(a, dtype == TXL_BF16, static_cast<cudaStream_t>(stream)));
}

size_t txl_linear_logprobs_workspace_bytes(long long rows, int K, int V) {
    if (linear_logprobs_sizes(rows, K, V) != TXL_OK || rows == 0) return 0;
    return std::max(txl::linear_logprobs_workspace_bytes(txl::linear_logprobs_plan((int)rows, K, V, false)),
                    txl::linear_logprobs_workspace_bytes(txl::linear_logprobs_plan((int)rows, K, V, true)));
}

int txl_linear_logprobs(const void* x, const void* w, const void* bias, const long long* tokens, long long rows, int K,
                        int V, float* logprob, float* lse, float* entropy, void* workspace, size_t ws_bytes,
                        void* stream) {
    const int rc = linear_logprobs_sizes(rows, K, V);
    if (rc != TXL_OK) return rc;
    if (rows == 0) return TXL_OK;
    if (!x || !w || !tokens || !logprob || !lse || !entropy) return TXL_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned_to(bias, 2) || !aligned_to(tokens, 8) || !aligned_to(logprob, 4) ||
        !aligned_to(lse, 4) || !aligned_to(entropy, 4))
        return TXL_ERR_MISALIGNED;
    const txl::LpPlan plan = txl::linear_logprobs_plan((int)rows, K, V, bias != nullptr);
    // (a workspace serves calls with a bias and without)
    const size_t need = std::max(txl::linear_logprobs_workspace_bytes(plan),
                                 txl::linear_logprobs_workspace_bytes(txl::linear_logprobs_plan((int)rows, K, V, bias == nullptr)));
    if (bad_workspace(workspace, ws_bytes, need)) return TXL_ERR_WORKSPACE;
    const size_t nr = (size_t)rows * sizeof(float);
    Range r[] = {range_of(x, (size_t)rows * K * 2, false), range_of(w, (size_t)V * K * 2, false),
                 range_of(bias, (size_t)V * 2, false),     range_of(tokens, 2 * nr, false),
                 range_of(logprob, nr, true),              range_of(lse, nr, true),
                 range_of(entropy, nr, true),              range_of(workspace, need, true)};
    if (any_written_overlap(r, sizeof(r) / sizeof(r[0]))) return TXL_ERR_ALIAS;
    int* status = dev_status_ptr();
    if (!status) return TXL_ERR_CUDA;
    return launch_status(txl::launch_linear_logprobs(plan, x, w, bias, K, tokens, logprob, lse, entropy, workspace, need, status,
                                                     static_cast<cudaStream_t>(stream)));
}

long long txl_adamw_state_elements(const txl_adamw_tensor* tensors, int n_tensors) {
    if (!tensors || n_tensors <= 0) return -1;
    long long blocks = 0;
    for (int i = 0; i < n_tensors; ++i) {
        if (tensors[i].n < 0 || tensors[i].n > (1ll << 38)) return -1;
        blocks += (tensors[i].n + txl::kAdamwBlock - 1) / txl::kAdamwBlock;
        if (blocks > (1ll << 30)) return -1;
    }
    return blocks * txl::kAdamwBlock;
}

size_t txl_adamw_workspace_bytes(const txl_adamw_tensor* tensors, int n_tensors) {
    const long long n = txl_adamw_state_elements(tensors, n_tensors);
    return n < 0 ? 0 : txl::adamw_workspace_bytes(n / txl::kAdamwBlock);
}

int txl_adamw_step(const txl_adamw_tensor* tensors, int n_tensors, int param_dtype, int grad_dtype,
                   int state_bits, float* master, void* exp_avg, float* exp_avg_scale, void* exp_avg_sq,
                   float* exp_avg_sq_scale, long long* steps, const float* lr, double beta1, double beta2,
                   double eps, double max_norm, unsigned seed, float* grad_norm, void* workspace,
                   size_t ws_bytes, void* stream) {
    const int ep = elem_size(param_dtype), eg = elem_size(grad_dtype);
    if (!ep || !eg || (state_bits != 8 && state_bits != 32)) return TXL_ERR_INVALID_ARG;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(eps) ||
        !(max_norm >= 0.0) || !std::isfinite(max_norm))
        return TXL_ERR_INVALID_ARG;
    // (the update's reciprocal counts an operand below 2^-126 as 0: 0 / eps would be NaN)
    if (eps > 0.0 && (float)eps < FLT_MIN) return TXL_ERR_INVALID_ARG;
    const long long total = txl_adamw_state_elements(tensors, n_tensors);
    if (total < 0 || !steps || !lr) return TXL_ERR_INVALID_ARG;
    const bool eight = state_bits == 8, bf16 = param_dtype == TXL_BF16;
    // (flat buffers of no elements may be null)
    if ((master && !bf16) || ((exp_avg_scale || exp_avg_sq_scale) && !eight)) return TXL_ERR_INVALID_ARG;
    if (total && (!exp_avg || !exp_avg_sq || (bf16 && !master) || (eight && (!exp_avg_scale || !exp_avg_sq_scale))))
        return TXL_ERR_INVALID_ARG;
    for (const void* p : {(const void*)master, (const void*)exp_avg, (const void*)exp_avg_scale,
                          (const void*)exp_avg_sq, (const void*)exp_avg_sq_scale})
        if (!aligned16(p)) return TXL_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(steps) & 7u) || (reinterpret_cast<uintptr_t>(lr) & 3u) ||
        (reinterpret_cast<uintptr_t>(grad_norm) & 3u))
        return TXL_ERR_MISALIGNED;
    const size_t need = txl_adamw_workspace_bytes(tensors, n_tensors);
    if (bad_workspace(workspace, ws_bytes, need)) return TXL_ERR_WORKSPACE;
    // (no exception leaves a C entry point)
    std::vector<Range> r;
    try {
        r.reserve(2 * (size_t)n_tensors + 9);
    } catch (const std::bad_alloc&) {
        return TXL_ERR_UNSUPPORTED;
    }
    for (int i = 0; i < n_tensors; ++i) {
        const txl_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        if (!t.param || !t.grad) return TXL_ERR_INVALID_ARG;
        if (!aligned16(t.param) || !aligned16(t.grad)) return TXL_ERR_MISALIGNED;
        r.push_back(range_of(t.param, (size_t)t.n * ep, true));
        r.push_back(range_of(t.grad, (size_t)t.n * eg, false));
    }
    const size_t state = (size_t)total * (eight ? 1 : 4), scales = (size_t)total / txl::kAdamwBlock * sizeof(float);
    r.push_back(range_of(master, (size_t)total * 4, true));
    r.push_back(range_of(exp_avg, state, true));
    r.push_back(range_of(exp_avg_sq, state, true));
    r.push_back(range_of(exp_avg_scale, scales, true));
    r.push_back(range_of(exp_avg_sq_scale, scales, true));
    r.push_back(range_of(steps, sizeof(long long), true));
    r.push_back(range_of(lr, sizeof(float), false));
    r.push_back(range_of(grad_norm, sizeof(float), true));
    r.push_back(range_of(workspace, need, true));
    if (any_written_overlap(r.data(), r.size())) return TXL_ERR_ALIAS;
    const txl::AdamwArgs a = {tensors,       n_tensors, bf16, grad_dtype == TXL_BF16, eight, master,
                              exp_avg,       exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, steps, lr,
                              beta1,         beta2,     eps,  max_norm, seed, grad_norm,
                              workspace};
    return cuda_status(txl::launch_adamw(a, static_cast<cudaStream_t>(stream)));
}

size_t txl_grad_norm_workspace_bytes(const txl_grad_tensor* tensors, int n_tensors) {
    return grad_tensors_status(tensors, n_tensors) == TXL_OK
               ? txl::grad_norm_workspace_bytes(txl::grad_norm_plan(tensors, n_tensors))
               : 0;
}

int txl_grad_norm(const txl_grad_tensor* tensors, int n_tensors, double max_norm, float* norm, float* norms,
                  void* workspace, size_t ws_bytes, void* stream) {
    if (!(max_norm >= 0.0) || !std::isfinite(max_norm) || (max_norm > 0.0 && max_norm < FLT_MIN) || max_norm > FLT_MAX ||
        !norm)
        return TXL_ERR_INVALID_ARG;
    const int rc = grad_tensors_status(tensors, n_tensors);
    if (rc != TXL_OK) return rc;
    if (!aligned_to(norm, 4) || !aligned_to(norms, 4)) return TXL_ERR_MISALIGNED;
    const txl::GradNormPlan plan = txl::grad_norm_plan(tensors, n_tensors);
    const size_t need = txl::grad_norm_workspace_bytes(plan);
    if (bad_workspace(workspace, ws_bytes, need)) return TXL_ERR_WORKSPACE;
    const Range own[] = {range_of(norm, sizeof(float), true), range_of(norms, (size_t)n_tensors * sizeof(float), true),
                         range_of(workspace, need, true)};
    bool rising = true;  // each tensor behind the one before: none overlaps another
    uintptr_t end = 0;
    for (int i = 0; i < n_tensors; ++i) {
        const txl_grad_tensor& t = tensors[i];
        if (t.n == 0) continue;
        if (!t.grad) return TXL_ERR_INVALID_ARG;
        if (!aligned16(t.grad)) return TXL_ERR_MISALIGNED;
        const Range g = range_of(t.grad, (size_t)t.n * elem_size(t.dtype), false);
        rising = rising && g.at >= end;
        end = g.end;
        for (const Range& o : own)
            if (o.at && o.at < g.end && g.at < o.end) return TXL_ERR_ALIAS;
    }
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (own[i].at && own[j].at && own[i].at < own[j].end && own[j].at < own[i].end) return TXL_ERR_ALIAS;
    if (max_norm > 0.0 && !rising) {
        std::vector<Range> r;
        try {
            r.reserve((size_t)n_tensors);
        } catch (const std::bad_alloc&) {
            return TXL_ERR_UNSUPPORTED;
        }
        for (int i = 0; i < n_tensors; ++i)
            if (tensors[i].n) r.push_back(range_of(tensors[i].grad, (size_t)tensors[i].n * elem_size(tensors[i].dtype), true));
        if (any_written_overlap(r.data(), r.size())) return TXL_ERR_ALIAS;
    }
    const txl::GradNormArgs a = {tensors, n_tensors, plan, max_norm, norm, norms, workspace};
    return cuda_status(txl::launch_grad_norm(a, static_cast<cudaStream_t>(stream)));
}

const char* txl_status_string(int status) {
    switch (status) {
        case TXL_OK: return "ok";
        case TXL_ERR_INVALID_ARG: return "invalid argument";
        case TXL_ERR_UNSUPPORTED: return "unsupported size";
        case TXL_ERR_MISALIGNED: return "pointer not 16-byte aligned";
        case TXL_ERR_ALIAS: return "output overlaps an input";
        case TXL_ERR_LAUNCH: return "kernel launch failed";
        case TXL_ERR_DEVICE_TIMEOUT: return "device-side wait timed out";
        case TXL_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        case TXL_ERR_CUDA: return "CUDA runtime/driver call failed";
        case TXL_ERR_SCRATCH_LIMIT: return "call needs more scratch than the static no-alloc buffer";
        case TXL_ERR_OUT_OF_BOUNDS: return "a bounds-checked kernel skipped an out-of-range access";
        default: return "unknown status";
    }
}

int txl_version(void) { return (1 << 16) | 0; }

int txl_bounds_status(unsigned long long* first) {
#ifndef TXL_CHECKED
    if (first) *first = 0;
    return TXL_ERR_UNSUPPORTED;  // this library was built without bounds checks
#else
    if (cudaDeviceSynchronize() != cudaSuccess) return TXL_ERR_CUDA;
    const unsigned long long words[] = {txl::bounds_word_attn_simt(),   txl::bounds_word_attn_tc(),
                                         txl::bounds_word_attn_bwd(),    txl::bounds_word_attn_bwd_tc(),
                                         txl::bounds_word_mem_update(),  txl::bounds_word_layer_norm(),
                                         txl::bounds_word_proj_gemm(),   txl::bounds_word_layer_norm_train(),
                                         txl::bounds_word_adamw(),       txl::bounds_word_linear_bwd(),
                                         txl::bounds_word_token_logprobs(), txl::bounds_word_grad_norm(),
                                         txl::bounds_word_linear_logprobs()};
    unsigned long long w = 0;
    for (unsigned long long x : words) {
        if (x == ~0ull) return TXL_ERR_CUDA;
        if (!w && x) w = x;
    }
    if (first) *first = w;
    return w ? TXL_ERR_OUT_OF_BOUNDS : TXL_OK;
#endif
}

int txl_debug_inject(int kind) {
    if (kind < 0 || kind > 1) return TXL_ERR_INVALID_ARG;
    g_inject = kind;
    return TXL_OK;
}

}  // extern "C"
