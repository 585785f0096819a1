// LayerNorm for training: the forward pass that keeps each row's statistics,
// and its gradients.  With z = x (+ y) a row of d elements,
//
//   mean = sum z / d,  rstd = (sum (z - mean)^2 / d + eps)^(-1/2)
//   out  = xh gamma + beta,  xh = (z - mean) rstd
//
// and for the gradient `dout` of out, with g = dout gamma,
//
//   dx     = rstd (g - sum(g) / d - xh sum(g xh) / d)  (+ dres)
//   dgamma = sum over rows of dout xh,  dbeta = sum over rows of dout
//
// (dx is the gradient of x and of y alike.)  bf16 or fp32 in and out, fp32
// arithmetic, statistics and parameter gradients.  dgamma and dbeta are summed
// in a fixed order (partial sums per row range, then their sum): the same
// inputs give the same bits.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "txl_device.cuh"

namespace txl {

namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(256) ln_fwd_kernel(const T* __restrict__ x, const T* __restrict__ y,
                                                     const T* __restrict__ gamma, const T* __restrict__ beta,
                                                     long long rows, int d, float eps, T* __restrict__ out,
                                                     float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= rows) return;
    const T* xr = x + r * d;
    const T* yr = y ? y + r * d : nullptr;
    float s = 0.f;
    for (int c = lane; c < d; c += 32) s += to_f(xr[c]) + (yr ? to_f(yr[c]) : 0.f);
    const float mean = warp_sum(s) / d;
    float q = 0.f;
    for (int c = lane; c < d; c += 32) {
        const float t = to_f(xr[c]) + (yr ? to_f(yr[c]) : 0.f) - mean;
        q = fmaf(t, t, q);
    }
    const float rstd = 1.f / sqrtf(warp_sum(q) / d + eps);
    for (int c = lane; c < d; c += 32) {
        const float t = to_f(xr[c]) + (yr ? to_f(yr[c]) : 0.f) - mean;
        out[r * d + c] = from_f<T>(fmaf(t * rstd, to_f(gamma[c]), to_f(beta[c])));
    }
    if (lane == 0) {
        mean_out[r] = mean;
        rstd_out[r] = rstd;
    }
}

// dx: one warp per row.
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_dx_kernel(const T* __restrict__ dout, const T* __restrict__ x,
                                                        const T* __restrict__ y, const T* __restrict__ gamma,
                                                        const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, const T* __restrict__ dres,
                                                        long long rows, int d, T* __restrict__ dx) {
    const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= rows) return;
    const float mu = mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = lane; c < d; c += 32) {
        const float z = to_f(x[r * d + c]) + (y ? to_f(y[r * d + c]) : 0.f);
        const float g = to_f(dout[r * d + c]) * to_f(gamma[c]);
        s1 += g;
        s2 = fmaf(g, (z - mu) * rs, s2);
    }
    s1 = warp_sum(s1) / d;
    s2 = warp_sum(s2) / d;
    for (int c = lane; c < d; c += 32) {
        const float z = to_f(x[r * d + c]) + (y ? to_f(y[r * d + c]) : 0.f);
        const float g = to_f(dout[r * d + c]) * to_f(gamma[c]);
        float v = rs * (g - s1 - (z - mu) * rs * s2);
        if (dres) v += to_f(dres[r * d + c]);
        dx[r * d + c] = from_f<T>(v);
    }
}

// Partial sums of dgamma and dbeta over one range of rows: part[range][2][d].
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_part_kernel(const T* __restrict__ dout, const T* __restrict__ x,
                                                          const T* __restrict__ y, const float* __restrict__ mean,
                                                          const float* __restrict__ rstd, long long rows, int d,
                                                          long long range, float* __restrict__ part) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= d) return;
    const long long r0 = blockIdx.y * range, r1 = r0 + range < rows ? r0 + range : rows;
    float a = 0.f, b = 0.f;
    for (long long r = r0; r < r1; ++r) {
        const float z = to_f(x[r * d + c]) + (y ? to_f(y[r * d + c]) : 0.f);
        const float g = to_f(dout[r * d + c]);
        a = fmaf(g, (z - mean[r]) * rstd[r], a);
        b += g;
    }
    part[(size_t)blockIdx.y * 2 * d + c] = a;
    part[(size_t)blockIdx.y * 2 * d + d + c] = b;
}

__global__ void __launch_bounds__(256) ln_bwd_sum_kernel(const float* __restrict__ part, int n_part, int d,
                                                         float* __restrict__ dgamma, float* __restrict__ dbeta) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= 2 * d) return;
    float a = 0.f;
    for (int p = 0; p < n_part; ++p) a += part[(size_t)p * 2 * d + c];
    if (c < d)
        dgamma[c] = a;
    else
        dbeta[c - d] = a;
}

constexpr int kPartRows = 64;  // rows of one partial sum, at least
constexpr int kMaxParts = 1024;

int ln_parts(long long rows) {
    const long long p = (rows + kPartRows - 1) / kPartRows;
    return (int)(p < 1 ? 1 : (p > kMaxParts ? kMaxParts : p));
}

template <typename T>
cudaError_t ln_fwd(const void* x, const void* y, const void* gamma, const void* beta, long long rows, int d,
                   float eps, void* out, float* mean, float* rstd, cudaStream_t stream) {
    if (rows <= 0) return cudaSuccess;
    ln_fwd_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(
        static_cast<const T*>(x), static_cast<const T*>(y), static_cast<const T*>(gamma),
        static_cast<const T*>(beta), rows, d, eps, static_cast<T*>(out), mean, rstd);
    return cudaGetLastError();
}

template <typename T>
cudaError_t ln_bwd(const void* dout, const void* x, const void* y, const void* gamma, const float* mean,
                   const float* rstd, const void* dres, long long rows, int d, void* dx, float* dgamma,
                   float* dbeta, float* part, cudaStream_t stream) {
    const T* dd = static_cast<const T*>(dout);
    const T* xx = static_cast<const T*>(x);
    const T* yy = static_cast<const T*>(y);
    const int parts = ln_parts(rows);
    if (rows > 0)
        ln_bwd_dx_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(
            dd, xx, yy, static_cast<const T*>(gamma), mean, rstd, static_cast<const T*>(dres), rows, d,
            static_cast<T*>(dx));
    ln_bwd_part_kernel<T><<<dim3((d + 255) / 256, parts), 256, 0, stream>>>(dd, xx, yy, mean, rstd, rows, d,
                                                                         (rows + parts - 1) / parts, part);
    ln_bwd_sum_kernel<<<(2 * d + 255) / 256, 256, 0, stream>>>(part, parts, d, dgamma, dbeta);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const void* x, const void* y, const void* gamma, const void* beta, long long rows,
                                  int d, float eps, void* out, float* mean, float* rstd, int bf16,
                                  cudaStream_t stream) {
    return bf16 ? ln_fwd<__nv_bfloat16>(x, y, gamma, beta, rows, d, eps, out, mean, rstd, stream)
                : ln_fwd<float>(x, y, gamma, beta, rows, d, eps, out, mean, rstd, stream);
}

size_t layer_norm_bwd_workspace_bytes(long long rows, int d) {
    return (size_t)ln_parts(rows) * 2 * d * sizeof(float);
}

cudaError_t launch_layer_norm_bwd(const void* dout, const void* x, const void* y, const void* gamma,
                                  const float* mean, const float* rstd, const void* dres, long long rows, int d,
                                  void* dx, float* dgamma, float* dbeta, void* workspace, int bf16,
                                  cudaStream_t stream) {
    float* part = static_cast<float*>(workspace);
    return bf16 ? ln_bwd<__nv_bfloat16>(dout, x, y, gamma, mean, rstd, dres, rows, d, dx, dgamma, dbeta, part, stream)
                : ln_bwd<float>(dout, x, y, gamma, mean, rstd, dres, rows, d, dx, dgamma, dbeta, part, stream);
}

TXL_BOUNDS_READER(bounds_word_layer_norm_train)

}  // namespace txl
