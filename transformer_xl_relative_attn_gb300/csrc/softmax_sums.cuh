// The running statistics of a softmax in one pass: of the values x seen so far
//
//   m = max x,   s = sum e^(x - m),   t = sum e^(x - m) (x - m)
//
// all in fp32, from which log-sum-exp = m + ln s and entropy = ln s - t / s.
// When the maximum moves from m to M, with d = m - M <= 0, the sums become
// s e^d and e^d (t + d s).  Differences are held at or above kLowest: what a value of
// -inf adds to t is then 0 times a finite number (e^kLowest is 0, and kLowest times 2^30
// values is finite), not 0 times -inf;
// and m starts at the lowest finite number, so that x - m of x = -inf is not NaN.
// A NaN or +inf among the values makes s and t NaN.
#pragma once
#include <cuda_bf16.h>

namespace txl {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -1e20f;

__device__ __forceinline__ float sm_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger of two, NaN if either is.
__device__ __forceinline__ float sm_max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Packed fp32 pairs, each half rounded as the scalar operation.
__device__ __forceinline__ float2 sm_add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 sm_mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 sm_fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}

struct SoftmaxSums {
    float m, s, t;
    __device__ __forceinline__ void clear() { m = -3.402823466e38f, s = 0.f, t = 0.f; }
    // The maximum becomes `to` where that is larger.
    __device__ __forceinline__ void raise(float to) {
        if (to > m) {
            const float d = fmaxf(m - to, kLowest), f = sm_ex2(d * kLog2e);
            t = f * fmaf(d, s, t);
            s = f * s;
            m = to;
        }
    }
    __device__ __forceinline__ void merge(const SoftmaxSums& o) {
        const float M = fmaxf(m, o.m);
        const float d = fmaxf(m - M, kLowest), e = fmaxf(o.m - M, kLowest);
        const float f = sm_ex2(d * kLog2e), g = sm_ex2(e * kLog2e);
        t = fmaf(f, fmaf(d, s, t), g * fmaf(e, o.s, o.t));
        s = fmaf(f, s, g * o.s);
        m = M;
    }
    // Over the warp, every lane with the same result (the same order of additions).
    __device__ __forceinline__ void merge_warp() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            SoftmaxSums b;
            b.m = __shfl_xor_sync(0xffffffffu, m, o);
            b.s = __shfl_xor_sync(0xffffffffu, s, o);
            b.t = __shfl_xor_sync(0xffffffffu, t, o);
            merge(b);
        }
    }
};

// Two values, neither above m, onto pairs of sums.
__device__ __forceinline__ void sm_add_pair(float2 x, float m, float2& s, float2& t) {
    float2 d = sm_add2(x, make_float2(-m, -m));
    d.x = sm_max_nan(d.x, kLowest);
    d.y = sm_max_nan(d.y, kLowest);
    const float2 y = sm_mul2(d, make_float2(kLog2e, kLog2e));
    const float2 e = make_float2(sm_ex2(y.x), sm_ex2(y.y));
    s = sm_add2(s, e);
    t = sm_fma2(e, d, t);
}

// What a row's sums say: log-sum-exp, entropy, and log p of a value of the row.  A row
// of nothing but -inf has no probabilities: log-sum-exp and log p are -inf, its entropy 0.
struct SoftmaxRow {
    float m, log_s, lse, entropy;
    __device__ __forceinline__ explicit SoftmaxRow(const SoftmaxSums& a) {
        m = a.m;
        log_s = logf(a.s);  // -inf where s is 0
        lse = a.m + log_s;
        const float h = log_s - a.t / a.s;
        entropy = a.s == 0.f || h < 0.f ? 0.f : h;
    }
    __device__ __forceinline__ float logprob(float x) const { return log_s == -INFINITY ? -INFINITY : (x - m) - log_s; }
};

}  // namespace txl
