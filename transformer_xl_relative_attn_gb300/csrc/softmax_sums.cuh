// The running statistics of a softmax in one pass: of the values x seen so far, with
// L = log2 e as fp32 has it,
//
//   m near max x,   r = m L (rounded),   s = sum 2^(x L - r),   t = sum 2^(x L - r) (x L - r)
//
// all in fp32, from which log-sum-exp = m + (log2 s - (m L - r)) / L and entropy = (log2 s - t / s) ln 2.
// The reference is r itself, so that its rounding is no error, and a term costs one fused
// product before its power of two; that L is off by 1.3e-8 of itself is a temperature off
// by as much.  When the reference moves from m to M, with d = r(m) - r(M) <= 0, the sums
// become s 2^d and 2^d (t + d s).  m need not be the maximum itself (moved each time, some lane of a
// warp had to in most of the steps), but log2 s and t / s then carry its distance, which cancels
// between them but for their roundings.  Where the values' maximum is at hand (token_logprobs) m
// follows it once it is kSlack above; where it is not (linear_logprobs) once the terms of a tile
// are four times as much as the columns they may be of.
//
// What is not ordinary: a value of -inf, or one so low that x L - r is, would make t NaN (0
// times -inf).  Either nothing below kLow is added, whose power is 0 and whose product with
// it too; or a batch is added with no look at its values, and once more with it where that
// was not fine (in linear_logprobs, where two instructions for each logit cost a tenth of the
// time).  A reference from +-kHuge on is the maximum: numbers lie 64 and more apart there, where
// r's rounding would leave the powers' range, and s counts those equal to it.  m starts at the
// lowest finite number, which is beyond -kHuge and equals no -inf.  A NaN or +inf among the
// values makes s and t NaN.
#pragma once
#include <cuda_bf16.h>

namespace txl {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLow = -1e38f;    // (bf16 and fp32 hold it, and x L - r of it is finite)
constexpr float kHuge = 0x1p29f;  // r is off by 32 at most below it
constexpr float kSlack = 4.f;
constexpr float kLowest = -1e20f;  // differences of references are held at or above it (times 2^30 terms it is finite)

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
// The largest of three, a NaN left out.
__device__ __forceinline__ float sm_max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

__device__ __forceinline__ bool sm_ordinary(float m) { return fabsf(m) < kHuge; }
__device__ __forceinline__ float sm_reference(float m) { return __fmul_rn(m, kLog2e); }

// What sums against the maximum m are worth against M >= m: the factor, and d of the above.
__device__ __forceinline__ float sm_factor(float m, float M, float& d) {
    d = fmaxf(sm_reference(m) - sm_reference(M), kLowest);
    if (sm_ordinary(M)) return sm_ex2(d);
    d = 0.f;
    return m == M ? 1.f : 0.f;
}

struct SoftmaxSums {
    float m, s, t;
    __device__ __forceinline__ void clear() { m = -3.402823466e38f, s = 0.f, t = 0.f; }
    // One more value.
    __device__ __forceinline__ void add(float x) {
        float d;
        if (x > m) {
            const float f = sm_factor(m, x, d);
            t = f * fmaf(d, s, t);
            s = f * s;
            m = x;
        }
        if (sm_ordinary(m)) {
            const float y = fmaf(sm_max_nan(x, kLow), kLog2e, -sm_reference(m)), e = sm_ex2(y);
            s += e;
            t = fmaf(e, y, t);
        } else {
            s += x == m ? (x - x) + 1.f : x != x ? x : 0.f;
        }
    }
    __device__ __forceinline__ void merge(const SoftmaxSums& o) {
        const float M = fmaxf(m, o.m);
        float d, e;
        const float f = sm_factor(m, M, d), g = sm_factor(o.m, M, e);
        t = fmaf(f, fmaf(d, s, t), g * fmaf(e, o.s, o.t));
        s = fmaf(f, s, g * o.s);
        m = M;
    }
    // Over the warp, every lane with the same result.
    __device__ __forceinline__ void merge_warp() {
        float M, d;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(M) : "f"(m));
        const float f = sm_factor(m, M, d);
        t = f * fmaf(d, s, t);
        s = f * s;
        m = M;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            t += __shfl_xor_sync(0xffffffffu, t, o);
        }
    }
};

// Sums of many values in pairs; SoftmaxSums once they are folded.
struct SoftmaxPairs {
    float m;
    float2 s, t;
    __device__ __forceinline__ void clear() { m = -3.402823466e38f, s = t = make_float2(0.f, 0.f); }
    // Ahead of values of which `to` is the largest.
    __device__ __forceinline__ void raise(float to) {
        if (to > m + kSlack) follow(to);
    }
    // The same sums against another reference, to >= m.
    __device__ __forceinline__ void follow(float to) {
        float d;
        const float f = sm_factor(m, to, d);
        const float2 ff = make_float2(f, f);
        t = sm_mul2(ff, sm_fma2(make_float2(d, d), s, t));
        s = sm_mul2(ff, s);
        m = to;
    }
    // Takes over the other's sums, whose reference is the same one.
    __device__ __forceinline__ void take(SoftmaxPairs& o) {
        s = sm_add2(s, o.s), t = sm_add2(t, o.t);
        o.s = o.t = make_float2(0.f, 0.f);
    }
    // Two values, m ordinary, r = sm_reference(m).
    __device__ __forceinline__ void add(float2 x, float r) {
        const float2 y = sm_fma2(x, make_float2(kLog2e, kLog2e), make_float2(-r, -r));
        const float2 e = make_float2(sm_ex2(y.x), sm_ex2(y.y));
        s = sm_add2(s, e);
        t = sm_fma2(e, y, t);
    }
    // The same where values may be below kLow.
    __device__ __forceinline__ void add_low(float2 x, float r) { add(make_float2(sm_max_nan(x.x, kLow), sm_max_nan(x.y, kLow)), r); }
    // Whether values that nothing was known of were added as they should: the sum is neither
    // `much`, for which the reference has to follow, nor NaN, and t is none either.
    __device__ __forceinline__ bool fine(float much) const {
        const float a = s.x + s.y, b = t.x + t.y;
        return a < much && b == b;
    }
    // One value not above m (or NaN), where m is not ordinary.
    __device__ __forceinline__ void add_far(float x) { s.x += x == m ? (x - x) + 1.f : x != x ? x : 0.f; }
    __device__ __forceinline__ SoftmaxSums fold() const { return {m, s.x + s.y, t.x + t.y}; }
};

// What a row's sums say: log-sum-exp, entropy, and log p of a value of the row.  A row
// of nothing but -inf has no probabilities: log-sum-exp and log p are -inf, its entropy 0.
// (log p is x - m, exact or nearly, less ln sum e^(x - m): over x L - r it would carry the
// roundings of a product of its own size.)
struct SoftmaxRow {
    float m, ln_s, lse, entropy;  // ln_s: of the sum against m itself
    __device__ __forceinline__ explicit SoftmaxRow(const SoftmaxSums& a) {
        m = a.m;
        const float log_s = log2f(a.s);  // -inf where s is 0
        // the sum is against r, which is m L but for this much
        const float off = sm_ordinary(m) ? fmaf(m, kLog2e, -sm_reference(m)) : 0.f;
        ln_s = (log_s - off) * (1.f / kLog2e);
        lse = m + ln_s;
        const float h = (log_s - a.t / a.s) * kLn2;
        entropy = a.s == 0.f || h < 0.f ? 0.f : h;
    }
    __device__ __forceinline__ float logprob(float x) const {
        const float l = (x - m) - ln_s;
        return ln_s == -INFINITY ? -INFINITY : l > 0.f ? 0.f : l;  // (a rounding above it where p is 1)
    }
};

}  // namespace txl
