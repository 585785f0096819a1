// One AdamW step over many tensors.  With g the gradient (times the clip
// factor c = min(1, max_norm / |all gradients|) where max_norm is given), t
// the step's number and every product and sum in fp32,
//
//   m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) g g
//   p = p - (lr wd p + lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// p is an fp32 parameter, or the fp32 master copy of a bf16 one (which is
// written as the master's rounding).  The decay is subtracted as lr wd p, not
// as a factor 1 - lr wd: with lr wd = 1e-6 that factor would be 6 % off in fp32.
//
// States.  The tensors' states lie one behind the other in flat buffers, each
// tensor starting at a multiple of 256 elements.  One warp owns one such block
// of 256 (8 elements per lane), so a block's scale in the 8-bit form needs one
// warp reduction and no shared memory.  In 32 bits the buffers hold m and v.
// In 8 bits they hold e4m3 codes of m / s and sqrt(v) / s', with s the block's
// largest magnitude / 448.  sqrt(v) rather than v because its range is half as
// many octaves, and e4m3 covers 18 of them.  Codes are rounded up or down at
// random with the value kept in the mean: under round-to-nearest, a moving
// average that changes by 0.1 % a step would never leave a code 3 mantissa bits
// wide.  The 32 random bits of an element are a hash of (seed, step, its index):
// the same inputs give the same bits.  A non-zero sqrt(v) is never rounded to 0,
// which bounds m / sqrt(v) of the next step.  A block whose largest magnitude is
// not above 2^-110 is stored as zeros; one that is not finite gets a scale that
// is not finite.
//
// The step's number, the learning rate and the clip factor are device values:
// a step can be captured in a graph and replayed.  A first launch sums g g
// (only with max_norm), a one-CTA launch turns it into the step's coefficients
// and advances the step, and the third launch updates.  A norm that is not finite
// leaves everything as it was.
//
// The tensor table travels in the kernel's parameters (32 bytes per tensor):
// no table in device memory to keep in step with the host's.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "adamw.h"
#include "txl_device.cuh"

namespace txl {

namespace {

// Blocks per CTA: as many as make full rounds of the CTAs that are resident at once (a
// last round with a few of them takes as long as a full one), with at most 256 blocks of
// 8 bits, whose prefetch wants a long run, or 64 of 32 bits; a multiple of the 8 warps.
// Measured at 226.7 M elements of 8 bits: at most 64 blocks 776 us, 256 blocks 757 us, in
// full rounds 750 us; at 37.8 M of 32 bits, which prefetch nothing: 64 blocks 199 us, 256
// blocks 212 us.
constexpr int kCtas8 = 3, kCtas32 = 4;  // per SM
unsigned blocks_per_cta(long long blocks, bool eight) {
    const long long most = eight ? 256 : 64, resident = (long long)current_sm_count() * (eight ? kCtas8 : kCtas32);
    const long long rounds = (blocks + resident * most - 1) / (resident * most);
    const long long per = rounds ? (blocks + resident * rounds - 1) / (resident * rounds) : 1;
    return (unsigned)((per + 7) / 8 * 8);
}

// What the update launch needs of this step, written by adamw_coef_kernel.
struct AdamwCoef {
    float clip;       // factor of the gradients
    float step_size;  // lr / (1 - b1^t)
    float root_corr;  // 1 / sqrt(1 - b2^t)
    float lr;
    unsigned key;  // hash key of the step
    int skip;      // the gradient norm is not finite
};

struct AdamwEntry {
    void* p;
    const void* g;
    long long n;
    unsigned start;  // first block, relative to the launch's first
    float wd;
};

// Tables of two sizes: a launch copies its parameters, so a short list should
// not pay for a long one.
template <int CAP>
struct AdamwTable {
    int n;
    AdamwEntry e[CAP];
};

struct AdamwFlat {
    unsigned blocks;  // of each buffer
    float* master;
    void* m;
    float* ms;
    void* v;
    float* vs;
};

// 32-bit integer hash: xor-shifts and odd multipliers, every input bit reaching
// every output bit.
__host__ __device__ __forceinline__ unsigned mix32(unsigned h) {
    h ^= h >> 16;
    h *= 0x6C8E9CF5u;
    h ^= h >> 15;
    h *= 0x2B7E1517u;
    return h ^ (h >> 16);
}

// The larger of two magnitudes, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Over the warp, in one instruction (five exchanges deep it was 2 of 88
// instructions an element, and their latency twice per block).
__device__ __forceinline__ float warp_max_nan(float a) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(a));
    return r;
}

// q >= 0 to a neighbouring e4m3 value, up with the probability of the fraction
// by 16 random bits (random20: those, followed by four zeros).  e4m3 keeps 3 mantissa bits, so 20 bits of the fp32
// pattern are cut off after the random bits were added below the cut; its
// subnormals (below 2^-6) step by 2^-9, which are the steps of the numbers
// from 2^-6 on, so they are moved there and back.
// (What is rounded up past 448 is left to the conversion, which saturates there.)
__device__ __forceinline__ float round_e4m3(float q, unsigned random20) {
    const float c = q < 0x1p-6f ? 0x1p-6f : 0.f;
    const float t = __uint_as_float((__float_as_uint(__fadd_rn(q, c)) + random20) & 0xFFF00000u);
    return __fadd_rn(t, -c);
}

// 1 / x to 1 ulp (an x below 2^-126 counts as 0).
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&f)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
template <typename T>
__device__ __forceinline__ float load1(const T* p) {
    return static_cast<float>(*p);
}
__device__ __forceinline__ void store1(float* p, float f) { *p = f; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }

// Elements 0 .. 3 of p, of which `left` are the tensor's (0 behind its end).
// `full`: the whole block is the tensor's.  at, n: the index of p in its tensor and the
// tensor's length, for the bounds-checked build alone.
template <typename T>
__device__ __forceinline__ void load4_tail(const T* p, bool full, int left, long long at, long long n, float (&f)[4]) {
    if (full) {
        if (TXL_BOUNDS(at >= 0 && at + 4 <= n, 1001, at)) load4(p, f);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = k < left && TXL_BOUNDS(at >= 0 && at + k < n, 1004, at) ? load1(p + k) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store4_tail(T* p, bool full, int left, long long at, long long n, const float (&f)[4]) {
    if (full) {
        if (TXL_BOUNDS(at >= 0 && at + 4 <= n, 1002, at)) store4(p, f);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left && TXL_BOUNDS(at >= 0 && at + k < n, 1005, at)) store1(p + k, f[k]);
    }
}

// The entry that block b lies in: the last whose start is not behind it.
template <int CAP>
__device__ __forceinline__ int find_entry(const AdamwTable<CAP>& t, unsigned b) {
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.e[mid].start <= b)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Sum of g g over each CTA's blocks: part[blockIdx.x] (of n_part left in the workspace).
template <typename G, int CAP>
__global__ void __launch_bounds__(256) adamw_norm_kernel(const __grid_constant__ AdamwTable<CAP> t,
                                                         unsigned n_blocks, unsigned per,
                                                         float* __restrict__ part, unsigned n_part) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float sh[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned b0 = blockIdx.x * per, end = min(n_blocks, b0 + per);
    int e = find_entry(t, b0);
    float s = 0.f;
    for (unsigned b = b0 + warp; b < end; b += 8) {
        while (e + 1 < t.n && t.e[e + 1].start <= b) ++e;
        const long long i = (long long)(b - t.e[e].start) * kAdamwBlock, n = t.e[e].n - i;
        const bool full = n >= kAdamwBlock;
        const int left = full ? kAdamwBlock : (int)n - lane * 4;
        const G* const gp = static_cast<const G*>(t.e[e].g) + i + lane * 4;
        float g[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            load4_tail(gp + 128 * h, full, left - 128 * h, i + lane * 4 + 128 * h, t.e[e].n, g[h]);
#pragma unroll
        for (int x = 0; x < 8; ++x) s = fmaf(g[x >> 2][x & 3], g[x >> 2][x & 3], s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sh[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float a = 0.f;
        for (int w = 0; w < 8; ++w) a += sh[w];
        if (TXL_BOUNDS(blockIdx.x < n_part, 1006, blockIdx.x)) part[blockIdx.x] = a;
    }
}

// The step's coefficients, from the partial sums of g g (clipped = 0: no clipping; max_norm
// may be 0 all the same, where it is below fp32's range).
// 1 - b^t = -expm1(t ln b) with ln b from the host: fp32 keeps it to 2^-22 however
// small, and double precision's pow alone took longer than a small update.
__global__ void __launch_bounds__(1024) adamw_coef_kernel(const float* __restrict__ part, unsigned n_part,
                                                          double ln_beta1, double ln_beta2, int clipped,
                                                          float max_norm, unsigned seed, const float* lr, long long* steps,
                                                          float* grad_norm, AdamwCoef* coef) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float sh[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long t = *steps + 1;
    const float rate = *lr;
    float s = 0.f;
    if (clipped) {
        for (unsigned i = threadIdx.x; i < n_part; i += blockDim.x) s += part[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sh[warp] = s;
        __syncthreads();
        s = lane < (int)(blockDim.x >> 5) ? sh[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    if (threadIdx.x != 0) return;
    AdamwCoef c = {1.f, 0.f, 0.f, rate, mix32(seed + (unsigned)t * 0x9E3779B1u), 0};
    if (clipped) {
        const float norm = sqrtf(s);
        if (grad_norm) *grad_norm = norm;
        c.skip = !(norm < INFINITY);
        c.clip = norm > max_norm ? max_norm / norm : 1.f;
    }
    c.step_size = rate / -expm1f((float)((double)t * ln_beta1));
    c.root_corr = 1.f / sqrtf(-expm1f((float)((double)t * ln_beta2)));
    if (!c.skip) *steps = t;
    *coef = c;
}

// One block's state in 8 bits: codes (4 per 32-bit word) and scale of x.
// ROOT: x is a square root, not negative, and what is not zero stays so.
// random: 16 bits of it from bit SHIFT on are each element's.
template <bool ROOT, int SHIFT>
__device__ __forceinline__ float quantize(const float (&x)[8], const unsigned (&random)[8], unsigned (&code)[2]) {
    float a = fabsf(x[0]);
#pragma unroll
    for (int k = 1; k < 8; ++k) a = max_nan(a, fabsf(x[k]));
    a = warp_max_nan(a);
    const bool fine = a > 0x1p-110f && a < INFINITY;
    const float inv = __fmul_rn(__frcp_rn(a), 448.f);
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float t = __fmul_rn(fabsf(x[k]), inv);
        q[k] = round_e4m3(t, ((random[k] >> SHIFT) & 0xFFFFu) * 16u);
        if (ROOT)
            q[k] = fmaxf(q[k], t > 0.f ? 0x1p-9f : 0.f);
        else
            q[k] = copysignf(q[k], x[k]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const unsigned lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h], q[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
        const unsigned hi =
            __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h + 2], q[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
        code[h] = fine ? lo | (hi << 16) : 0u;
    }
    // a NaN is not at the limit or below, and stays
    return a <= 0x1p-110f ? 0.f : __fmul_rn(a, 1.f / 448.f);
}

__device__ __forceinline__ void codes_to_float(unsigned w, float s, float* f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * h)), __NV_E4M3);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r));
        f[2 * h] = __fmul_rn(v.x, s);
        f[2 * h + 1] = __fmul_rn(v.y, s);
    }
}

// A lane's 8 elements of one block as they lie in memory, and where they go back.
template <typename P, typename G, bool EIGHT>
struct AdamwRaw {
    P* p;       // the lane's first element
    int left;   // elements of the tensor from there on, kAdamwBlock where the whole block is its
    long long i, n;  // index of p in its tensor, whose length is n (bounds-checked build)
    float wd;
    unsigned blk;  // block of the flat buffers
    float g[8], w[8];
    float m[EIGHT ? 1 : 8], v[EIGHT ? 1 : 8];
    unsigned mc[2], vc[2];
    float ms, vs;
};

template <typename P, typename G, bool EIGHT, int CAP>
__device__ __forceinline__ void adamw_load(const AdamwTable<CAP>& t, int& e, unsigned b, unsigned first,
                                           const AdamwFlat& flat, AdamwRaw<P, G, EIGHT>& r) {
    constexpr bool MASTER = sizeof(P) == 2;
    const int lane = threadIdx.x & 31;
    while (e + 1 < t.n && t.e[e + 1].start <= b) ++e;
    const long long i = (long long)(b - t.e[e].start) * kAdamwBlock, n = t.e[e].n - i;
    const bool full = n >= kAdamwBlock;
    r.left = full ? kAdamwBlock : (int)n - lane * 4;
    r.p = static_cast<P*>(t.e[e].p) + i + lane * 4;
    r.i = i + lane * 4;
    r.n = t.e[e].n;
    r.wd = t.e[e].wd;
    r.blk = first + b;
    if (!TXL_BOUNDS(r.blk < flat.blocks, 1003, r.blk)) r.blk = 0;
    const G* const gp = static_cast<const G*>(t.e[e].g) + i + lane * 4;
    const size_t at = (size_t)r.blk * kAdamwBlock + lane * 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        load4_tail(gp + 128 * h, full, r.left - 128 * h, r.i + 128 * h, r.n, *reinterpret_cast<float(*)[4]>(r.g + 4 * h));
        if (MASTER)
            load4(flat.master + at + 128 * h, *reinterpret_cast<float(*)[4]>(r.w + 4 * h));
        else
            load4_tail(reinterpret_cast<const float*>(r.p) + 128 * h, full, r.left - 128 * h, r.i + 128 * h, r.n,
                       *reinterpret_cast<float(*)[4]>(r.w + 4 * h));
        if constexpr (EIGHT) {
            r.mc[h] = *reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(flat.m) + at + 128 * h);
            r.vc[h] = *reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(flat.v) + at + 128 * h);
        } else {
            load4(static_cast<const float*>(flat.m) + at + 128 * h, *reinterpret_cast<float(*)[4]>(r.m + 4 * h));
            load4(static_cast<const float*>(flat.v) + at + 128 * h, *reinterpret_cast<float(*)[4]>(r.v + 4 * h));
        }
    }
    if constexpr (EIGHT) {
        r.ms = flat.ms[r.blk];
        r.vs = flat.vs[r.blk];
    }
}

template <typename P, typename G, bool EIGHT>
__device__ __forceinline__ void adamw_update(const AdamwRaw<P, G, EIGHT>& r, const AdamwFlat& flat,
                                             const AdamwCoef& c, float b1, float b1c, float b2, float b2c,
                                             float eps) {
    constexpr bool MASTER = sizeof(P) == 2;
    const int lane = threadIdx.x & 31;
    const size_t at = (size_t)r.blk * kAdamwBlock + lane * 4;
    const float decay = r.wd * c.lr;
    const bool full = r.left == kAdamwBlock;
    float m[8], v[8], p[8], root[8];
    if constexpr (EIGHT) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            codes_to_float(r.mc[h], r.ms, m + 4 * h);
            codes_to_float(r.vc[h], r.vs, v + 4 * h);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = __fmul_rn(v[x], v[x]);
    } else {
#pragma unroll
        for (int x = 0; x < 8; ++x) m[x] = r.m[x], v[x] = r.v[x];
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        // each product and sum rounded by itself: what the states become does not hang on
        // how the compiler fuses them
        const float gs = __fmul_rn(r.g[x], c.clip);
        m[x] = __fadd_rn(__fmul_rn(m[x], b1), __fmul_rn(gs, b1c));
        v[x] = __fadd_rn(__fmul_rn(v[x], b2), __fmul_rn(__fmul_rn(gs, gs), b2c));
        root[x] = __fsqrt_rn(v[x]);
        // the quotient to 2 ulp: it is added to p scaled by the step size
        const float u = m[x] * rcp_approx(fmaf(root[x], c.root_corr, eps));
        p[x] = r.w[x] - fmaf(r.w[x], decay, u * c.step_size);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float(&p4)[4] = *reinterpret_cast<const float(*)[4]>(p + 4 * h);
        store4_tail(r.p + 128 * h, full, r.left - 128 * h, r.i + 128 * h, r.n, p4);
        if (MASTER) store4(flat.master + at + 128 * h, p4);
    }
    if constexpr (EIGHT) {
        unsigned random[8], code[2];
#pragma unroll
        for (int x = 0; x < 8; ++x) random[x] = mix32((unsigned)at + 128u * (x >> 2) + (x & 3) + c.key);
        uint8_t* mc = static_cast<uint8_t*>(flat.m) + at;
        uint8_t* vc = static_cast<uint8_t*>(flat.v) + at;
        const float ms = quantize<false, 0>(m, random, code);
        *reinterpret_cast<unsigned*>(mc) = code[0];
        *reinterpret_cast<unsigned*>(mc + 128) = code[1];
        const float vs = quantize<true, 16>(root, random, code);
        *reinterpret_cast<unsigned*>(vc) = code[0];
        *reinterpret_cast<unsigned*>(vc + 128) = code[1];
        if (lane == 0) {
            flat.ms[r.blk] = ms;
            flat.vs[r.blk] = vs;
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            store4(static_cast<float*>(flat.m) + at + 128 * h, *reinterpret_cast<const float(*)[4]>(m + 4 * h));
            store4(static_cast<float*>(flat.v) + at + 128 * h, *reinterpret_cast<const float(*)[4]>(v + 4 * h));
        }
    }
}

// The update.  P: type of the parameters (bf16 with a master copy), G: of the
// gradients.  `first`: the launch's first block in the flat buffers.  With 8-bit
// states a block takes longer to compute than to fetch, so the next one's loads
// are issued before it.
template <typename P, typename G, bool EIGHT, int CAP>
__global__ void __launch_bounds__(256, EIGHT ? kCtas8 : kCtas32)
adamw_kernel(const __grid_constant__ AdamwTable<CAP> t, unsigned n_blocks, unsigned per, unsigned first,
             const AdamwFlat flat, float b1, float b1c, float b2, float b2c, float eps, const AdamwCoef* __restrict__ coef) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const unsigned warp = threadIdx.x >> 5, b0 = blockIdx.x * per;
    const AdamwCoef c = *coef;
    if (c.skip) return;
    const unsigned b1st = b0 + warp, end = min(n_blocks, b0 + per);
    if (b1st >= end) return;
    int e = find_entry(t, b1st);
    if constexpr (EIGHT) {
        AdamwRaw<P, G, EIGHT> next;
        adamw_load(t, e, b1st, first, flat, next);
#pragma unroll 1
        for (unsigned b = b1st; b < end; b += 8) {
            const AdamwRaw<P, G, EIGHT> cur = next;
            if (b + 8 < end) adamw_load(t, e, b + 8, first, flat, next);
            adamw_update(cur, flat, c, b1, b1c, b2, b2c, eps);
        }
    } else {
        for (unsigned b = b1st; b < end; b += 8) {
            AdamwRaw<P, G, EIGHT> cur;
            adamw_load(t, e, b, first, flat, cur);
            adamw_update(cur, flat, c, b1, b1c, b2, b2c, eps);
        }
    }
}

unsigned ctas(unsigned blocks, unsigned per) { return (blocks + per - 1) / per; }

// Launch with programmatic stream serialisation (every kernel here waits for
// the one before it before its first global access).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), unsigned grid, unsigned threads, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

size_t coef_bytes() { return 256; }

// Fills the table with the next tensors (at most CAP) and calls f(table, blocks, first block).
template <int CAP, typename F>
cudaError_t each_group(const AdamwArgs& a, F f) {
    AdamwTable<CAP> t;
    long long first = 0, at = 0;
    t.n = 0;
    cudaError_t err = cudaSuccess;
    auto flush = [&] {
        if (t.n && err == cudaSuccess) err = f(t, (unsigned)(at - first), (unsigned)first);
        first = at;
        t.n = 0;
    };
    for (int i = 0; i < a.n_tensors; ++i) {
        const txl_adamw_tensor& x = a.tensors[i];
        if (x.n <= 0) continue;
        t.e[t.n++] = {x.param, x.grad, x.n, (unsigned)(at - first), x.weight_decay};
        at += (x.n + kAdamwBlock - 1) / kAdamwBlock;
        if (t.n == CAP) flush();
    }
    flush();
    return err;
}

constexpr int kSmallTable = 32, kLargeTable = 480;

// One partial sum per CTA of each group of tensors (a group's last CTA may be partly
// filled: one more per group at most).
long long part_count(long long blocks) { return blocks / 8 + blocks / kSmallTable + 2; }

template <int CAP>
cudaError_t run(const AdamwArgs& a, long long blocks, cudaStream_t stream) {
    AdamwCoef* coef = static_cast<AdamwCoef*>(a.workspace);
    float* part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + coef_bytes());
    const unsigned per = blocks_per_cta(blocks, a.eight_bit);
    unsigned n_part = 0;
    cudaError_t e = cudaSuccess;
    if (a.max_norm > 0) {
        e = each_group<CAP>(a, [&](const AdamwTable<CAP>& t, unsigned n, unsigned) {
            float* to = part + n_part;
            const unsigned room = (unsigned)(part_count(blocks) - n_part);
            n_part += ctas(n, per);
            auto go = [&](auto kern) { return launch_pdl(kern, ctas(n, per), 256u, stream, t, n, per, to, room); };
            return a.bf16_grad ? go(adamw_norm_kernel<__nv_bfloat16, CAP>) : go(adamw_norm_kernel<float, CAP>);
        });
        if (e != cudaSuccess) return e;
    }
    e = launch_pdl(adamw_coef_kernel, 1, a.max_norm > 0 ? 1024u : 32u, stream, part, n_part, std::log(a.beta1),
                   std::log(a.beta2), (int)(a.max_norm > 0), (float)a.max_norm, a.seed, a.lr, a.steps, a.grad_norm, coef);
    if (e != cudaSuccess) return e;
    const AdamwFlat flat = {(unsigned)blocks, a.master, a.exp_avg, a.exp_avg_scale, a.exp_avg_sq, a.exp_avg_sq_scale};
    const float b1 = (float)a.beta1, b1c = (float)(1.0 - a.beta1), b2 = (float)a.beta2, b2c = (float)(1.0 - a.beta2);
    return each_group<CAP>(a, [&](const AdamwTable<CAP>& t, unsigned n, unsigned first) {
        auto go = [&](auto kern) {
            return launch_pdl(kern, ctas(n, per), 256u, stream, t, n, per, first, flat, b1, b1c, b2, b2c, (float)a.eps,
                              coef);
        };
        using B = __nv_bfloat16;
        if (a.eight_bit) {
            if (a.bf16_param) return a.bf16_grad ? go(adamw_kernel<B, B, true, CAP>) : go(adamw_kernel<B, float, true, CAP>);
            return a.bf16_grad ? go(adamw_kernel<float, B, true, CAP>) : go(adamw_kernel<float, float, true, CAP>);
        }
        if (a.bf16_param) return a.bf16_grad ? go(adamw_kernel<B, B, false, CAP>) : go(adamw_kernel<B, float, false, CAP>);
        return a.bf16_grad ? go(adamw_kernel<float, B, false, CAP>) : go(adamw_kernel<float, float, false, CAP>);
    });
}

}  // namespace

long long adamw_blocks(const txl_adamw_tensor* tensors, int n_tensors) {
    long long b = 0;
    for (int i = 0; i < n_tensors; ++i)
        if (tensors[i].n > 0) b += (tensors[i].n + kAdamwBlock - 1) / kAdamwBlock;
    return b;
}

size_t adamw_workspace_bytes(long long blocks) { return coef_bytes() + (size_t)part_count(blocks) * sizeof(float); }

cudaError_t launch_adamw(const AdamwArgs& a, cudaStream_t stream) {
    const long long blocks = adamw_blocks(a.tensors, a.n_tensors);
    return a.n_tensors <= kSmallTable ? run<kSmallTable>(a, blocks, stream) : run<kLargeTable>(a, blocks, stream);
}

TXL_BOUNDS_READER(bounds_word_adamw)

}  // namespace txl
