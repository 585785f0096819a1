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
// arithmetic, statistics and parameter gradients.
//
// Both passes are bound by memory: a row is read once, held in registers (E
// elements per lane, L lanes per row), reduced by shuffles and, with several
// warps per row, through shared memory, and written once.  Rows of a multiple of 16
// bytes move as 16-byte vectors, others by 4 or 2 bytes with the same code.
// The backward pass is persistent: bulk copies bring rows ahead into a ring of
// stages in shared memory, and each thread keeps its columns' sums of dout xh and
// dout in registers over all rows of its CTA, so dgamma and dbeta cost no second
// pass over the rows; the CTAs' sums go to the workspace and a second launch adds
// them, in a fixed order (the same inputs give the same bits).  With few rows other
// CTAs of the same launch read the rows again for these sums, column by column, and
// there is neither second launch nor workspace.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "txl_device.cuh"

namespace txl {

namespace {

// V consecutive elements as floats, 16 bytes at a time where V elements are 16 bytes.
template <typename T, int V>
struct Vec;
template <>
struct Vec<float, 4> {
    static __device__ __forceinline__ void load(const float* p, float* f) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <>
struct Vec<float, 1> {
    static __device__ __forceinline__ void load(const float* p, float* f) { f[0] = *p; }
    static __device__ __forceinline__ void store(float* p, const float* f) { *p = f[0]; }
};
template <>
struct Vec<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* f) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 x = __bfloat1622float2(h[e]);
            f[2 * e] = x.x, f[2 * e + 1] = x.y;
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Vec<__nv_bfloat16, 2> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* f) {
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
        f[0] = x.x, f[1] = x.y;
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(f[0], f[1]);
    }
};
template <>
struct Vec<__nv_bfloat16, 1> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* f) { f[0] = __bfloat162float(*p); }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) { *p = __float2bfloat16_rn(f[0]); }
};

// V sums, 16 bytes at a time where V allows it (one by one, V apart between lanes, they cost
// a CTA of 4096 columns 9 us).
template <int V>
__device__ __forceinline__ void store_sums(float* p, const float* f) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) Vec<float, 4>::store(p + 4 * i, f + 4 * i);
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else {
        *p = f[0];
    }
}

// Dynamic shared memory of this launch (bounds-checked build).
[[maybe_unused]] __device__ __forceinline__ uint32_t dynamic_bytes() {
    uint32_t n;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(n));
    return n;
}

// Two fp32 operations per instruction: the rows' arithmetic, not memory, bounded these
// kernels one element at a time (forward, bf16: 18 instructions per element, 68 % of the
// issue slots).  Arrays of E floats are taken as pairs.
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2& pair(float* f, int i) { return reinterpret_cast<float2*>(f)[i]; }

// 1 / sqrt(a) to about 1 ulp: the approximation and one Newton step (0 and infinities as
// they come from the approximation).
__device__ __forceinline__ float inv_sqrt(float a) {
    const float r = rsqrtf(a), h = 0.5f * a * r;
    return a > 0.f && a < INFINITY ? fmaf(r, fmaf(-h, r, 0.5f), r) : r;
}

// Over a warp, or its L lanes of a row.
template <int L = 32>
__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// A CTA's threads: R rows side by side, L lanes on each; T threads if they hold a row.
// The forward pass takes 128 (25600 x 1024 bf16: 19.8 us, with 256 21.1 us: its CTAs are
// short, and smaller ones leave and follow more evenly), the backward pass, whose CTAs
// stay and fold their sums at the end, 256 (11264 x 512 bf16: 13.8 us, with 128 15.0 us).
template <int L, int T = 256>
struct Shape {
    static constexpr int THREADS = L < T ? T : L;
    static constexpr int R = THREADS / L;
    static constexpr int TPR = L;  // threads per row
};

// Sum over the L lanes of a row.  sh: [2][THREADS / 32], `phase` alternates from
// call to call, so one barrier per call is enough.
template <int L>
__device__ __forceinline__ float row_sum(float s, float* sh, int phase) {
    s = warp_sum<L>(s);
    if (L <= 32) return s;
    constexpr int N = Shape<L, 128>::THREADS / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[phase * N + warp] = s;
    __syncthreads();
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < L / 32; ++w) a += sh[phase * N + warp / (L / 32) * (L / 32) + w];
    return a;
}
template <int L>
__device__ __forceinline__ float2 row_sum2(float2 s, float2* sh, int phase) {
    s = make_float2(warp_sum<L>(s.x), warp_sum<L>(s.y));
    if (L <= 32) return s;
    constexpr int N = Shape<L>::THREADS / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[phase * N + warp] = s;
    __syncthreads();
    float2 a = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < L / 32; ++w) {
        const float2 t = sh[phase * N + warp / (L / 32) * (L / 32) + w];
        a.x += t.x, a.y += t.y;
    }
    return a;
}

// E elements of a row, this thread's: vectors of V, the i-th `TPR V i` elements behind p,
// of which `left` (from p on) are the row's; 0 behind its end.
template <typename T, int V, int E, int TPR>
__device__ __forceinline__ void load_row(const T* p, int left, float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
        if (TPR * V * i < left && TXL_BOUNDS(TPR * V * i + V <= left, 901, left)) {
            Vec<T, V>::load(p + TPR * V * i, f + V * i);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) f[V * i + k] = 0.f;
        }
    }
}

// Threads of a forward CTA.  Rows of 8 elements per lane make many and short CTAs, which cost
// more to start than to run (400000 x 64 bf16: 256 threads 21.3 us, 128 26.4, 512 22.2).
template <int E>
constexpr int fwd_threads() {
    return E <= 8 ? 256 : 128;
}

template <typename T, int V, int E, int L>
__global__ void __launch_bounds__(Shape<L, fwd_threads<E>()>::THREADS)
ln_fwd_kernel(const T* __restrict__ x, const T* __restrict__ y, const T* __restrict__ gamma,
              const T* __restrict__ beta, long long rows, int d, float inv_d, float eps, T* __restrict__ out,
              float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    using S = Shape<L, fwd_threads<E>()>;
    __shared__ float sh[2 * S::THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = threadIdx.x % S::TPR;
    const long long r = (long long)blockIdx.x * S::R + threadIdx.x / S::TPR;
    const bool in = r < rows;  // (the barriers of a row are the CTA's)
    const int left = d - t * V;
    const long long at = r * d + t * V;
    alignas(8) float z[E];
    if (in) {
        load_row<T, V, E, S::TPR>(x + at, left, z);
        if (y) {
            alignas(8) float b[E];
            load_row<T, V, E, S::TPR>(y + at, left, b);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) pair(z, e) = __fadd2_rn(pair(z, e), pair(b, e));
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] = 0.f;
    }
    float2 s = both(0.f);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) s = __fadd2_rn(s, pair(z, e));
    const float mean = row_sum<L>(s.x + s.y, sh, 0) * inv_d;
    // (behind the row's end z is 0 and stays so)
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
        const float m = S::TPR * V * i < left ? -mean : 0.f;
        if (V == 1)
            z[i] += m;
        else
#pragma unroll
            for (int e = 0; e < V / 2; ++e) pair(z, V / 2 * i + e) = __fadd2_rn(pair(z, V / 2 * i + e), both(m));
    }
    float2 q = both(0.f);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) q = __ffma2_rn(pair(z, e), pair(z, e), q);
    const float rstd = inv_sqrt(fmaf(row_sum<L>(q.x + q.y, sh, 1), inv_d, eps));
    if (!in) return;
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
        constexpr int OFF = S::TPR * V;
        if (OFF * i < left && TXL_BOUNDS(OFF * i + V <= left && r < rows, 902, at)) {
            alignas(8) float g[V], b[V], o[V];
            Vec<T, V>::load(gamma + t * V + OFF * i, g);
            Vec<T, V>::load(beta + t * V + OFF * i, b);
            if (V == 1)
                o[0] = fmaf(z[i] * rstd, g[0], b[0]);
            else
#pragma unroll
                for (int e = 0; e < V / 2; ++e)
                    pair(o, e) = __ffma2_rn(__fmul2_rn(pair(z, V / 2 * i + e), both(rstd)), pair(g, e), pair(b, e));
            Vec<T, V>::store(out + at + OFF * i, o);
        }
    }
    if (t == 0) {
        mean_out[r] = mean;
        rstd_out[r] = rstd;
    }
}

// Shared memory of the rings of an SM, beside 2 KB a CTA for the rest.
constexpr size_t kRingRoom = 220 * 1024;

// CTAs per SM that the backward kernel is compiled for.
template <int E, int L>
constexpr int bwd_ctas() {
    return Shape<L>::THREADS > 256 ? 1 : (E <= 8 ? 3 : 2);
}

// dgamma and dbeta of a few columns by one CTA: CL lanes of V columns side by side, at least
// 32 bytes of a row, and as many threads below one another as the CTA has.
template <typename T, int V, int L>
struct Columns {
    static constexpr int THREADS = Shape<L>::THREADS;
    static constexpr int SECTOR = 32 / (int)sizeof(T) / V;
    static constexpr int CL = SECTOR > THREADS / 128 ? SECTOR : THREADS / 128;
    static constexpr int C = CL * V;           // columns of a CTA
    static constexpr int RG = THREADS / CL;    // rows at a time
    // Rows up to which this is done: 8 per thread, fp32 4, and 16 of narrow vectors.  Bf16 with y, once
    // against sums in the row CTAs and a second launch: 128 x 512 2.2 and 4.2 us, 1024 x 512
    // 4.0 and 5.1, 2048 x 512 8.2 and 5.5; 512 x 500 3.4 and 5.1, 1024 x 500 5.5 and 5.1;
    // 128 x 4096 3.3 and 13.2.
    static constexpr int ROWS = (V >= 4 ? 16 / (int)sizeof(T) : 16) * RG;
};

template <typename T, int V, int L>
__device__ __forceinline__ void ln_bwd_columns(const T* __restrict__ dout, const T* __restrict__ x,
                                               const T* __restrict__ y, const float* __restrict__ mean,
                                               const float* __restrict__ rstd, int rows, int d, int cta, float* sh,
                                               float* __restrict__ dgamma, float* __restrict__ dbeta) {
    using S = Columns<T, V, L>;
    const int cl = threadIdx.x % S::CL, c = cta * S::C + cl * V;
    float dg[V], db[V];
#pragma unroll
    for (int k = 0; k < V; ++k) dg[k] = db[k] = 0.f;
    if (c < d && TXL_BOUNDS(c + V <= d, 904, c)) {
#pragma unroll 2
        for (int r = threadIdx.x / S::CL; r < rows; r += S::RG) {
            const long long at = (long long)r * d + c;
            const float mu = mean[r], rs = rstd[r];
            alignas(8) float z[V], g[V];
            Vec<T, V>::load(x + at, z);
            Vec<T, V>::load(dout + at, g);
            if (y) {
                alignas(8) float b[V];
                Vec<T, V>::load(y + at, b);
#pragma unroll
                for (int k = 0; k < V; ++k) z[k] += b[k];
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                dg[k] = fmaf(g[k], (z[k] - mu) * rs, dg[k]);
                db[k] += g[k];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
        for (int o = S::CL; o < 32; o <<= 1) {
            dg[k] += __shfl_xor_sync(0xffffffffu, dg[k], o);
            db[k] += __shfl_xor_sync(0xffffffffu, db[k], o);
        }
    }
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < S::CL &&
        TXL_BOUNDS((warp + 1) * 2 * S::C * sizeof(float) <= dynamic_bytes() && cl * V + V <= S::C, 912, warp)) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            sh[warp * 2 * S::C + cl * V + k] = dg[k];
            sh[warp * 2 * S::C + S::C + cl * V + k] = db[k];
        }
    }
    __syncthreads();
    const int i = threadIdx.x, col = cta * S::C + i % S::C;
    if (i >= 2 * S::C || col >= d) return;
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < S::THREADS / 32; ++w) a += sh[w * 2 * S::C + i];
    (i < S::C ? dgamma : dbeta)[col] = a;
}

// How the rows come: from global memory row by row; the same, with CTAs from row_ctas on
// that take columns (part is not used); or ahead of their use through a ring of stages in
// shared memory.
enum BwdMode { kPlain, kFew, kRing };
constexpr int kMaxStages = 3;  // (25600 x 1024 bf16: 3 or 4 stages 33 us, 8 35 us)

// Whether rows that are not few come through the ring: where they did, plain loads waited for
// memory with 16 warps per SM (25600 x 1024 bf16 40 us, through the ring 33; 8000 x 3000 49
// and 37; 9001 x 1001 fp32 31.4 and 28.2).  A warp per row of bf16 has rows enough in flight
// (11264 x 512 12.8 us, with the ring 13.8), and bf16 by single elements has its instructions to
// wait for (9001 x 1001 20.4 us and 21.1).  32 warps leave 64 registers.
template <typename T, int V, int L>
constexpr bool takes_ring() {
    return L < 1024 && (sizeof(T) == 4 || (V == 8 && L > 32));
}

// A stage of the ring: `rows` consecutive rows of every tensor, whose bytes are a multiple of 16.
struct Ring {
    int rows, stages;
    int gamma;  // offset behind the stages
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <typename T, int V, int E, int L, int MODE>
__global__ void __launch_bounds__(Shape<L>::THREADS, bwd_ctas<E, L>())
ln_bwd_kernel(const T* __restrict__ dout, const T* __restrict__ x, const T* __restrict__ y,
              const T* __restrict__ gamma, const float* __restrict__ mean, const float* __restrict__ rstd,
              const T* __restrict__ dres, long long rows, int d, float inv_d, T* __restrict__ dx, int row_ctas,
              float* __restrict__ part, float* __restrict__ dgamma, float* __restrict__ dbeta, Ring ring, int* status) {
    using S = Shape<L>;
    using Col = Columns<T, V, L>;
    __shared__ float2 sh[2 * S::THREADS / 32];
    __shared__ __align__(8) uint64_t full[MODE == kRing ? kMaxStages : 1];
    __shared__ int abort_word;
    extern __shared__ __align__(128) unsigned char dynamic[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (MODE == kRing && threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) mbar_init(&full[s], 1);
        abort_word = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (MODE == kFew && (int)blockIdx.x >= row_ctas) {
        ln_bwd_columns<T, V, L>(dout, x, y, mean, rstd, (int)rows, d, (int)blockIdx.x - row_ctas,
                                reinterpret_cast<float*>(dynamic), dgamma, dbeta);
        return;
    }
    const int t = threadIdx.x % S::TPR, lr = threadIdx.x / S::TPR;
    // gamma stays in registers, or in shared memory beside a ring of whole fp32 vectors (in
    // registers it made that kernel spill, and beside the ring there is little L1 to spill to)
    constexpr bool GAMMA_SH = MODE == kRing && sizeof(T) == 4 && V == 4 && L >= 256;
    constexpr int G = GAMMA_SH ? V : E;
    alignas(8) float dg[E], db[E], gam[G];
    const int left = d - t * V;
    T* const gamma_sh = reinterpret_cast<T*>(dynamic + ring.gamma);
    if constexpr (GAMMA_SH) {
        for (int i = threadIdx.x; i < d; i += S::THREADS)
            if (TXL_BOUNDS(ring.gamma + (i + 1) * sizeof(T) <= dynamic_bytes(), 911, i)) gamma_sh[i] = gamma[i];
    } else {
        load_row<T, V, E, S::TPR>(gamma + t * V, left, gam);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) dg[e] = db[e] = 0.f;
    int phase = 0;
    // One row, this thread's elements of which lie at px, pd, py, pr and go to `to`.
    auto row = [&](const T* px, const T* pd, const T* py, const T* pr, T* to, bool in, float mu, float rs) {
        alignas(8) float xh[E], g[E];
        float2 s = both(0.f);
        if (in) {
            load_row<T, V, E, S::TPR>(px, left, xh);
            load_row<T, V, E, S::TPR>(pd, left, g);
            if (y) {
                alignas(8) float b[E];
                load_row<T, V, E, S::TPR>(py, left, b);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) pair(xh, e) = __fadd2_rn(pair(xh, e), pair(b, e));
            }
            // behind the row's end g is 0: what xh holds there reaches no sum
            float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                // (the mean is taken off before the product: it may be far larger than the rest)
                float2& h = pair(xh, e);
                float2& q = pair(g, e);
                h = __fmul2_rn(__fadd2_rn(h, both(-mu)), both(rs));
                if (MODE != kFew) {
                    pair(dg, e) = __ffma2_rn(q, h, pair(dg, e));
                    pair(db, e) = __fadd2_rn(pair(db, e), q);
                }
                if (GAMMA_SH && 2 * e % G == 0)
                    load_row<T, V, G, S::TPR>(gamma_sh + (t + S::TPR * (2 * e / V)) * V, left - S::TPR * (2 * e / V) * V,
                                              gam);
                q = __fmul2_rn(q, pair(gam, e % (G / 2)));
                s1 = __fadd2_rn(s1, q);
                s2 = __ffma2_rn(q, h, s2);
            }
            s = make_float2(s1.x + s1.y, s2.x + s2.y);
            // dres is added to rs g here: its loads run beside the reduction, and hold
            // no registers of their own through it
            if (dres) {
                alignas(8) float a[E];
                load_row<T, V, E, S::TPR>(pr, left, a);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) pair(g, e) = __ffma2_rn(pair(g, e), both(rs), pair(a, e));
            } else {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) pair(g, e) = __fmul2_rn(pair(g, e), both(rs));
            }
        }
        s = row_sum2<L>(s, sh, phase);
        phase ^= 1;
        if (!in) return;
        const float2 c1 = both(-rs * s.x * inv_d), c2 = both(-rs * s.y * inv_d);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) pair(g, e) = __fadd2_rn(__ffma2_rn(pair(xh, e), c2, pair(g, e)), c1);
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            constexpr int OFF = S::TPR * V;
            if (OFF * i < left && TXL_BOUNDS(OFF * i + V <= left, 903, left)) Vec<T, V>::store(to + OFF * i, g + V * i);
        }
    };
    if constexpr (MODE == kRing) {
        // This CTA's stages are blockIdx.x, blockIdx.x + row_ctas, ..  Thread 0 fills a slot
        // again when all threads are past their reads of it: with several warps per row
        // that is known from the row's own reduction.
        const long long n_stages = rows / ring.rows;
        const int count = (int)(n_stages > blockIdx.x ? (n_stages - blockIdx.x + row_ctas - 1) / row_ctas : 0);
        const uint32_t per = (uint32_t)ring.rows * d * sizeof(T);
        const uint32_t bytes = per * (2 + (y != nullptr) + (dres != nullptr));
        const uint32_t o_y = 2 * per, o_r = o_y + (y ? per : 0);
        auto fill = [&](int k, int slot) {
            const long long at = ((long long)k * row_ctas + blockIdx.x) * ring.rows * d;
            if (!TXL_BOUNDS(at + (long long)ring.rows * d <= rows * d, 905, at) ||
                !TXL_BOUNDS((slot + 1) * bytes <= dynamic_bytes(), 909, slot))
                return;
            unsigned char* const to = dynamic + slot * bytes;
            mbar_expect_tx(&full[slot], bytes);
            bulk_load(to, x + at, per, &full[slot]);
            bulk_load(to + per, dout + at, per, &full[slot]);
            if (y) bulk_load(to + o_y, y + at, per, &full[slot]);
            if (dres) bulk_load(to + o_r, dres + at, per, &full[slot]);
        };
        if (threadIdx.x == 0)
            for (int k = 0; k < ring.stages && k < count; ++k) fill(k, k);
        __syncthreads();  // the barriers are ready
        // The rows behind the last full stage are a stage of the CTA whose turn it is, copied
        // by its threads.
        const int rest = (int)(rows - n_stages * ring.rows);
        const int total = count + (rest && (long long)blockIdx.x == n_stages % row_ctas);
        bool ok = true;
        int slot = 0, parity = 0;
        long long r = (long long)blockIdx.x * ring.rows + lr;  // this thread's row
        float mu = 0.f, rs = 0.f;
        if (r < rows) mu = mean[r], rs = rstd[r];
#pragma unroll 1
        for (int k = 0; k < total; ++k) {
            T* const st = reinterpret_cast<T*>(dynamic + slot * bytes);
            int n = ring.rows;
            if (k == count) {
                n = rest;
                const long long at = n_stages * ring.rows * d;
                for (int i = threadIdx.x; i < n * d; i += S::THREADS) {
                    if (!TXL_BOUNDS(at + i < rows * d && (i + 1) * sizeof(T) <= per && (slot + 1) * bytes <= dynamic_bytes(), 910,
                                    at + i))
                        continue;
                    st[i] = x[at + i];
                    st[i + per / sizeof(T)] = dout[at + i];
                    if (y) st[i + o_y / sizeof(T)] = y[at + i];
                    if (dres) st[i + o_r / sizeof(T)] = dres[at + i];
                }
                __syncthreads();
            } else if (ok && !mbar_wait(&full[slot], parity, kDevTimeoutProducer, &abort_word, status)) {
                // (nothing is waited for or filled from here on; what is still on its way lands
                // before the CTA ends)
                ok = false;
                for (int i = k; threadIdx.x == 0 && i < count && i < k + ring.stages; ++i) {
                    const uint64_t t0 = globaltimer_ns();
                    const int at = i % ring.stages, odd = (i / ring.stages) & 1;
                    while (!mbar_try_wait(&full[at], odd) && globaltimer_ns() - t0 < kWaitLimitNs) {}
                }
            }
            const T* p = st + lr * d + t * V;
#pragma unroll 1
            for (int q = 0; q < n; q += S::R, p += S::R * d) {
                const float m = mu, s = rs;
                const bool in = q + lr < n;
                T* const to = dx + r * d + t * V;
                r += q + S::R >= n ? (long long)row_ctas * ring.rows - q : S::R;
                if (r < rows) mu = mean[r], rs = rstd[r];
                row(p, p + per / sizeof(T), p + o_y / sizeof(T), p + o_r / sizeof(T), to, in, m, s);
            }
            if (L <= 32) __syncthreads();
            if (threadIdx.x == 0 && ok && k + ring.stages < count) fill(k + ring.stages, slot);
            if (++slot == ring.stages) slot = 0, parity ^= 1;
        }
    } else {
        // where this thread's elements of its rows lie, row after row
        const long long first = (long long)blockIdx.x * S::R + lr, step = (long long)row_ctas * S::R, hop = step * d;
        long long at = first * d + t * V;
        int todo =
            (int)(rows > (long long)blockIdx.x * S::R ? (rows - (long long)blockIdx.x * S::R + step - 1) / step : 0);
        const float *mp = mean + first, *rp = rstd + first;
        long long past = rows - first;  // rows from this thread's on
#pragma unroll 1
        for (; todo > 0; --todo, at += hop, past -= step, mp += step, rp += step) {
            const bool in = past > 0;
            row(x + at, dout + at, y + at, dres + at, dx + at, in, in ? *mp : 0.f, in ? *rp : 0.f);
        }
    }
    if (MODE == kFew) return;
    // the CTA's rows fold in halves, into the first row's threads
    if (S::R > 1) {
        float* const fold = reinterpret_cast<float*>(dynamic);
#pragma unroll
        for (int half = S::R / 2; half > 0; half >>= 1) {
            __syncthreads();
            const int n = half * S::TPR;
            if (lr >= half && lr < 2 * half && TXL_BOUNDS(2 * E * n * sizeof(float) <= dynamic_bytes(), 907, n)) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    fold[(2 * e) * n + threadIdx.x - n] = dg[e];
                    fold[(2 * e + 1) * n + threadIdx.x - n] = db[e];
                }
            }
            __syncthreads();
            if (lr < half && TXL_BOUNDS(2 * E * n * sizeof(float) <= dynamic_bytes(), 908, n)) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    dg[e] += fold[(2 * e) * n + threadIdx.x];
                    db[e] += fold[(2 * e + 1) * n + threadIdx.x];
                }
            }
        }
    }
    if (lr > 0) return;
    float* to = part + (size_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
        const int c = (t + S::TPR * i) * V;
        if (c < d && TXL_BOUNDS(c + V <= d && (int)blockIdx.x < row_ctas, 906, c)) {
            store_sums<V>(to + c, dg + V * i);
            store_sums<V>(to + d + c, db + V * i);
        }
    }
}

// dgamma and dbeta: the CTAs' sums of 32 columns per CTA, 64 threads on each two, all of
// whose loads are on their way together (up to 384 parts).
__global__ void __launch_bounds__(1024) ln_bwd_sum_kernel(const float* __restrict__ part, int n_part, int d,
                                                          float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ float sh[32][33];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + (lane & 15) * 2;  // (2 d is even)
    float2 a = both(0.f);
    for (int p0 = threadIdx.x >> 4; c < 2 * d && p0 < n_part; p0 += 6 * 64) {
        float2 v[6];
#pragma unroll
        for (int i = 0; i < 6; ++i)
            v[i] = p0 + 64 * i < n_part && TXL_BOUNDS(c + 2 <= 2 * d, 913, c)
                       ? *reinterpret_cast<const float2*>(part + (size_t)(p0 + 64 * i) * 2 * d + c)
                       : both(0.f);
#pragma unroll
        for (int i = 0; i < 6; ++i) a = __fadd2_rn(a, v[i]);
    }
    a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
    if (lane < 16) {
        sh[w][2 * lane] = a.x;
        sh[w][2 * lane + 1] = a.y;
    }
    __syncthreads();
    const float s = warp_sum(sh[lane][w]);  // column w of this CTA's 32
    const int cw = blockIdx.x * 32 + w;
    if (lane == 0 && cw < 2 * d) {
        if (cw < d)
            dgamma[cw] = s;
        else
            dbeta[cw - d] = s;
    }
}

// Launch with programmatic stream serialisation (every kernel here waits for
// the one before it before its first global access).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), unsigned grid, unsigned threads, size_t dynamic, cudaStream_t stream,
                       Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = dynamic;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Calls f with the element and lane counts that a row of d elements takes: as few lanes as
// hold it at 32 elements each (forward) or 16 (backward, which keeps two sums per element
// besides), and short rows several to a warp (400000 x 64 bf16: forward 26 us, backward 37,
// with a warp to each row 102 and 115).
template <int E, int L>
struct Pick {
    static constexpr int e = E, l = L;
};
template <typename F>
cudaError_t pick_fwd(int d, F f) {
    if (d <= 64) return f(Pick<8, 8>());
    if (d <= 128) return f(Pick<8, 16>());
    if (d <= 256) return f(Pick<8, 32>());
    if (d <= 512) return f(Pick<16, 32>());
    if (d <= 1024) return f(Pick<32, 32>());
    if (d <= 2048) return f(Pick<32, 64>());
    if (d <= 4096) return f(Pick<32, 128>());
    if (d <= 8192) return f(Pick<32, 256>());
    return f(Pick<32, 512>());
}
template <typename F>
cudaError_t pick_bwd(int d, F f) {
    if (d <= 64) return f(Pick<8, 8>());
    if (d <= 128) return f(Pick<8, 16>());
    if (d <= 256) return f(Pick<8, 32>());
    if (d <= 512) return f(Pick<16, 32>());
    if (d <= 1024) return f(Pick<16, 64>());
    if (d <= 2048) return f(Pick<16, 128>());
    if (d <= 4096) return f(Pick<16, 256>());
    if (d <= 8192) return f(Pick<16, 512>());
    return f(Pick<16, 1024>());
}

// Calls f with the vector length of rows of d elements.
template <int V>
struct Width {
    static constexpr int v = V;
};
template <typename T, typename F>
auto pick_width(int d, F f) {
    if constexpr (sizeof(T) == 2)
        return d % 2 ? f(Width<1>()) : d % 8 ? f(Width<2>()) : f(Width<8>());
    else
        return d % 4 ? f(Width<1>()) : f(Width<4>());
}

// How the backward pass is launched: CTAs that take rows (one round of resident ones at
// most; none without rows, as a row CTA reads gamma before its first row), CTAs that take
// columns (0: the row CTAs sum them, into as many parts), and the rows of a ring's stage.
struct BwdGrid {
    int rows, columns, stage;
};
template <typename T>
BwdGrid bwd_grid(long long rows, int d) {
    BwdGrid g = {};
    pick_bwd(d, [&](auto k) {
        constexpr int E = decltype(k)::e, L = decltype(k)::l, R = Shape<L>::R;
        const long long most = (long long)bwd_ctas<E, L>() * current_sm_count();
        // as many rows as fill the CTA, start at 16 bytes, and make 4 KB where there are many
        g.stage = R;
        while ((long long)g.stage * d * sizeof(T) % 16) g.stage *= 2;
        while ((long long)g.stage * d * sizeof(T) < 4096 && rows / (2 * g.stage) >= 2 * most) g.stage *= 2;
        int by = R;
        pick_width<T>(d, [&](auto v) {
            constexpr int V = decltype(v)::v;
            using C = Columns<T, V, L>;
            // (two stages of four tensors may not fit: then the rows are dealt one by one)
            if (rows <= C::ROWS)
                g.columns = (d + C::C - 1) / C::C;
            else if (takes_ring<T, V, L>() &&
                     (size_t)(g.stage * 4 * 2 + 1) * d * sizeof(T) <= kRingRoom / bwd_ctas<E, L>())
                by = g.stage;
            return 0;
        });
        const long long want = (rows + by - 1) / by;
        g.rows = (int)(want < most ? want : most);
        return cudaSuccess;
    });
    return g;
}

template <typename T, int V>
cudaError_t ln_fwd(const void* x, const void* y, const void* gamma, const void* beta, long long rows, int d,
                   float eps, void* out, float* mean, float* rstd, cudaStream_t stream) {
    if (rows <= 0) return cudaSuccess;
    return pick_fwd(d, [&](auto k) {
        constexpr int E = decltype(k)::e, L = decltype(k)::l;
        using S = Shape<L, fwd_threads<E>()>;
        const long long ctas = (rows + S::R - 1) / S::R;
        if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
        return launch_pdl(ln_fwd_kernel<T, V, E, L>, (unsigned)ctas, (unsigned)S::THREADS, 0, stream,
                          static_cast<const T*>(x), static_cast<const T*>(y), static_cast<const T*>(gamma),
                          static_cast<const T*>(beta), rows, d, 1.f / d, eps, static_cast<T*>(out), mean, rstd);
    });
}

template <typename T, int V>
cudaError_t ln_bwd(const void* dout, const void* x, const void* y, const void* gamma, const float* mean,
                   const float* rstd, const void* dres, long long rows, int d, void* dx, float* dgamma,
                   float* dbeta, float* part, int* status, cudaStream_t stream) {
    // (no rows: column CTAs that add nothing write the zeros)
    const BwdGrid grid = bwd_grid<T>(rows, d);
    const cudaError_t e = pick_bwd(d, [&](auto k) {
        constexpr int E = decltype(k)::e, L = decltype(k)::l;
        using S = Shape<L>;
        auto go = [&](auto kern, size_t dynamic, Ring ring) {
            return launch_pdl(kern, (unsigned)(grid.rows + grid.columns), (unsigned)S::THREADS, dynamic, stream,
                              static_cast<const T*>(dout), static_cast<const T*>(x), static_cast<const T*>(y),
                              static_cast<const T*>(gamma), mean, rstd, static_cast<const T*>(dres), rows, d, 1.f / d,
                              static_cast<T*>(dx), grid.rows, part, dgamma, dbeta, ring, status);
        };
        if (grid.columns)
            return go(ln_bwd_kernel<T, V, E, L, kFew>, S::THREADS / 32 * 2 * Columns<T, V, L>::C * sizeof(float),
                      Ring{});
        const size_t fold = S::R > 1 ? S::THREADS * E * sizeof(float) : 0;
        const size_t stage = (size_t)grid.stage * d * sizeof(T) * (2 + (y != nullptr) + (dres != nullptr));
        if constexpr (takes_ring<T, V, L>()) {
            constexpr size_t kRoom = kRingRoom / bwd_ctas<E, L>();
            const size_t own = (size_t)d * sizeof(T), most = kRoom > own ? (kRoom - own) / stage : 0;
            const int stages = (int)(most < kMaxStages ? most : kMaxStages);
            if (stages >= 2) {
                static PerDeviceOnce attrs;
                const cudaError_t set = attrs.run([] {
                    return cudaFuncSetAttribute(ln_bwd_kernel<T, V, E, L, kRing>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRoom);
                });
                if (set != cudaSuccess) return set;
                const size_t bytes = stage * stages + own;
                return go(ln_bwd_kernel<T, V, E, L, kRing>, bytes > fold ? bytes : fold,
                          Ring{grid.stage, stages, (int)(stage * stages)});
            }
        }
        return go(ln_bwd_kernel<T, V, E, L, kPlain>, fold, Ring{});
    });
    if (e != cudaSuccess || grid.columns) return e;
    return launch_pdl(ln_bwd_sum_kernel, (unsigned)((2 * d + 31) / 32), 1024u, 0, stream, part, grid.rows, d, dgamma,
                      dbeta);
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const void* x, const void* y, const void* gamma, const void* beta, long long rows,
                                  int d, float eps, void* out, float* mean, float* rstd, int bf16,
                                  cudaStream_t stream) {
    auto go = [&](auto zero) {
        using T = decltype(zero);
        return pick_width<T>(d, [&](auto v) {
            return ln_fwd<T, decltype(v)::v>(x, y, gamma, beta, rows, d, eps, out, mean, rstd, stream);
        });
    };
    return bf16 ? go(__nv_bfloat16()) : go(float());
}

size_t layer_norm_bwd_workspace_bytes(long long rows, int d, int bf16) {
    const BwdGrid g = bf16 ? bwd_grid<__nv_bfloat16>(rows, d) : bwd_grid<float>(rows, d);
    return g.columns ? 0 : (size_t)g.rows * 2 * d * sizeof(float);
}

cudaError_t launch_layer_norm_bwd(const void* dout, const void* x, const void* y, const void* gamma,
                                  const float* mean, const float* rstd, const void* dres, long long rows, int d,
                                  void* dx, float* dgamma, float* dbeta, void* workspace, int bf16, int* status,
                                  cudaStream_t stream) {
    float* part = static_cast<float*>(workspace);
    auto go = [&](auto zero) {
        using T = decltype(zero);
        return pick_width<T>(d, [&](auto v) {
            return ln_bwd<T, decltype(v)::v>(dout, x, y, gamma, mean, rstd, dres, rows, d, dx, dgamma, dbeta, part, status,
                                               stream);
        });
    };
    return bf16 ? go(__nv_bfloat16()) : go(float());
}

TXL_BOUNDS_READER(bounds_word_layer_norm_train)

}  // namespace txl
