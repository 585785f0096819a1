// The 2-norm of many tensors, each one's and that of all together, and their scaling by
// min(1, max_norm / norm) in place.
//
// Two launches.  The first cuts the tensors into pieces, one per CTA, and leaves the sum
// of squares of each; in the second every CTA adds all pieces' sums, in the same order,
// so that each has the norm without a launch in between that finds it (but where tensors
// are many), and scales a piece of its own.  The pieces come in the opposite order then: the last ones read are still in
// L2.  Both are bound by memory; nothing is written where nothing is clipped.
//
// Sums are fp32 throughout, in chains of 128 additions and then of those, for a piece whose
// sum leaves [2^-80, 2^100] of squares scaled by a power of two that a second look at the
// piece finds, so that neither large nor small gradients leave the range.  A sum is kept as
// a number in [1, 4) and an even power of two.  (fp64 would have the range, but at a
// sixty-fourth of the rate.)
//
// The tensor table travels in the kernel's parameters, as AdamW's does.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "grad_norm.h"
#include "txl_device.cuh"

namespace txl {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLoads = 8;                          // 16-byte vectors on their way per thread
constexpr long long kStep = kThreads * 16;         // bytes that a CTA's threads load at once
// A thread's chain of additions ends after so many rounds of loads: 2^33 alike bf16 gradients in one
// chain per thread were off by 2.6e-5.  Pieces of no more rounds have code without that, whose loop
// takes less time (37.8 M bf16 gradients: 10.5 us, with it 11.2).
constexpr int kRounds = 16;
constexpr long long kShort = kRounds * kLoads * kStep;
// Up to so many pieces each CTA that scales adds all their sums itself; more, as many small tensors
// have, are added once in a launch of their own (clipped, us, without and with it: 1000 small tensors
// 20 and 22, 2000 39 and 37, 5000 112 and 85, 100000 16000 and 1700).
constexpr long long kFewPieces = 1800;
constexpr int kSmallTable = 32, kMiddleTable = 160, kLargeTable = 480;  // tensors per launch
constexpr int kNothing = -(1 << 20);               // exponent of a sum that is 0

struct GradEntry {
    void* p;
    long long n;
    unsigned start;  // first piece, relative to the launch's first
    int bf16;
};

template <int CAP>
struct GradTable {
    int n;
    unsigned pieces;
    GradEntry e[CAP];
};

// value = x 2^e, x in [1, 4) (or not finite) and e even; 0: e = kNothing.
struct Sum {
    float x;
    int e;
};

template <int CAP>
__device__ __forceinline__ int find_entry(const GradTable<CAP>& t, unsigned b) {
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

__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void store16(void* p, const uint4& v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ float2 bf16_pair(unsigned w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}

// Sum or maximum over the CTA, every thread with the result.
template <bool MAX>
__device__ __forceinline__ float over_cta(float a, float (&sh)[kWarps]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float b = __shfl_xor_sync(0xffffffffu, a, o);
        a = MAX ? max_nan(a, b) : a + b;
    }
    __syncthreads();  // the last use of sh is over
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
    __syncthreads();
    a = sh[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) a = MAX ? max_nan(a, sh[w]) : a + sh[w];
    return a;
}

// max_norm / norm as a factor, and a power of two (1 as a rule) that a value is multiplied by behind
// it: a quotient below 2^-126 would lose its bits, where the product need not.
struct Factor {
    float f, down;
    __device__ __forceinline__ Factor(float max_norm, float norm) : f(max_norm / norm), down(1.f) {
        if (f < 0x1p-126f) {
            const int m = ilogbf(max_norm), n = ilogbf(norm), a = (n - m) / 2 - 1;
            f = ldexpf(ldexpf(max_norm, -m) / ldexpf(norm, -n), -a);
            down = ldexpf(1.f, a - (n - m));
        }
    }
    // (rounded by the first product alone, unless the result is below 2^-126)
    __device__ __forceinline__ float operator()(float x) const { return x * f * down; }
};

// A piece of a tensor: elements [at, at + n) of `of`.
struct Piece {
    char* p;  // of the first element
    long long at, n, of;
};

template <int CAP>
__device__ __forceinline__ Piece piece_of(const GradTable<CAP>& t, int e, unsigned b, long long piece_bytes) {
    const int es = t.e[e].bf16 ? 2 : 4;
    const long long per = piece_bytes / es, at = (long long)(b - t.e[e].start) * per;
    return {static_cast<char*>(t.e[e].p) + at * es, at, min(per, t.e[e].n - at), t.e[e].n};
}

// f(vector) for each thread's vectors of the piece (zeros behind its end), g(value) for the
// last elements of a tensor (once, at any time); FOLD: fold() behind every kRounds rounds of loads.
template <bool BF16, bool FOLD, typename F, typename G, typename H>
__device__ __forceinline__ void each_vector(const Piece& c, F f, G g, H fold) {
    constexpr int N = BF16 ? 8 : 4, ES = BF16 ? 2 : 4;
    const long long vecs = c.n / N;
    const auto last = [&] {
        const int left = (int)(c.n - vecs * N);
        if ((int)threadIdx.x < left && TXL_BOUNDS(c.at + vecs * N + threadIdx.x < c.of, 1202, threadIdx.x)) {
            const char* const p = c.p + vecs * 16 + threadIdx.x * ES;
            g(BF16 ? __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p)) : *reinterpret_cast<const float*>(p));
        }
    };
    if (FOLD) last();  // (2^31 bf16 gradients took 612 us with it behind the loop, 589 ahead)
    int rounds = 0;
#pragma unroll 1
    for (long long base = threadIdx.x; base < vecs; base += (long long)kLoads * kThreads) {
        uint4 v[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const long long i = base + u * kThreads;
            v[u] = i < vecs && TXL_BOUNDS(c.at >= 0 && c.at + (i + 1) * N <= c.of, 1201, c.at + i * N) ? load16(c.p + i * 16)
                                                                                                  : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) f(v[u]);
        if (FOLD && ++rounds == kRounds) fold(), rounds = 0;
    }
    if (!FOLD) last();
}

template <bool BF16>
__device__ __forceinline__ float2 pair_of(const uint4& v, int i) {
    if (BF16) return bf16_pair(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
    return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                  : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
}

// Sum of (scale x)^2 over the piece, every thread with the result.
template <bool BF16, bool SCALED, bool LONG>
__device__ __forceinline__ float squares(const Piece& c, float scale, float (&sh)[kWarps]) {
    constexpr int PAIRS = BF16 ? 4 : 2;
    float2 a[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) a[i] = make_float2(0.f, 0.f);
    float s = 0.f;
    const auto fold = [&] {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) s += a[i].x + a[i].y, a[i] = make_float2(0.f, 0.f);
    };
    each_vector<BF16, LONG>(
        c,
        [&](const uint4& v) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                float2 x = pair_of<BF16>(v, i);
                if (SCALED) x.x *= scale, x.y *= scale;
                a[i] = fma2(x, x, a[i]);
            }
        },
        [&](float x) {
            if (SCALED) x *= scale;
            s = x * x;
        },
        fold);
    fold();
    return over_cta<false>(s, sh);
}

template <bool BF16, bool LONG>
__device__ __noinline__ Sum squares_scaled(const Piece c, float (&sh)[kWarps]) {
    float m = 0.f;
    each_vector<BF16, false>(
        c,
        [&](const uint4& v) {
#pragma unroll
            for (int i = 0; i < (BF16 ? 4 : 2); ++i) {
                const float2 x = pair_of<BF16>(v, i);
                m = max_nan(m, max_nan(fabsf(x.x), fabsf(x.y)));
            }
        },
        [&](float x) { m = max_nan(m, fabsf(x)); }, [] {});
    m = over_cta<true>(m, sh);
    if (m == 0.f) return {0.f, kNothing};
    if (!(m < INFINITY)) return {m, 0};
    const int k = max(ilogbf(m), -120);
    return {squares<BF16, true, LONG>(c, ldexpf(1.f, -k), sh), 2 * k};
}

// x 2^e with x in [1, 4), e even.
__device__ __forceinline__ Sum normalise(Sum s) {
    if (s.e == kNothing || !(s.x < INFINITY)) return s;
    if (s.x == 0.f) return {0.f, kNothing};
    const int k = ilogbf(s.x) & ~1;
    return {ldexpf(s.x, -k), s.e + k};
}

template <int CAP, bool LONG>
__global__ void __launch_bounds__(kThreads) grad_sums_kernel(const __grid_constant__ GradTable<CAP> t, long long piece_bytes,
                                                             Sum* __restrict__ part, unsigned n_part) {
    __shared__ float sh[kWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int e = find_entry(t, blockIdx.x);
    const Piece c = piece_of(t, e, blockIdx.x, piece_bytes);
    const bool bf16 = t.e[e].bf16;
    Sum s = {bf16 ? squares<true, false, LONG>(c, 1.f, sh) : squares<false, false, LONG>(c, 1.f, sh), 0};
    if (!(s.x >= 0x1p-80f && s.x <= 0x1p100f)) s = bf16 ? squares_scaled<true, LONG>(c, sh) : squares_scaled<false, LONG>(c, sh);
    if (threadIdx.x == 0 && TXL_BOUNDS(blockIdx.x < n_part, 1203, blockIdx.x)) part[blockIdx.x] = normalise(s);
}

// Sum of n sums by `width` threads (a warp, or the CTA), in an order that n alone decides; each
// thread adds its own against the largest exponent, whose parts then meet.
struct Total {
    float x;
    int e;  // kNothing: 0
    __device__ __forceinline__ float norm() const { return e == kNothing ? 0.f : ldexpf(sqrtf(x), e / 2); }
};

__device__ __forceinline__ Total total_by_warp(const Sum* part, unsigned n) {
    const int lane = threadIdx.x & 31;
    int most = kNothing;
    for (unsigned i = lane; i < n; i += 32) most = max(most, part[i].e);
    most = __reduce_max_sync(0xffffffffu, most);
    float x = 0.f;
    for (unsigned i = lane; i < n; i += 32) {
        const Sum s = part[i];
        x += ldexpf(s.x, max(s.e - most, -200));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return {x, most};
}

__device__ __forceinline__ Total total_by_cta(const Sum* part, unsigned n, float (&sh)[kWarps], int (&she)[kWarps]) {
    constexpr int R = 6;  // kept in registers per thread: the second look at the others is at L2
    Sum own[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const unsigned i = threadIdx.x + k * kThreads;
        own[k] = i < n ? part[i] : Sum{0.f, kNothing};
    }
    int most = kNothing;
#pragma unroll
    for (int k = 0; k < R; ++k) most = max(most, own[k].e);
    for (unsigned i = threadIdx.x + R * kThreads; i < n; i += kThreads) most = max(most, part[i].e);
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) she[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) most = max(most, she[w]);
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < R; ++k) x += ldexpf(own[k].x, max(own[k].e - most, -200));
    for (unsigned i = threadIdx.x + R * kThreads; i < n;) {  // (in chains of 64, as many tensors are many sums)
        const unsigned end = n - i > 64 * kThreads ? i + 64 * kThreads : n;
        float chain = 0.f;
        for (; i < end; i += kThreads) {
            const Sum s = part[i];
            chain += ldexpf(s.x, max(s.e - most, -200));
        }
        x += chain;
    }
    return {over_cta<false>(x, sh), most};
}

// The total of n sums, which stands in their place for the scaling where they are many.
__global__ void __launch_bounds__(kThreads) grad_total_kernel(const Sum* __restrict__ part, unsigned n, Sum* __restrict__ total) {
    __shared__ float sh[kWarps];
    __shared__ int she[kWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Total t = total_by_cta(part, n, sh, she);
    if (threadIdx.x == 0) *total = {t.x, t.e};
}

// Norms from the sums, and a piece's scaling.  `all`, `n_all`: the sums of every launch's pieces, or
// their total; `part`: this one's.
template <int CAP, bool CLIP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ GradTable<CAP> t, long long piece_bytes,
                                                             const Sum* __restrict__ all, unsigned n_all,
                                                             const Sum* __restrict__ part, float max_norm, float* norm,
                                                             float* norms) {
    __shared__ float sh[kWarps];
    __shared__ int she[kWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (norms) {  // a warp per tensor
        for (int e = blockIdx.x * kWarps + warp; e < t.n; e += gridDim.x * kWarps) {
            const unsigned end = e + 1 < t.n ? t.e[e + 1].start : t.pieces;
            const Total s = total_by_warp(part + t.e[e].start, end - t.e[e].start);
            if (lane == 0) norms[e] = s.norm();
        }
    }
    if (!CLIP && (blockIdx.x || !norm)) return;
    const Total s = total_by_cta(all, n_all, sh, she);
    const float length = s.norm();
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = length;
    if (!CLIP || !(length > max_norm && length < INFINITY) || blockIdx.x >= t.pieces) return;
    const Factor scaled(max_norm, length);
    const unsigned b = t.pieces - 1 - blockIdx.x;
    const int e = find_entry(t, b);
    const Piece c = piece_of(t, e, b, piece_bytes);
    const bool bf16 = t.e[e].bf16;
    const int n = bf16 ? 8 : 4;
    const long long vecs = c.n / n;
#pragma unroll 1
    for (long long base = threadIdx.x; base < vecs; base += (long long)kLoads * kThreads) {
        uint4 v[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const long long i = base + u * kThreads;
            if (i < vecs && TXL_BOUNDS(c.at >= 0 && c.at + (i + 1) * n <= c.of, 1204, c.at + i * n)) v[u] = load16(c.p + i * 16);
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const long long i = base + u * kThreads;
            uint4 o;
            if (bf16) {
                unsigned w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = bf16_pair(w[k]);
                    w[k] = pack_bf16x2(scaled(f.x), scaled(f.y));
                }
                o = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                o = make_uint4(__float_as_uint(scaled(__uint_as_float(v[u].x))), __float_as_uint(scaled(__uint_as_float(v[u].y))),
                               __float_as_uint(scaled(__uint_as_float(v[u].z))), __float_as_uint(scaled(__uint_as_float(v[u].w))));
            }
            if (i < vecs && TXL_BOUNDS(c.at >= 0 && c.at + (i + 1) * n <= c.of, 1205, c.at + i * n))
                store16(c.p + i * 16, o);
        }
    }
    const int left = (int)(c.n - vecs * n);
    if ((int)threadIdx.x < left && TXL_BOUNDS(c.at + vecs * n + threadIdx.x < c.of, 1206, threadIdx.x)) {
        if (bf16) {
            __nv_bfloat16* const p = reinterpret_cast<__nv_bfloat16*>(c.p + vecs * 16) + threadIdx.x;
            *p = __float2bfloat16_rn(scaled(__bfloat162float(*p)));
        } else {
            float* const p = reinterpret_cast<float*>(c.p + vecs * 16) + threadIdx.x;
            *p = scaled(*p);
        }
    }
}

// ------------------------------------------------------------ host side
long long bytes_of(const txl_grad_tensor& t) { return t.n * (t.dtype == TXL_BF16 ? 2 : 4); }

// Bytes of a piece: as many as make 8 pieces per SM, whole steps of a CTA, 4 at least (a
// piece that is loaded in a few rounds costs less than its CTA's begin and end).  37.8 M gradients
// of both types, clipped: 27.5 us with 8 per SM, 29.7 with 5, 29.1 with 10, 31.2 with 16.
long long piece_bytes_of(const txl_grad_tensor* tensors, int n) {
    long long total = 0;
    for (int i = 0; i < n; ++i) total += bytes_of(tensors[i]);
    const long long most = 8ll * current_sm_count();
    return std::max(4ll, (total + most * kStep - 1) / (most * kStep)) * kStep;
}
long long pieces_of(const txl_grad_tensor& t, long long piece_bytes) {
    const long long n = bytes_of(t);
    return n <= piece_bytes ? n > 0 : (n + piece_bytes - 1) / piece_bytes;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), unsigned grid, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Calls f(table, first piece, first tensor) for the tensors, CAP at a time.
template <int CAP, typename F>
cudaError_t each_group(const GradNormArgs& a, long long piece_bytes, F f) {
    GradTable<CAP> t;
    long long first = 0;
    for (int i = 0; i < a.n_tensors;) {
        const int i0 = i;
        long long at = 0;
        t.n = 0;
        for (; i < a.n_tensors && t.n < CAP; ++i) {
            const txl_grad_tensor& x = a.tensors[i];
            t.e[t.n++] = {x.grad, x.n, (unsigned)at, x.dtype == TXL_BF16};
            at += pieces_of(x, piece_bytes);
        }
        t.pieces = (unsigned)at;
        const cudaError_t e = f(t, first, i0);
        if (e != cudaSuccess) return e;
        first += at;
    }
    return cudaSuccess;
}

template <int CAP>
cudaError_t run(const GradNormArgs& a, cudaStream_t stream) {
    const long long piece = a.plan.piece_bytes, pieces = a.plan.pieces;
    Sum* const part = static_cast<Sum*>(a.workspace);
    cudaError_t e = each_group<CAP>(a, piece, [&](const GradTable<CAP>& t, long long first, int) {
        return t.pieces ? launch_pdl(piece > kShort ? grad_sums_kernel<CAP, true> : grad_sums_kernel<CAP, false>, t.pieces, stream, t,
                                     piece, part + first, (unsigned)(pieces - first))
                        : cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    const Sum* all = part;
    unsigned n_all = (unsigned)pieces;
    if (a.max_norm > 0 && pieces > kFewPieces) {
        e = launch_pdl(grad_total_kernel, 1, stream, (const Sum*)part, n_all, part + pieces);
        if (e != cudaSuccess) return e;
        all = part + pieces, n_all = 1;
    }
    return each_group<CAP>(a, piece, [&](const GradTable<CAP>& t, long long first, int i0) {
        float* const norm = i0 ? nullptr : a.norm;
        float* const norms = a.norms ? a.norms + i0 : nullptr;
        const unsigned by_norms = (unsigned)(t.n + kWarps - 1) / kWarps;
        if (a.max_norm > 0)
            return launch_pdl(grad_norm_kernel<CAP, true>, std::max(1u, t.pieces), stream, t, piece, all, n_all,
                              (const Sum*)(part + first), (float)a.max_norm, norm, norms);
        return launch_pdl(grad_norm_kernel<CAP, false>, norms ? by_norms : 1u, stream, t, piece, all, n_all,
                          (const Sum*)(part + first), 0.f, norm, norms);
    });
}

}  // namespace

GradNormPlan grad_norm_plan(const txl_grad_tensor* tensors, int n) {
    GradNormPlan p = {piece_bytes_of(tensors, n), 0};
    for (int i = 0; i < n; ++i) p.pieces += pieces_of(tensors[i], p.piece_bytes);
    return p;
}

size_t grad_norm_workspace_bytes(const GradNormPlan& plan) {
    const long long sums = plan.pieces + (plan.pieces > kFewPieces);  // (the total)
    return ((size_t)sums * sizeof(Sum) + 255) / 256 * 256;
}

cudaError_t launch_grad_norm(const GradNormArgs& a, cudaStream_t stream) {
    if (a.n_tensors <= kSmallTable) return run<kSmallTable>(a, stream);
    return a.n_tensors <= kMiddleTable ? run<kMiddleTable>(a, stream) : run<kLargeTable>(a, stream);
}

TXL_BOUNDS_READER(bounds_word_grad_norm)

}  // namespace txl
