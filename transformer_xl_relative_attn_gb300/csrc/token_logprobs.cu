// Log probabilities of given tokens from a row's logits, with what a sampler or a loss
// wants besides, and their gradient.  Of a row x of V logits and its token,
//
//   lse = ln sum e^x,   logprob = x_token - lse,   entropy = -sum p ln p,   p = e^(x - lse)
//   the `top` largest logits (of equal ones the lower index first) and their x - lse
//
//   dx_j = dlogprob (delta_j - p_j) + dlse p_j - dentropy p_j ((x_j - lse) + entropy)
//
// The forward pass reads each logit once (softmax_sums.cuh has the statistics); what
// bounds it is that read.  A row goes to a warp where it is short, to a CTA, or, where
// rows are few, to a cluster of CTAs, each with a part of the row: the parts meet in the
// first CTA's shared memory, so there is one launch, no workspace, and the order of the
// additions depends on the sizes alone.
//
// The best `top` of a warp lie sorted in its lanes, one each, as 64-bit keys (the value's
// order, then the complement of the index: no two are alike).  A vector of logits whose
// maximum is below the last of them costs one comparison and a vote.
//
// The gradient is a pass of its own, read once and written once, in place where the
// caller wants it.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "softmax_sums.cuh"
#include "token_logprobs.h"
#include "txl_device.cuh"

namespace txl {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr unsigned kAll = 0xffffffffu;

// 16 bytes of logits, read once.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    uint4 q;
    __device__ __forceinline__ static uint4 nothing() { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
    __device__ __forceinline__ static float2 halves(unsigned w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    __device__ __forceinline__ float2 pair(int i) const {  // i known at compile time
        return halves(i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w);
    }
    __device__ __forceinline__ float max() const {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
        const float2 f = halves(*reinterpret_cast<const unsigned*>(&m));
        return sm_max_nan(f.x, f.y);
    }
    __device__ __forceinline__ float at(int j) const {
        const unsigned w = j & 4 ? (j & 2 ? q.w : q.z) : (j & 2 ? q.y : q.x);
        return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    uint4 q;
    __device__ __forceinline__ static uint4 nothing() { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
    __device__ __forceinline__ float2 pair(int i) const {
        return i == 0 ? make_float2(__uint_as_float(q.x), __uint_as_float(q.y))
                      : make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
    }
    __device__ __forceinline__ float max() const {
        return sm_max_nan(sm_max_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                          sm_max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
    __device__ __forceinline__ float at(int j) const {
        return __uint_as_float(j & 2 ? (j & 1 ? q.w : q.z) : (j & 1 ? q.y : q.x));
    }
};

__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// A row as its 16-byte vectors and the elements before and behind them.
struct RowCut {
    int head, vecs, loose;  // elements before the first vector; vectors; elements outside of them
    template <typename T>
    __device__ __forceinline__ RowCut(const T* row, int V) {
        const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T);
        head = min(V, (int)((Vec<T>::N - off) % Vec<T>::N));
        vecs = (V - head) / Vec<T>::N;
        loose = V - vecs * Vec<T>::N;
    }
    // index of the i-th element outside the vectors (fewer than 2 Vec<T>::N)
    template <typename T>
    __device__ __forceinline__ int index(int i) const {
        return i < head ? i : i + vecs * Vec<T>::N;
    }
};

// ------------------------------------------------------------ alternatives
// The order of fp32 values as that of unsigned integers: -0 as 0, NaN above all, and 0
// below what any value gives.
__device__ __forceinline__ unsigned order_of(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const unsigned b = __float_as_uint(x + 0.f);
    return b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// The best keys that a warp has seen, lane i with the i-th; `last` is the k-th.
struct Best {
    unsigned long long key, last;
    float bar;  // value of the k-th, -inf while there are fewer
    __device__ __forceinline__ void clear() { key = last = 0, bar = -INFINITY; }
    // One candidate per lane (0: none).
    __device__ __forceinline__ void offer(unsigned long long c, int k) {
        const int lane = threadIdx.x & 31;
        unsigned more = __ballot_sync(kAll, c > last);
        if (!more) return;
        do {
            const int src = __ffs(more) - 1;
            const unsigned long long n = __shfl_sync(kAll, c, src);
            const unsigned long long up = __shfl_up_sync(kAll, key, 1);
            const int at = __popc(__ballot_sync(kAll, key > n));
            key = lane < at ? key : lane == at ? n : up;
            last = __shfl_sync(kAll, key, k - 1);
            if (lane == src) c = 0;
            more = __ballot_sync(kAll, c > last);
        } while (more);
        bar = last ? value_of((unsigned)(last >> 32)) : -INFINITY;
    }
    __device__ __forceinline__ void offer(bool valid, float x, unsigned index, int k) {
        offer(valid ? (unsigned long long)order_of(x) << 32 | (unsigned)~index : 0ull, k);
    }
    // Whether a vector of this maximum may hold one of the best.
    __device__ __forceinline__ bool worth(float max) const { return !(max < bar); }
};

// ------------------------------------------------------------ one warp's share of a row
// Vectors first + 32 warp + lane + i step, i = 0, 1, .., below `end`, and, with `loose`,
// the elements outside the vectors.
template <typename T, bool TOP, int U>
__device__ __forceinline__ void scan(const T* row, int V, const RowCut& cut, int first, int end, int step, bool loose, int k,
                                     SoftmaxSums& sums, Best& best) {
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x & 31;
    const T* const vec0 = row + cut.head;
    float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
    // sums' own s and t stay 0 until the end: the pairs hold them
#pragma unroll 1
    for (int base = first; base < end; base += U * step) {
        Vec<T> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * step + lane;
            v[u].q = i < end && TXL_BOUNDS(i >= 0 && cut.head + (long long)(i + 1) * N <= V, 1101, i)
                         ? load_stream(vec0 + (size_t)i * N)
                         : Vec<T>::nothing();
        }
        float most[U], all = v[0].max();
        most[0] = all;
#pragma unroll
        for (int u = 1; u < U; ++u) {
            most[u] = v[u].max();
            all = sm_max_nan(all, most[u]);
        }
        if (all > sums.m) {
            const float d = fmaxf(sums.m - all, kLowest), f = sm_ex2(d * kLog2e);
            const float2 ff = make_float2(f, f);
            t = sm_mul2(ff, sm_fma2(make_float2(d, d), s, t));
            s = sm_mul2(ff, s);
            sums.m = all;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N / 2; ++i) sm_add_pair(v[u].pair(i), sums.m, s, t);
        if (TOP) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!__any_sync(kAll, best.worth(most[u]))) continue;
                const int i = base + u * step + lane;
#pragma unroll 1
                for (int j = 0; j < N; ++j) best.offer(i < end, v[u].at(j), cut.head + i * N + j, k);
            }
        }
    }
    sums.s = s.x + s.y;
    sums.t = t.x + t.y;
    if (loose) {
        const bool mine = lane < cut.loose;
        const int at = mine ? cut.index<T>(lane) : 0;
        const float x = mine && TXL_BOUNDS(at < V, 1102, at) ? load_one(row + at) : -INFINITY;
        sums.raise(x);
        const float d = sm_max_nan(x - sums.m, kLowest), e = sm_ex2(d * kLog2e);
        sums.s += e;
        sums.t = fmaf(e, d, sums.t);
        if (TOP) best.offer(mine, x, at, k);
    }
}

// A row's results from its sums and the best keys (of one warp, all lanes of it here).
template <typename T, bool TOP>
__device__ __forceinline__ void finish(const TokenLogprobs& a, long long r, const SoftmaxSums& sums, const Best& best, long long token,
                                       float given) {
    const int lane = threadIdx.x & 31;
    const SoftmaxRow row(sums);
    if (lane == 0) {
        a.lse[r] = row.lse;
        a.entropy[r] = row.entropy;
        a.logprob[r] = token < 0 ? 0.f : token < a.V ? row.logprob(given) : __uint_as_float(0x7FFFFFFFu);
    }
    if (TOP && lane < a.top) {
        a.top_index[r * a.top + lane] = (unsigned)~(unsigned)best.key;
        a.top_logprob[r * a.top + lane] = row.logprob(value_of((unsigned)(best.key >> 32)));
    }
}

template <typename T>
__device__ __forceinline__ float given_logit(const T* row, long long token, int V) {
    return token >= 0 && token < V ? load_one(row + token) : 0.f;
}

// One row per warp.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads) logprobs_warp_kernel(const TokenLogprobs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long r = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (r >= a.rows) return;
    const T* const row = static_cast<const T*>(a.logits) + r * a.ld;
    const long long token = a.tokens[r];
    const float given = given_logit(row, token, a.V);
    const RowCut cut(row, a.V);
    SoftmaxSums sums;
    Best best;
    sums.clear();
    best.clear();
    scan<T, TOP, 2>(row, a.V, cut, 0, cut.vecs, 32, true, a.top, sums, best);
    sums.merge_warp();
    finish<T, TOP>(a, r, sums, best, token, given);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

struct RowShared {
    SoftmaxSums sums[kWarps];
    unsigned long long best[kWarps][kTopMost];
    // of the cluster's CTAs, in its first one
    SoftmaxSums part[kMaxCluster];
    unsigned long long part_best[kMaxCluster][kTopMost];
};

// One row per CTA, or per cluster of CTAs.
template <typename T, bool TOP, bool CLUSTER>
__global__ void __launch_bounds__(kThreads) logprobs_cta_kernel(const TokenLogprobs a) {
    __shared__ RowShared sh;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (CLUSTER) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = CLUSTER ? cluster_size() : 1, rank = CLUSTER ? cluster_rank() : 0;
    const long long r = blockIdx.x / ctas;
    const T* const row = static_cast<const T*>(a.logits) + r * a.ld;
    const long long token = a.tokens[r];
    const float given = given_logit(row, token, a.V);
    const RowCut cut(row, a.V);
    const int from = (int)((long long)cut.vecs * rank / ctas), to = (int)((long long)cut.vecs * (rank + 1) / ctas);
    SoftmaxSums sums;
    Best best;
    sums.clear();
    best.clear();
    scan<T, TOP, 32 / Vec<T>::N>(row, a.V, cut, from + 32 * warp, to, kThreads, rank == 0 && warp == 0, a.top, sums, best);
    sums.merge_warp();
    if (lane == 0) sh.sums[warp] = sums;
    if (TOP) sh.best[warp][lane] = best.key;
    // every CTA of the cluster runs by now: its shared memory may be written
    if (CLUSTER) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    __syncthreads();
    if (warp == 0) {
        sums = sh.sums[lane & (kWarps - 1)];
        if (lane >= kWarps) sums.clear();
        sums.merge_warp();
        if (TOP)
#pragma unroll 1
            for (int w = 1; w < kWarps; ++w) best.offer(lane < a.top ? sh.best[w][lane] : 0ull, a.top);
        if (CLUSTER) {
            uint32_t to_sums, to_best;
            asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to_sums) : "r"(smem_u32(&sh.part[rank])));
            asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to_best) : "r"(smem_u32(&sh.part_best[rank][lane])));
            if (lane == 0) {
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to_sums), "f"(sums.m) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to_sums + 4), "f"(sums.s) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to_sums + 8), "f"(sums.t) : "memory");
            }
            if (TOP) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to_best), "l"(best.key) : "memory");
        } else {
            finish<T, TOP>(a, r, sums, best, token, given);
        }
    }
    if (CLUSTER) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank == 0 && warp == 0) {
            if (lane < ctas)
                sums = sh.part[lane];
            else
                sums.clear();
            sums.merge_warp();
            if (TOP)
#pragma unroll 1
                for (int c = 1; c < ctas; ++c) best.offer(lane < a.top ? sh.part_best[c][lane] : 0ull, a.top);
            finish<T, TOP>(a, r, sums, best, token, given);
        }
    }
}

// ------------------------------------------------------------ gradient
// What a row's gradient is made of: dx = p (a - h (x - lse)), plus g at the token.
struct RowGrad {
    float lse, a, h, g;
    bool none;  // nothing reaches the row, or it has no probabilities: zeros
};

__device__ __forceinline__ RowGrad row_grad(const TokenLogprobsBwd& a, long long r, long long token) {
    RowGrad o;
    o.lse = a.lse[r];
    o.g = a.dlogprob && token >= 0 ? a.dlogprob[r] : 0.f;
    const float l = a.dlse ? a.dlse[r] : 0.f;
    o.h = a.dentropy ? a.dentropy[r] : 0.f;
    o.none = (o.g == 0.f && l == 0.f && o.h == 0.f) || o.lse == -INFINITY;
    o.a = l - o.g;
    if (a.dentropy && o.h != 0.f) o.a = fmaf(-o.h, a.entropy[r], o.a);
    if (token >= a.V && o.g != 0.f) o.a = __uint_as_float(0x7FFFFFFFu);  // no such token
    return o;
}

template <bool ENT>
__device__ __forceinline__ float2 grad_pair(float2 x, const RowGrad& o) {
    float2 d = sm_add2(x, make_float2(-o.lse, -o.lse));
    const float2 y = sm_mul2(d, make_float2(kLog2e, kLog2e));
    const float2 p = make_float2(sm_ex2(y.x), sm_ex2(y.y));
    if (!ENT) return sm_mul2(p, make_float2(o.a, o.a));
    // (below -1e4 p is 0, and its factor finite)
    d.x = sm_max_nan(d.x, -1e4f);
    d.y = sm_max_nan(d.y, -1e4f);
    return sm_mul2(p, sm_fma2(make_float2(-o.h, -o.h), d, make_float2(o.a, o.a)));
}

__device__ __forceinline__ void store_one(float* p, float f) { *p = f; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }

// A warp takes `U` vectors per lane of one row; segment 0 also what lies outside the vectors.
template <typename T, bool ENT, int U>
__global__ void __launch_bounds__(kThreads) logprobs_bwd_kernel(const TokenLogprobsBwd a, unsigned segments, long long items) {
    constexpr int N = Vec<T>::N;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= items) return;
    const long long r = item / segments;
    const int seg = (int)(item - r * segments);
    const T* const row = static_cast<const T*>(a.logits) + r * a.ld;
    T* const out = static_cast<T*>(a.dlogits) + r * a.ldd;
    const RowCut cut(row, a.V);
    const int first = seg * 32 * U + lane;
    // (x and its gradient may lie differently against 16 bytes: then they leave one by one)
    const bool whole = (reinterpret_cast<uintptr_t>(out + cut.head) & 15u) == 0;
    const long long token = a.tokens[r];
    const RowGrad o = row_grad(a, r, token);
    Vec<T> v[U];
    if (!o.none) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = first + 32 * u;
            v[u].q = i < cut.vecs && TXL_BOUNDS(cut.head + (long long)(i + 1) * N <= a.V, 1103, i)
                         ? load_stream(row + cut.head + (size_t)i * N)
                         : Vec<T>::nothing();
        }
    }
    const int t0 = cut.head + (first - lane) * N;
    const bool here = token >= t0 && token < t0 + 32ll * U * N;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = first + 32 * u;
        float f[N];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const float2 p = o.none ? make_float2(0.f, 0.f) : grad_pair<ENT>(v[u].pair(j), o);
            f[2 * j] = p.x, f[2 * j + 1] = p.y;
        }
        if (here && !o.none) {
            const long long at = token - (cut.head + (long long)i * N);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (at == j) f[j] += o.g;
        }
        if (i >= cut.vecs || !TXL_BOUNDS(cut.head + (long long)(i + 1) * N <= a.V, 1104, i)) continue;
        T* const to = out + cut.head + (size_t)i * N;
        if (whole) {
            uint4 q;
            if constexpr (N == 8)
                q = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
            else
                q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            *reinterpret_cast<uint4*>(to) = q;
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) store_one(to + j, f[j]);
        }
    }
    if (seg == 0 && lane < cut.loose) {
        const int at = cut.index<T>(lane);
        if (TXL_BOUNDS(at < a.V, 1105, at)) {
            float f = 0.f;
            if (!o.none) {
                const float x = load_one(row + at);
                f = grad_pair<ENT>(make_float2(x, x), o).x;
                if (at == token) f += o.g;
            }
            store_one(out + at, f);
        }
    }
}

// ------------------------------------------------------------ host side
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), long long grid, unsigned cluster, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

constexpr int kWarpRowBytes = 4096;  // rows of up to so many bytes go to a warp each

template <typename T, bool TOP>
cudaError_t forward(const TokenLogprobs& a, cudaStream_t stream) {
    if ((long long)a.V * (long long)sizeof(T) <= kWarpRowBytes)
        return launch(logprobs_warp_kernel<T, TOP>, (a.rows + kWarps - 1) / kWarps, 1, stream, a);
    // as many CTAs per row as give every SM two, each with a vector per thread at least
    int ctas = 1;
    while (ctas < kMaxCluster && a.rows * ctas < 2ll * current_sm_count() &&
           (long long)a.V * (long long)sizeof(T) >= 2ll * ctas * kThreads * 16)
        ctas *= 2;
    if (ctas == 1) return launch(logprobs_cta_kernel<T, TOP, false>, a.rows, 1, stream, a);
    return launch(logprobs_cta_kernel<T, TOP, true>, a.rows * ctas, ctas, stream, a);
}

template <typename T, bool ENT>
cudaError_t backward(const TokenLogprobsBwd& a, cudaStream_t stream) {
    constexpr int U = 4;
    const long long per = 32ll * U * Vec<T>::N, segments = std::max(1ll, (a.V + per - 1) / per), items = segments * a.rows;
    return launch(logprobs_bwd_kernel<T, ENT, U>, (items + kWarps - 1) / kWarps, 1, stream, a, (unsigned)segments, items);
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenLogprobs& a, bool bf16, cudaStream_t stream) {
    if (bf16) return a.top ? forward<__nv_bfloat16, true>(a, stream) : forward<__nv_bfloat16, false>(a, stream);
    return a.top ? forward<float, true>(a, stream) : forward<float, false>(a, stream);
}

cudaError_t launch_token_logprobs_bwd(const TokenLogprobsBwd& a, bool bf16, cudaStream_t stream) {
    if (bf16) return a.dentropy ? backward<__nv_bfloat16, true>(a, stream) : backward<__nv_bfloat16, false>(a, stream);
    return a.dentropy ? backward<float, true>(a, stream) : backward<float, false>(a, stream);
}

TXL_BOUNDS_READER(bounds_word_token_logprobs)

}  // namespace txl
