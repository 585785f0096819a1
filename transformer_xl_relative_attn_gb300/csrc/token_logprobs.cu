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
// additions depends on sizes and alignment alone.
//
// Alternatives are ordered as 64-bit keys: the value's order, then the complement of the
// index, so that no two are alike.  In the pass over the row a thread only notes which two
// of its 16-byte vectors have the largest values, and the largest of the others (10
// instructions a vector; keeping the best in order as they come took the kernel twice its
// time).  Behind it the threads' best elements are put in order, by sorting within warps
// and by rank among the warps' lists, and the k-th of them is a bar: a second element of a
// thread can only count where one reaches it.  Then its warp looks at its two vectors each
// again, and at all vectors of a thread whose third one reaches the bar too.
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
    // the same with nothing below kLow
    __device__ __forceinline__ float2 pair_from_low(int i) const {
        const unsigned w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w, low = 0xFE96FE96u;  // kLow, cut to bf16
        const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&low));
        return halves(*reinterpret_cast<const unsigned*>(&m));
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
    __device__ __forceinline__ float2 pair_from_low(int i) const {
        const float2 p = pair(i);
        return make_float2(sm_max_nan(p.x, kLow), sm_max_nan(p.y, kLow));
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
// 16 bytes that this kernel does not look at again, past L1 (through it the gradient of 11264 x
// 32768 bf16 took 233 us, past it 204).
__device__ __forceinline__ void store_stream(void* p, const uint4& v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
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

__device__ __forceinline__ unsigned long long key_of(float x, unsigned index) {
    return (unsigned long long)order_of(x) << 32 | (unsigned)~index;
}

// The larger of each two lanes `apart` goes to the one whose `down` is false.
__device__ __forceinline__ unsigned long long exchange(unsigned long long a, int apart, bool down) {
    const unsigned long long b = __shfl_xor_sync(kAll, a, apart);
    return (a > b) == down ? b : a;
}
// The best 32 of a falling list (a key per lane) and of one candidate per lane, falling.
// (A call: inlined where it is needed, code of several times the size missed its cache.)
__device__ __noinline__ unsigned long long merge_all(unsigned long long key, unsigned long long c) {
    const int lane = threadIdx.x & 31;
    // sorted upwards, so that against the list's order each lane keeps the larger of two:
    // the best 32 of both, rising and then falling, to be sorted downwards
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int apart = size / 2; apart > 0; apart /= 2)
            c = exchange(c, apart, ((lane & apart) == 0) == ((lane & size) == 0));
    key = c > key ? c : key;
#pragma unroll
    for (int apart = 16; apart > 0; apart /= 2) key = exchange(key, apart, (lane & apart) != 0);
    return key;
}

// The keys of a warp's lanes in falling order, the first k of them at least (0: none).
__device__ __forceinline__ unsigned long long in_order(unsigned long long c, int k) {
    if (k > 8) return merge_all(0ull, c);
    // one by one: a round takes fewer instructions than two steps of the sort
    const int lane = threadIdx.x & 31;
    unsigned long long key = 0;
#pragma unroll 1
    for (int i = 0; i < k; ++i) {
        const unsigned hi = (unsigned)(c >> 32), top = __reduce_max_sync(kAll, hi);
        const unsigned low = __reduce_max_sync(kAll, hi == top ? (unsigned)c : 0u);
        const unsigned long long n = (unsigned long long)top << 32 | low;
        if (lane == i) key = n;
        if (c == n) c = 0;
    }
    return key;
}

// The best keys that a warp has seen, lane i with the i-th.
struct Best {
    unsigned long long key, last;  // `last`: the k-th, or what a key has to be above to count
    float bar;                     // its value, -inf where there is none
    __device__ __forceinline__ void settle(int k, unsigned long long floor) {
        const unsigned long long n = __shfl_sync(kAll, key, k - 1);
        last = n > floor ? n : floor;
        bar = last ? value_of((unsigned)(last >> 32)) : -INFINITY;
    }
    // One candidate per lane (0: none), no key twice; all lanes of the warp together.
    __device__ __forceinline__ void offer(unsigned long long c, int k, unsigned long long floor) {
        const int lane = threadIdx.x & 31;
        unsigned more = __ballot_sync(kAll, c > last);
        if (!more) return;
        if (__popc(more) > kSingly) {
            key = merge_all(key, c);
            settle(k, floor);
            return;
        }
#pragma unroll 1
        do {
            const int src = __ffs(more) - 1;
            const unsigned long long n = __shfl_sync(kAll, c, src);
            const unsigned long long up = __shfl_up_sync(kAll, key, 1);
            const int at = __popc(__ballot_sync(kAll, key > n));
            key = lane < at ? key : lane == at ? n : up;
            settle(k, floor);
            if (lane == src) c = 0;
            more = __ballot_sync(kAll, c > last);
        } while (more);
    }
    // Whether a vector of this maximum may hold one of the best.
    __device__ __forceinline__ bool worth(float max) const { return !(max < bar); }

    // Candidates are taken one by one up to this many at a time, sorted together beyond: an
    // insertion is a chain of some 110 cycles, a sort and merge one of 700.
    static constexpr int kSingly = 4;
};

// How many of a falling list of k keys are above `key`.
__device__ __forceinline__ int above(const unsigned long long* list, int k, unsigned long long key) {
    int n = 0;
#pragma unroll
    for (int step = kTopMost; step > 0; step /= 2)
        if (n + step <= k && list[n + step - 1] > key) n += step;
    return n;
}

// ------------------------------------------------------------ one warp's share of a row
// What a thread notes for the alternatives: its vectors' three largest values, and the
// vectors of the first two (of equal ones the first that came).  A NaN is left out here: the
// thread's sums show it, and all its vectors are then looked at again.
struct Noted {
    float most, next, third;
    int at, at2;
    __device__ __forceinline__ void clear(int first) { most = next = third = -INFINITY, at = first, at2 = -1; }
    __device__ __forceinline__ void see(float max, int vec) {
        third = fmaxf(third, fminf(max, next));
        at2 = max > most ? at : max > next ? vec : at2;
        next = fmaxf(next, fminf(max, most));
        at = max > most ? vec : at;
        most = fmaxf(max, most);
    }
};

constexpr int kBatches = 64;  // even, as they are taken two by two

// A warp's vectors are first + lane + i step, i = 0, 1, .., below `end`; with `loose` it has
// the elements outside the vectors too.
struct Share {
    int first, end, step;
    bool loose;
    int vecs;  // of the row
};

template <typename T, bool TOP, int U>
__device__ __forceinline__ void scan(const T* row, int V, const RowCut& cut, const Share& sh, SoftmaxSums& sums, Noted& noted) {
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x & 31;
    const T* const vec0 = row + cut.head;
    SoftmaxPairs acc;
    acc.clear();
    if (TOP) noted.clear(sh.first + lane);
    auto load = [&](Vec<T>(&v)[U], int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * sh.step + lane;
            v[u].q = i < sh.end && TXL_BOUNDS(i >= 0 && cut.head + (long long)(i + 1) * N <= V, 1101, i)
                         ? load_stream(vec0 + (size_t)i * N)
                         : Vec<T>::nothing();
        }
    };
    auto take = [&](const Vec<T>(&v)[U], int base) {
        float all = v[0].max();
        if (TOP) noted.see(all, base + lane);
#pragma unroll
        for (int u = 1; u < U; ++u) {
            const float most = v[u].max();
            if (TOP) noted.see(most, base + u * sh.step + lane);
            all = sm_max_nan(all, most);
        }
        acc.raise(all);
        if (sm_ordinary(acc.m)) {
            const float r = sm_reference(acc.m);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < N / 2; ++i) acc.add(v[u].pair_from_low(i), r);
        } else {
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                Vec<T> x = v[0];
#pragma unroll
                for (int i = 1; i < U; ++i)
                    if (u == i) x = v[i];
#pragma unroll 1
                for (int j = 0; j < N; ++j) acc.add_far(x.at(j));
            }
        }
    };
    const int stride = U * sh.step;
    Vec<T> v[U];
    // A chain of additions has kBatches batches at most; the chains are added one by one.
    int base = sh.first;
    do {
        const int end = sh.end - base > kBatches * stride ? base + kBatches * stride : sh.end;
        if constexpr (sizeof(T) == 2) {
#pragma unroll 1
            for (; base < end; base += stride) {
                load(v, base);
                take(v, base);
            }
        } else {
            // A batch is on its way while the one before is worked on (1001 x 50021: 37 us, one at
            // a time 55; in bf16, whose batches have twice the elements and whose CTAs would be
            // fewer, 11264 x 32768 took 134 us so and 112 one at a time).
            Vec<T> w[U];
            if (base < end) load(v, base);
#pragma unroll 1
            for (; base < end; base += 2 * stride) {
                if (base + stride < end) load(w, base + stride);
                take(v, base);
                if (base + 2 * stride < end) load(v, base + 2 * stride);
                if (base + stride < end) take(w, base + stride);
            }
        }
        if (end <= sh.first + kBatches * stride) {
            sums = acc.fold();
        } else {
            sums.merge(acc.fold());
        }
        acc.clear();
    } while (base < sh.end);
    if (sh.loose && lane < cut.loose) {
        const int at = cut.index<T>(lane);
        if (TXL_BOUNDS(at < V, 1102, at)) sums.add(load_one(row + at));
    }
}

// A thread's best vector once more.
template <typename T>
__device__ __forceinline__ Vec<T> best_vector(const T* row, int V, const RowCut& cut, const Share& sh, const Noted& noted) {
    Vec<T> v;
    v.q = sh.first + (int)(threadIdx.x & 31) < sh.end &&
                  TXL_BOUNDS(noted.at >= 0 && cut.head + (long long)(noted.at + 1) * Vec<T>::N <= V, 1106, noted.at)
              ? load_stream(row + cut.head + (size_t)noted.at * Vec<T>::N)
              : Vec<T>::nothing();
    return v;
}

// The key of a thread's best element in its vectors (0: it has none), of whose best vector v is
// the content; `next` becomes the largest order that another of them may have, and `third` that
// of one outside the two noted vectors.  (With a NaN, `nan`, both are the highest, and the key
// is one of the thread's elements all the same.)
template <typename T>
__device__ __forceinline__ unsigned long long best_of(const Vec<T>& v, const RowCut& cut, const Share& sh, const Noted& noted, bool nan,
                                                      unsigned& next, unsigned& third) {
    constexpr int N = Vec<T>::N;
    if (sh.first + (int)(threadIdx.x & 31) >= sh.end) {
        next = third = 0;
        return 0;
    }
    float most = -INFINITY, second = noted.next;
    int at = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float2 p = v.pair(j / 2);
        const float x = j & 1 ? p.y : p.x;
        second = fmaxf(second, fminf(x, most));
        at = x > most ? j : at;
        most = fmaxf(x, most);
    }
    next = nan ? 0xFFFFFFFFu : order_of(second);
    third = nan ? 0xFFFFFFFFu : order_of(noted.third);
    return key_of(v.at(at), cut.head + noted.at * N + at);
}

// The best keys of a warp as they stand behind best_of: its lanes' best, `mine`, and the
// elements outside the vectors.
template <typename T>
__device__ __forceinline__ unsigned long long first_list(const T* row, int V, const RowCut& cut, const Share& sh, unsigned long long mine,
                                                         int k) {
    const int lane = threadIdx.x & 31;
    unsigned long long list = in_order(mine, k);
    if (sh.loose && cut.loose) {
        const int at = lane < cut.loose ? cut.index<T>(lane) : 0;
        list = merge_all(list, lane < cut.loose && TXL_BOUNDS(at < V, 1107, at) ? key_of(load_one(row + at), at) : 0ull);
    }
    return list;
}

// A warp's noted vectors once more, two per lane, for what else is among its best `k` and not
// below the order `bar`; and all vectors of the lanes that `whole` names, each of which the
// warp shares out.  `list`: its best so far (a key per lane, falling), the threads' best,
// `mine`, among them.
template <typename T>
__device__ __noinline__ unsigned long long look_again(const T* vec0, int head, const Share sh, int at, int at2, unsigned whole,
                                                      unsigned long long list, unsigned long long mine, unsigned bar, int k) {
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x & 31;
    const unsigned long long floor = (unsigned long long)bar << 32;
    Best best;
    best.key = list;
    best.settle(k, floor);
    auto load = [&](int i) {
        Vec<T> v;
        v.q = i >= 0 && i < sh.end && TXL_BOUNDS(i < sh.vecs, 1108, i) ? load_stream(vec0 + (size_t)i * N) : Vec<T>::nothing();
        return v;
    };
    if (sh.first + lane >= sh.end) at = -1;
    if (at2 == at || at2 >= sh.end) at2 = -1;
    // a vector per lane at a time: first the noted ones, then the shared-out ones
    int i = at, from = -1, skip = -1, skip2 = -1, round = 0;
    Vec<T> x = load(at);
    const Vec<T> second = load(at2);
#pragma unroll 1
    for (;;) {
        unsigned bits = 0;  // elements that may count
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float2 p = x.pair(j / 2);
            bits |= best.worth(j & 1 ? p.y : p.x) ? 1u << j : 0u;
        }
        if (i < 0) bits = 0;
        while (__any_sync(kAll, bits != 0)) {
            const int j = bits ? __ffs(bits) - 1 : 0;
            const unsigned long long c = bits ? key_of(x.at(j), head + i * N + j) : 0ull;
            best.offer(c == mine ? 0ull : c, k, floor);
            bits &= bits - 1;
        }
        if (++round == 1) {
            x = second, i = at2;
            continue;
        }
        if (from < 0 || from + 32 * sh.step >= sh.end) {  // the next lane's
            if (!whole) return best.key;
            const int src = __ffs(whole) - 1;
            whole &= whole - 1;
            from = sh.first + src;
            skip = __shfl_sync(kAll, at, src), skip2 = __shfl_sync(kAll, at2, src);
        } else {
            from += 32 * sh.step;
        }
        i = from + lane * sh.step;
        if (i >= sh.end || i == skip || i == skip2) i = -1;
        x = load(i);
    }
}

__device__ __forceinline__ void write_statistics(const TokenLogprobs& a, long long r, const SoftmaxRow& row, long long token, float given) {
    a.lse[r] = row.lse;
    a.entropy[r] = row.entropy;
    a.logprob[r] = token < 0 ? 0.f : token < a.V ? row.logprob(given) : __uint_as_float(0x7FFFFFFFu);
}
__device__ __forceinline__ void write_best(const TokenLogprobs& a, long long r, const SoftmaxRow& row, int i, unsigned long long key) {
    a.top_index[r * a.top + i] = (unsigned)~(unsigned)key;
    a.top_logprob[r * a.top + i] = row.logprob(value_of((unsigned)(key >> 32)));
}

template <typename T>
__device__ __forceinline__ float given_logit(const T* row, long long token, int V) {
    return token >= 0 && token < V ? load_one(row + token) : 0.f;
}

// One row per warp, U vectors per lane at a time.
template <typename T, bool TOP, int U>
__global__ void __launch_bounds__(kThreads) logprobs_warp_kernel(const TokenLogprobs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (r >= a.rows) return;
    const T* const row = static_cast<const T*>(a.logits) + r * a.ld;
    const long long token = a.tokens[r];
    const float given = given_logit(row, token, a.V);
    const RowCut cut(row, a.V);
    const Share sh = {0, cut.vecs, 32, true, cut.vecs};
    SoftmaxSums sums;
    Noted noted;
    scan<T, TOP, U>(row, a.V, cut, sh, sums, noted);
    Vec<T> v;
    if (TOP) v = best_vector(row, a.V, cut, sh, noted);
    const bool nan = sums.s != sums.s;
    sums.merge_warp();
    const SoftmaxRow out(sums);
    if (lane == 0) write_statistics(a, r, out, token, given);
    if (TOP) {
        unsigned next, third;
        const unsigned long long mine = best_of(v, cut, sh, noted, nan, next, third);
        unsigned long long key = first_list(row, a.V, cut, sh, mine, a.top);
        const unsigned bar = (unsigned)(__shfl_sync(kAll, key, a.top - 1) >> 32);
        if (__any_sync(kAll, next >= bar))
            key = look_again(row + cut.head, cut.head, sh, noted.at, noted.at2, __ballot_sync(kAll, third >= bar), key, mine, bar, a.top);
        if (lane < a.top) write_best(a, r, out, lane, key);
    }
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

// Lists of keys, one behind the other without a gap.
template <int THREADS>
struct RowShared {
    unsigned bar;  // order of the k-th best of the threads' best
    SoftmaxSums sums[THREADS / 32];
    unsigned long long best[THREADS];
    // of the cluster's CTAs, in its first one
    SoftmaxSums part[kMaxCluster];
    unsigned long long part_best[kMaxCluster * kTopMost];
};
static_assert(kMaxCluster * kTopMost <= kThreads, "a CTA's threads hold a key of each of the cluster's lists");

// Of n lists of k keys, this thread's (below n k) and how many of all are above it.
__device__ __forceinline__ int rank_of(const unsigned long long* lists, int n, int k, unsigned long long& key) {
    key = lists[threadIdx.x];
    int above_it = 0;
#pragma unroll 4
    for (int l = 0; l < n; ++l) above_it += above(lists + l * k, k, key);
    return above_it;
}

// One row per CTA, or per cluster of CTAs.
template <typename T, bool TOP, bool CLUSTER, int THREADS>
__global__ void __launch_bounds__(THREADS, (sizeof(T) == 2 ? (TOP ? 5 : 6) : (TOP ? 4 : 3)) * (kThreads / THREADS))
logprobs_cta_kernel(const TokenLogprobs a) {
    constexpr int WARPS = THREADS / 32;
    static_assert(!CLUSTER || THREADS == kThreads, "clusters are of the larger CTAs");
    __shared__ RowShared<THREADS> sh;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (CLUSTER) {
        if (TOP) sh.part_best[threadIdx.x] = 0;  // (lists of less than k keys: 0 in place of the rest)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = a.top;
    const int ctas = CLUSTER ? cluster_size() : 1, rank = CLUSTER ? cluster_rank() : 0;
    const long long r = blockIdx.x / ctas;
    const T* const row = static_cast<const T*>(a.logits) + r * a.ld;
    const long long token = a.tokens[r];
    const float given = given_logit(row, token, a.V);
    const RowCut cut(row, a.V);
    const int from = (int)((long long)cut.vecs * rank / ctas), to = (int)((long long)cut.vecs * (rank + 1) / ctas);
    const Share share = {from + 32 * warp, to, THREADS, rank == 0 && warp == 0, cut.vecs};
    SoftmaxSums sums;
    Noted noted;
    scan<T, TOP, 4>(row, a.V, cut, share, sums, noted);
    Vec<T> v;
    if (TOP) v = best_vector(row, a.V, cut, share, noted);
    const bool nan = sums.s != sums.s;
    sums.merge_warp();
    if (lane == 0) sh.sums[warp] = sums;
    unsigned next = 0, third = 0;
    unsigned long long mine = 0, list = 0;
    if (TOP) {
        mine = best_of(v, cut, share, noted, nan, next, third);
        list = first_list(row, a.V, cut, share, mine, k);
        if (lane < k) sh.best[warp * k + lane] = list;
        if (threadIdx.x == 0) sh.bar = 0;
    }
    // every CTA of the cluster runs by now: its shared memory may be written
    if (CLUSTER) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();
    sums = sh.sums[lane & (WARPS - 1)];  // every warp for itself
    if (lane >= WARPS) sums.clear();
    sums.merge_warp();
    const bool listed = TOP && (int)threadIdx.x < WARPS * k;
    unsigned long long key = 0;
    int place = THREADS;
    if (TOP) {
        if (listed) {
            place = rank_of(sh.best, WARPS, k, key);
            if (place == k - 1) sh.bar = (unsigned)(key >> 32);
        }
        __syncthreads();
        const unsigned bar = sh.bar;
        const bool again = __any_sync(kAll, next >= bar);
        if (__syncthreads_or(again)) {
            if (again) {
                list = look_again(row + cut.head, cut.head, share, noted.at, noted.at2, __ballot_sync(kAll, third >= bar), list, mine, bar, k);
                if (lane < k) sh.best[warp * k + lane] = list;
            }
            __syncthreads();
            if (listed) place = rank_of(sh.best, WARPS, k, key);
        }
    }
    if (!CLUSTER) {
        const SoftmaxRow out(sums);
        if (threadIdx.x == 0) write_statistics(a, r, out, token, given);
        if (place < k && key) write_best(a, r, out, place, key);
        return;
    }
    if (threadIdx.x == 0) {
        uint32_t to_sums;
        asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to_sums) : "r"(smem_u32(&sh.part[rank])));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to_sums), "f"(sums.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to_sums + 4), "f"(sums.s) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to_sums + 8), "f"(sums.t) : "memory");
    }
    if (place < k && key) {
        uint32_t to_best;
        asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to_best) : "r"(smem_u32(&sh.part_best[rank * k + place])));
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to_best), "l"(key) : "memory");
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank) return;
    if (lane < ctas)
        sums = sh.part[lane];
    else
        sums.clear();
    sums.merge_warp();
    const SoftmaxRow out(sums);
    if (threadIdx.x == 0) write_statistics(a, r, out, token, given);
    if (TOP && (int)threadIdx.x < ctas * k) {
        const int i = rank_of(sh.part_best, ctas, k, key);
        if (i < k && key) write_best(a, r, out, i, key);
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
            store_stream(to, q);
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
template <int THREADS = kThreads, typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), long long grid, unsigned cluster, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
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

// Rows of up to so many bytes go to a warp each: where rows are many (us, top 8, a warp and a CTA
// of 128 threads: 10000 x 1024 fp32 17 and 34, 10000 x 4096 bf16 24 and 38), and where they are
// few and a warp's steps one after the other count (300 x 2048 bf16, top 32: 17 and 6).
constexpr int kWarpRowBytes = 8192, kWarpFewRowBytes = 1024, kManyRows = 8;  // rows per SM

template <typename T, bool TOP>
cudaError_t forward(const TokenLogprobs& a, cudaStream_t stream) {
    const long long bytes = (long long)a.V * (long long)sizeof(T);
    if (bytes <= (a.rows >= (long long)kManyRows * current_sm_count() ? kWarpRowBytes : kWarpFewRowBytes))
        return launch(bytes <= 512 ? logprobs_warp_kernel<T, TOP, 1> : bytes <= 1024 ? logprobs_warp_kernel<T, TOP, 2> : logprobs_warp_kernel<T, TOP, 4>,
                      (a.rows + kWarps - 1) / kWarps, 1, stream, a);
    // as many CTAs per row as give every SM two, each with a vector per thread at least
    int ctas = 1;
    while (ctas < kMaxCluster && a.rows * ctas < 2ll * current_sm_count() &&
           bytes >= 2ll * ctas * kThreads * 16)
        ctas *= 2;
    // CTAs of half the threads, and so twice as many rows at once, with alternatives, whose
    // search behind the pass leaves other rows' loads to fill the time (us, top 8, 256 and 128
    // threads: 11264 x 32768 bf16 186 and 133, 1001 x 50021 fp32 45 and 38).  Without, where
    // rows are many: short ones, where a CTA's begin and end weigh (1520 x 4200 bf16 6.3 and 4.9,
    // 1824 x 24576 bf16 16 and 14, 1520 x 8200 fp32 9.5 and 7.3, 8000 x 12288 fp32 68 and 59; with
    // 1300 x 16384 bf16 8.8 and 10, 1520 about even), and by a little others (8000 x 32768 bf16
    // 79 and 77, fp32 146 and 143; 2432 x 32768 bf16 27.7 and 28.8).  The longest take as long or
    // less with all threads (8000 x 65536 bf16 149 and 150, 4100 124 and 130 with 100000).
    const long long per_sm = a.rows / current_sm_count();
    const bool half = TOP || (bytes <= 48 * 1024 ? per_sm >= 10 : bytes <= 128 * 1024 && per_sm >= 27);
    if (ctas == 1 && half) return launch<kThreads / 2>(logprobs_cta_kernel<T, TOP, false, kThreads / 2>, a.rows, 1, stream, a);
    if (ctas == 1) return launch(logprobs_cta_kernel<T, TOP, false, kThreads>, a.rows, 1, stream, a);
    return launch(logprobs_cta_kernel<T, TOP, true, kThreads>, a.rows * ctas, ctas, stream, a);
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
