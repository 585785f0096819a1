// Log probabilities of given tokens straight from hidden states, on the sm_103a tensor
// cores: with logits z = x W^T + bias (bf16 in, fp32 accumulation, never written to memory)
//
//   lse = ln sum e^z,   logprob = z_token - lse,   entropy = -sum p ln p,   p = e^(z - lse)
//
// A persistent GEMM whose epilogue keeps each row's running maximum and sums
// (softmax_sums.cuh) in registers: a thread of the epilogue owns a row, which is how
// tensor memory hands an accumulator out, so a row's statistics need no exchange.  An item
// is a tile of rows and a run of column tiles; items are dealt run by run, so that all
// SMs read the same part of W at about the same time and it comes from memory once.
// An item's (m, s, t) go to the workspace, and a second launch adds a row's in the order of
// the runs.  What bounds it: the MMAs with many rows (an accumulator of 128 x 256 takes the
// epilogue less time than 512 elements of K the tensor cores), the read of W with few.
//
// Two CTAs of a cluster share a tile of 256 rows (cta_group::2), or one CTA takes 128.  A
// tile has 256 columns, or fewer (a multiple of 64) where that fills the units more evenly.
// Both operands are K-major, 64 elements of K per stage: two TMA instructions a CTA.  Rows,
// columns and K need not fill their tiles: TMA fills with zeros behind the ends, and columns
// behind V count as -inf.
//
// Roles (384 threads, one CTA per SM): warp 0 lane 0 issues the TMA loads, warp 1 the
// MMAs, warps 4-11 the epilogue; two accumulators let an epilogue overlap the next tile's
// MMAs.  Every wait is bounded (1 s) and reports through the device status word.
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "linear_logprobs.h"
#include "pair_mma.cuh"
#include "softmax_sums.cuh"
#include "txl_device.cuh"

namespace txl {

namespace lp {
constexpr int BM = 128;  // rows of a CTA's accumulator
constexpr int BK = 64;   // K per stage
constexpr int MAX_BN = 256;
constexpr int NTHREADS = 384;
constexpr uint32_t SZ_A = BM * BK * 2;  // 16 KB; the second operand's slot: 128 bytes per column of the CTA's
constexpr int MAX_STAGES = 8;
constexpr uint32_t TMEM_COLS = 2 * MAX_BN;

// A tile's width is known at compile time: with the width, the stages and the descriptors'
// steps as variables the MMAs' issuing loop took 7 % longer (11264 rows, 512 -> 32768: 241
// us as constants, 260).
template <bool PAIR, int BN>
struct Cfg {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TM = BM * CTAS;                      // rows of a tile
    static constexpr uint32_t SZ_B = BN / CTAS * BK * 2;      // of a pair's columns each CTA holds half
    static constexpr int FIT = 220 * 1024 / (SZ_A + SZ_B);
    static constexpr int STAGES = FIT < MAX_STAGES ? FIT : MAX_STAGES;
    static constexpr uint32_t OFF_B = STAGES * SZ_A;
    static constexpr uint32_t OFF_BAR = OFF_B + STAGES * SZ_B;
    static constexpr uint32_t OFF_BIAS = OFF_BAR + 512;       // of each epilogue warp's columns, fp32
    static constexpr uint32_t SMEM_BYTES = OFF_BIAS + 8 * (BN / 2) * 4 + 1024;
    static constexpr uint32_t IDESC = idesc_bf16_f32(TM, BN, 0, 0);
    static_assert(SMEM_BYTES <= 232448, "shared memory budget of one sm_103a CTA");
};
}  // namespace lp

struct LpMaps {
    CUtensorMap x, w;  // (element, row), boxes of 64 x 128 and of 64 x a CTA's columns
};

struct LpShared {
    uint64_t full[lp::MAX_STAGES];  // a pair's: those of its first CTA
    uint64_t empty[lp::MAX_STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];  // a pair's: those of its first CTA
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// An item: a tile of rows and column tiles [v0, v1), the runs outermost.
struct LpItem {
    int r, run, v0, v1;
};

__device__ __forceinline__ LpItem lp_item(const LpParams& p, int i) {
    LpItem it;
    it.run = i / p.n_rt;
    it.r = i - it.run * p.n_rt;
    it.v0 = it.run * p.per;
    it.v1 = min(it.v0 + p.per, p.n_vt);
    return it;
}

// Whether a part or a token's logit lies in the workspace.
template <typename T>
__device__ __forceinline__ bool lp_in_workspace(const LpParams& p, const T* at) {
    return reinterpret_cast<const char*>(at) >= reinterpret_cast<const char*>(p.part) &&
           reinterpret_cast<const char*>(at + 1) <= p.ws_end;
}

// One column of an accumulator, a row per lane.
__device__ __forceinline__ float lp_tmem_column(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(taddr) : "memory");
    return __uint_as_float(r);
}
// The same, of zeros.
__device__ __forceinline__ void lp_tmem_clear_column(uint32_t taddr) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(0u) : "memory");
}

// (BIAS: unused, the bias' code cost a call without one 4 %.)
template <bool PAIR, int BN, bool BIAS>
__global__ void __launch_bounds__(lp::NTHREADS, 1) linear_logprobs_kernel(const __grid_constant__ LpMaps maps, const LpParams p) {
    using namespace lp;
    using C = Cfg<PAIR, BN>;
    constexpr int CTAS = C::CTAS, TM = C::TM, STAGES = C::STAGES;
    constexpr uint32_t SZ_B = C::SZ_B, OFF_B = C::OFF_B;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    LpShared* sh = reinterpret_cast<LpShared*>(smem + C::OFF_BAR);
    const uint32_t s_base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? lb_cta_rank() : 0;

    if (warp == 1) lb_tmem_alloc<PAIR>(&sh->tmem_base, TMEM_COLS);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], 8 * CTAS);  // one arrival per epilogue warp
        }
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
    }
    tc_fence_before();
    if (PAIR) __syncthreads();
    lb_sync<PAIR>();
    tc_fence_after();
    // (not before the CTA has its tensor memory: a kernel that got ahead would hold it and wait for this one)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = sh->tmem_base;
    volatile int* abort = &sh->abort;
    const int unit = blockIdx.x / CTAS, units = gridDim.x / CTAS, items = p.n_rt * p.chunks;

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        // A pair's full barriers are its first CTA's, which expects both CTAs' bytes; the
        // second's loads may land before it does (the barrier waits for the arrival).
        if (lane == 0) {
            bool ok = true;
            // One thread's instructions per stage bound the loads, so what does not change is
            // kept out of the loop.
            uint32_t s = 0, phase = 1;  // slot, parity of its empty barrier (a fresh one passes for 1)
            long long loads = 0;
            const uint32_t full0 = PAIR ? lb_mapa(&sh->full[0], 0) : smem_u32(&sh->full[0]);
            const uint32_t bytes = (SZ_A + SZ_B) * CTAS;
            uint32_t to_a = s_base, to_b = s_base + OFF_B, bar = full0;
            const int K = p.ksteps * BK;
            for (int i = unit; ok && i < items; i += units) {
                const LpItem it = lp_item(p, i);
                const int r0 = it.r * TM + BM * rank;
                for (int v = it.v0; ok && v < it.v1; ++v) {
                    const int n0 = v * BN + BN / CTAS * rank;
                    for (int k = 0; k < K; k += BK) {
                        if (!mbar_wait(&sh->empty[s], phase, kDevTimeoutProducer, abort, p.status)) {
                            ok = false;
                            break;
                        }
                        if (rank == 0) mbar_expect_tx(&sh->full[s], bytes);
                        lb_load_2d<PAIR>(to_a, &maps.x, bar, k, r0);
                        lb_load_2d<PAIR>(to_b, &maps.w, bar, k, n0);
                        to_a += SZ_A, to_b += SZ_B, bar += 8;
                        if (++s == STAGES) s = 0, phase ^= 1, to_a = s_base, to_b = s_base + OFF_B, bar = full0;
                        ++loads;
                    }
                }
            }
            // the last load into each slot has landed before the CTAs exit
            for (int i = 0; i < STAGES && rank == 0; ++i) {
                const long long c = loads - 1 - i;
                if (c >= 0) lb_wait_landed(&sh->full[c % STAGES], (c / STAGES) & 1, p.status);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        if (rank == 0) {
            const uint32_t leader = elect_one();
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, kDevTimeoutMma, abort, p.status));
                return ok;
            };
            const uint64_t dA0 = smem_desc_sw128(s_base, 16, 1024);
            const uint64_t dB0 = smem_desc_sw128(s_base + OFF_B, 16, 1024);
            uint32_t s = 0, phase = 0;  // slot, parity of its full barrier
            int j = 0;                  // accumulators filled
            for (int i = unit; ok && i < items; i += units) {
                const LpItem it = lp_item(p, i);
                for (int v = it.v0; ok && v < it.v1; ++v) {
                    const int acc = j & 1;
                    if (j >= 2 && !wait(&sh->acc_empty[acc], ((j >> 1) - 1) & 1)) break;
                    tc_fence_after();
                    const uint32_t d_acc = tmem + acc * MAX_BN;
                    uint32_t more_than_first = 0;
                    auto step = [&](int n) {
                        if (!wait(&sh->full[s], phase)) return false;
                        tc_fence_after();
                        const uint64_t ad = dA0 + s * (SZ_A >> 4), bd = dB0 + s * (SZ_B >> 4);
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            if (kk < n) {
                                lb_mma<PAIR>(d_acc, ad + 2 * kk, bd + 2 * kk, C::IDESC, more_than_first, leader);
                                more_than_first = 1;
                            }
                        if (leader) lb_commit<PAIR>(&sh->empty[s]);
                        if (++s == STAGES) s = 0, phase ^= 1;
                        return true;
                    };
                    for (int k = 1; k < p.ksteps; ++k)
                        if (!step(BK / 16)) break;
                    if (ok) step(p.klast);
                    if (!ok) break;
                    if (leader) lb_commit<PAIR>(&sh->acc_full[acc]);
                    ++j;
                }
            }
            if (leader) lb_commit<PAIR>(&sh->drain);
            lb_wait_landed(&sh->drain, 0, p.status);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------- epilogue
        const int wq = warp & 3;
        const int chalf = (warp - 4) >> 2;
        constexpr int chunks = BN / 64, half = 32 * chunks;  // 32-column chunks per warp; its columns
        const uint32_t t_row = tmem + ((uint32_t)(wq * 32) << 16) + half * chalf;
        const uint32_t acc_empty0 = PAIR ? lb_mapa(&sh->acc_empty[0], 0) : 0;
        float4* const my_bias = reinterpret_cast<float4*>(smem + C::OFF_BIAS) + (warp - 4) * (half / 4);
        bool ok = true;
        int j = 0;
        for (int i = unit; ok && i < items; i += units) {
            const LpItem it = lp_item(p, i);
            const int row = it.r * TM + BM * rank + 32 * wq + lane;
            const long long token = row < p.rows ? p.tokens[row] : -1;
            // a tile's sums, and those of the tiles before it: one chain of additions through all of
            // a run would round each way as often as it has columns.  Both against one reference, which
            // follows the maximum of a chunk with which a tile's terms are `much` (262144 logits in one
            // run, alike but for the first 32, which lie 15.5 lower: their entropy was off by 3.3e-4 with
            // 2^30 as much, and is by 1.4e-6; by 3.6e-5 at most where they lie 1.25 lower, which makes the
            // others' terms just less than much.  A look at the sums behind each tile too would make that
            // 1e-5, for a 140th of the time)
            constexpr float much = 4.f * half;
            SoftmaxPairs sums, before;
            sums.clear();
            before.clear();
            auto add = [&](const float (&z)[32]) {
                const SoftmaxPairs was = sums;
                if (sm_ordinary(sums.m)) {
                    const float r = sm_reference(sums.m);
#pragma unroll
                    for (int x = 0; x < 32; x += 2) sums.add(make_float2(z[x], z[x + 1]), r);
                    if (sums.fine(much)) return;
                    sums = was;
                }
                float most = fmaxf(z[0], z[1]);
#pragma unroll
                for (int x = 2; x < 32; x += 2) most = sm_max3(most, z[x], z[x + 1]);
                if (most > sums.m) sums.follow(most), before.follow(most);
                if (sm_ordinary(sums.m)) {
                    const float r = sm_reference(sums.m);
#pragma unroll
                    for (int x = 0; x < 32; x += 2) sums.add_low(make_float2(z[x], z[x + 1]), r);
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) sums.add_far(z[x]);
                }
                const float terms = sums.s.x + sums.s.y;
                if (terms > 2.f * half) {  // made much by the chunks before: on to where all are on average
                    const float to = sums.m + __logf(terms / half);
                    if (sm_ordinary(to)) sums.follow(to), before.follow(to);
                }
            };
            // A chunk of the accumulator, columns n .. n + 31 of the logits, c of this warp's.  (Two
            // copies of the sums: with what the end of V changes in the first, it took 2 % longer.)
            auto take = [&](const uint32_t (&q)[32], int n, int c) {
                float z[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) z[x] = __uint_as_float(q[x]);
                if (!BIAS && n + 32 <= p.V) {
                    add(z);
                    return;
                }
                float w[32];
#pragma unroll
                for (int x = 0; x < 32; x += 4) {
                    if (BIAS) {
                        const float4 b = my_bias[8 * c + x / 4];
                        const float2 lo = sm_add2(make_float2(z[x], z[x + 1]), make_float2(b.x, b.y));
                        const float2 hi = sm_add2(make_float2(z[x + 2], z[x + 3]), make_float2(b.z, b.w));
                        w[x] = lo.x, w[x + 1] = lo.y, w[x + 2] = hi.x, w[x + 3] = hi.y;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[x + k] = n + x + k < p.V ? z[x + k] : -INFINITY;
                    }
                }
                add(w);
            };
            // The bias of this warp's columns from n on, four per lane; -inf behind V, which masks them.
            auto load_bias = [&](int n) {
                float4 b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                n += 4 * lane;
                if (4 * lane >= half || n >= p.V) return b;
                if (p.wide_bias && n + 4 <= p.V) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.bias + n));
                    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
                }
                b.x = __bfloat162float(p.bias[n]);
                if (n + 1 < p.V) b.y = __bfloat162float(p.bias[n + 1]);
                if (n + 2 < p.V) b.z = __bfloat162float(p.bias[n + 2]);
                if (n + 3 < p.V) b.w = __bfloat162float(p.bias[n + 3]);
                return b;
            };
            float4 ahead = make_float4(0.f, 0.f, 0.f, 0.f);  // the next tile's
            if (BIAS) ahead = load_bias(it.v0 * BN + half * chalf);
            for (int v = it.v0; v < it.v1; ++v, ++j) {
                const int acc = j & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(&sh->acc_full[acc], (j >> 1) & 1, kDevTimeoutSoftmax, abort, p.status));
                if (!ok) break;
                tc_fence_after();
                const int n0 = v * BN + half * chalf;
                if (BIAS) {
                    __syncwarp();  // the last tile's has been read
                    if (4 * lane < half &&
                        TXL_BOUNDS(smem_u32(my_bias + lane + 1) <= smem_u32(smem_raw) + C::SMEM_BYTES, 1304, lane))
                        my_bias[lane] = ahead;
                    __syncwarp();
                    if (v + 1 < it.v1) ahead = load_bias((v + 1) * BN + half * chalf);
                }
                const uint32_t from = t_row + acc * MAX_BN;
                // the logits of the tokens that lie in these columns, row by row (few do)
                for (unsigned has = __ballot_sync(0xffffffffu, token >= n0 && token < n0 + half && token < p.V); has; has &= has - 1) {
                    const int src = __ffs(has) - 1, n = __shfl_sync(0xffffffffu, (int)token, src);
                    if (!TXL_BOUNDS(n - v * BN >= 0 && n - v * BN < BN && acc * MAX_BN + n - v * BN < (int)TMEM_COLS, 1306, n)) continue;
                    float g = lp_tmem_column(from + (n - n0));
                    if (BIAS) g += __bfloat162float(p.bias[n]);
                    if (lane == src && TXL_BOUNDS(lp_in_workspace(p, p.given + row), 1301, row)) p.given[row] = g;
                }
                // Columns behind V hold 0 times x, which is NaN where x is not finite, and that with the bias
                // of -inf too.  (Selected in the sums instead, wherever in them, 4 % more time with K of 256.)
                if (BIAS && n0 + half > p.V && __any_sync(0xffffffffu, lp_tmem_column(from + half - 1) != 0.f)) {
#pragma unroll 1
                    for (int c = max(0, p.V - n0); c < half; ++c) lp_tmem_clear_column(from + c);
                    tmem_wait_st();
                }
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    uint32_t q[32];
                    tmem_ld32(from + 32 * c, q);
                    tmem_wait_ld();
                    if (c == chunks - 1) {  // the accumulator is the MMAs' again
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (PAIR)
                                lb_arrive_remote(acc_empty0 + 8 * acc);
                            else
                                mbar_arrive(&sh->acc_empty[acc]);
                        }
                    }
                    take(q, n0 + 32 * c, c);
                }
                before.take(sums);
            }
            if (ok && row < p.rows) {
                const int slot = 2 * it.run + chalf;
                float4* const to = p.part + ((long long)row * (2 * p.chunks) + slot);
                if (TXL_BOUNDS(slot < 2 * p.chunks && lp_in_workspace(p, to) && to < reinterpret_cast<const float4*>(p.given), 1302, slot))
                    *to = make_float4(before.m, before.s.x + before.s.y, before.t.x + before.t.y, 0.f);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    // the second CTA's barriers have had the last of the first one's commits
    if (PAIR && rank == 1 && warp == 1) lb_wait_landed(&sh->drain, 0, p.status);
    __syncwarp();
    lb_sync<PAIR>();  // no CTA of a pair exits while the other may signal it or read its operands
    if (warp == 1) {
        tc_fence_after();
        lb_tmem_dealloc<PAIR>(tmem, TMEM_COLS);
    }
}

// A row's results from its parts: a warp per row, its lanes on the parts.
__global__ void __launch_bounds__(256) linear_logprobs_join_kernel(const LpParams p, float* logprob, float* lse, float* entropy) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, r = blockIdx.x * 8 + (threadIdx.x >> 5), n = 2 * p.chunks;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (r >= p.rows) return;
    const long long token = p.tokens[r];
    const float4* const q = p.part + (long long)r * n;
    const float given = token >= 0 && token < p.V && TXL_BOUNDS(lp_in_workspace(p, p.given + r), 1305, r) ? p.given[r] : 0.f;
    SoftmaxSums a;
    a.clear();
    for (int i = lane; i < n; i += 32 * 8) {  // 8 on their way at a time
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = i + 32 * u < n && TXL_BOUNDS(lp_in_workspace(p, q + i + 32 * u), 1303, r)
                       ? q[i + 32 * u]
                       : make_float4(-3.402823466e38f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const SoftmaxSums b = {v[u].x, v[u].y, v[u].z};
            a.merge(b);
        }
    }
    a.merge_warp();
    if (lane == 0) {
        const SoftmaxRow o(a);
        lse[r] = o.lse;
        entropy[r] = o.entropy;
        logprob[r] = token < 0 ? 0.f : token < p.V ? o.logprob(given) : __uint_as_float(0x7FFFFFFFu);
    }
}

// ---------------------------------------------------------------- host side
namespace {

typedef CUresult (*LpEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

LpEncodeFn lp_encode_fn() {
    static LpEncodeFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<LpEncodeFn>(ptr);
        return static_cast<LpEncodeFn>(nullptr);
    }();
    return fn;
}

// [rows, K] bf16 as boxes of 64 elements x `high` rows.
bool lp_encode(CUtensorMap* map, const void* base, long long rows, int K, int high) {
    LpEncodeFn fn = lp_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)K * 2};
    const cuuint32_t box[2] = {lp::BK, (cuuint32_t)high}, es[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Microseconds that a tile takes, as measured over K of 64 to 1024 and tiles of 64 to 256
// columns: its stages, or, where those are few, what lies between two of its accumulators (a
// pair's hand-over goes through both CTAs) and the epilogue.  A single CTA's stages take longer, as
// it loads as many rows of W for half the rows of x, its hand-over half the time: 11264 rows to
// 32768 columns take pairs and single CTAs 156 and 111 us with K of 256, 199 and 219 with 512.
double lp_tile_us(bool pair, int bn, int ksteps, bool lines, bool bias) {
    const double w = (double)bn / lp::MAX_BN;
    // (rows of W that do not begin on 128-byte lines take longer to load)
    const double step = pair ? (0.10 + 0.23 * w) * (lines ? 1.0 : 1.3) : (0.16 + 0.20 * w) * (lines ? 1.0 : 1.5);
    const double apart = (pair ? 0.9 + (0.75 + 0.14 * ksteps) * w : 0.25 + w) + (bias ? 0.4 * w : 0.0);
    return std::max(step * ksteps, apart);
}
constexpr double kItem = 1.0;  // that an item's end adds
constexpr int kMostTiles = 2048;  // of an item, whose sums are added one after the other

}  // namespace

LpPlan linear_logprobs_plan(int rows, int K, int V, bool bias) {
    LpPlan pl = {};
    LpParams& p = pl.p;
    p.rows = rows;
    p.V = V;
    p.ksteps = (K + lp::BK - 1) / lp::BK;
    p.klast = (K - (p.ksteps - 1) * lp::BK + 15) / 16;
    const int sms = current_sm_count();
    // The tile and the run with the least time by this model: rounds of items over the units.
    double best = -1;
    for (int ctas : {2, 1}) {
        const int most = sms / ctas, tile = lp::BM * ctas;
        if (most < 1) continue;
        const int rt = (int)(((long long)rows + tile - 1) / tile);
        // (narrower tiles only where the units have few)
        const bool few = (double)rt * ((double)V / lp::MAX_BN) < 16.0 * most;
        for (int bn = lp::MAX_BN; bn >= (few ? 64 : lp::MAX_BN); bn -= 64) {
            const int vt = (int)(((long long)V + bn - 1) / bn);
            const double us = lp_tile_us(ctas == 2, bn, p.ksteps, K % lp::BK == 0, bias);
            for (int rounds = 1; rounds <= (few ? 4 : 24); ++rounds) {
                const int runs = (int)std::max(1ll, std::min<long long>(vt, (long long)most * rounds / rt));
                const int per = std::min((vt + runs - 1) / runs, kMostTiles), chunks = (vt + per - 1) / per;
                const long long items = (long long)rt * chunks, units = std::min<long long>(items, most);
                const double cost = (double)((items + units - 1) / units) * (per * us + kItem);
                if (best >= 0 && cost >= best) continue;
                best = cost;
                pl.pair = ctas == 2;
                pl.grid = (int)units * ctas;
                p.bn = bn;
                p.n_rt = rt;
                p.n_vt = vt;
                p.per = per;
                p.chunks = chunks;
            }
        }
    }
    return pl;
}

size_t linear_logprobs_workspace_bytes(const LpPlan& pl) { return ((size_t)pl.p.chunks * 2 * sizeof(float4) + sizeof(float)) * pl.p.rows; }

namespace {

template <bool PAIR, int BN, bool BIAS>
cudaError_t lp_launch(const LpMaps& maps, const LpPlan& pl, cudaStream_t stream) {
    using C = lp::Cfg<PAIR, BN>;
    static PerDeviceOnce attrs;
    const cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(linear_logprobs_kernel<PAIR, BN, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.grid);
    cfg.blockDim = dim3(lp::NTHREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_logprobs_kernel<PAIR, BN, BIAS>, maps, pl.p);
}

template <bool PAIR, bool BIAS>
cudaError_t lp_launch(const LpMaps& maps, const LpPlan& pl, cudaStream_t stream) {
    switch (pl.p.bn) {
        case 64: return lp_launch<PAIR, 64, BIAS>(maps, pl, stream);
        case 128: return lp_launch<PAIR, 128, BIAS>(maps, pl, stream);
        case 192: return lp_launch<PAIR, 192, BIAS>(maps, pl, stream);
        default: return lp_launch<PAIR, 256, BIAS>(maps, pl, stream);
    }
}

}  // namespace

cudaError_t launch_linear_logprobs(LpPlan pl, const void* x, const void* w, const void* bias, int K, const long long* tokens,
                                   float* logprob, float* lse, float* entropy, void* workspace, size_t ws_bytes, int* status,
                                   cudaStream_t stream) {
    LpParams& p = pl.p;
    p.tokens = tokens;
    p.bias = static_cast<const __nv_bfloat16*>(bias);
    p.wide_bias = (reinterpret_cast<uintptr_t>(bias) & 7u) == 0;
    p.part = static_cast<float4*>(workspace);
    p.given = reinterpret_cast<float*>(p.part + (size_t)p.chunks * 2 * p.rows);
    p.ws_end = static_cast<const char*>(workspace) + ws_bytes;
    p.status = status;
    LpMaps maps;
    if (!lp_encode(&maps.x, x, p.rows, K, lp::BM) || !lp_encode(&maps.w, w, p.V, K, p.bn / (pl.pair ? 2 : 1))) return cudaErrorInvalidValue;
    const cudaError_t e = pl.pair ? (bias ? lp_launch<true, true>(maps, pl, stream) : lp_launch<true, false>(maps, pl, stream))
                                  : (bias ? lp_launch<false, true>(maps, pl, stream) : lp_launch<false, false>(maps, pl, stream));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.rows + 7ll) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_logprobs_join_kernel, p, logprob, lse, entropy);
}

TXL_BOUNDS_READER(bounds_word_linear_logprobs)

}  // namespace txl
