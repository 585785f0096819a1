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
// Two CTAs of a cluster share a 256 x 256 tile (cta_group::2), or one CTA takes 128 x 128
// where there are few rows.  Both operands are K-major, 128 rows of 64 elements per stage
// and CTA: two TMA instructions of 16 KB.  Rows, columns and K need not fill their tiles:
// TMA fills with zeros behind the ends, and columns behind V count as -inf.
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
constexpr int NTHREADS = 384;
constexpr uint32_t SZ_A = BM * BK * 2;  // 16 KB
constexpr uint32_t SZ_B = 128 * BK * 2;  // of a pair's 256 columns, each CTA holds half
constexpr int STAGES = 6;
constexpr uint32_t OFF_A = 0;
constexpr uint32_t OFF_B = STAGES * SZ_A;
constexpr uint32_t OFF_BAR = OFF_B + STAGES * SZ_B;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 512 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget of one sm_103a CTA");

template <bool PAIR>
struct Cfg {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TM = BM * CTAS;  // tile
    static constexpr int BN = PAIR ? 256 : 128;
    static constexpr uint32_t TMEM_COLS = 2 * BN;
    static constexpr uint32_t IDESC = idesc_bf16_f32(TM, BN, 0, 0);
};
}  // namespace lp

struct LpMaps {
    CUtensorMap x, w;  // (element, row), boxes of 64 x 128
};

struct LpShared {
    uint64_t full[lp::STAGES];  // a pair's: those of its first CTA
    uint64_t empty[lp::STAGES];
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

template <bool PAIR>
__global__ void __launch_bounds__(lp::NTHREADS, 1) linear_logprobs_kernel(const __grid_constant__ LpMaps maps, const LpParams p) {
    using namespace lp;
    using C = Cfg<PAIR>;
    constexpr int BN = C::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    LpShared* sh = reinterpret_cast<LpShared*>(smem + OFF_BAR);
    const uint32_t s_base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? lb_cta_rank() : 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 1) lb_tmem_alloc<PAIR>(&sh->tmem_base, C::TMEM_COLS);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], 8 * C::CTAS);  // one arrival per epilogue warp
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
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = sh->tmem_base;
    volatile int* abort = &sh->abort;
    const int unit = blockIdx.x / C::CTAS, units = gridDim.x / C::CTAS, items = p.n_rt * p.chunks;

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        // A pair's full barriers are its first CTA's, which expects both CTAs' bytes; the
        // second's loads may land before it does (the barrier waits for the arrival).
        if (lane == 0) {
            bool ok = true;
            uint32_t s = 0, phase = 1;  // slot, parity of its empty barrier (a fresh one passes for 1)
            long long loads = 0;
            const uint32_t full0 = PAIR ? lb_mapa(&sh->full[0], 0) : smem_u32(&sh->full[0]);
            for (int i = unit; ok && i < items; i += units) {
                const LpItem it = lp_item(p, i);
                const int r0 = it.r * C::TM + BM * rank;
                for (int v = it.v0; ok && v < it.v1; ++v) {
                    const int n0 = v * BN + 128 * rank;
                    for (int k = 0; k < p.ksteps; ++k) {
                        if (!mbar_wait(&sh->empty[s], phase, kDevTimeoutProducer, abort, p.status)) {
                            ok = false;
                            break;
                        }
                        if (rank == 0) mbar_expect_tx(&sh->full[s], (SZ_A + SZ_B) * C::CTAS);
                        lb_load_2d<PAIR>(s_base + OFF_A + s * SZ_A, &maps.x, full0 + 8 * s, k * BK, r0);
                        lb_load_2d<PAIR>(s_base + OFF_B + s * SZ_B, &maps.w, full0 + 8 * s, k * BK, n0);
                        if (++s == STAGES) s = 0, phase ^= 1;
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
            const uint64_t dA0 = smem_desc_sw128(s_base + OFF_A, 16, 1024);
            const uint64_t dB0 = smem_desc_sw128(s_base + OFF_B, 16, 1024);
            uint32_t s = 0, phase = 0;  // slot, parity of its full barrier
            int j = 0;                  // accumulators filled
            for (int i = unit; ok && i < items; i += units) {
                const LpItem it = lp_item(p, i);
                for (int v = it.v0; ok && v < it.v1; ++v) {
                    const int acc = j & 1;
                    if (j >= 2 && !wait(&sh->acc_empty[acc], ((j >> 1) - 1) & 1)) break;
                    tc_fence_after();
                    const uint32_t d_acc = tmem + acc * BN;
                    for (int k = 0; k < p.ksteps; ++k) {
                        if (!wait(&sh->full[s], phase)) break;
                        tc_fence_after();
                        const uint64_t ad = dA0 + s * (SZ_A >> 4), bd = dB0 + s * (SZ_B >> 4);
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            lb_mma<PAIR>(d_acc, ad + 2 * kk, bd + 2 * kk, C::IDESC, (k > 0 || kk > 0) ? 1u : 0u, leader);
                        if (leader) lb_commit<PAIR>(&sh->empty[s]);
                        if (++s == STAGES) s = 0, phase ^= 1;
                    }
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
        constexpr int CPW = BN / 64;  // 32-column chunks per warp
        const uint32_t t_row = tmem + ((uint32_t)(wq * 32) << 16) + 32 * CPW * chalf;
        const uint32_t acc_empty0 = PAIR ? lb_mapa(&sh->acc_empty[0], 0) : 0;
        bool ok = true;
        int j = 0;
        for (int i = unit; ok && i < items; i += units) {
            const LpItem it = lp_item(p, i);
            const int row = it.r * C::TM + BM * rank + 32 * wq + lane;
            const long long token = row < p.rows ? p.tokens[row] : -1;
            SoftmaxSums sums;
            sums.clear();
            float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
            for (int v = it.v0; v < it.v1; ++v, ++j) {
                const int acc = j & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(&sh->acc_full[acc], (j >> 1) & 1, kDevTimeoutSoftmax, abort, p.status));
                if (!ok) break;
                tc_fence_after();
                const int n0 = v * BN + 32 * CPW * chalf;
#pragma unroll 1
                for (int cc = 0; cc < CPW; ++cc) {
                    uint32_t q[32];
                    tmem_ld32(t_row + acc * BN + 32 * cc, q);
                    tmem_wait_ld();
                    if (cc == CPW - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (PAIR)
                                lb_arrive_remote(acc_empty0 + 8 * acc);
                            else
                                mbar_arrive(&sh->acc_empty[acc]);
                        }
                    }
                    const int n = n0 + 32 * cc;
                    float z[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) z[x] = __uint_as_float(q[x]);
                    if (p.bias) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (n + x < p.V) z[x] += __bfloat162float(p.bias[n + x]);
                    }
                    if (n + 32 > p.V) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (n + x >= p.V) z[x] = -INFINITY;
                    }
                    if (token >= n && token < n + 32 && token < p.V) {
                        const int at = (int)token - n;
                        float g = z[0];
#pragma unroll
                        for (int x = 1; x < 32; ++x) g = at == x ? z[x] : g;
                        if (TXL_BOUNDS(row < p.ld, 1301, row)) p.given[row] = g;
                    }
                    float most = z[0];
#pragma unroll
                    for (int x = 1; x < 32; ++x) most = fmaxf(most, z[x]);
                    if (most > sums.m) {
                        const float d = fmaxf(sums.m - most, kLowest), f = sm_ex2(d * kLog2e);
                        const float2 ff = make_float2(f, f);
                        t = sm_mul2(ff, sm_fma2(make_float2(d, d), s, t));
                        s = sm_mul2(ff, s);
                        sums.m = most;
                    }
#pragma unroll
                    for (int x = 0; x < 32; x += 2) sm_add_pair(make_float2(z[x], z[x + 1]), sums.m, s, t);
                }
            }
            if (ok && row < p.rows) {
                const long long slot = 2 * it.run + chalf;
                if (TXL_BOUNDS(row < p.ld && slot < 2 * p.chunks, 1302, slot)) {
                    float* const to = p.part + slot * 3 * p.ld + row;
                    to[0] = sums.m;
                    to[p.ld] = s.x + s.y;
                    to[2 * p.ld] = t.x + t.y;
                }
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
        lb_tmem_dealloc<PAIR>(tmem, C::TMEM_COLS);
    }
}

// A row's results from its parts: 32 rows per CTA, a warp's lanes on a row each and its
// parts dealt to the 32 warps.
__global__ void __launch_bounds__(1024) linear_logprobs_join_kernel(const LpParams p, float* logprob, float* lse, float* entropy) {
    __shared__ SoftmaxSums sh[32][33];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * 32 + lane;
    SoftmaxSums a;
    a.clear();
    if (row < p.rows) {
#pragma unroll 4
        for (int slot = warp; slot < 2 * p.chunks; slot += 32) {
            const float* const q = p.part + (long long)slot * 3 * p.ld + row;
            const SoftmaxSums b = {q[0], q[p.ld], q[2 * p.ld]};
            a.merge(b);
        }
    }
    sh[warp][lane] = a;
    __syncthreads();
    const int r = blockIdx.x * 32 + warp;  // now a warp per row
    a = sh[lane][warp];
    a.merge_warp();
    if (lane == 0 && r < p.rows) {
        const SoftmaxRow o(a);
        const long long token = p.tokens[r];
        lse[r] = o.lse;
        entropy[r] = o.entropy;
        logprob[r] = token < 0 ? 0.f : token < p.V ? o.logprob(p.given[r]) : __uint_as_float(0x7FFFFFFFu);
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

// [rows, K] bf16 as boxes of 64 elements x 128 rows.
bool lp_encode(CUtensorMap* map, const void* base, long long rows, int K) {
    LpEncodeFn fn = lp_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)K * 2};
    const cuuint32_t box[2] = {lp::BK, 128}, es[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Microseconds that a stage takes a pair or a CTA, and that an item's end adds.
constexpr double kStepPair = 0.36, kStepOne = 0.27, kItem = 1.0;

}  // namespace

LpPlan linear_logprobs_plan(int rows, int K, int V) {
    LpPlan pl = {};
    LpParams& p = pl.p;
    p.rows = rows;
    p.V = V;
    p.ksteps = (K + lp::BK - 1) / lp::BK;
    const int sms = current_sm_count();
    // The tile and the run with the least time by this model: rounds of items over the units.
    double best = -1;
    for (int ctas : {2, 1}) {
        const int most = sms / ctas, tile = lp::BM * ctas;
        if (most < 1) continue;
        const int rt = (int)(((long long)rows + tile - 1) / tile), vt = (int)(((long long)V + tile - 1) / tile);
        // (runs of each length that some number of rounds gives, up to 64 rounds)
        for (int rounds = 1; rounds <= 64; ++rounds) {
            const long long runs = std::max(1ll, (long long)most * rounds / rt);
            const int per = (int)((vt + runs - 1) / runs), chunks = (vt + per - 1) / per;
            const long long items = (long long)rt * chunks, units = std::min<long long>(items, most);
            const double cost = (double)((items + units - 1) / units) * (per * p.ksteps * (ctas == 2 ? kStepPair : kStepOne) + kItem);
            if (best >= 0 && cost >= best) continue;
            best = cost;
            pl.pair = ctas == 2;
            pl.grid = (int)units * ctas;
            p.n_rt = rt;
            p.n_vt = vt;
            p.per = per;
            p.chunks = chunks;
            p.ld = (long long)rt * tile;
        }
    }
    return pl;
}

size_t linear_logprobs_workspace_bytes(const LpPlan& pl) { return ((size_t)pl.p.chunks * 6 + 1) * pl.p.ld * sizeof(float); }

namespace {

template <bool PAIR>
cudaError_t lp_launch(const LpMaps& maps, const LpPlan& pl, cudaStream_t stream) {
    static PerDeviceOnce attrs;
    const cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(linear_logprobs_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, lp::SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.grid);
    cfg.blockDim = dim3(lp::NTHREADS);
    cfg.dynamicSmemBytes = lp::SMEM_BYTES;
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
    return cudaLaunchKernelEx(&cfg, linear_logprobs_kernel<PAIR>, maps, pl.p);
}

}  // namespace

cudaError_t launch_linear_logprobs(LpPlan pl, const void* x, const void* w, const void* bias, int K, const long long* tokens,
                                   float* logprob, float* lse, float* entropy, void* workspace, int* status,
                                   cudaStream_t stream) {
    LpParams& p = pl.p;
    p.tokens = tokens;
    p.bias = static_cast<const __nv_bfloat16*>(bias);
    p.part = static_cast<float*>(workspace);
    p.given = p.part + (size_t)p.chunks * 6 * p.ld;
    p.status = status;
    LpMaps maps;
    if (!lp_encode(&maps.x, x, p.rows, K) || !lp_encode(&maps.w, w, p.V, K)) return cudaErrorInvalidValue;
    const cudaError_t e = pl.pair ? lp_launch<true>(maps, pl, stream) : lp_launch<false>(maps, pl, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.rows + 31ll) / 32));
    cfg.blockDim = dim3(1024);
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
