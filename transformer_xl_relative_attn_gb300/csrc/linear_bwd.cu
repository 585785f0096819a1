// Gradients of a Linear layer out = x W^T + b on the sm_103a tensor cores, bf16
// in, fp32 accumulation:
//
//   dx = dy W          [T, K] = [T, N] [N, K]   bf16 (where x came out of a ReLU: times [x > 0])
//   dw = dy^T x        [N, K] = [N, T] [T, K]   fp32
//   db = sum over rows of dy                    fp32
//
// One persistent launch holds both products.  In both the second operand (W for
// dx, x for dw) is read with K contiguous and its other axis reduced over (MN-major
// for the tensor core) and the output is tiled 128 x BN with BN along K, so one
// pipeline serves both: 64-row boxes of 64 columns land in shared memory the same
// way, and only dy's view differs (K-major with the rows as M for dx, MN-major
// with the columns as M for dw).  Nothing is transposed in memory.
//
// The ReLU mask is a factor of the epilogue of dx, read from x.  db comes from the
// dy tiles of the dw product while they lie in shared memory (two warps add up the
// columns of the first column tile's stages): dy is not read again for it.
//
// dw has few tiles and a long reduction (base512's second feed-forward layer: 32
// tiles over 11264 rows), so its rows are split over several CTAs, each writing an
// fp32 partial tile to the workspace; a second launch adds the parts in a fixed
// order (the same inputs give the same bits).
//
// Roles (384 threads, one CTA per SM): warp 0 lane 0 issues the TMA loads, warp 1
// the MMAs, warps 2-3 the column sums, warps 4-11 the epilogue; two accumulators
// let an epilogue overlap the next tile's MMAs.  Every wait is bounded (1 s) and
// reports through the device status word.  Rows, N and K need not fill tiles: TMA
// fills with zeros behind the ends and clips its stores.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "linear_bwd.h"
#include "txl_device.cuh"

namespace txl {

namespace lb {
constexpr int BM = 128;
constexpr int BR = 64;  // reduction per stage
constexpr int NTHREADS = 384;
constexpr uint32_t SZ_BOX = 64 * 64 * 2;  // 64 rows of 64 bf16: 8 KB
constexpr uint32_t SZ_A = 2 * SZ_BOX;
constexpr int MAX_STAGES = 6;

template <int BN_>
struct Cfg {
    static constexpr int BN = BN_;
    static constexpr int STAGES = BN_ == 256 ? 4 : 6;
    static constexpr uint32_t SZ_B = BN_ / 64 * SZ_BOX;
    static constexpr uint32_t OFF_A = 0;
    static constexpr uint32_t OFF_B = STAGES * SZ_A;
    static constexpr uint32_t OFF_STG = OFF_B + STAGES * SZ_B;  // 4 KB per epilogue warp
    static constexpr uint32_t OFF_BAR = OFF_STG + 8 * 4096;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 256 + 1024;
    static constexpr uint32_t TMEM_COLS = 2 * BN_;
    static constexpr uint32_t IDESC_DX = idesc_bf16_f32(BM, BN_, 1, 0);
    static constexpr uint32_t IDESC_DW = idesc_bf16_f32(BM, BN_, 1, 1);
    static_assert(SMEM_BYTES <= 232448, "shared memory budget of one sm_103a CTA");
};
}  // namespace lb

struct LbParams {
    int T, B;       // rows per batch row, batch rows (rows layout: all rows, 1)
    int K, N;
    int heads;      // x and dx are [B, K / 64, T, 64]
    int relu;
    int n_kt, n_nt, n_tt;  // tiles along K, N and T (per batch row)
    int t_steps;           // 64-row steps per batch row
    int n_steps;           // 64-column steps of N
    int splits;            // of dw's reduction
    int n_w, n_d;          // dw items (tiles * splits), dx tiles
    int heavy, extra;      // see LbSchedule
    int want_db;
    const __nv_bfloat16* x;
    float* db;             // [splits, N]
    int* status;
};

struct LbMaps {
    CUtensorMap dy;  // (column, row, batch row)
    CUtensorMap w;   // (column, row)
    CUtensorMap x;   // (element, row, 64-column slice, batch row); rows layout: one slice of K
    CUtensorMap dx;  // the same, boxes of 32 rows
    CUtensorMap dw;  // (column, row, split), boxes of 32 x 32
};

struct LbShared {
    uint64_t full[lb::MAX_STAGES];
    uint64_t empty[lb::MAX_STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// The items of one CTA, the same sequence for every role.  dw items are dealt in
// turn first (the long ones).  Where they do not divide evenly, the CTAs from
// `heavy` on have one less: they take `extra` dx tiles each ahead of the rest, which
// is then dealt in turn from the last CTA down.
struct LbSchedule {
    const LbParams& p;
    int c, g, light, head;  // CTA, CTAs, CTAs with one dw item less, dx tiles dealt to them ahead
    int w, e, d;            // next dw item, next extra tile, next dx tile
    __device__ __forceinline__ explicit LbSchedule(const LbParams& p_) : p(p_) {
        c = blockIdx.x;
        g = gridDim.x;
        light = p.heavy ? g - p.heavy : 0;
        head = min(p.n_d, light * p.extra);
        w = c;
        e = light && c >= p.heavy ? c - p.heavy : head;
        d = head + (g - 1 - c);
    }
    // The next item: dw = true with its index, or a dx tile.
    __device__ __forceinline__ bool next(bool& dw, int& item) {
        if (w < p.n_w) {
            dw = true;
            item = w;
            w += g;
            return true;
        }
        dw = false;
        if (e < head) {
            item = e;
            e += light;
            return true;
        }
        if (d < p.n_d) {
            item = d;
            d += g;
            return true;
        }
        return false;
    }
};

// What an item covers: output tile (m0, k0), the reduction steps [s0, s1), and for
// dx the batch row, for dw the split.
struct LbItem {
    int m0, k0, s0, s1, b, split;
};

template <int BN>
__device__ __forceinline__ LbItem lb_item(const LbParams& p, bool dw, int i) {
    LbItem it;
    it.k0 = (i % p.n_kt) * BN;
    int rest = i / p.n_kt;
    if (dw) {
        it.m0 = (rest % p.n_nt) * lb::BM;
        it.split = rest / p.n_nt;
        it.b = 0;
        const long long total = (long long)p.B * p.t_steps;
        it.s0 = (int)(total * it.split / p.splits);
        it.s1 = (int)(total * (it.split + 1) / p.splits);
    } else {
        it.m0 = (rest % p.n_tt) * lb::BM;
        it.b = rest / p.n_tt;
        it.split = 0;
        it.s0 = 0;
        it.s1 = p.n_steps;
    }
    return it;
}

namespace {

__device__ __forceinline__ void lb_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                           int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void lb_store_4d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void lb_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void lb_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void lb_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace

template <int BN_>
__global__ void __launch_bounds__(lb::NTHREADS, 1)
linear_bwd_kernel(const __grid_constant__ LbMaps maps, const LbParams p) {
    using namespace lb;
    using C = Cfg<BN_>;
    constexpr int BN = C::BN, STAGES = C::STAGES;
    constexpr uint32_t SZ_B = C::SZ_B;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    LbShared* sh = reinterpret_cast<LbShared*>(smem + C::OFF_BAR);
    const uint32_t s_base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 1) {
        tmem_alloc(&sh->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], p.want_db ? 3 : 1);  // the MMAs' commit, and the two summing warps
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], 8);
        }
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.dy);
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.x);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = sh->tmem_base;
    volatile int* abort = &sh->abort;
    LbSchedule sched(p);
    bool dw;
    int item;

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (lane == 0) {
            bool ok = true;
            int c = 0;
            while (ok && sched.next(dw, item)) {
                const LbItem it = lb_item<BN>(p, dw, item);
                for (int st = it.s0; st < it.s1; ++st, ++c) {
                    const int s = c % STAGES;
                    if (c >= STAGES &&
                        !mbar_wait(&sh->empty[s], ((c / STAGES) & 1) ^ 1, kDevTimeoutProducer, abort, p.status)) {
                        ok = false;
                        break;
                    }
                    uint64_t* bar = &sh->full[s];
                    mbar_expect_tx(bar, SZ_A + SZ_B);
                    uint8_t* a = smem + C::OFF_A + s * SZ_A;
                    const uint32_t bt = s_base + C::OFF_B + s * SZ_B;
                    if (dw) {
                        const int b = st / p.t_steps, t = (st - b * p.t_steps) * BR;
                        tma_load_3d(a, &maps.dy, bar, it.m0, t, b);
                        tma_load_3d(a + SZ_BOX, &maps.dy, bar, it.m0 + 64, t, b);
#pragma unroll
                        for (int j = 0; j < BN / 64; ++j) {
                            const int k = it.k0 + 64 * j;
                            lb_load_4d(bt + j * SZ_BOX, &maps.x, bar, p.heads ? 0 : k, t, p.heads ? k >> 6 : 0, b);
                        }
                    } else {
                        const int n = st * BR;
                        tma_load_3d(a, &maps.dy, bar, n, it.m0, it.b);
                        tma_load_3d(a + SZ_BOX, &maps.dy, bar, n, it.m0 + 64, it.b);
#pragma unroll
                        for (int j = 0; j < BN / 64; ++j)
                            tma_load_2d(smem + C::OFF_B + s * SZ_B + j * SZ_BOX, &maps.w, bar, it.k0 + 64 * j, n);
                    }
                }
            }
            // the last load into each slot has landed before the CTA exits
            for (int i = c - STAGES; i < c; ++i)
                if (i >= 0) {
                    const uint64_t t0n = globaltimer_ns();
                    while (!mbar_try_wait(&sh->full[i % STAGES], (i / STAGES) & 1))
                        if (globaltimer_ns() - t0n > kWaitLimitNs) {
                            record_status(p.status, kDevTimeoutDrain);
                            break;
                        }
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        const uint32_t leader = elect_one();
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, kDevTimeoutMma, abort, p.status));
            return ok;
        };
        const uint64_t dA0 = smem_desc_sw128(s_base + C::OFF_A, 16, 1024);          // K-major: rows of dy
        const uint64_t dAm = smem_desc_sw128(s_base + C::OFF_A, SZ_BOX, 1024);      // MN-major: columns of dy
        const uint64_t dB0 = smem_desc_sw128(s_base + C::OFF_B, SZ_BOX, 1024);      // MN-major
        int c = 0, j = 0;
        for (; ok && sched.next(dw, item); ++j) {
            const LbItem it = lb_item<BN>(p, dw, item);
            const int acc = j & 1;
            if (j >= 2 && !wait(&sh->acc_empty[acc], ((j >> 1) - 1) & 1)) break;
            tc_fence_after();
            const uint32_t d_acc = tmem + acc * BN;
            for (int st = it.s0; st < it.s1; ++st, ++c) {
                const int s = c % STAGES;
                if (!wait(&sh->full[s], (c / STAGES) & 1)) break;
                tc_fence_after();
                const uint64_t bd = dB0 + s * (SZ_B >> 4);
                if (dw) {
                    const uint64_t a = dAm + s * (SZ_A >> 4);
#pragma unroll
                    for (int kk = 0; kk < BR / 16; ++kk)
                        mma_ss_elect(d_acc, a + 128 * kk, bd + 128 * kk, C::IDESC_DW,
                                     (st > it.s0 || kk > 0) ? 1u : 0u, leader);
                } else {
                    const uint64_t a = dA0 + s * (SZ_A >> 4);
#pragma unroll
                    for (int kk = 0; kk < BR / 16; ++kk)
                        mma_ss_elect(d_acc, a + 2 * kk, bd + 128 * kk, C::IDESC_DX,
                                     (st > it.s0 || kk > 0) ? 1u : 0u, leader);
                }
                if (leader) mma_commit(&sh->empty[s]);
            }
            if (!ok) break;
            if (leader) mma_commit(&sh->acc_full[acc]);
        }
        if (leader) mma_commit(&sh->drain);
        const uint64_t t0n = globaltimer_ns();
        while (!mbar_try_wait(&sh->drain, 0))
            if (globaltimer_ns() - t0n > kWaitLimitNs) {
                record_status(p.status, kDevTimeoutDrain);
                break;
            }
        __syncwarp();
    } else if (warp < 4) {
        // ---------------------------------------------------- column sums of dy
        // Warp 2 + h: columns 64 h .. of the tile, two per lane; 64 rows are summed
        // by themselves before they join the running sum, which keeps its rounding
        // errors to those of chains of 64.
        if (p.want_db) {
            const int h = warp - 2;
            bool ok = true;
            int c = 0;
            while (ok && sched.next(dw, item)) {
                const LbItem it = lb_item<BN>(p, dw, item);
                const bool mine = dw && it.k0 == 0;
                float s0 = 0.f, s1 = 0.f;
                for (int st = it.s0; st < it.s1; ++st, ++c) {
                    const int s = c % STAGES;
                    ok = __all_sync(0xffffffffu, mbar_wait(&sh->full[s], (c / STAGES) & 1, kDevTimeoutSoftmax, abort,
                                                           p.status));
                    if (!ok) break;
                    if (mine) {
                        const uint8_t* a = smem + C::OFF_A + s * SZ_A + h * SZ_BOX + (lane & 3) * 4;
                        float a0 = 0.f, a1 = 0.f;
#pragma unroll 16
                        for (int t = 0; t < BR; ++t) {
                            const __nv_bfloat162 v =
                                *reinterpret_cast<const __nv_bfloat162*>(a + t * 128 + (((lane >> 2) ^ (t & 7)) << 4));
                            const float2 f = __bfloat1622float2(v);
                            a0 += f.x;
                            a1 += f.y;
                        }
                        s0 += a0;
                        s1 += a1;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->empty[s]);
                }
                const int n = it.m0 + 64 * h + 2 * lane;  // N is even
                if (ok && mine && n < p.N &&
                    TXL_BOUNDS(it.split < p.splits && n + 2 <= p.N, 801, (long long)it.split * p.N + n))
                    *reinterpret_cast<float2*>(p.db + (size_t)it.split * p.N + n) = make_float2(s0, s1);
            }
        }
    } else {
        // ---------------------------------------------------- epilogue
        const int wq = warp & 3;
        const int chalf = (warp - 4) >> 2;
        constexpr int CPW = BN / 64;  // 32-column chunks per warp
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t stg = s_base + C::OFF_STG + (uint32_t)(warp - 4) * 4096;
        bool store_pending = false, ok = true;
        for (int j = 0; ok && sched.next(dw, item); ++j) {
            const LbItem it = lb_item<BN>(p, dw, item);
            const int acc = j & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&sh->acc_full[acc], (j >> 1) & 1, kDevTimeoutSoftmax, abort, p.status));
            if (!ok) break;
            tc_fence_after();
            const int m = it.m0 + 32 * wq;  // first row of this warp's 32
#pragma unroll 1
            for (int cc = CPW * chalf; cc < CPW * chalf + CPW; ++cc) {
                uint32_t v[32];
                tmem_ld32(tmem + lane_off + acc * BN + 32 * cc, v);
                tmem_wait_ld();
                if (cc == CPW * chalf + CPW - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->acc_empty[acc]);
                }
                const int k = it.k0 + 32 * cc;
                if (!dw && p.relu && m + lane < p.T) {
                    // x [row, k ..]: rows layout (K columns) or heads (64)
                    const size_t row = (size_t)it.b * p.T + m + lane;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int kq = k + 8 * q;  // K is a multiple of 8
                        const size_t at = p.heads ? (((size_t)it.b * (p.K >> 6) + (kq >> 6)) * p.T + m + lane) * 64 + (kq & 63)
                                                  : row * p.K + kq;
                        if (kq >= p.K || !TXL_BOUNDS(at + 8 <= (size_t)p.B * p.T * p.K, 802, at)) continue;
                        const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(p.x + at));
                        const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&w4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = __bfloat1622float2(h2[e]);
                            if (!(f.x > 0.f)) v[8 * q + 2 * e] = 0;
                            if (!(f.y > 0.f)) v[8 * q + 2 * e + 1] = 0;
                        }
                    }
                }
                // a staged slice is 32 rows of 128 bytes (64 bf16 or 32 fp32 columns), its
                // 16-byte chunk c at c ^ (row & 7): the swizzle of the store's map
                if (dw || (cc & 1) == 0) {
                    if (store_pending) lb_wait_read();
                    store_pending = false;
                    __syncwarp();
                }
                if (dw) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        st_shared_v4(stg + lane * 128 + ((q ^ (lane & 7)) << 4), v[4 * q], v[4 * q + 1], v[4 * q + 2],
                                     v[4 * q + 3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c16 = 4 * (cc & 1) + q;
                        st_shared_v4(stg + lane * 128 + ((c16 ^ (lane & 7)) << 4),
                                     pack_bf16x2(__uint_as_float(v[8 * q + 0]), __uint_as_float(v[8 * q + 1])),
                                     pack_bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                                     pack_bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                                     pack_bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7])));
                    }
                }
                if (dw || (cc & 1)) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    const int k1 = dw ? k : k - 32;  // the slice's first column
                    if (lane == 0 && k1 < p.K && m < (dw ? p.N : p.T)) {
                        if (dw)
                            lb_store_3d(&maps.dw, stg, k1, m, it.split);
                        else
                            lb_store_4d(&maps.dx, stg, p.heads ? 0 : k1, m, p.heads ? k1 >> 6 : 0, it.b);
                        store_pending = true;
                    }
                }
            }
        }
        if (lane == 0) lb_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// dw and db from their parts, in the order of the splits.
__global__ void __launch_bounds__(256) linear_bwd_sum_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                             long long n4, int splits, const float* __restrict__ db_part,
                                                             float* __restrict__ db, int n_db) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i < n4) {
        const float4* q = reinterpret_cast<const float4*>(part) + i;
        float4 a = q[0];
        for (int s = 1; s < splits; ++s) {
            const float4 b = q[s * n4];
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        }
        reinterpret_cast<float4*>(dw)[i] = a;
    }
    if (i < n_db) {
        float a = db_part[i];
        for (int s = 1; s < splits; ++s) a += db_part[(size_t)s * n_db + i];
        db[i] = a;
    }
}

// ---------------------------------------------------------------- host side
namespace {

typedef CUresult (*LbEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

LbEncodeFn lb_encode_fn() {
    static LbEncodeFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<LbEncodeFn>(ptr);
        return static_cast<LbEncodeFn>(nullptr);
    }();
    return fn;
}

bool lb_encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
               const cuuint64_t* strides, const cuuint32_t* box) {
    LbEncodeFn fn = lb_encode_fn();
    if (!fn) return false;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(map, type, rank, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// How the call is cut: tile width, splits of dw's reduction, schedule.
struct LbPlan {
    int bn, splits, grid;
    LbParams p;
};

LbPlan lb_plan(int B, int T, int K, int N, int heads, bool want_dx, bool want_dw) {
    LbPlan pl;
    LbParams& p = pl.p;
    p = {};
    p.T = heads ? T : B * T;
    p.B = heads ? B : 1;
    p.K = K;
    p.N = N;
    p.heads = heads;
    p.n_nt = ceil_div(N, lb::BM);
    p.n_tt = ceil_div(p.T, lb::BM);
    p.t_steps = ceil_div(p.T, lb::BR);
    p.n_steps = ceil_div(N, lb::BR);
    const int sms = current_sm_count();
    const long long total = (long long)p.B * p.t_steps;
    // 256 columns per tile unless that leaves SMs without a tile
    const auto tiles = [&](int bn) {
        const long long kt = ceil_div(K, bn);
        return (want_dx ? (long long)p.B * p.n_tt * kt : 0) + (want_dw ? (long long)p.n_nt * kt : 0);
    };
    pl.bn = tiles(256) >= sms ? 256 : 128;
    p.n_kt = ceil_div(K, pl.bn);
    p.n_d = want_dx ? (int)((long long)p.B * p.n_tt * p.n_kt) : 0;
    // Splits: the CTA with most to do has max(whole dw items, an even share + half a
    // dx tile) steps; a split costs its part's write and read (about 1.7 MB per
    // 0.34 us step) and the second launch.
    const int wt = p.n_nt * p.n_kt;
    double best = 0;
    p.splits = 1;
    for (int s = 1; want_dw && s <= 32 && s <= total; ++s) {
        const double a = (double)ceil_div(total, s);
        const double share = (wt * (double)total + (double)p.n_d * p.n_steps) / sms + (p.n_d ? p.n_steps * 0.5 : 0.0);
        double cost = (double)ceil_div((long long)wt * s, sms) * a;
        if (cost < share) cost = share;
        if (s > 1) cost += 6.0 + (double)s * N * K * 8.0 / 1.7e6;
        if (s == 1 || cost < best) {
            best = cost;
            p.splits = s;
        }
    }
    p.n_w = want_dw ? wt * p.splits : 0;
    const long long items = (long long)p.n_w + p.n_d;
    pl.grid = (int)(items < sms ? items : sms);
    p.heavy = p.n_w % pl.grid;
    p.extra = p.heavy ? (int)(total / p.splits / p.n_steps) : 0;
    return pl;
}

template <int BN>
cudaError_t lb_launch(const LbMaps& maps, const LbPlan& pl, cudaStream_t stream) {
    using C = lb::Cfg<BN>;
    static PerDeviceOnce attrs;
    const cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(linear_bwd_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.grid);
    cfg.blockDim = dim3(lb::NTHREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_bwd_kernel<BN>, maps, pl.p);
}

size_t part_bytes(int N, int K, int splits) {
    return splits > 1 ? ((size_t)splits * N * K * 4 + 255) / 256 * 256 : 0;
}

}  // namespace

size_t linear_bwd_workspace_bytes(int heads, int B, int T, int K, int N, bool want_dx, bool want_dw) {
    if (!want_dw) return 0;
    const LbPlan pl = lb_plan(B, T, K, N, heads, want_dx, true);
    return pl.p.splits > 1 ? part_bytes(N, K, pl.p.splits) + (size_t)pl.p.splits * N * 4 : 0;
}

cudaError_t launch_linear_bwd(const void* dy, const void* x, int heads, int B, int T, int K, const void* w, int N,
                              int relu, void* dx, float* dw, float* db, void* workspace, int* status,
                              cudaStream_t stream) {
    LbPlan pl = lb_plan(B, T, K, N, heads, dx != nullptr, dw != nullptr);
    LbParams& p = pl.p;
    p.relu = relu;
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.status = status;
    p.want_db = db != nullptr;
    const bool split = p.splits > 1;
    float* part = split ? static_cast<float*>(workspace) : dw;
    float* db_part = split ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part_bytes(N, K, p.splits)) : db;
    p.db = db_part;
    LbMaps maps;
    const cuuint64_t Tt = p.T, Bb = p.B, Kk = K, Nn = N;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    {
        const cuuint64_t dims[3] = {Nn, Tt, Bb}, strides[2] = {Nn * 2, Tt * Nn * 2};
        const cuuint32_t box[3] = {64, 64, 1};
        if (!lb_encode(&maps.dy, bf, dy, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t dims[2] = {Kk, Nn}, strides[1] = {Kk * 2};
        const cuuint32_t box[2] = {64, 64};
        if (!lb_encode(&maps.w, bf, w, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t rows_dims[4] = {Kk, Tt, 1, 1}, rows_str[3] = {Kk * 2, Tt * Kk * 2, Tt * Kk * 2};
        const cuuint64_t heads_dims[4] = {64, Tt, Kk / 64, Bb}, heads_str[3] = {128, Tt * 128, Tt * Kk * 2};
        const cuuint32_t box[4] = {64, 64, 1, 1}, out_box[4] = {64, 32, 1, 1};
        if (!lb_encode(&maps.x, bf, x, 4, heads ? heads_dims : rows_dims, heads ? heads_str : rows_str, box))
            return cudaErrorInvalidValue;
        if (!lb_encode(&maps.dx, bf, dx ? dx : x, 4, heads ? heads_dims : rows_dims, heads ? heads_str : rows_str, out_box))
            return cudaErrorInvalidValue;
    }
    if (dw) {
        const cuuint64_t dims[3] = {Kk, Nn, (cuuint64_t)p.splits}, strides[2] = {Kk * 4, Nn * Kk * 4};
        const cuuint32_t box[3] = {32, 32, 1};
        if (!lb_encode(&maps.dw, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, part, 3, dims, strides, box)) return cudaErrorInvalidValue;
    } else {
        maps.dw = maps.dx;
    }
    cudaError_t e = pl.bn == 256 ? lb_launch<256>(maps, pl, stream) : lb_launch<128>(maps, pl, stream);
    if (e != cudaSuccess || !split) return e;
    const long long n4 = (long long)N * K / 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n4 + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_bwd_sum_kernel, (const float*)part, dw, n4, p.splits, (const float*)db_part, db,
                              db ? N : 0);
}

TXL_BOUNDS_READER(bounds_word_linear_bwd)

}  // namespace txl
