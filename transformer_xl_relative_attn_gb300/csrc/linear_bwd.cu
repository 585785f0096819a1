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
// The ReLU mask is a factor of the epilogue of dx, read from x before the tile's
// MMAs end.  db is summed by two warps of every CTA that have no part in the products,
// from dy in global memory (L2 mostly: the products read it at the same time).
//
// dw has few tiles and a long reduction (base512's second feed-forward layer: 32
// tiles over 11264 rows), so its rows are split over several CTAs, each writing an
// fp32 partial tile to the workspace; a second launch adds the parts, and db's, in a
// fixed order (the same inputs give the same bits).  The tensor core cuts off what it
// adds to an accumulator (1.7e-8 of the result per MMA on random data, measured), so
// a dw accumulator takes 1024 rows at a time and the epilogue adds these in registers:
// at 6144 rows the error went from 3.3e-6 to below that of an fp32 product.
//
// A TMA instruction costs its issuing thread some 100 cycles whatever it loads, and an
// L2 miss far more: a stage of 48 KB is two instructions where the widths are
// multiples of 64 (boxes of several 64-column slices), six otherwise.
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
constexpr int BR = 64;   // reduction per stage
constexpr int CHAIN = 16;  // stages that one dw accumulator takes
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
    int k64, n64;          // K, N are multiples of 64: boxes of several slices
    int db_rows;           // parts of db (row ranges); 0: no db
    const __nv_bfloat16* x;
    const __nv_bfloat16* dy;
    float* db;             // [db_rows, N]
    int* status;
};

struct LbMaps {
    CUtensorMap dy;   // (column, row, batch row), boxes of 64 x 128: dx's first operand
    CUtensorMap dyc;  // dw's: (element, row, 64-column slice, batch row), boxes of two slices of 64 rows;
                      // N not a multiple of 64: one slice of N, boxes of 64 x 64
    CUtensorMap w;    // (element, row, slice), boxes of BN / 64 slices of 64 rows; K not a multiple of 64: one slice
    CUtensorMap x;    // the same, with the batch row
    CUtensorMap dx;   // (element, row, slice, batch row), boxes of 32 rows; rows layout: one slice of K
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

__device__ __forceinline__ void lb_load_4d(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                           int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
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
// tmem_ld32 for 16 columns (the running sums leave no registers for 32).
__device__ __forceinline__ void lb_tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
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
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], 8);
        }
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.dy);
        tma_prefetch_desc(&maps.dyc);
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
                int b = dw ? it.s0 / p.t_steps : it.b;
                int r = (dw ? it.s0 - b * p.t_steps : it.s0) * BR;  // row of dy and x, or column of dy and row of w
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
                    uint8_t* bt = smem + C::OFF_B + s * SZ_B;
                    if (dw) {
                        if (p.n64) {
                            lb_load_4d(a, &maps.dyc, bar, 0, r, it.m0 >> 6, b);
                        } else {
                            lb_load_4d(a, &maps.dyc, bar, it.m0, r, 0, b);
                            lb_load_4d(a + SZ_BOX, &maps.dyc, bar, it.m0 + 64, r, 0, b);
                        }
                        if (p.k64) {
                            lb_load_4d(bt, &maps.x, bar, 0, r, it.k0 >> 6, b);
                        } else {
#pragma unroll
                            for (int j = 0; j < BN / 64; ++j)
                                lb_load_4d(bt + j * SZ_BOX, &maps.x, bar, it.k0 + 64 * j, r, 0, b);
                        }
                        r += BR;
                        if (r >= p.T) r = 0, ++b;
                    } else {
                        tma_load_3d(a, &maps.dy, bar, r, it.m0, b);
                        if (p.k64) {
                            tma_load_3d(bt, &maps.w, bar, 0, r, it.k0 >> 6);
                        } else {
#pragma unroll
                            for (int j = 0; j < BN / 64; ++j)
                                tma_load_3d(bt + j * SZ_BOX, &maps.w, bar, it.k0 + 64 * j, r, 0);
                        }
                        r += BR;
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
        int c = 0, j = 0;  // stages consumed, accumulators filled
        while (ok && sched.next(dw, item)) {
            const LbItem it = lb_item<BN>(p, dw, item);
            int st = it.s0;
            do {
                const int first = st, last = dw ? min(it.s1, st + CHAIN) : it.s1;
                const int acc = j & 1;
                if (j >= 2 && !wait(&sh->acc_empty[acc], ((j >> 1) - 1) & 1)) break;
                tc_fence_after();
                const uint32_t d_acc = tmem + acc * BN;
                for (; st < last; ++st, ++c) {
                    const int s = c % STAGES;
                    if (!wait(&sh->full[s], (c / STAGES) & 1)) break;
                    tc_fence_after();
                    const uint64_t bd = dB0 + s * (SZ_B >> 4);
                    if (dw) {
                        const uint64_t a = dAm + s * (SZ_A >> 4);
#pragma unroll
                        for (int kk = 0; kk < BR / 16; ++kk)
                            mma_ss_elect(d_acc, a + 128 * kk, bd + 128 * kk, C::IDESC_DW,
                                         (st > first || kk > 0) ? 1u : 0u, leader);
                    } else {
                        const uint64_t a = dA0 + s * (SZ_A >> 4);
#pragma unroll
                        for (int kk = 0; kk < BR / 16; ++kk)
                            mma_ss_elect(d_acc, a + 2 * kk, bd + 128 * kk, C::IDESC_DX,
                                         (st > first || kk > 0) ? 1u : 0u, leader);
                    }
                    if (leader) mma_commit(&sh->empty[s]);
                }
                if (!ok) break;
                if (leader) mma_commit(&sh->acc_full[acc]);
                ++j;
            } while (st < it.s1);
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
        // A warp adds 256 columns (8 per lane) over one of db_rows ranges of rows.
        if (p.db_rows) {
            const int groups = (p.N + 255) >> 8;
            const long long rows = (long long)p.B * p.T;
            for (int u = blockIdx.x * 2 + warp - 2; u < groups * p.db_rows; u += 2 * gridDim.x) {
                const int part = u / groups, n = (u - part * groups) * 256 + lane * 8;  // N is a multiple of 8
                if (n >= p.N) continue;
                const long long r0 = rows * part / p.db_rows, r1 = rows * (part + 1) / p.db_rows;
                float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
                for (long long r = r0; r < r1; ++r) {
                    if (!TXL_BOUNDS(r < rows && n + 8 <= p.N, 801, r * p.N + n)) continue;
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.dy + r * p.N + n));
                    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = __bfloat1622float2(h[e]);
                        a[2 * e] += f.x;
                        a[2 * e + 1] += f.y;
                    }
                }
                float4* to = reinterpret_cast<float4*>(p.db + (size_t)part * p.N + n);
                to[0] = make_float4(a[0], a[1], a[2], a[3]);
                to[1] = make_float4(a[4], a[5], a[6], a[7]);
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
        int j = 0;
        auto wait_acc = [&](int acc) {
            ok = __all_sync(0xffffffffu, mbar_wait(&sh->acc_full[acc], (j >> 1) & 1, kDevTimeoutSoftmax, abort, p.status));
            tc_fence_after();
            return ok;
        };
        auto free_acc = [&](int acc) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->acc_empty[acc]);
        };
        // the staged slice may be overwritten: its last store has read it
        auto stage_free = [&] {
            if (store_pending) lb_wait_read();
            store_pending = false;
            __syncwarp();
        };
        // A staged slice is 32 rows of 128 bytes (64 bf16 or 32 fp32 columns), its
        // 16-byte chunk c at c ^ (row & 7): the swizzle of the store's map.
        auto chunk_at = [&](int c16) { return stg + lane * 128 + ((c16 ^ (lane & 7)) << 4); };
        while (ok && sched.next(dw, item)) {
            const LbItem it = lb_item<BN>(p, dw, item);
            const int m = it.m0 + 32 * wq;  // first row of this warp's 32
            if (dw) {
                float sum[CPW][32];
#pragma unroll
                for (int cc = 0; cc < CPW; ++cc)
#pragma unroll
                    for (int x = 0; x < 32; ++x) sum[cc][x] = 0.f;
#pragma unroll 1
                for (int st = it.s0; st < it.s1; st += CHAIN, ++j) {
                    const int acc = j & 1;
                    if (!wait_acc(acc)) break;
#pragma unroll
                    for (int h = 0; h < 2 * CPW; ++h) {
                        uint32_t v[16];
                        lb_tmem_ld16(tmem + lane_off + acc * BN + 32 * CPW * chalf + 16 * h, v);
                        tmem_wait_ld();
                        if (h == 2 * CPW - 1) free_acc(acc);
#pragma unroll
                        for (int x = 0; x < 16; ++x) sum[h >> 1][16 * (h & 1) + x] += __uint_as_float(v[x]);
                    }
                }
                if (!ok) break;
#pragma unroll
                for (int cc = 0; cc < CPW; ++cc) {
                    const int k = it.k0 + 32 * (CPW * chalf + cc);
                    stage_free();
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        st_shared_v4(chunk_at(q), __float_as_uint(sum[cc][4 * q]), __float_as_uint(sum[cc][4 * q + 1]),
                                     __float_as_uint(sum[cc][4 * q + 2]), __float_as_uint(sum[cc][4 * q + 3]));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && k < p.K && m < p.N) {
                        lb_store_3d(&maps.dw, stg, k, m, it.split);
                        store_pending = true;
                    }
                }
                continue;
            }
            // The ReLU mask of the warp's 32 rows, fetched while the MMAs run: x comes in as
            // whole lines (a lane per 8 columns), a byte per lane goes through the staging
            // area, and each thread takes its row's: bit x of keep[cc] for column x of chunk
            // cc.  (With each thread reading its own row of x, one line per lane and load,
            // the epilogue took longer than the tile: 44 us instead of 22 without the mask.)
            uint32_t keep[CPW];
            if (p.relu) {
                constexpr int G = 4 * CPW, ROWS = 32 / G;  // 8-column groups of a row; rows per load
                stage_free();
                const int g = lane % G, kq = it.k0 + 32 * CPW * chalf + 8 * g;  // K is a multiple of 8
                constexpr int BATCH = 8;  // loads in flight per thread
#pragma unroll 1
                for (int i0 = 0; i0 < 32 / ROWS; i0 += BATCH) {
                    uint4 w4[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int row = ROWS * (i0 + i) + lane / G;
                        const size_t at = p.heads
                                              ? (((size_t)it.b * (p.K >> 6) + (kq >> 6)) * p.T + m + row) * 64 + (kq & 63)
                                              : ((size_t)it.b * p.T + m + row) * p.K + kq;
                        w4[i] = make_uint4(0, 0, 0, 0);
                        if (m + row < p.T && kq < p.K && TXL_BOUNDS(at + 8 <= (size_t)p.B * p.T * p.K, 802, at))
                            w4[i] = __ldg(reinterpret_cast<const uint4*>(p.x + at));
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&w4[i]);
                        uint32_t bits = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = __bfloat1622float2(h2[e]);
                            bits |= (f.x > 0.f ? 1u : 0u) << (2 * e);
                            bits |= (f.y > 0.f ? 1u : 0u) << (2 * e + 1);
                        }
                        const int row = ROWS * (i0 + i) + lane / G;
                        asm volatile("st.shared.u8 [%0], %1;" ::"r"(stg + row * G + g), "r"(bits) : "memory");
                    }
                }
                __syncwarp();
#pragma unroll
                for (int cc = 0; cc < CPW; ++cc)
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(keep[cc]) : "r"(stg + lane * G + 4 * cc) : "memory");
                __syncwarp();
            }
            const int acc = j & 1;
            if (!wait_acc(acc)) break;
#pragma unroll
            for (int cc = 0; cc < CPW; ++cc) {
                uint32_t v[32];
                tmem_ld32(tmem + lane_off + acc * BN + 32 * (CPW * chalf + cc), v);
                tmem_wait_ld();
                if (cc == CPW - 1) free_acc(acc);
                if (p.relu) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = (keep[cc] >> x) & 1u ? v[x] : 0u;
                }
                if ((cc & 1) == 0) stage_free();
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_shared_v4(chunk_at(4 * (cc & 1) + q),
                                 pack_bf16x2(__uint_as_float(v[8 * q + 0]), __uint_as_float(v[8 * q + 1])),
                                 pack_bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                                 pack_bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                                 pack_bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7])));
                if (cc & 1) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    const int k = it.k0 + 32 * (CPW * chalf + cc - 1);  // the slice's first column
                    if (lane == 0 && k < p.K && m < p.T) {
                        lb_store_4d(&maps.dx, stg, p.heads ? 0 : k, m, p.heads ? k >> 6 : 0, it.b);
                        store_pending = true;
                    }
                }
            }
            ++j;
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

// dw from its parts, in the order of the splits (the first n_dw CTAs), and db from
// its row ranges (32 columns per CTA, 8 threads on each).
__global__ void __launch_bounds__(256) linear_bwd_sum_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                             long long n4, int splits, int n_dw,
                                                             const float* __restrict__ db_part, float* __restrict__ db,
                                                             int N, int db_rows) {
    __shared__ float sh[8][33];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x < n_dw) {
        const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
        if (i >= n4) return;
        const float4* q = reinterpret_cast<const float4*>(part) + i;
        float4 a = q[0];
#pragma unroll 4
        for (int s = 1; s < splits; ++s) {
            const float4 b = q[s * n4];
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        }
        reinterpret_cast<float4*>(dw)[i] = a;
        return;
    }
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int n = ((int)blockIdx.x - n_dw) * 32 + lane;
    float a = 0.f;
    if (n < N) {
#pragma unroll 8
        for (int r = w; r < db_rows; r += 8) a += db_part[(size_t)r * N + n];
    }
    sh[w][lane] = a;
    __syncthreads();
    if (w == 0 && n < N) {
#pragma unroll
        for (int k = 1; k < 8; ++k) a += sh[k][lane];
        db[n] = a;
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
    int bn, grid;
    LbParams p;
};

// Microseconds that a stage takes by tile width, and that the parts of one more split
// cost per byte of dw (write and read, through L2); measured on base512's and large384's
// layers.
constexpr double kStep256 = 0.40, kStep128 = 0.25, kSplitPerByte = 0.4e-6, kSumLaunch = 2.0;

LbPlan lb_plan(int B, int T, int K, int N, int heads, bool want_dx, bool want_dw) {
    LbPlan pl;
    LbParams& p = pl.p;
    p = {};
    p.T = heads ? T : B * T;
    p.B = heads ? B : 1;
    p.K = K;
    p.N = N;
    p.heads = heads;
    p.k64 = K % 64 == 0;
    p.n64 = N % 64 == 0;
    p.n_nt = ceil_div(N, lb::BM);
    p.n_tt = ceil_div(p.T, lb::BM);
    p.t_steps = ceil_div(p.T, lb::BR);
    p.n_steps = ceil_div(N, lb::BR);
    const int sms = current_sm_count();
    const long long total = (long long)p.B * p.t_steps;
    // The tile width and the splits with the least time by this model: the CTA with
    // most to do has all its dw items, or an even share of all stages and half a dx
    // tile; splits add their parts' traffic and the second launch.
    double best = 0;
    pl.bn = 0;
    for (int bn : {256, 128}) {
        const double step = bn == 256 ? kStep256 : kStep128;
        const long long kt = ceil_div(K, bn), n_d = want_dx ? (long long)p.B * p.n_tt * kt : 0, wt = p.n_nt * kt;
        for (int s = 1; s <= (want_dw ? 32 : 1) && s <= total; ++s) {
            const double even = ((want_dw ? wt * (double)total : 0.0) + (double)n_d * p.n_steps) / sms;
            double steps = even + (n_d ? p.n_steps * 0.5 : 0.0);
            if (n_d && steps < p.n_steps) steps = p.n_steps;
            if (want_dw) {
                const double most = (double)((wt * s + sms - 1) / sms) * ceil_div(total, s);
                if (steps < most) steps = most;
            }
            const double cost = steps * step + (s > 1 ? kSumLaunch + s * (N * 4.0 * K) * kSplitPerByte : 0.0);
            if (!pl.bn || cost < best) {
                best = cost;
                pl.bn = bn;
                p.splits = s;
            }
        }
    }
    p.n_kt = ceil_div(K, pl.bn);
    p.n_d = want_dx ? (int)((long long)p.B * p.n_tt * p.n_kt) : 0;
    p.n_w = want_dw ? p.n_nt * p.n_kt * p.splits : 0;
    const long long items = (long long)p.n_w + p.n_d;
    pl.grid = (int)(items < sms ? items : sms);
    p.heavy = p.n_w % pl.grid;
    p.extra = p.heavy ? (int)(total / p.splits / p.n_steps) : 0;
    // row ranges of db: as many as give each of the two summing warps per CTA one, of 16
    // rows at least
    const long long rows = (long long)B * T, groups = (N + 255) / 256;
    long long parts = 2ll * pl.grid / groups;
    if (parts > rows / 16) parts = rows / 16;
    p.db_rows = parts < 1 ? 1 : (int)parts;
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

size_t part_bytes(const LbPlan& pl) {
    return pl.p.splits > 1 ? ((size_t)pl.p.splits * pl.p.N * pl.p.K * 4 + 255) / 256 * 256 : 0;
}

cudaError_t lb_sum(const float* part, float* dw, int splits, const float* db_part, float* db, int N, int K, int db_rows,
                   cudaStream_t stream) {
    const long long n4 = splits > 1 ? (long long)N * K / 4 : 0;
    const long long n_dw = (n4 + 255) / 256, ctas = n_dw + (db ? (N + 31) / 32 : 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_bwd_sum_kernel, part, dw, n4, splits, (int)n_dw, db_part, db, N, db_rows);
}

}  // namespace

size_t linear_bwd_workspace_bytes(int heads, int B, int T, int K, int N, bool want_dx, bool want_dw, bool want_db) {
    if (!want_dw) return 0;
    const LbPlan pl = lb_plan(B, T, K, N, heads, want_dx, true);
    return part_bytes(pl) + (want_db ? (size_t)pl.p.db_rows * N * 4 : 0);
}

cudaError_t launch_linear_bwd(const void* dy, const void* x, int heads, int B, int T, int K, const void* w, int N,
                              int relu, void* dx, float* dw, float* db, void* workspace, int* status,
                              cudaStream_t stream) {
    LbPlan pl = lb_plan(B, T, K, N, heads, dx != nullptr, dw != nullptr);
    LbParams& p = pl.p;
    p.relu = relu;
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.dy = static_cast<const __nv_bfloat16*>(dy);
    p.status = status;
    if (!db) p.db_rows = 0;
    const bool split = p.splits > 1;
    float* part = split ? static_cast<float*>(workspace) : dw;
    p.db = db ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part_bytes(pl)) : nullptr;
    LbMaps maps;
    const cuuint64_t Tt = p.T, Bb = p.B, Kk = K, Nn = N;
    const cuuint32_t slices = pl.bn / 64;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    {
        const cuuint64_t dims[3] = {Nn, Tt, Bb}, strides[2] = {Nn * 2, Tt * Nn * 2};
        const cuuint32_t box[3] = {64, 128, 1};
        if (!lb_encode(&maps.dy, bf, dy, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t cut[4] = {64, Tt, Nn / 64, Bb}, cut_str[3] = {Nn * 2, 128, Tt * Nn * 2};
        const cuuint64_t one[4] = {Nn, Tt, 1, Bb}, one_str[3] = {Nn * 2, Tt * Nn * 2, Tt * Nn * 2};
        const cuuint32_t cut_box[4] = {64, 64, 2, 1}, one_box[4] = {64, 64, 1, 1};
        if (!lb_encode(&maps.dyc, bf, dy, 4, p.n64 ? cut : one, p.n64 ? cut_str : one_str, p.n64 ? cut_box : one_box))
            return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t cut[3] = {64, Nn, Kk / 64}, cut_str[2] = {Kk * 2, 128};
        const cuuint64_t one[3] = {Kk, Nn, 1}, one_str[2] = {Kk * 2, Nn * Kk * 2};
        const cuuint32_t cut_box[3] = {64, 64, slices}, one_box[3] = {64, 64, 1};
        if (!lb_encode(&maps.w, bf, w, 3, p.k64 ? cut : one, p.k64 ? cut_str : one_str, p.k64 ? cut_box : one_box))
            return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t rows_dims[4] = {Kk, Tt, 1, 1}, rows_str[3] = {Kk * 2, Tt * Kk * 2, Tt * Kk * 2};
        const cuuint64_t cut_dims[4] = {64, Tt, Kk / 64, Bb};
        const cuuint64_t heads_str[3] = {128, Tt * 128, Tt * Kk * 2}, cut_str[3] = {Kk * 2, 128, Tt * Kk * 2};
        const cuuint32_t box[4] = {64, 64, p.k64 ? slices : 1, 1}, out_box[4] = {64, 32, 1, 1};
        if (!lb_encode(&maps.x, bf, x, 4, p.k64 ? cut_dims : rows_dims, heads ? heads_str : p.k64 ? cut_str : rows_str, box))
            return cudaErrorInvalidValue;
        if (!lb_encode(&maps.dx, bf, dx ? dx : x, 4, heads ? cut_dims : rows_dims, heads ? heads_str : rows_str, out_box))
            return cudaErrorInvalidValue;
    }
    if (dw) {
        const cuuint64_t dims[3] = {Kk, Nn, (cuuint64_t)p.splits}, strides[2] = {Kk * 4, Nn * Kk * 4};
        const cuuint32_t box[3] = {32, 32, 1};
        if (!lb_encode(&maps.dw, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, part, 3, dims, strides, box)) return cudaErrorInvalidValue;
    } else {
        maps.dw = maps.dx;
    }
    const cudaError_t e = pl.bn == 256 ? lb_launch<256>(maps, pl, stream) : lb_launch<128>(maps, pl, stream);
    if (e != cudaSuccess || (!split && !db)) return e;
    return lb_sum(part, dw, p.splits, p.db, db, N, K, p.db_rows, stream);
}

TXL_BOUNDS_READER(bounds_word_linear_bwd)

}  // namespace txl
