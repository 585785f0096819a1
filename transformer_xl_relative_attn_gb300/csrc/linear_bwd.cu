// Gradients of a Linear layer out = x W^T + b on the sm_103a tensor cores, bf16
// in, fp32 accumulation:
//
//   dx = dy W          [T, K] = [T, N] [N, K]   bf16 (where x came out of a ReLU: 0 unless x > 0)
//   dw = dy^T x        [N, K] = [N, T] [T, K]   fp32
//   db = sum over rows of dy                    fp32
//
// One persistent launch holds both products.  In both the second operand (W for
// dx, x for dw) is read with K contiguous and its other axis reduced over (MN-major
// for the tensor core), so one pipeline serves both: 64-row boxes of 64 columns land
// in shared memory the same way, and only dy's view differs (K-major with the rows as M
// for dx, MN-major with the columns as M for dw).  Nothing is transposed in memory.
// Two CTAs of a cluster share a 256 x 256 tile (cta_group::2), or one CTA takes 128 x
// 128 where the larger tiles would leave SMs idle.
//
// The ReLU mask is applied in the epilogue of dx (by bits: a masked element is 0 also where
// the product is not finite), read from x before the tile's MMAs end.  db is summed by two warps of every CTA that have no part in the products,
// from dy in global memory (L2 mostly: the products read it at the same time).
//
// dw has few tiles and a long reduction (base512's second feed-forward layer: 16
// tiles over 11264 rows), so its rows are split over several pairs, each writing an
// fp32 partial tile to the workspace; a second launch adds the parts, and db's, in a
// fixed order (the same inputs give the same bits).  The tensor core cuts off what it
// adds to an accumulator (1.7e-8 of the result per MMA on random data, measured), so
// a dw accumulator takes 1024 rows at a time and the epilogue adds these in registers:
// at 6144 rows the error went from 3.3e-6 to 1.0e-6 (an fp32 library product's: 0.8e-6).
// dx, which is rounded to bf16, takes its whole reduction in one accumulator (2048
// columns: 2e-6 against the rounding's 2e-3).
//
// TMA is what the loads need all of: an instruction costs its issuing thread some
// 100 cycles whatever it loads, so a stage of 32 KB is two instructions where the widths
// are multiples of 64 (boxes of two 64-column slices), up to four otherwise; and results
// leave through plain stores of whole lines (a warp turns its rows in shared memory)
// rather than TMA stores, which held the loads up (base512's second feed-forward layer
// without its mask: 22.5 us with them).
//
// Roles (384 threads, one CTA per SM): warp 0 lane 0 issues the TMA loads, warp 1
// the MMAs, warps 2-3 the column sums, warps 4-11 the epilogue; two accumulators
// let an epilogue overlap the next tile's MMAs.  Every wait is bounded (1 s) and
// reports through the device status word.  Rows, N and K need not fill tiles: TMA
// fills with zeros behind the ends.
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "linear_bwd.h"
#include "pair_mma.cuh"
#include "txl_device.cuh"

namespace txl {

namespace lb {
constexpr int BM = 128;  // rows of a CTA's accumulator
constexpr int BR = 64;   // reduction per stage
constexpr int CHAIN = 16;  // stages that one dw accumulator takes
constexpr int DB_CHAIN = 1024;  // rows that one accumulator of db takes
constexpr int NTHREADS = 384;
constexpr uint32_t SZ_BOX = 64 * 64 * 2;  // 64 rows of 64 bf16: 8 KB
constexpr uint32_t SZ_A = 2 * SZ_BOX;     // 128 of M
constexpr uint32_t SZ_B = 2 * SZ_BOX;     // 128 of N: of a pair's 256, each CTA holds half
constexpr int STAGES = 6;
constexpr uint32_t SZ_SLOT = 4096;        // a staged slice: 32 rows of 128 bytes
constexpr uint32_t OFF_A = 0;
constexpr uint32_t OFF_B = STAGES * SZ_A;
constexpr uint32_t OFF_STG = OFF_B + STAGES * SZ_B;  // a slot per epilogue warp
constexpr uint32_t OFF_BAR = OFF_STG + 8 * SZ_SLOT;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 512 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget of one sm_103a CTA");

// Two CTAs of a cluster work one 256 x 256 tile (PAIR), or one CTA a 128 x 128 tile.
// Either way a CTA loads 128 + 128 columns per stage; as a pair the tensor cores read
// each other's half of the second operand, and do twice the work on the same loads.
template <bool PAIR>
struct Cfg {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TM = BM * CTAS;  // tile
    static constexpr int BN = PAIR ? 256 : 128;
    static constexpr uint32_t TMEM_COLS = 2 * BN;
    static constexpr uint32_t IDESC_DX = idesc_bf16_f32(TM, BN, 1, 0);
    static constexpr uint32_t IDESC_DW = idesc_bf16_f32(TM, BN, 1, 1);
};
}  // namespace lb

struct LbMaps {
    CUtensorMap dy;   // (column, row, batch row), boxes of 64 x 128: dx's first operand
    CUtensorMap dyc;  // dw's: (element, row, 64-column slice, batch row), boxes of two slices of 64 rows;
                      // N not a multiple of 64: one slice of N, boxes of 64 x 64
    CUtensorMap w;    // (element, row, slice), boxes of two slices of 64 rows; K not a multiple of 64: one slice
    CUtensorMap x;    // the same, with the batch row
};

struct LbShared {
    uint64_t full[lb::STAGES];  // a pair's: those of its first CTA
    uint64_t empty[lb::STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];  // a pair's: those of its first CTA
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// The items of one CTA (or pair), the same sequence for every role.  dw items are dealt in
// turn first (the long ones).  Where they do not divide evenly, the CTAs from
// `heavy` on have one less: they take `extra` dx tiles each ahead of the rest, which
// is then dealt in turn from the last CTA down.
struct LbSchedule {
    const LbParams& p;
    int c, g, light, head;  // CTA, CTAs, CTAs with one dw item less, dx tiles dealt to them ahead
    int w, e, d;            // next dw item, next extra tile, next dx tile
    __device__ __forceinline__ LbSchedule(const LbParams& p_, int ctas) : p(p_) {
        c = blockIdx.x / ctas;
        g = gridDim.x / ctas;
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

template <bool PAIR>
__device__ __forceinline__ LbItem lb_item(const LbParams& p, bool dw, int i) {
    using C = lb::Cfg<PAIR>;
    LbItem it;
    it.k0 = (i % p.n_kt) * C::BN;
    int rest = i / p.n_kt;
    if (dw) {
        it.m0 = (rest % p.n_nt) * C::TM;
        it.split = rest / p.n_nt;
        it.b = 0;
        const long long total = (long long)p.B * p.t_steps;
        it.s0 = (int)(total * it.split / p.splits);
        it.s1 = (int)(total * (it.split + 1) / p.splits);
    } else {
        it.m0 = (rest % p.n_tt) * C::TM;
        it.b = rest / p.n_tt;
        it.split = 0;
        it.s0 = 0;
        it.s1 = p.n_steps;
    }
    return it;
}

namespace {

// tmem_ld32 for 16 columns (the running sums leave no registers for 32).
__device__ __forceinline__ void lb_tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ uint4 lb_ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// 16 bytes that are read once, past L1: beside 230 KB of shared memory L1 is too small for
// the loads on their way to wait in (base512's second feed-forward layer 49.5 us through L1,
// 47.9 past it).
__device__ __forceinline__ uint4 lb_load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// Eight bf16 onto eight sums; eight sums to memory.
__device__ __forceinline__ void lb_add8(float (&a)[8], const uint4& v) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = __bfloat1622float2(h[e]);
        a[2 * e] += f.x;
        a[2 * e + 1] += f.y;
    }
}
__device__ __forceinline__ void lb_put8(float* p, const float (&a)[8]) {
    float4* to = reinterpret_cast<float4*>(p);
    to[0] = make_float4(a[0], a[1], a[2], a[3]);
    to[1] = make_float4(a[4], a[5], a[6], a[7]);
}

}  // namespace

template <bool PAIR, bool RELU>
__global__ void __launch_bounds__(lb::NTHREADS, 1)
linear_bwd_kernel(const __grid_constant__ LbMaps maps, const LbParams p) {
    using namespace lb;
    using C = Cfg<PAIR>;
    constexpr int BN = C::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    LbShared* sh = reinterpret_cast<LbShared*>(smem + OFF_BAR);
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
        tma_prefetch_desc(&maps.dy);
        tma_prefetch_desc(&maps.dyc);
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.x);
    }
    tc_fence_before();
    if (PAIR) __syncthreads();
    lb_sync<PAIR>();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = sh->tmem_base;
    volatile int* abort = &sh->abort;
    LbSchedule sched(p, C::CTAS);
    bool dw;
    int item;
    // Registers: the launch's 384 * 168 = 64512 as 128 * 80 + 256 * 208 (1024 to spare).  An
    // epilogue thread keeps 128 running sums of dw besides what it unpacks; a single spilled
    // register costs more than the split (with 230 KB of shared memory in use L1 holds little).
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 0) {
            // ---------------------------------------------------- TMA producer
            // A pair's full barriers are its first CTA's, which expects both CTAs' bytes; the
            // second's loads may land before it does (the barrier waits for the arrival).
            // One thread's instructions per stage bound the loads (at 870 cycles a stage took
            // longer than its MMAs), so what does not change is kept out of the loops.
            if (lane == 0) {
                bool ok = true;
                uint32_t s = 0, phase = 1;  // slot, parity of its empty barrier (a fresh one passes for 1)
                long long loads = 0;
                const uint32_t full0 = PAIR ? lb_mapa(&sh->full[0], 0) : smem_u32(&sh->full[0]);
                auto next_slot = [&](uint32_t& a, uint32_t& b, uint32_t& bar) {
                    if (!mbar_wait(&sh->empty[s], phase, kDevTimeoutProducer, abort, p.status)) return ok = false;
                    if (rank == 0) mbar_expect_tx(&sh->full[s], (SZ_A + SZ_B) * C::CTAS);
                    a = s_base + OFF_A + s * SZ_A;
                    b = s_base + OFF_B + s * SZ_B;
                    bar = full0 + 8 * s;
                    if (++s == STAGES) s = 0, phase ^= 1;
                    ++loads;
                    return true;
                };
                const bool n64 = p.n64, k64 = p.k64;
                while (ok && sched.next(dw, item)) {
                    const LbItem it = lb_item<PAIR>(p, dw, item);
                    const int m = it.m0 + BM * rank, k = it.k0 + 128 * rank;  // this CTA's share
                    uint32_t a, b, bar;
                    if (dw) {
                        const int m_el = n64 ? 0 : m, m_sl = n64 ? m >> 6 : 0;
                        const int k_el = k64 ? 0 : k, k_sl = k64 ? k >> 6 : 0;
                        int bt = it.s0 / p.t_steps, t = (it.s0 - bt * p.t_steps) * BR;
                        const int T = p.T;
                        for (int n = it.s1 - it.s0; n > 0 && next_slot(a, b, bar); --n) {
                            lb_load_4d<PAIR>(a, &maps.dyc, bar, m_el, t, m_sl, bt);
                            lb_load_4d<PAIR>(b, &maps.x, bar, k_el, t, k_sl, bt);
                            if (!n64) lb_load_4d<PAIR>(a + SZ_BOX, &maps.dyc, bar, m_el + 64, t, 0, bt);
                            if (!k64) lb_load_4d<PAIR>(b + SZ_BOX, &maps.x, bar, k_el + 64, t, 0, bt);
                            t += BR;
                            if (t >= T) t = 0, ++bt;
                        }
                    } else {
                        const int k_el = k64 ? 0 : k, k_sl = k64 ? k >> 6 : 0;
                        int r = 0;  // column of dy, row of w
                        for (int n = it.s1; n > 0 && next_slot(a, b, bar); --n) {
                            lb_load_3d<PAIR>(a, &maps.dy, bar, r, m, it.b);
                            lb_load_3d<PAIR>(b, &maps.w, bar, k_el, r, k_sl);
                            if (!k64) lb_load_3d<PAIR>(b + SZ_BOX, &maps.w, bar, k_el + 64, r, 0);
                            r += BR;
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
                const uint64_t dA0 = smem_desc_sw128(s_base + OFF_A, 16, 1024);      // K-major: rows of dy
                const uint64_t dAm = smem_desc_sw128(s_base + OFF_A, SZ_BOX, 1024);  // MN-major: columns of dy
                const uint64_t dB0 = smem_desc_sw128(s_base + OFF_B, SZ_BOX, 1024);  // MN-major
                uint32_t s = 0, phase = 0;  // slot, parity of its full barrier
                int j = 0;                  // accumulators filled
                while (ok && sched.next(dw, item)) {
                    const LbItem it = lb_item<PAIR>(p, dw, item);
                    // dx's first operand steps along its rows (32 bytes per MMA), dw's and every
                    // second one by 16 rows of 128 bytes
                    const uint64_t dA = dw ? dAm : dA0;
                    const uint64_t a_step = dw ? 128 : 2;
                    const uint32_t idesc = dw ? C::IDESC_DW : C::IDESC_DX;
                    int left = it.s1 - it.s0;
                    do {
                        const int acc = j & 1, n = dw ? min(left, CHAIN) : left;
                        if (j >= 2 && !wait(&sh->acc_empty[acc], ((j >> 1) - 1) & 1)) break;
                        tc_fence_after();
                        const uint32_t d_acc = tmem + acc * BN;
                        uint32_t more_than_first = 0;
                        for (int i = 0; i < n; ++i) {
                            if (!wait(&sh->full[s], phase)) break;
                            tc_fence_after();
                            const uint64_t ad = dA + s * (SZ_A >> 4), bd = dB0 + s * (SZ_B >> 4);
#pragma unroll
                            for (int kk = 0; kk < BR / 16; ++kk) {
                                lb_mma<PAIR>(d_acc, ad + a_step * kk, bd + 128 * kk, idesc, more_than_first, leader);
                                more_than_first = 1;
                            }
                            if (leader) lb_commit<PAIR>(&sh->empty[s]);
                            if (++s == STAGES) s = 0, phase ^= 1;
                        }
                        if (!ok) break;
                        if (leader) lb_commit<PAIR>(&sh->acc_full[acc]);
                        ++j;
                        left -= n;
                    } while (left > 0);
                }
                if (leader) lb_commit<PAIR>(&sh->drain);
                lb_wait_landed(&sh->drain, 0, p.status);
            }
            __syncwarp();
        } else {
            // ---------------------------------------------------- column sums of dy
            // Many rows: a warp adds 256 columns (8 per lane) over one of db_rows ranges of rows.
            // Few: 16 columns over all of them, 16 lanes on a column, with nothing left to add.
            if (p.db_rows) {
                const int groups = (p.N + 255) >> 8;
                const long long rows = (long long)p.B * p.T;
                for (int u = blockIdx.x * 2 + warp - 2; u < groups * p.db_rows; u += 2 * gridDim.x) {
                    const int part = u / groups, n = (u - part * groups) * 256 + lane * 8;  // N is a multiple of 8
                    if (n >= p.N) continue;
                    const long long r0 = rows * part / p.db_rows, r1 = rows * (part + 1) / p.db_rows;
                    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    // (a wide dy has few ranges, of many rows: a chain of additions ends after
                    // DB_CHAIN, so that its roundings stay those of DB_CHAIN + rows / DB_CHAIN)
                    for (long long r = r0; r < r1;) {
                        const long long end = min(r1, r + DB_CHAIN);
                        float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
                        for (; r < end; ++r) {
                            if (!TXL_BOUNDS(r < rows && n + 8 <= p.N, 801, r * p.N + n)) continue;
                            const uint4 v = lb_load_once(p.dy + r * p.N + n);
                            lb_add8(a, v);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum[e] += a[e];
                    }
                    if (TXL_BOUNDS(n + 8 <= p.N && part < p.db_rows, 805, n)) lb_put8(p.db + (size_t)part * p.N + n, sum);
                }
            } else if (p.db) {
                const int rows = p.B * p.T;
                for (int u = blockIdx.x * 2 + warp - 2; u * 16 < p.N; u += 2 * gridDim.x) {
                    const int n = u * 16 + (lane & 1) * 8, end = n < p.N ? rows : 0;
                    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int r = lane >> 1; r < end; r += 16 * 8) {  // 8 rows on their way at a time
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] = r + 16 * i < end && TXL_BOUNDS(n + 8 <= p.N, 804, n)
                                       ? lb_load_once(p.dy + (long long)(r + 16 * i) * p.N + n)
                                       : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 8; ++i) lb_add8(a, v[i]);
                    }
#pragma unroll
                    for (int o = 2; o < 32; o <<= 1)
#pragma unroll
                        for (int e = 0; e < 8; ++e) a[e] += __shfl_xor_sync(0xffffffffu, a[e], o);
                    if (lane < 2 && n < p.N && TXL_BOUNDS(n + 8 <= p.N, 806, n)) lb_put8(p.db + n, a);
                }
            }
        }
    } else {
        // ---------------------------------------------------- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int wq = warp & 3;
        const int chalf = (warp - 4) >> 2;
        constexpr int CPW = BN / 64;  // 32-column chunks per warp
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t stg = s_base + OFF_STG + (uint32_t)(warp - 4) * SZ_SLOT;
        const uint32_t acc_empty0 = PAIR ? lb_mapa(&sh->acc_empty[0], 0) : 0;
        bool ok = true;
        int j = 0;
        auto wait_acc = [&](int acc) {
            ok = __all_sync(0xffffffffu, mbar_wait(&sh->acc_full[acc], (j >> 1) & 1, kDevTimeoutSoftmax, abort, p.status));
            tc_fence_after();
            return ok;
        };
        auto free_acc = [&](int acc) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR)
                    lb_arrive_remote(acc_empty0 + 8 * acc);
                else
                    mbar_arrive(&sh->acc_empty[acc]);
            }
        };
        // A slice of results, 32 rows of 128 bytes (64 bf16 or 32 fp32 columns), is written
        // a row per thread and read back as whole lines, 8 threads on a row: 16-byte chunk c
        // of a row lies at c ^ (row & 7), so that neither way two threads share a bank.
        auto chunk_at = [&](int row, int c16) { return stg + row * 128 + ((c16 ^ (row & 7)) << 4); };
        const int lrow = lane >> 3, lc = lane & 7;  // row (of 4 at a time) and chunk of this thread's line accesses
        const uint32_t t_row = tmem + lane_off + 32 * CPW * chalf;
        bool more = sched.next(dw, item);
        for (; ok && more && dw; more = sched.next(dw, item)) {
                const LbItem it = lb_item<PAIR>(p, true, item);
                const int m = it.m0 + BM * rank + 32 * wq;  // first row of this warp's 32
                const int k = it.k0 + 32 * CPW * chalf;     // its first column
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
                        lb_tmem_ld16(t_row + acc * BN + 16 * h, v);
                        tmem_wait_ld();
                        if (h == 2 * CPW - 1) free_acc(acc);
#pragma unroll
                        for (int x = 0; x < 16; ++x) sum[h >> 1][16 * (h & 1) + x] += __uint_as_float(v[x]);
                    }
                }
                if (!ok) break;
                float* const out = p.dw + (size_t)it.split * p.N * p.K;
#pragma unroll
                for (int cc = 0; cc < CPW; ++cc) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        st_shared_v4(chunk_at(lane, q), __float_as_uint(sum[cc][4 * q]),
                                     __float_as_uint(sum[cc][4 * q + 1]), __float_as_uint(sum[cc][4 * q + 2]),
                                     __float_as_uint(sum[cc][4 * q + 3]));
                    __syncwarp();
                    const int c = k + 32 * cc + 4 * lc;  // K is a multiple of 8
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = 4 * i + lrow;
                        const uint4 v = lb_ld_shared_v4(chunk_at(row, lc));
                        const size_t at = (size_t)(m + row) * p.K + c;
                        if (m + row < p.N && c < p.K &&
                            TXL_BOUNDS(at + 4 <= (size_t)p.N * p.K && it.split < p.splits, 803, at))
                            *reinterpret_cast<uint4*>(out + at) = v;
                    }
                    __syncwarp();
                }
        }
        // dx: this thread's lines of a tile, in x and dx: rows row, row + 4, .. + 28 and 8
        // columns from c on of each 64-column slice
        constexpr int SL = CPW / 2;  // slices
        struct Lines {
            long long at;  // of the first line
            int rows, cols;  // rows of T and columns of K from there on
        };
        const int row_stride = p.heads ? 64 : p.K;
        const long long slice_stride = p.heads ? 64ll * p.T : 64;
        auto lines_of = [&](int i) {
            const LbItem it = lb_item<PAIR>(p, false, i);
            const int row = it.m0 + BM * rank + 32 * wq + lrow, c = it.k0 + 32 * CPW * chalf + 8 * lc;
            const long long col = p.heads ? (((long long)it.b * (p.K >> 6) + (c >> 6)) * p.T) * 64 + (c & 63)
                                          : (long long)it.b * p.T * p.K + c;
            return Lines{col + (long long)row * row_stride, p.T - row, p.K - c};
        };
        auto line_in = [&](const Lines& l, int sl, int i) {  // K is a multiple of 8
            return 4 * i < l.rows && 64 * sl < l.cols &&
                   TXL_BOUNDS(l.at + sl * slice_stride + (long long)(4 * i) * row_stride + 8 <= (long long)p.B * p.T * p.K, 802,
                              l.at);
        };
        // The ReLU mask of the lines, 8 bits each, from x: fetched a tile ahead, while that
        // tile's results leave (fetched at the tile's start it took longer than the MMAs).
        auto fetch = [&](uint4 (&x4)[8], const Lines& l, int sl) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x4[i] = line_in(l, sl, i) ? lb_load_once(p.x + l.at + sl * slice_stride + (long long)(4 * i) * row_stride)
                                          : make_uint4(0, 0, 0, 0);
        };
        auto mask_of = [&](uint4 (&x4)[8], uint32_t (&keep)[2]) {
            keep[0] = keep[1] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // (not moved ahead of what was issued since the fetch)
                asm volatile("" : "+r"(x4[i].x), "+r"(x4[i].y), "+r"(x4[i].z), "+r"(x4[i].w));
                const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&x4[i]);
                uint32_t four = 0;  // bit e for the low half of word e, bit 16 + e for its high half
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    four |= __hgt2_mask(h2[e], __floats2bfloat162_rn(0.f, 0.f)) & (0x00010001u << e);
                keep[i >> 2] += four << (4 * (i & 3));
            }
        };
        Lines cur = {}, next = {};
        // Each slice of the next tile is on its way for a slice's time and packed behind it, the
        // last one only when the next tile begins.
        uint32_t keep[SL][2];
        uint4 x4[8];
        if (ok && more) {
            next = lines_of(item);
            if (RELU) {
#pragma unroll
                for (int sl = 0; sl < SL; ++sl) {
                    if (sl) mask_of(x4, keep[sl - 1]);
                    fetch(x4, next, sl);
                }
            }
        }
        while (ok && more) {
            cur = next;
            more = sched.next(dw, item);
            if (more) next = lines_of(item);
            uint32_t first[2];  // the next tile's first mask, until this one's is used
            if (RELU) {
                mask_of(x4, keep[SL - 1]);
                if (more) fetch(x4, next, 0);
            }
            const int acc = j & 1;
            if (!wait_acc(acc)) break;
#pragma unroll
            for (int sl = 0; sl < SL; ++sl) {
#pragma unroll
                for (int hc = 0; hc < 2; ++hc) {
                    uint32_t v[32];
                    tmem_ld32(t_row + acc * BN + 64 * sl + 32 * hc, v);
                    tmem_wait_ld();
                    if (sl == SL - 1 && hc == 1) free_acc(acc);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        st_shared_v4(chunk_at(lane, 4 * hc + q),
                                     pack_bf16x2(__uint_as_float(v[8 * q + 0]), __uint_as_float(v[8 * q + 1])),
                                     pack_bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                                     pack_bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                                     pack_bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7])));
                }
                __syncwarp();
                __nv_bfloat16* const to = p.dx + cur.at + sl * slice_stride;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint4 v = lb_ld_shared_v4(chunk_at(4 * i + lrow, lc));
                    if (RELU) {
                        uint32_t* o = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // the two bits to the tops of the halves, and these over the halves
                            uint32_t on = keep[sl][i >> 2] << (15 - 4 * (i & 3) - e);
                            asm("prmt.b32 %0, %0, 0, 0xBB99;" : "+r"(on));
                            o[e] &= on;
                        }
                    }
                    if (line_in(cur, sl, i)) *reinterpret_cast<uint4*>(to + (long long)(4 * i) * row_stride) = v;
                }
                __syncwarp();
                if (RELU && more && sl + 1 < SL) {
                    mask_of(x4, first);
                    fetch(x4, next, sl + 1);
                }
            }
            if (SL > 1) keep[0][0] = first[0], keep[0][1] = first[1];
            ++j;
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
            if (!TXL_BOUNDS(i + s * n4 < n4 * splits, 807, i + s * n4)) continue;
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
        for (int r = w; r < db_rows; r += 8)
            if (TXL_BOUNDS((long long)r * N + n < (long long)db_rows * N, 808, n)) a += db_part[(size_t)r * N + n];
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

// Microseconds that a stage takes a pair or a CTA, that a dx tile's and a dw item's end
// add to the last of a unit, that the parts of one more split cost per byte of dw (write
// and read, through L2), and that the second launch costs; measured on base512's and
// large384's layers.
constexpr double kStepPair = 0.36, kStepOne = 0.27, kTail = 3.0, kSplitPerByte = 0.4e-6, kSumLaunch = 2.0;

// Up to this many rows db is summed without parts, which is what a second launch would be
// for where dw has none (512 -> 2048, 1024 rows: 10.1 us against 11.3, 2048 rows 11.5 against
// 13.3, 4096 rows 23.3 against 19.4), or has one for dw's anyway (512 -> 512, 1536 rows: 10.0
// us against 8.8).
constexpr long long kDbOnce = 2048, kDbOnceSplit = 1024;

}  // namespace

LbPlan linear_bwd_plan(int heads, int B, int T, int K, int N, bool want_dx, bool want_dw) {
    LbPlan pl = {};
    LbParams& p = pl.p;
    p.T = heads ? T : B * T;
    p.B = heads ? B : 1;
    p.K = K;
    p.N = N;
    p.heads = heads;
    p.k64 = K % 64 == 0;
    p.n64 = N % 64 == 0;
    p.t_steps = ceil_div(p.T, lb::BR);
    p.n_steps = ceil_div(N, lb::BR);
    const int sms = current_sm_count();
    const long long total = (long long)p.B * p.t_steps;
    // Tiles, splits and schedule with the least time by this model: the stages of the
    // unit (pair or CTA) with most to do, and the parts' traffic.
    double best = -1;
    for (int ctas : {2, 1}) {
        const int most_units = sms / ctas, tile = lb::BM * ctas;
        if (most_units < 1) continue;
        const int kt = ceil_div(K, tile), nt = ceil_div(N, tile), tt = ceil_div(p.T, tile);
        const long long n_d = want_dx ? (long long)p.B * tt * kt : 0;
        for (int s = 1; s <= (want_dw ? 32 : 1) && s <= total; ++s) {
            const long long n_w = want_dw ? (long long)nt * kt * s : 0;
            const int units = (int)(n_w + n_d < most_units ? n_w + n_d : most_units);
            const int heavy = (int)(n_w % units), light = heavy ? units - heavy : 0;
            const double len = (double)total / s;  // stages of a dw item
            // (no more than there are: light * extra stays an int)
            const int extra = light ? (int)std::min(len / p.n_steps, (double)(n_d / light + 1)) : 0;
            const long long head = n_d < (long long)light * extra ? n_d : (long long)light * extra, rest = n_d - head;
            const double all = (double)(n_w / units) * len, turn = (double)((rest + units - 1) / units) * p.n_steps;
            const double fewer = (double)(rest / units) * p.n_steps;
            const double hi = all + (heavy ? len : 0.0) + (rest % units > light || !light ? turn : fewer);
            const double lo = all + (light ? (double)((head + light - 1) / light) * p.n_steps : 0.0) + turn;
            const double cost = (hi > lo ? hi : lo) * (ctas == 2 ? kStepPair : kStepOne) + kTail +
                                (s > 1 ? kSumLaunch + s * (N * 4.0 * K) * kSplitPerByte : 0.0);
            if (best >= 0 && cost >= best) continue;
            best = cost;
            pl.pair = ctas == 2;
            pl.grid = units * ctas;
            p.splits = s;
            p.n_kt = kt;
            p.n_nt = nt;
            p.n_tt = tt;
            p.n_w = (int)n_w;
            p.n_d = (int)n_d;
            p.heavy = heavy;
            p.extra = extra;
        }
    }
    // row ranges of db: as many as give each of the two summing warps per CTA one
    const long long rows = (long long)B * T, groups = (N + 255) / 256;
    const long long parts = std::max(1ll, std::min(2ll * pl.grid / groups, rows / 16));
    p.db_rows = rows <= (p.splits > 1 ? kDbOnceSplit : kDbOnce) ? 0 : (int)parts;
    return pl;
}

namespace {

template <bool PAIR, bool RELU>
cudaError_t lb_launch(const LbMaps& maps, const LbPlan& pl, cudaStream_t stream) {
    static PerDeviceOnce attrs;
    const cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(linear_bwd_kernel<PAIR, RELU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    lb::SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.grid);
    cfg.blockDim = dim3(lb::NTHREADS);
    cfg.dynamicSmemBytes = lb::SMEM_BYTES;
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
    return cudaLaunchKernelEx(&cfg, linear_bwd_kernel<PAIR, RELU>, maps, pl.p);
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

size_t linear_bwd_workspace_bytes(const LbPlan& pl, bool want_db) {
    return part_bytes(pl) + (want_db ? (size_t)pl.p.db_rows * pl.p.N * 4 : 0);
}

cudaError_t launch_linear_bwd(LbPlan pl, const void* dy, const void* x, const void* w, int relu, void* dx, float* dw,
                              float* db, void* workspace, int* status, cudaStream_t stream) {
    LbParams& p = pl.p;
    const int K = p.K, N = p.N, heads = p.heads;
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.dy = static_cast<const __nv_bfloat16*>(dy);
    p.dx = static_cast<__nv_bfloat16*>(dx);
    p.status = status;
    if (!db) p.db_rows = 0;
    const bool split = p.splits > 1;
    float* part = split ? static_cast<float*>(workspace) : dw;
    p.dw = part;
    p.db = p.db_rows ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part_bytes(pl)) : db;
    LbMaps maps;
    const cuuint64_t Tt = p.T, Bb = p.B, Kk = K, Nn = N;
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
        const cuuint32_t cut_box[3] = {64, 64, 2}, one_box[3] = {64, 64, 1};
        if (!lb_encode(&maps.w, bf, w, 3, p.k64 ? cut : one, p.k64 ? cut_str : one_str, p.k64 ? cut_box : one_box))
            return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t rows_dims[4] = {Kk, Tt, 1, 1}, rows_str[3] = {Kk * 2, Tt * Kk * 2, Tt * Kk * 2};
        const cuuint64_t cut_dims[4] = {64, Tt, Kk / 64, Bb};
        const cuuint64_t heads_str[3] = {128, Tt * 128, Tt * Kk * 2}, cut_str[3] = {Kk * 2, 128, Tt * Kk * 2};
        const cuuint32_t box[4] = {64, 64, p.k64 ? 2u : 1u, 1};
        if (!lb_encode(&maps.x, bf, x, 4, p.k64 ? cut_dims : rows_dims, heads ? heads_str : p.k64 ? cut_str : rows_str, box))
            return cudaErrorInvalidValue;
    }
    const cudaError_t e = pl.pair ? (relu ? lb_launch<true, true> : lb_launch<true, false>)(maps, pl, stream)
                                  : (relu ? lb_launch<false, true> : lb_launch<false, false>)(maps, pl, stream);
    if (e != cudaSuccess || (!split && !p.db_rows)) return e;
    return lb_sum(part, dw, p.splits, p.db, p.db_rows ? db : nullptr, N, K, p.db_rows, stream);
}

TXL_BOUNDS_READER(bounds_word_linear_bwd)

}  // namespace txl
