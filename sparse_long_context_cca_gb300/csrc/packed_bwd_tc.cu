// Gradients of attention over packed sequences on the sm_103a tensor cores (bf16, d = 128 or 64): dS =
// P (dO . v - D) with P recomputed from the forward's LSE and D = dO . O given.
//
// Two persistent kernels of one CTA per SM, 320 threads: warp 0 issues the copies, warp 1 the products (one
// elected lane), warps 2..9 do the element-wise work, two warps to 32 rows, 64 columns each.  A CTA's
// items come from the batch's plan, heaviest first, dealt to and fro, and the roles run through them without a
// barrier between: rings of tiles and phases count on from item to item, an item's first copies start when
// the last products that read the ones before are done, and its first products run while the results of the
// item before are read out of tensor memory.  (A CTA per item spent 6.4 us, for dK and dV 10, on its launch,
// first copies and last stores: 5 or 6 tiles of work.)
//
//  dq: an item is 128 query rows of one head, over its key tiles (cores, then the band):
//     S = Q K^T, dP = dO V^T  ->  dS (bf16);   dQ += dS K
//  TMEM: S | dP | dS | Q | dQ.  The element-wise warps take S and dP of a tile into registers at once, and both
//  products of the next tile run while they form dS; Q, the left side of every S, is copied to tensor memory,
//  where it takes no shared-memory bandwidth.
//
//  dkv: an item is 128 keys (raw tokens or cores) of one KV head, over the rows of its query heads that see any:
//     S^T = K Q^T, dP^T = V dO^T  ->  P^T over S^T, dS^T over dP^T (bf16);   dV += P^T dO,  dK += dS^T Q
//  TMEM: S^T | dP^T | dK | dV.  The rows of a core tile are split over items, whose sums are added up in order
//  later; those of few tokens' tiles over two, the second of which to end adds the other's sums.
//
// What bounds them (32 heads over 8, 16 K tokens in five sequences, window 1024): dq 370-373 us, dkv of the tokens 382-385
// and of the cores 79, the tensor pipe active 50 and 57% of the time.  S and dP, and the exponentials, are formed in both
// kernels: with the forward nine products for a tile where seven would do, and tiles hold 19% more pairs than are
// visible.  One kernel for all three sums was not built: at d = 128 tensor memory has no room for dQ beside dK and dV.  With its parts taken out in turn, dq (376 us then) took
// 372 us without copies, 370 without exponentials, 343 without dQ's product, 310 without any product, and 229 with
// nothing but waits, tensor-memory reads and writes, and dS: the chain of a tile through the eight element-wise
// warps.  Sixteen of them gained nothing.  dkv without any product took 315 us of 388, and with nothing but waits,
// tensor-memory traffic and dS 271; paired arithmetic (391), dP read at once (408) and slots handed over by the
// barriers of P and dS (417) gained nothing either.
//
// P and dS are rounded to bf16 for the tensor cores (off by at most half a step, 2^-8 relative, each); everything between is fp32.
//
// Results leave once, in bf16 (a core's in fp32), from the thread that holds the row, with the pooling's share:
// rows of a tile behind the sequence's end belong to the next one and must stay as they are.  Read, they
// would reach sums over rows as 0 * NaN: the producer waits for such a tile (one at the end of a sequence) and
// sets those rows to zero before it hands it over; scores of masked pairs take part in nothing.
//
// Every wait is bounded; a time-out sets the CTA's abort flag, which ends every other wait: the issuer then waits
// (bounded) for the products it has issued, the producer for its copies in flight, TMEM is freed and
// CCA_ERR_TIMEOUT reported.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "packed.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.h"

namespace cca {

extern unsigned long long g_wait_limit_ns;
extern int g_skip_q_load;

namespace {

constexpr int BT = 128;                       // rows of a tile (queries or keys)
constexpr uint32_t HALF_BYTES = BT * 64 * 2;  // 64 columns of a tile, as one swizzled box
constexpr uint32_t IDESC_SS = ptx::idesc_bf16_f32(128, 128, 0, 0);  // K-major A and B
constexpr float LOG2E = 1.4426950408889634f;
constexpr int THREADS = 320;
constexpr int LONG_ST = 3, SHORT_ST = 2;  // stages of the operand that is read twice (K; Q), and of the other (V; dO)

struct Args {
    Plan plan;
    Rows<__nv_bfloat16> dQ, dK, dV;
    PackedBwdSpace space;
    const float *LSE;
    int Hq, Hkv, r;  // r: query heads of a KV head
    FastDiv by_Hq, by_Hkv, by_r, by_per;  // per: items of a dkv tile
    int per;
    float tau;
    int cores;  // whether any core is seen
    unsigned long long wait_limit_ns;
    int skip_loads;  // test hook: issue no copies, so the first wait runs out
};

// Shared memory: two resident tiles (Q and dO; K and V), the rings, the tile's LSE and D (dkv), barriers.
template <int HD>
struct Layout {
    static constexpr uint32_t TILE = BT * HD * 2;
    static constexpr uint32_t LONG = 2 * TILE, SHORT = LONG + LONG_ST * TILE;
    static constexpr uint32_t SLOT = SHORT + SHORT_ST * TILE;
    static constexpr uint32_t BAR = SLOT + 2 * BT * 4;
    static constexpr uint32_t TMEM = BAR + 32 * 8, ABORT = TMEM + 4, ITEMS = ABORT + 4;
    static constexpr uint32_t SMEM = ITEMS + 3 * 4 + 1024;  // + slack for the 1024-byte alignment
    static_assert(SMEM <= 232448, "shared memory budget");
};
// Barriers of both kernels.
constexpr int B_RES = 0;                    // resident tiles are there
constexpr int B_RESFREE = 1;                // ... have been read
constexpr int B_LFULL = 2, B_LEMPTY = 5;    // LONG_ST each
constexpr int B_SFULL_RING = 8, B_SEMPTY = 10;  // SHORT_ST each
constexpr int B_S = 12;                     // dkv: S is there
constexpr int B_READ = 13;                  // dq: S and dP are in registers
constexpr int B_DP = 14;                    // dP is there (dq: S too)
constexpr int B_P = 15;                     // dkv: P is there
constexpr int B_DS = 16;                    // dS is there
constexpr int B_DSFREE = 17;                // dq: dS has been read
constexpr int B_DONE = 18;                  // the item's sums are there
constexpr int B_ACCFREE = 19;               // ... have been read
constexpr int B_Q = 20, B_QT = 21;          // dq: the queries are in shared memory; in tensor memory
constexpr int B_DRAIN = 22, B_CUT = 23;
constexpr int B_ITEM = 24, B_ITEMFREE = 26;  // dkv: 2 each, the next item's number is there; has been read
constexpr int N_BARS = 28;

template <int HD>
__device__ __forceinline__ void load_tile(const void *map, uint32_t bar, uint32_t dst, int y, int z) {
#pragma unroll
    for (int x = 0; x < HD / 64; ++x) ptx::tma_load_3d(map, bar, dst + x * HALF_BYTES, 64 * x, y, z);
}

// load_tile by a whole warp, with the tile's rows from `rows` on set to zero before it is handed over on
// `full` (an arrival like that of a plain tile, whose copies complete the phase).  `own` is a barrier for
// these copies alone, `phase` its phase.  false: the wait ran out.
template <int HD>
__device__ __forceinline__ bool load_cut_tile(const void *map, uint32_t full, uint32_t own, uint32_t &phase, uint32_t dst, int y, int z,
                                              int rows, volatile int *abort_flag, uint64_t lim) {
    const int lane = threadIdx.x & 31;
    if (rows >= BT) {
        if (lane == 0) {
            ptx::mbar_arrive_expect_tx(full, BT * HD * 2);
            load_tile<HD>(map, full, dst, y, z);
        }
        __syncwarp();
        return true;
    }
    if (lane == 0) {
        ptx::mbar_arrive_expect_tx(own, BT * HD * 2);
        load_tile<HD>(map, own, dst, y, z);
    }
    __syncwarp();
    // the copies land in any case: the wait that may give up is followed by one that only time ends
    if (!__all_sync(0xffffffffu, ptx::wait_bounded(own, phase & 1, abort_flag, lim))) {
        volatile int never = 0;
        ptx::wait_bounded(own, phase & 1, &never, lim);
        return false;
    }
    ++phase;
    for (int i = rows * 8 + lane; i < BT * 8; i += 32)
#pragma unroll
        for (int x = 0; x < HD / 64; ++x) ptx::st_shared_v4(dst + x * HALF_BYTES + i * 16, 0.f, 0.f, 0.f, 0.f);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(full);
    return true;
}

// D = A B^T over the HD columns of two K-major tiles.
template <int HD>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc) {
    if constexpr (HD == 128) ptx::mma_ss_k128_warp(d_tmem, a_desc, b_desc, IDESC_SS, 0u);
    else ptx::mma_ss_k64_warp(d_tmem, a_desc, b_desc, IDESC_SS, 0u);
}

// COLS fp32 sums in registers times `scale`, plus xs * x + ys * y (rows of fp32, either may be nullptr), as bf16.
__device__ __forceinline__ void store32_bf16(const uint32_t (&v)[32], float scale, const float *x, float xs, const float *y, float ys,
                                             __nv_bfloat16 *out) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v[8 * q + k]) * scale;
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            if (x != nullptr) {
                const float4 a = *reinterpret_cast<const float4 *>(x + 8 * q + k);
                f[k] = fmaf(xs, a.x, f[k]), f[k + 1] = fmaf(xs, a.y, f[k + 1]);
                f[k + 2] = fmaf(xs, a.z, f[k + 2]), f[k + 3] = fmaf(xs, a.w, f[k + 3]);
            }
            if (y != nullptr) {
                const float4 a = *reinterpret_cast<const float4 *>(y + 8 * q + k);
                f[k] = fmaf(ys, a.x, f[k]), f[k + 1] = fmaf(ys, a.y, f[k + 1]);
                f[k + 2] = fmaf(ys, a.z, f[k + 2]), f[k + 3] = fmaf(ys, a.w, f[k + 3]);
            }
        }
        *reinterpret_cast<uint4 *>(out + 8 * q) = make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]),
                                                             ptx::pack_bf16x2(f[4], f[5]), ptx::pack_bf16x2(f[6], f[7]));
    }
}
__device__ __forceinline__ void store32_f32(const uint32_t (&v)[32], float scale, float *out) {
#pragma unroll
    for (int q = 0; q < 32; q += 4)
        *reinterpret_cast<float4 *>(out + q) = make_float4(__uint_as_float(v[q]) * scale, __uint_as_float(v[q + 1]) * scale,
                                                           __uint_as_float(v[q + 2]) * scale, __uint_as_float(v[q + 3]) * scale);
}

// Zero where a column's bit is not set; `whole`: all bits of all lanes are.
__device__ __forceinline__ void clear_unseen(uint32_t (&v)[32], uint32_t seen, bool whole) {
    if (whole) return;
#pragma unroll
    for (int k = 0; k < 32; ++k)
        if (!(seen & (1u << k))) v[k] = 0u;
}

// What every role has.
template <int HD>
struct Cta {
    using L = Layout<HD>;
    uint32_t base, tmem;
    volatile int *abort_flag;
    uint64_t lim;
    uint8_t *gb;
    __device__ __forceinline__ uint32_t bar(int k) const { return base + L::BAR + 8u * k; }
    __device__ __forceinline__ uint32_t res(int k) const { return base + k * L::TILE; }
    __device__ __forceinline__ uint32_t stage_l(uint32_t g) const { return base + L::LONG + g % LONG_ST * L::TILE; }
    __device__ __forceinline__ uint32_t stage_s(uint32_t g) const { return base + L::SHORT + g % SHORT_ST * L::TILE; }
    // a warp's wait; the same answer in every lane
    __device__ __forceinline__ bool wait(uint32_t b, uint32_t parity) const {
        return __all_sync(0xffffffffu, ptx::wait_bounded(b, parity, abort_flag, lim));
    }
};

template <int HD>
__device__ __forceinline__ Cta<HD> setup(uint8_t *smem_raw, const Args &p) {
    using L = Layout<HD>;
    Cta<HD> c;
    const uint32_t r0 = ptx::smem_addr(smem_raw);
    c.base = (r0 + 1023u) & ~1023u;
    c.gb = smem_raw + (c.base - r0);
    c.abort_flag = reinterpret_cast<volatile int *>(c.gb + L::ABORT);
    c.lim = p.wait_limit_ns;
    if (threadIdx.x == 0) {
        for (int k = 0; k < N_BARS; ++k)  // one arrival, but for those of the eight element-wise warps
            ptx::mbar_init(c.bar(k), k == B_READ || k == B_P || k == B_DS || k == B_ACCFREE || k == B_QT ? 8
                                        : k == B_ITEMFREE || k == B_ITEMFREE + 1                                        ? 2
                                                                                                                        : 1);
        *c.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (threadIdx.x < 32) {
        ptx::tmem_alloc(c.base + L::TMEM, 512);
        ptx::tmem_relinquish();
    }
    // Everything above runs while the kernel before ends.  This one does not let the next begin early, for the same
    // reason as the forward: with it the training step with cores took 1233 us instead of 1209.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    c.tmem = *reinterpret_cast<uint32_t *>(c.gb + L::TMEM);
    return c;
}

template <int HD>
__device__ __forceinline__ void finish(const Cta<HD> &c, const Args &p) {
    ptx::tc_fence_before();
    __syncthreads();
    if (*c.abort_flag && threadIdx.x == 0) report(p.plan.status, CCA_ERR_TIMEOUT);
    if (threadIdx.x < 32) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(c.tmem, 512);
    }
}

// The producer's wait for its last copies: `nl`, `ns` tiles were asked for, `nr` times the resident ones.  Not only where the
// abort flag is set: whoever gives up later than this may leave copies that nobody else waits for.
template <int HD>
__device__ __forceinline__ void drain_copies(const Cta<HD> &c, uint32_t nl, uint32_t ns, uint32_t nr) {
    volatile int never = 0;
    if (nr > 0) ptx::wait_bounded(c.bar(B_RES), (nr - 1) & 1, &never, c.lim);
    for (uint32_t g = nl > LONG_ST ? nl - LONG_ST : 0; g < nl; ++g)
        ptx::wait_bounded(c.bar(B_LFULL + g % LONG_ST), (g / LONG_ST) & 1, &never, c.lim);
    for (uint32_t g = ns > SHORT_ST ? ns - SHORT_ST : 0; g < ns; ++g)
        ptx::wait_bounded(c.bar(B_SFULL_RING + g % SHORT_ST), (g / SHORT_ST) & 1, &never, c.lim);
}

// ---------------------------------------------------------------- dQ

struct DqItem {
    int h, kv, n, row0, core0, i0, lo0, Tc, T;
    __device__ __forceinline__ DqItem(const Args &p, int item) {
        const int tile = p.by_Hq.div(item);
        const int4 e = p.plan.tiles[tile];
        h = item - tile * p.Hq;
        kv = p.by_r.div(h);
        row0 = e.x, n = e.y, core0 = e.w;
        i0 = e.z * BT;
        const int i1 = min(i0 + BT, n) - 1;
        lo0 = p.plan.start_of(i0);
        Tc = (p.plan.cores_of(i1) + BT - 1) / BT;                    // core tiles
        T = Tc + (i1 - lo0) / BT + 1;                                // + band tiles
    }
    __device__ __forceinline__ int tile_y(int x) const { return x < Tc ? x * BT : lo0 + (x - Tc) * BT; }
};

template <int HD>
__global__ void __launch_bounds__(THREADS, 1)
    packed_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                        const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmKc, const __grid_constant__ CUtensorMap tmVc,
                        const __grid_constant__ Args p) {
    extern __shared__ uint8_t smem_raw[];
    const Cta<HD> c = setup<HD>(smem_raw, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_items = plan_counts(p.plan).y * p.Hq;
    constexpr uint32_t T_DP = 128, T_DS = 256, T_Q = 320, T_DQ = 384;  // TMEM columns; S at 0

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        if (lane == 0) {
            ptx::prefetch_tmap(&tmQ);
            ptx::prefetch_tmap(&tmdO);
            ptx::prefetch_tmap(&tmK);
            ptx::prefetch_tmap(&tmV);
            ptx::prefetch_tmap(&tmKc);
            ptx::prefetch_tmap(&tmVc);
        }
        uint32_t g = 0, nl = 0, ns = 0, nq = 0, it = 0, cut = 0;
        bool ok = !p.skip_loads;
        for (int round = 0, item; ok && (item = item_of_round(round)) < n_items; ++round) {
            const DqItem d(p, item);
            const int groups = p.plan.by_g.div(d.n);
            if (!c.wait(c.bar(B_QT), (it & 1) ^ 1)) break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(c.bar(B_Q), Layout<HD>::TILE);
                load_tile<HD>(&tmQ, c.bar(B_Q), c.res(0), d.row0 + d.i0, d.h);
            }
            nq = it + 1;
            if (!c.wait(c.bar(B_RESFREE), (it & 1) ^ 1)) break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(c.bar(B_RES), Layout<HD>::TILE);
                load_tile<HD>(&tmdO, c.bar(B_RES), c.res(1), d.row0 + d.i0, d.h);
            }
            ++it;
            for (int x = 0; x < d.T; ++x, ++g) {
                const bool core = x < d.Tc;
                const int y = (core ? d.core0 : d.row0) + d.tile_y(x);
                const int left = (core ? groups : d.n) - d.tile_y(x);
                // only K takes part in a sum over keys; V's products stay in their column
                if (!(ok = c.wait(c.bar(B_LEMPTY + g % LONG_ST), ((g / LONG_ST) & 1) ^ 1))) break;
                if (!(ok = load_cut_tile<HD>(core ? (const void *)&tmKc : (const void *)&tmK, c.bar(B_LFULL + g % LONG_ST), c.bar(B_CUT), cut,
                                             c.stage_l(g), y, d.kv, left, c.abort_flag, c.lim)))
                    break;
                nl = g + 1;
                if (!(ok = c.wait(c.bar(B_SEMPTY + g % SHORT_ST), ((g / SHORT_ST) & 1) ^ 1))) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(c.bar(B_SFULL_RING + g % SHORT_ST), Layout<HD>::TILE);
                    load_tile<HD>(core ? (const void *)&tmVc : (const void *)&tmV, c.bar(B_SFULL_RING + g % SHORT_ST), c.stage_s(g), y, d.kv);
                }
                ns = g + 1;
            }
        }
        __syncwarp();
        if (!p.skip_loads) {
            drain_copies(c, nl, ns, it);
            volatile int never = 0;
            if (nq > 0) ptx::wait_bounded(c.bar(B_Q), (nq - 1) & 1, &never, c.lim);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        constexpr uint32_t IDESC_TS = ptx::idesc_bf16_f32(128, HD, 0, 1);  // A in TMEM, B MN-major
        const uint64_t ddOd = ptx::smem_desc_sw128(c.res(1), 16, 1024);
        // S(g) = Q K(g)^T and dP(g) = dO V(g)^T of the first or a later tile of item `it`
        auto products = [&](uint32_t g, uint32_t it, bool first) -> bool {
            if (!c.wait(c.bar(B_LFULL + g % LONG_ST), (g / LONG_ST) & 1)) return false;
            if (first && !c.wait(c.bar(B_QT), it & 1)) return false;
            if (g > 0 && !c.wait(c.bar(B_READ), (g - 1) & 1)) return false;
            ptx::tc_fence_after();
            const uint64_t k = ptx::smem_desc_sw128(c.stage_l(g), 16, 1024);
            if constexpr (HD == 128) ptx::mma_ts_nt_k128_warp(c.tmem, c.tmem + T_Q, k, IDESC_SS);
            else ptx::mma_ts_nt_k64_warp(c.tmem, c.tmem + T_Q, k, IDESC_SS);
            if (!c.wait(c.bar(B_SFULL_RING + g % SHORT_ST), (g / SHORT_ST) & 1)) return false;
            if (first && !c.wait(c.bar(B_RES), it & 1)) return false;
            ptx::tc_fence_after();
            mma_ss<HD>(c.tmem + T_DP, ddOd, ptx::smem_desc_sw128(c.stage_s(g), 16, 1024));
            ptx::tc_commit_warp(c.bar(B_DP));
            ptx::tc_commit_warp(c.bar(B_SEMPTY + g % SHORT_ST));
            return true;
        };
        uint32_t g = 0, it = 0;
        bool ok = true;
        for (int item; ok && (item = item_of_round(it)) < n_items; ++it) {
            const DqItem d(p, item);
            if (!(ok = products(g, it, true))) break;
            for (int x = 0; x < d.T; ++x, ++g) {
                if (x + 1 < d.T) {
                    if (!(ok = products(g + 1, it, false))) break;
                } else {
                    ptx::tc_commit_warp(c.bar(B_RESFREE));
                }
                if (!(ok = c.wait(c.bar(B_DS), g & 1))) break;
                if (x == 0 && !(ok = c.wait(c.bar(B_ACCFREE), (it & 1) ^ 1))) break;
                ptx::tc_fence_after();
                ptx::mma_ts_k128_warp(c.tmem + T_DQ, c.tmem + T_DS, ptx::smem_desc_sw128(c.stage_l(g), HALF_BYTES, 1024), IDESC_TS,
                                      x > 0 ? 1u : 0u);
                ptx::tc_commit_warp(c.bar(B_DSFREE));
                ptx::tc_commit_warp(c.bar(B_LEMPTY + g % LONG_ST));
            }
            if (ok) ptx::tc_commit_warp(c.bar(B_DONE));
        }
        // whatever was issued must complete before tensor memory is freed
        ptx::tc_commit_warp(c.bar(B_DRAIN));
        volatile int never = 0;
        ptx::wait_bounded(c.bar(B_DRAIN), 0, &never, c.lim);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- element-wise
        const int ch = (warp - 2) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const int h0 = ch * 64;  // this warp's 64 key columns of the tile
        const uint32_t lane_addr = c.tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const float c1 = p.tau * LOG2E;
        const uint64_t c2 = ptx::f2(c1, c1);
        // this warp's half of its rows' queries of item `it`, from the swizzled tile to tensor memory
        auto copy_q = [&](uint32_t it) -> bool {
            if (!c.wait(c.bar(B_Q), it & 1)) return false;
            const uint32_t src = c.res(0) + (HD == 128 ? ch * HALF_BYTES : 0) + row * 128;
#pragma unroll
            for (int k = 0; k < HD / 64; ++k) {
                uint32_t q[16];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int piece = (HD == 128 ? 4 * k : 4 * ch) + x;
                    const uint4 v = ptx::ld_shared_v4(src + ((piece ^ (row & 7)) << 4));
                    q[4 * x] = v.x, q[4 * x + 1] = v.y, q[4 * x + 2] = v.z, q[4 * x + 3] = v.w;
                }
                ptx::tmem_st16(lane_addr + T_Q + ch * (HD / 4) + 16 * k, q);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(c.bar(B_QT));
            return true;
        };
        uint32_t g = 0, it = 0;
        bool ok = item_of_round(0) >= n_items || copy_q(0);
        for (int item; ok && (item = item_of_round(it)) < n_items; ++it) {
            const DqItem d(p, item);
            const int i = d.i0 + row;
            const bool valid = i < d.n;
            float lse2 = 0.f, Di = 0.f;
            if (valid) {
                const int64_t u = static_cast<int64_t>(d.h) * p.plan.T + d.row0 + i;
                lse2 = p.LSE[u] * LOG2E;
                Di = p.space.D[u];
            }
            const uint64_t nl2 = ptx::f2(-lse2, -lse2);
            uint64_t nd2 = ptx::f2(-Di, -Di);
            const int lo_i = p.plan.start_of(i), nc_i = p.plan.cores_of(i);
            for (int x = 0; x < d.T; ++x, ++g) {
                // the row's visible key columns of this tile
                const int y0 = d.tile_y(x);
                int c_lo = 0, c_hi = BT - 1;
                if (x < d.Tc) {
                    c_hi = min(nc_i - y0, BT) - 1;
                } else {
                    c_lo = max(lo_i - y0, 0);
                    c_hi = min(i - y0, BT - 1);
                }
                if (!valid) c_hi = -1;
                const uint32_t seen[2] = {ptx::bits(c_lo - h0, c_hi - h0), ptx::bits(c_lo - h0 - 32, c_hi - h0 - 32)};
                const bool whole[2] = {__all_sync(0xffffffffu, seen[0] == 0xffffffffu) != 0, __all_sync(0xffffffffu, seen[1] == 0xffffffffu) != 0};
                if (!(ok = c.wait(c.bar(B_DP), g & 1))) break;  // S was issued before dP
                ptx::tc_fence_after();
                if (d.T == 1) {
                    // Few keys: D is formed from them, sum_j P_ij dP_ij.  dO . O carries the roundings of P and O to bf16,
                    // which for a few large weights are as much as dS itself is rounded (three tokens: dQ 0.0037 off
                    // instead of 0.0024, 2-norms, with 0.0017 the rounding of dQ).  Each warp goes over all 128 columns.
                    float sum = 0.f;
#pragma unroll 1
                    for (int j = 0; j < BT; j += 16) {
                        uint32_t s[16], dp[16];
                        ptx::tmem_ld16(lane_addr + j, s);
                        ptx::tmem_ld16(lane_addr + T_DP + j, dp);
                        ptx::tmem_wait_ld16(s);
                        ptx::tmem_wait_ld16(dp);
                        const uint32_t m = ptx::bits(c_lo - j, c_hi - j);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float w = ptx::ex2(fmaf(__uint_as_float(s[k]), c1, -lse2));
                            if (m & (1u << k)) sum = fmaf(w, __uint_as_float(dp[k]), sum);
                        }
                    }
                    nd2 = ptx::f2(-sum, -sum);
                    if (valid && ch == 0) p.space.D[static_cast<int64_t>(d.h) * p.plan.T + d.row0 + i] = sum;  // for dK and dV
                }
                uint32_t s[2][32], dp[2][32];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    ptx::tmem_ld32(lane_addr + h0 + 32 * j, s[j]);
                    ptx::tmem_ld32(lane_addr + T_DP + h0 + 32 * j, dp[j]);
                }
                ptx::tmem_wait_ld(s[0]);
                ptx::reg_touch(dp[0]);
                ptx::reg_touch(s[1]);
                ptx::reg_touch(dp[1]);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(c.bar(B_READ));  // the next S and dP may come
                // the product that reads the dS of the tile before is done
                if (g > 0 && !(ok = c.wait(c.bar(B_DSFREE), (g - 1) & 1))) break;
                ptx::tc_fence_after();
                // P = 2^(S tau log2e - LSE), dS = P (dP - D) as bf16 pairs; nothing of a masked value gets on, not as
                // 0 * NaN either
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float a, b;
                        ptx::f2_split(ptx::fma2(ptx::f2(__uint_as_float(s[j][k]), __uint_as_float(s[j][k + 1])), c2, nl2), a, b);
                        s[j][k] = __float_as_uint(ptx::ex2(a));
                        s[j][k + 1] = __float_as_uint(ptx::ex2(b));
                    }
                    clear_unseen(s[j], seen[j], whole[j]);
                    clear_unseen(dp[j], seen[j], whole[j]);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint64_t x2 = ptx::add2(ptx::f2(__uint_as_float(dp[j][2 * k]), __uint_as_float(dp[j][2 * k + 1])), nd2);
                        float a, b;
                        ptx::f2_split(ptx::mul2(ptx::f2(__uint_as_float(s[j][2 * k]), __uint_as_float(s[j][2 * k + 1])), x2), a, b);
                        pk[k] = ptx::pack_bf16x2(a, b);
                    }
                    ptx::tmem_st16(lane_addr + T_DS + ch * 32 + 16 * j, pk);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(c.bar(B_DS));
            }
            // the last S of this item is done: its queries give way to the next one's
            if (ok && item_of_round(it + 1) < n_items) ok = copy_q(it + 1);
            if (!ok || !(ok = c.wait(c.bar(B_DONE), it & 1))) break;
            ptx::tc_fence_after();
            const int c0 = ch * (HD / 2);
            uint32_t v[HD / 64][32];
#pragma unroll
            for (int k = 0; k < HD / 64; ++k) ptx::tmem_ld32(lane_addr + T_DQ + c0 + 32 * k, v[k]);
            ptx::tmem_wait_ld(v[0]);
            if constexpr (HD == 128) ptx::reg_touch(v[1]);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(c.bar(B_ACCFREE));
            if (valid) {
                // a group-last row that is pooled into a core some row sees has the pooling's share too
                const int j = p.plan.by_g.div(i);
                const bool last = p.cores != 0 && i - j * p.plan.g == p.plan.g - 1 && j < p.plan.seen_of(d.n);
                const float *add = last ? p.space.dqs + (static_cast<int64_t>(d.kv) * p.plan.G + d.core0 + j) * HD + c0 : nullptr;
                __nv_bfloat16 *out = p.dQ.at(d.h, d.row0 + i) + c0;
#pragma unroll
                for (int k = 0; k < HD / 64; ++k)
                    store32_bf16(v[k], p.tau, last ? add + 32 * k : nullptr, 1.f, nullptr, 0.f, out + 32 * k);
            }
        }
    }
    finish(c, p);
}

// ---------------------------------------------------------------- dK, dV

// Whose keys an item's are, and how items are dealt.
//  CORES: each CTA's first item is its own, later ones go to whoever comes (92 -> 79 us).
//  TOKENS: dealt to and fro, as dq's: items differ little where there are many, and handing numbers on costs 2%.
//  FEW_TOKENS (up to two tiles an SM): as cores; items of more than HALVED_PAIRS (query tile, head) pairs are two,
//  which share the rows: the longest one would be as long as the launch.  Six sequences of up to 2543 tokens, 16
//  heads over 4: 128 us whole, 115 so (from 64 pairs on 113, 32 119, 16 125); one of 4 K tokens 193 and 132 (125, 121, 115).
enum Kind { CORES, TOKENS, FEW_TOKENS };
constexpr int HALVED_PAIRS = 48;
template <Kind KIND>
struct DkvItem {
    int kv, n, row0, core0, y0, n_keys, qt_hi, n_it, split, tile;
    bool halved;   // another item has the rest of the rows of these tokens
    bool nothing;  // the second item of tokens that are not halved
    __device__ __forceinline__ DkvItem(const Args &p, int item) {
        constexpr bool CORE = KIND == CORES;
        const int splits = CORE ? p.space.splits : KIND == FEW_TOKENS ? 2 : 1;
        tile = p.by_per.div(item);
        const int4 e = (CORE ? p.plan.cores : p.plan.tiles)[tile];
        kv = item - tile * p.per;
        split = p.by_Hkv.div(kv);
        kv -= split * p.Hkv;
        row0 = e.x, n = e.y, core0 = e.w;
        n_keys = CORE ? p.plan.seen_of(n) : n;
        y0 = ((n_keys + BT - 1) / BT - 1 - e.z) * BT;  // the list's order is by the rows behind a key
        // the query rows [lo, hi] that see at least one key of the tile
        int lo = y0, hi = n - 1;
        if (CORE) {
            lo = static_cast<int>(static_cast<int64_t>(y0 + 1) * p.plan.g + p.plan.w - 1);  // core j is seen from row (j+1)g + w - 1 on
        } else {
            const int64_t last = last_row(p, min(y0 + BT, n) - 1);
            if (last < hi) hi = static_cast<int>(last);
        }
        int qt_lo = lo / BT;
        qt_hi = hi / BT;
        halved = KIND == FEW_TOKENS && (qt_hi - qt_lo + 1) * p.r > HALVED_PAIRS && qt_hi > qt_lo;
        nothing = KIND == FEW_TOKENS && !halved && split > 0;
        if (CORE ? splits > 1 : halved) {  // this item's part of the tiles (it may be none: its sums are zero)
            const int part = (qt_hi - qt_lo + splits) / splits;
            qt_hi -= part * split;
            qt_lo = max(qt_lo, qt_hi - part + 1);
        }
        // (query tile, head) pairs from the last tile down, heads fastest: the CTAs of a KV head then read
        // the same Q and dO tiles at about the same time, so they come from L2
        n_it = max(qt_hi - qt_lo + 1, 0) * p.r;
    }
    // the last row whose window holds token m (it may lie behind the sequence)
    __device__ static __forceinline__ int64_t last_row(const Args &p, int m) {
        return p.plan.window_mode ? static_cast<int64_t>(p.plan.by_g.div(m) + 1) * p.plan.g + p.plan.w - 2 : static_cast<int64_t>(m) + p.plan.w - 1;
    }
};
// The (query tile, head) pairs of an item in order.
struct Walk {
    int h, i0, first, r;
    template <typename I>
    __device__ __forceinline__ Walk(const Args &p, const I &d) : h(d.kv * p.r), i0(d.qt_hi * BT), first(d.kv * p.r), r(p.r) {}
    __device__ __forceinline__ void next() {
        if (++h == first + r) {
            h = first;
            i0 -= BT;
        }
    }
};

template <int HD, Kind KIND>
__global__ void __launch_bounds__(THREADS, 1)
    packed_dkv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                         const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ Args p) {
    using L = Layout<HD>;
    using Dkv = DkvItem<KIND>;
    constexpr bool CORE = KIND == CORES, BY_NEED = KIND != TOKENS;
    extern __shared__ uint8_t smem_raw[];
    const Cta<HD> c = setup<HD>(smem_raw, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int3 counts = plan_counts(p.plan);
    const int n_items = (CORE ? counts.z : counts.y) * p.per;
    volatile int *const slot_item = reinterpret_cast<volatile int *>(c.gb + L::ITEMS);  // two of the producer's, and the element-wise warps'
    constexpr uint32_t T_DP = 128, T_DK = 256, T_DV = 384;  // TMEM columns; S^T at 0

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        if (lane == 0) {
            ptx::prefetch_tmap(&tmK);
            ptx::prefetch_tmap(&tmV);
            ptx::prefetch_tmap(&tmQ);
            ptx::prefetch_tmap(&tmdO);
        }
        uint32_t g = 0, nl = 0, ns = 0, nr = 0, cut = 0;
        bool ok = !p.skip_loads;
        for (int round = 0; ok; ++round) {
            // the next item (n_items or more: none)
            int item = item_of_round(round);
            if constexpr (BY_NEED) {
                if (lane == 0 && round > 0) item = gridDim.x + atomicAdd(p.space.taken + (CORE ? 0 : 1), 1);
                item = __shfl_sync(0xffffffffu, item, 0);
                if (!(ok = c.wait(c.bar(B_ITEMFREE + (round & 1)), ((round >> 1) & 1) ^ 1))) break;
                if (lane == 0) {
                    slot_item[round & 1] = item;
                    ptx::mbar_arrive(c.bar(B_ITEM + (round & 1)));
                }
                __syncwarp();
            }
            if (item >= n_items) break;
            const Dkv d(p, item);
            if (d.n_it == 0 || d.nothing) continue;
            if (!c.wait(c.bar(B_RESFREE), (nr & 1) ^ 1)) break;
            if (lane == 0) {
                const int y = (CORE ? d.core0 : d.row0) + d.y0;
                ptx::mbar_arrive_expect_tx(c.bar(B_RES), 2 * L::TILE);
                load_tile<HD>(&tmK, c.bar(B_RES), c.res(0), y, d.kv);
                load_tile<HD>(&tmV, c.bar(B_RES), c.res(1), y, d.kv);
            }
            ++nr;
            Walk at(p, d);
            for (int x = 0; x < d.n_it; ++x, ++g, at.next()) {
                const int i0 = at.i0, h = at.h;
                if (!(ok = c.wait(c.bar(B_LEMPTY + g % LONG_ST), ((g / LONG_ST) & 1) ^ 1))) break;
                if (!(ok = load_cut_tile<HD>(&tmQ, c.bar(B_LFULL + g % LONG_ST), c.bar(B_CUT), cut, c.stage_l(g), d.row0 + i0, h, d.n - i0,
                                             c.abort_flag, c.lim)))
                    break;
                nl = g + 1;
                if (!(ok = c.wait(c.bar(B_SEMPTY + g % SHORT_ST), ((g / SHORT_ST) & 1) ^ 1))) break;
                if (!(ok = load_cut_tile<HD>(&tmdO, c.bar(B_SFULL_RING + g % SHORT_ST), c.bar(B_CUT), cut, c.stage_s(g), d.row0 + i0, h,
                                             d.n - i0, c.abort_flag, c.lim)))
                    break;
                ns = g + 1;
            }
        }
        __syncwarp();
        if (!p.skip_loads) drain_copies(c, nl, ns, nr);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        constexpr uint32_t IDESC_TS = ptx::idesc_bf16_f32(128, HD, 0, 1);  // A in TMEM, B MN-major
        const uint64_t dKk = ptx::smem_desc_sw128(c.res(0), 16, 1024), dVk = ptx::smem_desc_sw128(c.res(1), 16, 1024);
        // The MMAs of one thread complete in issue order, so S^T(g) and dP^T(g), issued after dV(g - 1) and dK(g - 1),
        // never overwrite what those read.
        auto issue_s = [&](uint32_t g) -> bool {  // S^T(g) = K Q(g)^T
            if (!c.wait(c.bar(B_LFULL + g % LONG_ST), (g / LONG_ST) & 1)) return false;
            ptx::tc_fence_after();
            mma_ss<HD>(c.tmem, dKk, ptx::smem_desc_sw128(c.stage_l(g), 16, 1024));
            ptx::tc_commit_warp(c.bar(B_S));
            return true;
        };
        auto issue_dp = [&](uint32_t g) -> bool {  // dP^T(g) = V dO(g)^T
            if (!c.wait(c.bar(B_SFULL_RING + g % SHORT_ST), (g / SHORT_ST) & 1)) return false;
            ptx::tc_fence_after();
            mma_ss<HD>(c.tmem + T_DP, dVk, ptx::smem_desc_sw128(c.stage_s(g), 16, 1024));
            ptx::tc_commit_warp(c.bar(B_DP));
            return true;
        };
        uint32_t g = 0, it = 0, nr = 0;
        bool ok = true;
        for (int round = 0; ok; ++round) {
            int item = item_of_round(round);
            if constexpr (BY_NEED) {
                if (!(ok = c.wait(c.bar(B_ITEM + (round & 1)), (round >> 1) & 1))) break;
                item = slot_item[round & 1];
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(c.bar(B_ITEMFREE + (round & 1)));
            }
            if (item >= n_items) break;
            const Dkv d(p, item);
            if (d.nothing) continue;
            if (d.n_it > 0) {
                if (!(ok = c.wait(c.bar(B_RES), nr & 1) && issue_s(g) && issue_dp(g))) break;
                ++nr;
                if (d.n_it == 1) ptx::tc_commit_warp(c.bar(B_RESFREE));
            }
            // the sums of the item before have been read (every item waits, so that no phase is passed over)
            if (d.n_it == 0 && !(ok = c.wait(c.bar(B_ACCFREE), (it & 1) ^ 1))) break;
            for (int x = 0; x < d.n_it; ++x, ++g) {
                const bool more = x + 1 < d.n_it;
                if (!(ok = c.wait(c.bar(B_P), g & 1))) break;
                if (x == 0 && !(ok = c.wait(c.bar(B_ACCFREE), (it & 1) ^ 1))) break;
                ptx::tc_fence_after();
                ptx::mma_ts_k128_split_warp(c.tmem + T_DV, c.tmem, ptx::smem_desc_sw128(c.stage_s(g), HALF_BYTES, 1024), IDESC_TS,
                                            x > 0 ? 1u : 0u);  // dV += P^T dO
                ptx::tc_commit_warp(c.bar(B_SEMPTY + g % SHORT_ST));
                if (more && !(ok = issue_s(g + 1))) break;
                if (!(ok = c.wait(c.bar(B_DS), g & 1))) break;
                ptx::tc_fence_after();
                ptx::mma_ts_k128_split_warp(c.tmem + T_DK, c.tmem + T_DP, ptx::smem_desc_sw128(c.stage_l(g), HALF_BYTES, 1024),
                                            IDESC_TS, x > 0 ? 1u : 0u);  // dK += dS^T Q
                ptx::tc_commit_warp(c.bar(B_LEMPTY + g % LONG_ST));
                if (more) {
                    if (!(ok = issue_dp(g + 1))) break;
                    if (x + 2 == d.n_it) ptx::tc_commit_warp(c.bar(B_RESFREE));
                }
            }
            if (ok) ptx::tc_commit_warp(c.bar(B_DONE));
            ++it;
        }
        // whatever was issued must complete before tensor memory is freed
        ptx::tc_commit_warp(c.bar(B_DRAIN));
        volatile int never = 0;
        ptx::wait_bounded(c.bar(B_DRAIN), 0, &never, c.lim);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- element-wise
        const int ch = (warp - 2) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const int h0 = ch * 64;  // this warp's 64 query columns of the tile
        const uint32_t lane_addr = c.tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const float c1 = p.tau * LOG2E;
        const int e = (warp - 2) * 32 + lane;  // this thread's value of the slot: LSE (log2 units) of query e, or D of e - 128
        float *const slot_f = reinterpret_cast<float *>(c.gb + L::SLOT);
        const float4 *const slot4 = reinterpret_cast<const float4 *>(slot_f);
        uint32_t g = 0, it = 0;
        bool ok = true;
        // Every element-wise thread runs every iteration of an item and all their named barriers, so that a time-out (which
        // skips the work) cannot leave a barrier short of threads.
        for (int round = 0;; ++round) {
            int item = item_of_round(round);
            if constexpr (BY_NEED) {
                // one warp waits for the item and passes it on, so that all leave together after a time-out
                if (warp == 2) {
                    const bool got = c.wait(c.bar(B_ITEM + (round & 1)), (round >> 1) & 1);
                    if (lane == 0) {
                        slot_item[2] = got ? slot_item[round & 1] : 0x7fffffff;
                        ptx::mbar_arrive(c.bar(B_ITEMFREE + (round & 1)));
                    }
                    __syncwarp();
                }
                ptx::named_bar_sync(1, 256);
                item = slot_item[2];
                ptx::named_bar_sync(1, 256);
            }
            if (item >= n_items) break;
            const Dkv d(p, item);
            if (d.nothing) continue;
            const int m = d.y0 + row;  // this thread's key (core or token of the sequence)
            const bool valid = m < d.n_keys;
            const int64_t key_last = CORE ? 0 : Dkv::last_row(p, m);
            Walk at(p, d);  // the tile whose LSE and D come next
            auto slot_value = [&]() -> float {
                const int iq = at.i0 + (e & (BT - 1));
                if (iq >= d.n) return 0.f;
                const int64_t off = static_cast<int64_t>(at.h) * p.plan.T + d.row0 + iq;
                return e < BT ? p.LSE[off] * LOG2E : p.space.D[off];
            };
            if (d.n_it > 0) slot_f[e] = slot_value();  // nobody reads the slot behind the last item's last barrier
            ptx::named_bar_sync(1, 256);
            // the pooling's share of a raw token: a_m dKc_j + (tau/r) ds_m qsum_j and a_m dVc_j, j its group
            const int c0 = ch * (HD / 2), j = valid ? p.plan.by_g.div(m) : 0;
            const bool fuse = !CORE && p.cores != 0 && valid && j < p.plan.seen_of(d.n);
            const int64_t uj = (static_cast<int64_t>(d.kv) * p.plan.G + d.core0 + j) * HD + c0;
            float am = 0.f, cm = 0.f;
            if (fuse) {
                const int64_t um = static_cast<int64_t>(d.kv) * p.plan.T + d.row0 + m;
                am = p.space.a[um];
                cm = p.space.cds[um];
            }
            for (int x = 0; x < d.n_it; ++x, ++g) {
                const int i0 = at.i0;
                at.next();
                const float v_next = x + 1 < d.n_it ? slot_value() : 0.f;
                if (fuse && x == d.n_it - 1) {
                    // bring this row's half of dKc_j, dVc_j and qsum_j into L1 for the end
#pragma unroll
                    for (int l = 0; l < HD / 64; ++l) {
                        ptx::prefetch_l1(p.space.dKc + uj + 32 * l);
                        ptx::prefetch_l1(p.space.dVc + uj + 32 * l);
                        ptx::prefetch_l1(p.space.qsum + uj + 32 * l);
                    }
                }
                if (ok) ok = c.wait(c.bar(B_S), g & 1);
                uint32_t pa[32], pb[32];
                // this key's visible query columns [q_lo, q_hi] of the tile
                int q_lo = 0, q_hi = -1;
                if (valid && CORE) {
                    q_lo = max((m + 1) * p.plan.g + p.plan.w - 1 - i0, 0);
                    q_hi = min(d.n - 1 - i0, BT - 1);
                } else if (valid) {
                    const int last_i = static_cast<int>(key_last < d.n - 1 ? key_last : d.n - 1);
                    q_lo = max(m - i0, 0);
                    q_hi = min(last_i - i0, BT - 1);
                }
                const uint32_t seen[2] = {ptx::bits(q_lo - h0, q_hi - h0), ptx::bits(q_lo - h0 - 32, q_hi - h0 - 32)};
                const bool whole[2] = {__all_sync(0xffffffffu, seen[0] == 0xffffffffu) != 0, __all_sync(0xffffffffu, seen[1] == 0xffffffffu) != 0};
                if (ok) {
                    ptx::tc_fence_after();
                    const uint32_t sS = lane_addr + h0;
                    ptx::tmem_ld32(sS, pa);
                    ptx::tmem_ld32(sS + 32, pb);
                    ptx::tmem_wait_ld(pa);
                    ptx::reg_touch(pb);
                    // P^T = 2^(S^T tau log2e - LSE), zero off the visible columns (the LSE of four columns per
                    // shared-memory load, the same address across the warp)
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float4 la = slot4[h0 / 4 + q], lb = slot4[h0 / 4 + 8 + q];
                        const float lsa[4] = {la.x, la.y, la.z, la.w}, lsb[4] = {lb.x, lb.y, lb.z, lb.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            pa[4 * q + k] = __float_as_uint(ptx::ex2(fmaf(__uint_as_float(pa[4 * q + k]), c1, -lsa[k])));
                            pb[4 * q + k] = __float_as_uint(ptx::ex2(fmaf(__uint_as_float(pb[4 * q + k]), c1, -lsb[k])));
                        }
                    }
                    clear_unseen(pa, seen[0], whole[0]);
                    clear_unseen(pb, seen[1], whole[1]);
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) pk[k] = ptx::pack_bf16x2(__uint_as_float(pa[2 * k]), __uint_as_float(pa[2 * k + 1]));
                    ptx::tmem_st16(sS, pk);  // P^T over S^T columns [h0, h0 + 16), already read
#pragma unroll
                    for (int k = 0; k < 16; ++k) pk[k] = ptx::pack_bf16x2(__uint_as_float(pb[2 * k]), __uint_as_float(pb[2 * k + 1]));
                    ptx::tmem_st16(sS + 16, pk);
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(c.bar(B_P));
                }
                if (ok) ok = c.wait(c.bar(B_DP), g & 1);
                if (ok) {
                    ptx::tc_fence_after();
                    // dS^T = P^T (dP^T - D), bf16 pairs over dP^T columns [h0, h0 + 32), which this warp has already
                    // read; nothing of a masked value gets on, not as 0 * NaN either
                    const uint32_t sD = lane_addr + T_DP + h0;
                    uint32_t dp[32], dd[16];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        ptx::tmem_ld32(sD + 32 * j, dp);
                        ptx::tmem_wait_ld(dp);
                        clear_unseen(dp, seen[j], whole[j]);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float4 dv = slot4[(BT + h0) / 4 + 8 * j + q];
                            const float Dv[4] = {dv.x, dv.y, dv.z, dv.w};
                            const uint32_t *pp = j ? pb : pa;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int x = 4 * q + 2 * k;
                                dd[2 * q + k] = ptx::pack_bf16x2(__uint_as_float(pp[x]) * (__uint_as_float(dp[x]) - Dv[2 * k]),
                                                                 __uint_as_float(pp[x + 1]) * (__uint_as_float(dp[x + 1]) - Dv[2 * k + 1]));
                            }
                        }
                        ptx::tmem_st16(sD + 16 * j, dd);
                    }
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(c.bar(B_DS));
                }
                // the slot moves on to the next tile once every warp is done with this one
                ptx::named_bar_sync(1, 256);
                slot_f[e] = v_next;
                ptx::named_bar_sync(1, 256);
            }
            if (ok) ok = c.wait(c.bar(B_DONE), it & 1);
            ++it;
            if (!ok) continue;
            // dK * tau and dV, in pieces of 32 columns: of dK, then of dV
            auto store = [&](const uint32_t (&v)[32], int k) {
                const bool of_v = k >= HD / 64;
                const int x0 = c0 + 32 * (k % (HD / 64));
                const float scale = of_v ? 1.f : p.tau;
                if (CORE) {
                    const int64_t at = ((static_cast<int64_t>(d.split) * p.Hkv + d.kv) * p.plan.G + d.core0 + m) * HD + x0;
                    store32_f32(v, scale, (of_v ? p.space.dVc : p.space.dKc) + at);
                } else {
                    const float *add = fuse ? (of_v ? p.space.dVc : p.space.dKc) + uj + 32 * (k % (HD / 64)) : nullptr;
                    const float *qs = fuse && !of_v ? p.space.qsum + uj + 32 * (k % (HD / 64)) : nullptr;
                    store32_bf16(v, scale, add, am, qs, cm, (of_v ? p.dV : p.dK).at(d.kv, d.row0 + m) + x0);
                }
            };
            // Of two items that share these tokens, the warp that comes second adds the other's sums to its own and
            // stores; nobody waits, and a sum of two does not depend on their order.
            int32_t *const there = p.space.there + (static_cast<int64_t>(d.tile) * p.Hkv + d.kv) * 8 + (warp - 2);
            float4 *const parts = reinterpret_cast<float4 *>(p.space.parts) +
                                  ((static_cast<int64_t>(d.tile) * p.Hkv + d.kv) * 8 + (warp - 2)) * 2 * (HD * 8) + lane;
            float4 *const mine = parts + d.split * (HD * 8), *const other = parts + (1 - d.split) * (HD * 8);
            bool second = false;
            if (d.halved) {
                int count = 0;
                if (lane == 0) count = *static_cast<volatile int32_t *>(there);
                second = __shfl_sync(0xffffffffu, count, 0) == 1;
                __threadfence();
            }
            ptx::tc_fence_after();
            // a core tile that no query row sees gets zeros
#pragma unroll
            for (int k = 0; k < HD / 32; ++k) {
                const bool of_v = k >= HD / 64;
                const int x0 = c0 + 32 * (k % (HD / 64));
                uint32_t v[32];
                if (d.n_it > 0) {
                    ptx::tmem_ld32(lane_addr + (of_v ? T_DV : T_DK) + x0, v);
                    ptx::tmem_wait_ld(v);
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q) v[q] = 0u;
                }
                if (k == HD / 32 - 1) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(c.bar(B_ACCFREE));
                }
                if (d.halved) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        if (second) {
                            const float4 o = __ldcg(other + (k * 8 + q) * 32);
                            v[4 * q] = __float_as_uint(__uint_as_float(v[4 * q]) + o.x);
                            v[4 * q + 1] = __float_as_uint(__uint_as_float(v[4 * q + 1]) + o.y);
                            v[4 * q + 2] = __float_as_uint(__uint_as_float(v[4 * q + 2]) + o.z);
                            v[4 * q + 3] = __float_as_uint(__uint_as_float(v[4 * q + 3]) + o.w);
                        } else {
                            __stcg(mine + (k * 8 + q) * 32, make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                                                        __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])));
                        }
                    }
                }
                if (valid && (!d.halved || second)) store(v, k);
            }
            if (d.halved && !second) {
                __threadfence();
                __syncwarp();
                int count = 0;
                if (lane == 0) count = atomicAdd(there, 1);
                if (__shfl_sync(0xffffffffu, count, 0) == 1) {  // both came at the same time: this one is the later
                    __threadfence();
#pragma unroll 1
                    for (int k = 0; k < HD / 32; ++k) {
                        uint32_t v[32];
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float4 a = __ldcg(mine + (k * 8 + q) * 32), b = __ldcg(other + (k * 8 + q) * 32);
                            v[4 * q] = __float_as_uint(a.x + b.x), v[4 * q + 1] = __float_as_uint(a.y + b.y);
                            v[4 * q + 2] = __float_as_uint(a.z + b.z), v[4 * q + 3] = __float_as_uint(a.w + b.w);
                        }
                        if (valid) store(v, k);
                    }
                }
            }
        }
    }
    finish(c, p);
}

template <int HD>
cudaError_t launch(const PackedArgs &a, const PackedBwdSpace &w, int part, cudaStream_t stream) {
    EncodeTiledFn enc = get_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    static std::mutex mu;
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev & 63]) {
            e = cudaFuncSetAttribute(packed_dq_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<HD>::SMEM);
            auto room = [](auto kernel) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<HD>::SMEM); };
            if (e == cudaSuccess) e = room(packed_dkv_tc_kernel<HD, CORES>);
            if (e == cudaSuccess) e = room(packed_dkv_tc_kernel<HD, TOKENS>);
            if (e == cudaSuccess) e = room(packed_dkv_tc_kernel<HD, FEW_TOKENS>);
            if (e != cudaSuccess) return e;
            done[dev & 63] = true;
        }
    }
    CUtensorMap mQ, mdO, mK, mV, mKc, mVc;
    if (!encode_packed_bf16(enc, &mQ, a.Q, HD, a.plan.T, a.Hq) || !encode_packed_bf16(enc, &mdO, a.dO, HD, a.plan.T, a.Hq) ||
        !encode_packed_bf16(enc, &mK, a.K, HD, a.plan.T, a.Hkv) || !encode_packed_bf16(enc, &mV, a.V, HD, a.plan.T, a.Hkv))
        return cudaErrorInvalidValue;
    mKc = mK;  // without cores no tile of them is loaded
    mVc = mV;
    if (a.Kc != nullptr) {
        const int64_t head = static_cast<int64_t>(a.plan.G) * HD;
        const cca_packed_rows_t kc = {const_cast<void *>(a.Kc), head, HD}, vc = {const_cast<void *>(a.Vc), head, HD};
        if (!encode_packed_bf16(enc, &mKc, kc, HD, a.plan.G, a.Hkv) || !encode_packed_bf16(enc, &mVc, vc, HD, a.plan.G, a.Hkv))
            return cudaErrorInvalidValue;
    }
    Args p = {};
    p.plan = a.plan;
    p.dQ = rows_of<__nv_bfloat16>(a.dQ);
    p.dK = rows_of<__nv_bfloat16>(a.dK);
    p.dV = rows_of<__nv_bfloat16>(a.dV);
    p.space = w;
    p.LSE = a.LSE;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.r = a.Hq / a.Hkv;
    p.tau = a.scale;
    p.per = a.Hkv * (part == 0 ? w.splits : w.token_splits);
    p.by_Hq = fast_div(a.Hq);
    p.by_Hkv = fast_div(a.Hkv);
    p.by_r = fast_div(p.r);
    p.by_per = fast_div(p.per);
    p.cores = a.Kc != nullptr;
    p.wait_limit_ns = g_wait_limit_ns;
    p.skip_loads = g_skip_q_load;
    const int64_t most = part == 1 ? static_cast<int64_t>(a.plan.max_tiles) * a.Hq
                                   : static_cast<int64_t>(part == 0 ? a.plan.max_cores : a.plan.max_tiles) * p.per;
    if (most > 0x7fffffff) return cudaErrorNotSupported;
    const int sms = device_sms();
    if (sms < 1) return cudaErrorNoDevice;
    const unsigned grid = static_cast<unsigned>(most < sms ? most : sms);
    if (part == 1)
        return start_dependent(packed_dq_tc_kernel<HD>, dim3(grid), THREADS, Layout<HD>::SMEM, stream, mQ, mdO, mK, mV, mKc, mVc, p);
    auto dkv = [&](auto kernel) {
        return start_dependent(kernel, dim3(grid), THREADS, Layout<HD>::SMEM, stream, mQ, mdO, part == 0 ? mKc : mK, part == 0 ? mVc : mV, p);
    };
    if (part == 0) return dkv(packed_dkv_tc_kernel<HD, CORES>);
    return w.token_splits == 2 ? dkv(packed_dkv_tc_kernel<HD, FEW_TOKENS>) : dkv(packed_dkv_tc_kernel<HD, TOKENS>);
}

}  // namespace

cudaError_t launch_packed_bwd_tc(const PackedArgs &a, const PackedBwdSpace &w, int part, cudaStream_t stream) {
    return a.d == 128 ? launch<128>(a, w, part, stream) : launch<64>(a, w, part, stream);
}

}  // namespace cca
