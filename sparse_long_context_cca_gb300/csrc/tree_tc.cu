// Tree attention on the tcgen05 tensor cores: bf16, d = 128 or 64.  What it computes, the key list
// and the split over the grid are those of tree.cuh; this file is the walk of one CTA over its
// run of 128-key tiles.
//
// One CTA holds HALVES * 128 rows (T nodes times the query heads that share a KV head), so up
// to 256 rows read K and V once; the rows that a small tree leaves empty cost nothing, as the
// loads bound it.  Per tile an SM's share of HBM needs 64 KB / 44 GB/s = 1.5 us (2800 cycles).
// Measured: one half 2300 cycles a tile from L2, so HBM is the bound (64 sequences of one token,
// 32 heads, 8 K: 246 us with weights of one part, 0.94 of the copy bandwidth, 270 us with the two
// that so few rows have); two halves 3500 cycles: 16 sequences x 64 nodes, 32 heads
// over 8, 128 K, 135 us, 4.4 TB/s and 1.1 PFLOP/s.  That is the chain of a half: its softmax (2100
// cycles, two passes over the scores, as 512 threads leave a thread no room for a row), then its
// product, its next scores and the hand-offs (about 1370 in the prefill kernel).  Tensor work is
// 2048, and the operands that the products read from shared memory (192 KB at 128 B a cycle, next to
// 64 KB of copies) take no longer.  64-key tiles with two score buffers per half
// free the softmax from waiting for its product, but their N = 64 products took 740 cycles each:
// 201 us.  A call on little work is a chain: the CTA's run 1.8 us, page look-up and first copy
// 2.5 us, first softmax 1.4 us, output 1.5 us, then the join (one token of 32 heads at 32 K,
// 49 MB: 19.2 us warm, 24.0 us from HBM).
// At d = 64 a tile is half as long to copy (1400 cycles) and its softmax (2100) is the bound: 8
// sequences of 24 nodes, 32 heads over 8, up to 32 K: 23.6 us (38.4 by mma.sync).
//
// Roles (warpgroups of four warps):
//   0 .. HALVES-1   softmax and output of a half; thread t owns row t of it (TMEM lane t).
//                   They also bring their half's queries, while the last tile's product runs.
//   HALVES          producers, 32 keys of a tile per warp, page look-ups a tile ahead.  Tiles of
//                   runs (whole boxes of consecutive rows of a page) come by TMA, a box per
//                   lane; the rest, one to four tiles of a list, by cp.async, a key per lane to
//                   look up and 16 lanes to a row to copy, so any page size and alignment goes.
//                   Both fill 128-byte-swizzled tiles.
//   HALVES+1        its first warp issues the MMAs.
// K(t) and V(t) take two consecutive slots of a ring of NS tiles and are freed apart: K
// when its scores are done, V when its product is (both at once cost a load's latency per tile:
// 230 us in place of 158 at the time).
//
// Up to TWO_PART_ROWS rows the weights keep two parts: lanes 16 .. 31 of the first warp hold the
// same rows again (their queries too, so their scores and weights are the same to the bit) and put
// the weights' low parts into P, and the two outputs of a row are added at the list's end.  That
// costs three instructions for two weights and no matrix work: one token of 32 heads at 32 K 18.0 -> 19.2
// us, 64 sequences of one token at 8 K 246 -> 270, with 32 heads over 8 69 -> 75.
//
// Two halves: S_A | S_B | O_A | O_B fill the tensor memory; the halves' softmaxes and MMAs
// alternate.  P_h overwrites S_h, and S_h of the next tile is issued after the product that
// reads P_h, so a finished S_h means that all earlier products of the half are done.
// One half: two score buffers, so that the next tile's scores are made during this one's
// softmax; the softmax then waits for the earlier product itself before it touches O.
//
// Every wait is bounded: on a time-out the CTA stops, drains, frees its tensor memory and
// reports CCA_ERR_TIMEOUT.  The warps of a role may disagree on whether a wait ran out (one looks
// before the barrier completes and sees another role's time-out, the next looks after), so nothing
// but such waits joins them between the CTA's two __syncthreads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/cca.h"
#include "internal.h"
#include "paged.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.h"
#include "tree.cuh"

namespace cca {
namespace tree {
namespace {

constexpr int BN = 128;                       // keys per tile
constexpr uint32_t HALF_BYTES = BN * 128;     // 64 columns of a tile
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_O = 256;
constexpr float LAZY_RESCALE_LOG2 = 16.0f;  // keep a stale max while it is within 2^16
constexpr uint32_t IDESC_QK = ptx::idesc_bf16_f32(128, BN, 0, 0);  // Q, K both K-major
constexpr int METAS = 8;

// What the softmax needs to know of a tile's keys, a bit for each.
struct TileMeta {
    uint32_t gone[4];  // there is no such key: no page, or past the end of the list
    uint32_t odd[4];   // its V holds an infinity or NaN, and not every row sees it
};

template <int HALVES, int D>
struct Layout {
    static constexpr uint32_t TILE_BYTES = BN * D * 2;
    // ring slots: what 227 KB leave next to the queries and the bookkeeping; four tiles are enough
    static constexpr int NS = D == 64 ? 8 : HALVES == 2 ? 4 : 5;
    static_assert(METAS >= NS / 2 + 2, "a tile's bits stay until its softmax is over");
    static constexpr int THREADS = (HALVES + 2) * 128;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_RING = HALVES * TILE_BYTES;
    static constexpr uint32_t OFF_META = OFF_RING + NS * TILE_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_META + METAS * sizeof(TileMeta);
    static constexpr int B_FULL = 0;                  // NS
    static constexpr int B_EMPTY = B_FULL + NS;       // NS
    static constexpr int B_QFULL = B_EMPTY + NS;      // HALVES
    static constexpr int B_SFULL = B_QFULL + HALVES;  // 2: per half, or per score buffer
    static constexpr int B_PFULL = B_SFULL + 2;       // HALVES
    static constexpr int B_PVDONE = B_PFULL + HALVES; // HALVES: two halves per list, one half per tile
    static constexpr int B_OFREE = B_PVDONE + HALVES; // HALVES
    static constexpr int B_DRAIN = B_OFREE + HALVES;
    static constexpr int NUM_BARS = B_DRAIN + 1;
    static constexpr uint32_t OFF_TMEMPTR = OFF_BAR + NUM_BARS * 8;
    static constexpr uint32_t OFF_ABORT = OFF_TMEMPTR + 4;
    static constexpr uint32_t OFF_START = (OFF_ABORT + 4 + 15) / 16 * 16;
    static constexpr uint32_t OFF_NODES = (OFF_START + sizeof(Start) + 15) / 16 * 16;
    // then, per half: bits of every row [128][words]; per softmax warp: parents [T]
    static uint32_t bytes(int T) { return OFF_NODES + HALVES * (128 * 4 * ((T + 31) / 32) + 4 * 2 * ((T + 1) / 2 * 2)) + 1024; }
};

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// TWO_PARTS: up to TWO_PART_ROWS rows (with one half).
template <int HALVES, int D, bool TWO_PARTS>
__global__ void __launch_bounds__((HALVES + 2) * 128, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmKc, const __grid_constant__ CUtensorMap tmVc, const TreeArgs a,
                   const unsigned long long lim, const int skip_loads) {
    using L = Layout<HALVES, D>;
    constexpr int NS = L::NS;
    constexpr uint32_t TILE_BYTES = L::TILE_BYTES;
    constexpr uint32_t IDESC_PV = ptx::idesc_bf16_f32(128, D, 0, 1);  // P in tensor memory, V MN-major
    constexpr int CHUNKS = D / 8;              // 16-byte chunks of a row
    constexpr int ROWS_AT_ONCE = 32 / CHUNKS;  // rows that a warp copies at once
    constexpr int BM = HALVES * 128;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    auto bar = [&](int idx) -> uint32_t { return base + L::OFF_BAR + 8u * idx; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + L::OFF_ABORT);
    TileMeta *metas = reinterpret_cast<TileMeta *>(gbase + L::OFF_META);
    Start &st = *reinterpret_cast<Start *>(gbase + L::OFF_START);
    const int words = (a.T + 31) >> 5;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wg = warp >> 2;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(bar(L::B_FULL + s), 4);  // producer warps
            ptx::mbar_init(bar(L::B_EMPTY + s), 1);
        }
        for (int h = 0; h < HALVES; ++h) {
            ptx::mbar_init(bar(L::B_QFULL + h), 4);  // softmax warps
            ptx::mbar_init(bar(L::B_PFULL + h), 4);
            ptx::mbar_init(bar(L::B_PVDONE + h), 1);
            ptx::mbar_init(bar(L::B_OFREE + h), 4);
        }
        // the scores are done, and the issuer's own arrival: what the producers wrote about the
        // tile before they handed it over is visible behind it
        ptx::mbar_init(bar(L::B_SFULL), 2);
        ptx::mbar_init(bar(L::B_SFULL + 1), 2);
        ptx::mbar_init(bar(L::B_DRAIN), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc(base + L::OFF_TMEMPTR, TMEM_COLS);
        ptx::tmem_relinquish();
    }
    if (warp == HALVES * 4 && lane < 4) ptx::prefetch_tmap(lane == 0 ? &tmK : lane == 1 ? &tmV : lane == 2 ? &tmKc : &tmVc);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<uint32_t *>(gbase + L::OFF_TMEMPTR);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int mt = blockIdx.x % a.n_mt, group = blockIdx.x / a.n_mt;
    const Run run = find_run(a, group, st);
    const int x0 = run.x0, x1 = run.x1;
    const bool half_used[2] = {true, HALVES == 2 && mt * BM + 128 < a.R};
    int last_bulk = -1;  // of a producer warp: the last slot fill that went by TMA

    if (wg == HALVES) {
        // ------------------------------------------------------------ producers
        const int pw = warp & 3;
        const int sub = lane / CHUNKS, chunk = lane % CHUNKS;
        bool ok = x0 < x1 && !skip_loads;
        Item it = run.item;
        // the tile to load next: a lane's box of runs, or a lane's key of the rest
        bool runs = false, core = false;
        int box_y = 0;
        const char *kp = nullptr, *vp = nullptr;
        uint32_t gone = 0, mixed = 0;  // per key of this warp: not there; seen by some rows only
        const int per_warp = a.box_log2 > 0 ? 32 >> a.box_log2 : 0;  // boxes of a warp
        auto look_up = [&](int x) {
            const int tile = x - it.first;
            runs = tile < it.k.run_tiles;
            mixed = 0;
            if (runs) {
                int64_t row = 0;
                if (lane < per_warp) {
                    row = find_box(a, it.k, it.b, it.kv, (tile * 4 + pw) * per_warp + lane, core);
                    // no page: past the pool's end, where the copy fills in zeros
                    box_y = static_cast<int>(row >= 0 ? row : static_cast<int64_t>(core ? a.n_cpages : a.n_pages) * a.Hkv * (core ? a.crows : a.rows));
                }
                gone = __ballot_sync(kFull, row < 0);  // a bit per box; usually none
                if (gone != 0) gone = __ballot_sync(kFull, (gone >> (lane >> a.box_log2)) & 1u);
                return;
            }
            const Key key = settled(a, it.b, find_key(a, it.k, it.b, it.kv, (tile - it.k.run_tiles) * BN + pw * 32 + lane));
            kp = key.row < 0 ? nullptr : static_cast<const char *>(key.core ? a.Kc : a.K) + key.row * (D * 2);
            vp = key.row < 0 ? nullptr : static_cast<const char *>(key.core ? a.Vc : a.V) + key.row * (D * 2);
            gone = __ballot_sync(kFull, key.kind == 4);
            mixed = __ballot_sync(kFull, key.kind != 0 && key.kind != 4);
        };
        // a slot whose cp.async copies are in flight behind the one being filled
        int held = -1, held_meta = 0;
        uint32_t held_mixed = 0;
        bool held_v = false;
        auto land = [&]() {  // its copies (of this thread) have arrived
            if (held < 0) return;
            if (held_v && held_mixed != 0) {
                // infinities and NaN in the V of a key that only some rows see would reach the others
                // as 0 * NaN: they leave the tile, and the rows that see the key add them themselves
                auto at = [&](int r) {
                    return reinterpret_cast<uint4 *>(gbase + L::OFF_RING + held * TILE_BYTES + (chunk >> 3) * HALF_BYTES +
                                                     (pw * 32 + r) * 128 + (((chunk & 7) ^ (r & 7)) << 4));
                };
                // an exponent of all ones carries into the sign's place
                auto carry = [](uint32_t v) { return (v & 0x7f807f80u) + 0x00800080u; };
                uint32_t any = 0;
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
                    const uint4 v = *at(ROWS_AT_ONCE * j + sub);
                    any |= carry(v.x) | carry(v.y) | carry(v.z) | carry(v.w);
                }
                for (int j = 0; (any & 0x80008000u) != 0 && j < CHUNKS; ++j) {
                    const int r = ROWS_AT_ONCE * j + sub, row = pw * 32 + r;
                    if (!((held_mixed >> r) & 1u)) continue;
                    uint4 *p = at(r);
                    uint32_t v[4] = {p->x, p->y, p->z, p->w};
                    bool hit = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if ((v[i] & 0x7f80u) == 0x7f80u) {
                            v[i] &= 0xffff0000u;
                            hit = true;
                        }
                        if ((v[i] & 0x7f800000u) == 0x7f800000u) {
                            v[i] &= 0xffffu;
                            hit = true;
                        }
                    }
                    if (hit) {
                        *p = make_uint4(v[0], v[1], v[2], v[3]);
                        atomicOr(&metas[held_meta].odd[row >> 5], 1u << (row & 31));
                    }
                }
            }
            ptx::fence_proxy_async_smem();  // the MMAs read what this thread has written
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(L::B_FULL + held));
            held = -1;
        };
        if (ok) look_up(x0);
        for (int u = 0; ok && u < 2 * (x1 - x0); ++u) {
            const int x = x0 + (u >> 1), slot = u % NS;
            const bool is_v = u & 1;
            // Before it waits for room, or fills a slot by TMA, what is in flight is handed over: the
            // room may depend on it.
            const uint32_t parity = ((u / NS) & 1) ^ 1;
            if (held >= 0 && (runs || !__all_sync(kFull, ptx::mbar_try_wait(bar(L::B_EMPTY + slot), parity)))) {
                cp_wait<0>();
                land();
            }
            if (!__all_sync(kFull, ptx::wait_bounded(bar(L::B_EMPTY + slot), parity, abort_flag, lim))) {
                ok = false;
                break;
            }
            if (!is_v && lane == 0) {
                // The tile of METAS before: its softmax is over, as the scores that freed this slot were
                // issued behind it.
                metas[(x - x0) & (METAS - 1)].gone[pw] = gone;
                metas[(x - x0) & (METAS - 1)].odd[pw] = 0;
            }
            __syncwarp();
            const uint32_t dst = base + L::OFF_RING + slot * TILE_BYTES;
            if (runs) {
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar(L::B_FULL + slot), 32 * D * 2);
                __syncwarp();
                if (lane < per_warp) {
                    const uint32_t at = dst + (pw * 32 + (lane << a.box_log2)) * 128;
                    const void *map = is_v ? (core ? static_cast<const void *>(&tmVc) : static_cast<const void *>(&tmV))
                                           : (core ? static_cast<const void *>(&tmKc) : static_cast<const void *>(&tmK));
                    ptx::tma_load_2d(map, bar(L::B_FULL + slot), at, 0, box_y);
                    if constexpr (D == 128) ptx::tma_load_2d(map, bar(L::B_FULL + slot), at + HALF_BYTES, 64, box_y);
                }
                last_bulk = u;
                __syncwarp();
            } else {
                const unsigned long long mine = reinterpret_cast<unsigned long long>(is_v ? vp : kp);
#pragma unroll 4
                for (int j = 0; j < CHUNKS; ++j) {
                    const int row = pw * 32 + ROWS_AT_ONCE * j + sub;
                    const char *p = reinterpret_cast<const char *>(__shfl_sync(kFull, mine, ROWS_AT_ONCE * j + sub));
                    cp16(dst + (chunk >> 3) * HALF_BYTES + row * 128 + (((chunk & 7) ^ (row & 7)) << 4),
                         p == nullptr ? static_cast<const char *>(a.K) : p + chunk * 16, p != nullptr);
                }
                cp_commit();
                if (held >= 0) {
                    cp_wait<1>();
                    land();
                }
                held = slot;
                held_v = is_v;
                held_mixed = mixed;
                held_meta = (x - x0) & (METAS - 1);
            }
            if (is_v && x + 1 < x1) {
                if (x + 1 >= it.first + it.k.tiles) next_item(a, it);
                look_up(x + 1);
            }
        }
        cp_wait<0>();
        if (ok) land();
        __syncwarp();
    } else if (wg == HALVES + 1) {
        // ------------------------------------------------------------ MMA issuer
        if ((warp & 3) == 0) {
            auto wwait = [&](int b, uint32_t parity) -> bool {
                return __all_sync(kFull, ptx::wait_bounded(bar(b), parity, abort_flag, lim));
            };
            auto slot_full = [&](int u) -> bool { return wwait(L::B_FULL + u % NS, (u / NS) & 1); };
            const uint64_t dq = ptx::smem_desc_sw128(base + L::OFF_Q, 16, 1024);
            const uint64_t dk = ptx::smem_desc_sw128(base + L::OFF_RING, 16, 1024);
            const uint64_t dv = ptx::smem_desc_sw128(base + L::OFF_RING, HALF_BYTES, 1024);
            constexpr uint64_t STEP = TILE_BYTES >> 4;
            bool ok = true;
            uint32_t seg = 0, pcount = 0;  // lists; tiles whose P was waited for
            Item it = run.item;
            int x = x0;
            // S = Q_h K(t)^T into score buffer `buf`; K(t) has been waited for
            auto scores = [&](int h, int buf, int t) {
                ptx::tc_fence_after();
                const uint64_t k = dk + (2 * (t - x0) % NS) * STEP;
                if constexpr (D == 128) ptx::mma_ss_k128_warp(tmem + buf * 128, dq + h * STEP, k, IDESC_QK, 0u);
                else ptx::mma_ss_k64_warp(tmem + buf * 128, dq + h * STEP, k, IDESC_QK, 0u);
                ptx::tc_commit_warp(bar(L::B_SFULL + buf));
                if (lane == 0) ptx::mbar_arrive(bar(L::B_SFULL + buf));
                __syncwarp();
            };
            while (ok && x < x1) {
                const int end = min(it.first + it.k.tiles, x1);
                if constexpr (HALVES == 2) {
                    for (int h = 0; ok && h < 2; ++h) {
                        if (!half_used[h]) continue;
                        ok = wwait(L::B_QFULL + h, seg & 1) && slot_full(2 * (x - x0));
                        if (ok) scores(h, h, x);
                    }
                    if (!ok) break;
                    ptx::tc_commit_warp(bar(L::B_EMPTY + 2 * (x - x0) % NS));
                    for (int t = x; ok && t < end; ++t) {
                        const int u = 2 * (t - x0) + 1;
                        if (!slot_full(u)) {
                            ok = false;
                            break;
                        }
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            if (!half_used[h]) continue;
                            if (!wwait(L::B_PFULL + h, pcount & 1) || (t == x && !wwait(L::B_OFREE + h, (seg & 1) ^ 1))) {
                                ok = false;
                                break;
                            }
                            ptx::tc_fence_after();
                            ptx::mma_ts_k128_warp(tmem + TM_O + h * 128, tmem + h * 128, dv + (u % NS) * STEP, IDESC_PV, t == x ? 0u : 1u);
                            if (t + 1 < end) {
                                if (!slot_full(u + 1)) {
                                    ok = false;
                                    break;
                                }
                                scores(h, h, t + 1);
                            } else {
                                ptx::tc_commit_warp(bar(L::B_PVDONE + h));
                            }
                        }
                        if (!ok) break;
                        ptx::tc_commit_warp(bar(L::B_EMPTY + u % NS));
                        if (t + 1 < end) ptx::tc_commit_warp(bar(L::B_EMPTY + (u + 1) % NS));
                        ++pcount;
                    }
                } else {
                    ok = wwait(L::B_QFULL, seg & 1);
                    for (int t = x; ok && t <= end; ++t) {
                        // the scores of tile t, then the product of tile t - 1
                        if (t < end) {
                            const int u = 2 * (t - x0);
                            if (!slot_full(u)) {
                                ok = false;
                                break;
                            }
                            scores(0, (t - x0) & 1, t);
                            ptx::tc_commit_warp(bar(L::B_EMPTY + u % NS));
                        }
                        if (t == x) continue;
                        const int u = 2 * (t - 1 - x0) + 1;
                        if (!slot_full(u) || !wwait(L::B_PFULL, pcount & 1) || (t - 1 == x && !wwait(L::B_OFREE, (seg & 1) ^ 1))) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        ptx::mma_ts_k128_warp(tmem + TM_O, tmem + ((t - 1 - x0) & 1) * 128, dv + (u % NS) * STEP, IDESC_PV, t - 1 == x ? 0u : 1u);
                        ptx::tc_commit_warp(bar(L::B_PVDONE));
                        ptx::tc_commit_warp(bar(L::B_EMPTY + u % NS));
                        ++pcount;
                    }
                }
                ++seg;
                x = end;
                if (x < x1) next_item(a, it);
            }
            // Whatever was issued must complete before tensor memory is freed.
            ptx::tc_commit_warp(bar(L::B_DRAIN));
            volatile int never = 0;
            ptx::wait_bounded(bar(L::B_DRAIN), 0, &never, lim);
        }
        __syncwarp();
    } else if (wg == 0 || half_used[1]) {
        // ------------------------------------------------------------ softmax and output
        const int h = HALVES == 2 ? wg : 0;
        const int quarter = warp & 3;
        // A lane's row among its warp's 32; with two parts lane 16 + r has row r again, for the low ones.
        auto row_of = [](int r) { return TWO_PARTS ? r & (TWO_PART_ROWS - 1) : r; };
        const int in = h * 128 + quarter * 32 + row_of(lane);  // row of the CTA
        const int row = mt * BM + in;                          // row of the KV head
        const bool live = row < a.R;
        const bool mine = live && row_of(lane) == lane;        // it writes the row
        const uint32_t cut = row_of(lane) == lane ? 0u : 0xffff0000u;
        const float more = row_of(lane) == lane ? 1.f : LOW_MORE;
        const bool idle = mt * BM + h * 128 + quarter * 32 >= a.R;  // no row of this warp
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tO = tmem + lane_addr + TM_O + h * 128;
        uint32_t *const sees = reinterpret_cast<uint32_t *>(gbase + L::OFF_NODES) + (h * 128 + quarter * 32 + lane) * words;
        int16_t *const up = reinterpret_cast<int16_t *>(gbase + L::OFF_NODES + HALVES * 512 * words) + (h * 4 + quarter) * ((a.T + 1) / 2 * 2);
        const int node = live ? row % a.T : 0;
        bool ok = true;
        uint32_t seg = 0, n_s = 0;  // lists and tiles of this half so far
        Item it = run.item, nxt = run.item;
        int tree_of = -1;
        int start = 0, cores = -1;  // this row's first raw token; its visible cores, -1: empty node
        const int heads = a.Hq / a.Hkv;
        auto list_row = [&](const Item &i) { return (static_cast<int64_t>(i.b) * a.Hq + static_cast<int64_t>(i.kv) * heads) * a.T; };
        // The queries of this warp's rows, 16 lanes to a row, swizzled like the keys.  The scores of
        // the last tile are done, so nothing reads the old ones.
        auto load_q = [&](const Item &i) {
            const char *q = static_cast<const char *>(a.Q) + (list_row(i) + mt * BM + h * 128 + quarter * 32) * (D * 2);
            const int sub = lane / CHUNKS, chunk = lane % CHUNKS;
#pragma unroll 4
            for (int j = 0; j < CHUNKS; ++j) {
                const int r = ROWS_AT_ONCE * j + sub;
                const bool there = mt * BM + h * 128 + quarter * 32 + row_of(r) < a.R;
                cp16(base + L::OFF_Q + h * TILE_BYTES + (chunk >> 3) * HALF_BYTES + (quarter * 32 + r) * 128 + (((chunk & 7) ^ (r & 7)) << 4),
                     there ? q + row_of(r) * (D * 2) + chunk * 16 : static_cast<const char *>(a.Q), there);
            }
            cp_commit();
        };
        auto hand_q = [&]() {
            cp_wait<0>();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(L::B_QFULL + h));
        };
        // The list's tree: parents in this warp's own shared memory, each row walks its own chain.
        auto read_nodes = [&]() {
            if (it.b == tree_of) return;
            tree_of = it.b;
            __syncwarp();  // the old parents have been used
            for (int t = lane; t < a.T; t += 32) up[t] = static_cast<int16_t>(parent_of(a, it.b, t));
            __syncwarp();
            for (int i = 0; i < words; ++i) sees[i] = 0;
            const Chain c = walk_chain(up, sees, node);
            const int lo = window_lo(it.k.len + c.depth, a.w), vis = a.by_g.div(lo);
            cores = live && c.whole && it.k.n > 0 ? vis : -1;
            start = a.window_mode ? vis * a.g : lo;
        };
        // Bits of the 32 keys from key `x` of the rest on that this row sees.
        auto seen = [&](int x) {
            const int A = it.k.n_all, nc = it.k.cores_some - it.k.cores_all, nr = it.k.raw_all - it.k.raw_some;
            const int vc = min(max(cores - it.k.cores_all, 0), nc);      // of the cores that some see: the first vc
            const int sr = min(max(start - it.k.raw_some, 0), nr);       // of the raw tokens: all but the first sr
            uint32_t m = low_bits(A + vc - x) | (low_bits(A + nc + nr - x) & ~low_bits(A + nc + sr - x));
            const int n0 = x - (A + nc + nr);                            // node of bit 0
            if (n0 > -32 && n0 < a.T) {
                const int w0 = n0 >> 5;
                const uint32_t lo = w0 >= 0 ? sees[w0] : 0u, hi = w0 + 1 < words ? sees[w0 + 1] : 0u;
                m |= __funnelshift_r(lo, hi, n0 & 31);
            }
            return m;
        };
        if (x0 < x1) {
            load_q(it);
            hand_q();
            read_nodes();  // while the first scores are under way
        }
        int x = x0;
        while (ok && x < x1) {
            const int end = min(it.first + it.k.tiles, x1);
            float m = -INFINITY, l = 0.f;
            bool has_odd = false;
            float *const part = part_at(a, group, mt, x0 >= it.first ? 0 : 1, BM, D);
            if (it.k.n == 0 && threadIdx.x == 0) report(a.status, CCA_ERR_INVALID_ARG);
            for (int t = x; t < end; ++t, ++n_s) {
                const int buf = HALVES == 2 ? h : (t - x0) & 1;
                if (!__all_sync(kFull, ptx::wait_bounded(bar(L::B_SFULL + buf), HALVES == 2 ? n_s & 1 : (n_s >> 1) & 1, abort_flag, lim))) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                if (t + 1 == end && end < x1) {  // the last tile of this list: its scores have read the queries
                    nxt = it;
                    next_item(a, nxt);
                    load_q(nxt);
                }
                const uint32_t tS = tmem + lane_addr + buf * 128;
                const TileMeta &tm = metas[(t - x0) & (METAS - 1)];
                const int rest = t - it.first - it.k.run_tiles;  // tile of the rest, < 0: runs
                const uint4 gone = *reinterpret_cast<const uint4 *>(tm.gone);
                const bool masked = rest >= 0 || (gone.x | gone.y | gone.z | gone.w) != 0;
                auto mask_of = [&](int c) {  // of columns 32c .. 32c + 31
                    return (rest >= 0 ? seen(rest * BN + c * 32) : 0xffffffffu) & ~tm.gone[c];
                };
                if (!idle) {
                    // the row's maximum; 64 columns at a time, which keeps the code short (a launch
                    // begins with cold instruction caches) and the registers few.  A masked tile has
                    // a pass of its own: -inf into the scores that the row does not see, here and
                    // where they are.
                    float mx = -INFINITY;
                    auto maximum = [&](auto with_masks) {
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            uint32_t s[2][32];
                            ptx::tmem_ld32(tS + c * 64, s[0]);
                            ptx::tmem_ld32(tS + c * 64 + 32, s[1]);
                            uint32_t see[2] = {};
                            if constexpr (with_masks.value) {
                                see[0] = mask_of(2 * c);
                                see[1] = mask_of(2 * c + 1);
                            }
                            ptx::tmem_wait_ld(s[0]);
                            ptx::reg_touch(s[1]);
                            if constexpr (with_masks.value) {
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    if (__all_sync(kFull, see[j] == 0xffffffffu)) continue;
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        if (!((see[j] >> k) & 1u)) s[j][k] = __float_as_uint(-INFINITY);
                                    ptx::tmem_st16(tS + c * 64 + j * 32, reinterpret_cast<const uint32_t(&)[16]>(s[j][0]));
                                    ptx::tmem_st16(tS + c * 64 + j * 32 + 16, reinterpret_cast<const uint32_t(&)[16]>(s[j][16]));
                                }
                            }
                            float mp[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                mp[q] = fmaxf(__uint_as_float(s[q >> 1][(q & 1) * 16]), __uint_as_float(s[q >> 1][(q & 1) * 16 + 1]));
#pragma unroll
                                for (int k = 2; k < 16; k += 2)
                                    mp[q] = ptx::max3(mp[q], __uint_as_float(s[q >> 1][(q & 1) * 16 + k]), __uint_as_float(s[q >> 1][(q & 1) * 16 + k + 1]));
                            }
                            mx = fmaxf(ptx::max3(mx, mp[0], mp[1]), fmaxf(mp[2], mp[3]));
                        }
                    };
                    if (masked) {
                        maximum(std::true_type());
                        ptx::tmem_wait_st();
                    } else {
                        maximum(std::false_type());
                    }
                    const float m_new = fmaxf(m, mx * a.scale_log2);
                    bool rescale = false;
                    if (m == -INFINITY) {
                        m = m_new;  // nothing accumulated yet for this row
                    } else if (m_new > m + LAZY_RESCALE_LOG2) {
                        rescale = true;
                    }
                    if (__any_sync(kFull, rescale)) {
                        if constexpr (HALVES == 1) {  // the earlier product must be done with O
                            if (!__all_sync(kFull, ptx::wait_bounded(bar(L::B_PVDONE), (n_s & 1) ^ 1, abort_flag, lim))) {
                                ok = false;
                                break;
                            }
                            ptx::tc_fence_after();
                        }
                        const float f = rescale ? ptx::ex2(m - m_new) : 1.f;
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            ptx::tmem_ld16(tO + c * 16, o);
                            ptx::tmem_wait_ld16(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            ptx::tmem_st16(tO + c * 16, o);
                        }
                        if (rescale) {
                            l *= f;
                            m = m_new;
                        }
                    }
                    const float mu = m == -INFINITY ? 0.f : m;
                    if (rest >= 0) {
                        // V(t)'s slot is not filled again before this softmax is over: what the producers
                        // took out of it is known now
                        const int u = 2 * (t - x0) + 1;
                        if (!__all_sync(kFull, ptx::wait_bounded(bar(L::B_FULL + u % NS), (u / NS) & 1, abort_flag, lim))) {
                            ok = false;
                            break;
                        }
                    }
                    if (rest >= 0 && (tm.odd[0] | tm.odd[1] | tm.odd[2] | tm.odd[3]) != 0) {
                        // what the producers took out of V, for the rows that see it: the sums of
                        // infinities and NaN wait in this row of the CTA's partial for the output
#pragma unroll 1
                        for (int col = 0; col < BN; ++col) {
                            if (!((tm.odd[col >> 5] >> (col & 31)) & 1u)) continue;
                            __syncwarp();
                            uint32_t sc;
                            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(sc) : "r"(tS + col));
                            if (!mine || __uint_as_float(sc) == -INFINITY) continue;
                            const float p = ptx::ex2(fmaf(__uint_as_float(sc), a.scale_log2, -mu));
                            const Key key = find_key(a, it.k, it.b, it.kv, rest * BN + col);
                            const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(key.core ? a.Vc : a.V) + key.row * D;
                            for (int e = 0; e < D; ++e) {
                                const float f = __bfloat162float(v[e]);
                                float &sum = part[part_col(BM, in, e)];
                                const float before = has_odd ? sum : 0.f;
                                sum = f - f != 0.f ? before + p * f : before;
                            }
                            has_odd = true;
                        }
                        __syncwarp();
                    }
                    // p = 2^(s*scale - mu), two columns per packed FMA; P rounds to bf16 (see
                    // TWO_PART_ROWS), the sum does not
                    const uint64_t sc2 = ptx::f2(a.scale_log2, a.scale_log2);
                    const uint64_t nm2 = ptx::f2(-mu, -mu);
                    uint64_t lp[2] = {0, 0};
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t s[2][32];
                        ptx::tmem_ld32(tS + c * 64, s[0]);
                        ptx::tmem_ld32(tS + c * 64 + 32, s[1]);
                        ptx::tmem_wait_ld(s[0]);
                        ptx::reg_touch(s[1]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t pk[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int col = (q & 1) * 16 + 2 * k;
                                const uint64_t x2 = ptx::fma2(ptx::f2(__uint_as_float(s[q >> 1][col]), __uint_as_float(s[q >> 1][col + 1])), sc2, nm2);
                                float y0, y1;
                                ptx::f2_split(x2, y0, y1);
                                float p0 = ptx::ex2(y0);
                                float p1 = ptx::ex2(y1);
                                lp[k & 1] = ptx::add2(lp[k & 1], ptx::f2(p0, p1));
                                if constexpr (TWO_PARTS) {
                                    low_parts(p0, p1, cut, more);
                                    pk[k] = ptx::cut_bf16x2(p0, p1);
                                } else {
                                    pk[k] = ptx::pack_bf16x2(p0, p1);
                                }
                            }
                            ptx::tmem_st8(tS + c * 32 + q * 8, pk);  // P over scores that have been read
                        }
                    }
                    float a0, a1, b0, b1;
                    ptx::f2_split(lp[0], a0, a1);
                    ptx::f2_split(lp[1], b0, b1);
                    l += (a0 + a1) + (b0 + b1);
                    ptx::tmem_wait_st();
                }
                if constexpr (HALVES == 1) {
                    // the product of the tile before: done by now, and its barrier must not run ahead
                    if (n_s > 0 && !__all_sync(kFull, ptx::wait_bounded(bar(L::B_PVDONE), (n_s & 1) ^ 1, abort_flag, lim))) {
                        ok = false;
                        break;
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(L::B_PFULL + h));
            }
            if (!ok) break;
            if (end < x1) hand_q();  // the next list's
            const bool empty = cores < 0;
            if (!__all_sync(kFull, ptx::wait_bounded(bar(L::B_PVDONE + h), HALVES == 2 ? seg & 1 : (n_s & 1) ^ 1, abort_flag, lim))) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            if (__any_sync(kFull, has_odd)) {
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t v[16];
                    ptx::tmem_ld16(tO + c * 16, v);
                    ptx::tmem_wait_ld16(v);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) + (has_odd ? part[part_col(BM, in, c * 16 + k)] : 0.f));
                    ptx::tmem_st16(tO + c * 16, v);
                }
                ptx::tmem_wait_st();
            }
            if (empty) {
                m = -INFINITY;
                l = 0.f;
            }
            const bool nothing = l == 0.f;  // no visible key in this part (or an empty node)
            const bool whole = x0 <= it.first && it.first + it.k.tiles <= x1;
            const float scale = nothing ? 0.f : whole ? 1.f / l : 1.f;
            const int64_t out = list_row(it) + row;
            if (!idle) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    __syncwarp();
                    uint32_t o[32];
                    ptx::tmem_ld32(tO + c * 32, o);
                    ptx::tmem_wait_ld(o);
                    if constexpr (TWO_PARTS) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) + __shfl_down_sync(kFull, __uint_as_float(o[k]), TWO_PART_ROWS));
                    }
                    if (!mine) continue;
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = nothing ? 0u : __float_as_uint(__uint_as_float(o[k]) * scale);
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.O) + out * D + c * 32);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                v[k] = ptx::pack_bf16x2(__uint_as_float(o[8 * q + 2 * k]), __uint_as_float(o[8 * q + 2 * k + 1]));
                            dst[q] = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(part + part_col(BM, in, c * 32));
#pragma unroll
                        for (int q = 0; q < 8; ++q) dst[q * BM] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(L::B_OFREE + h));
            if (mine) {
                if (whole) {
                    a.LSE[out] = nothing ? -INFINITY : (m + log2f(l)) * kLn2;
                } else {
                    part[BM * D + in] = m;
                    part[BM * D + BM + in] = l;
                }
            }
            if (threadIdx.x == 0 && mt == 0) note_span(a, it, group, x0, x1);
            ++seg;
            x = end;
            if (x < x1) {
                it = nxt;
                read_nodes();
            }
        }
        cp_wait<0>();
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (*abort_flag && wg == HALVES && lane == 0) {
        // Bulk copies already issued land before the CTA's memory is given back.  A producer may have
        // been through before another role gave up, so this is asked behind the barrier.  A fill that
        // other warps left unfinished never completes: one such wait is long enough for all.
        volatile int never = 0;
        for (int u = last_bulk >= NS ? last_bulk - NS + 1 : 0; u <= last_bulk; ++u)
            if (!ptx::wait_bounded(bar(L::B_FULL + u % NS), (u / NS) & 1, &never, lim)) break;
    }
    if (*abort_flag && threadIdx.x == 0) report(a.status, CCA_ERR_TIMEOUT);
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int HALVES, int D, bool TWO_PARTS = false>
cudaError_t launch_halves(const CUtensorMap (&map)[4], const TreeArgs &a, unsigned long long lim, int skip_loads, cudaStream_t stream) {
    static std::atomic<int> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev].load(std::memory_order_relaxed) == 0) {
        e = cudaFuncSetAttribute(tree_tc_kernel<HALVES, D, TWO_PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(1, std::memory_order_relaxed);
    }
    return start_dependent(tree_tc_kernel<HALVES, D, TWO_PARTS>, dim3(static_cast<unsigned>(a.groups) * a.n_mt), Layout<HALVES, D>::THREADS,
                           static_cast<int>(Layout<HALVES, D>::bytes(a.T)), stream, map[0], map[1], map[2], map[3], a, lim, skip_loads);
}

}  // namespace

int tc_rows(int R) { return R <= 128 ? 128 : 256; }

cudaError_t launch_tc(TreeArgs a, int d, unsigned long long wait_limit_ns, int skip_loads, cudaStream_t stream) {
    // Runs: boxes of 32, 16 or 8 rows, the most that both page sizes are made of; rows of a pool
    // are 32-bit coordinates of its tensor map.  Otherwise every tile comes by cp.async.
    CUtensorMap map[4];
    const int64_t rows = static_cast<int64_t>(a.n_pages) * a.Hkv * a.rows, crows = static_cast<int64_t>(a.n_cpages) * a.Hkv * a.crows;
    a.box_log2 = 0;
    for (int lg = 5; lg >= 3 && a.box_log2 == 0; --lg)
        if (((a.rows | a.crows) & ((1 << lg) - 1)) == 0) a.box_log2 = lg;
    if (rows > 0x7fffffff - 32 || crows > 0x7fffffff - 32) a.box_log2 = 0;
    EncodeTiledFn enc = get_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    const uint32_t box = a.box_log2 > 0 ? 1u << a.box_log2 : 8u;
    const uint64_t n = a.box_log2 > 0 ? rows : 8, nc = a.box_log2 > 0 ? crows : 8;
    if (!encode_rows_bf16(enc, &map[0], a.K, d, n, box) || !encode_rows_bf16(enc, &map[1], a.V, d, n, box) ||
        !encode_rows_bf16(enc, &map[2], a.Kc, d, nc, box) || !encode_rows_bf16(enc, &map[3], a.Vc, d, nc, box))
        return cudaErrorInvalidValue;
    const bool one = tc_rows(a.R) == 128;
    if (d == 64)
        return one ? launch_halves<1, 64>(map, a, wait_limit_ns, skip_loads, stream) : launch_halves<2, 64>(map, a, wait_limit_ns, skip_loads, stream);
    if (a.R <= TWO_PART_ROWS) return launch_halves<1, 128, true>(map, a, wait_limit_ns, skip_loads, stream);
    return one ? launch_halves<1, 128>(map, a, wait_limit_ns, skip_loads, stream) : launch_halves<2, 128>(map, a, wait_limit_ns, skip_loads, stream);
}

}  // namespace tree
}  // namespace cca
