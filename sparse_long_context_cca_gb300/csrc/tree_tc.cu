// Tree attention on the tcgen05 tensor cores: bf16, d = 128, more than 16 query rows per KV
// head (T nodes times the query heads that share it).  What it computes, the key list and
// the split over the grid are those of tree.cuh; this file is the walk of one CTA over its
// run of 128-key tiles.
//
// One CTA holds HALVES * 128 rows, so up to 256 rows read K and V once.  Per tile of 128
// keys an SM's share of HBM needs 64 KB / 44 GB/s = 1.5 us, the MMAs of 256 rows 0.7 us for
// each product: with one half the loads bound it, with two the MMAs and loads are level.
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
// K(t) and V(t) take two consecutive slots of a ring of NS 32 KB slots.
//
// Two halves: S_A | S_B | O_A | O_B fill the tensor memory; the halves' softmaxes and MMAs
// alternate.  P_h overwrites S_h, and S_h of the next tile is issued after the product that
// reads P_h, so a finished S_h means that all earlier products of the half are done.
// One half: two score buffers, so that the next tile's scores are made during this one's
// softmax; the softmax then waits for the earlier product itself before it touches O.
//
// Every wait is bounded: on a time-out the CTA stops, drains, frees its tensor memory and
// reports CCA_ERR_TIMEOUT.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/cca.h"
#include "internal.h"
#include "paged.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.h"
#include "tree.cuh"

namespace cca {
namespace tree {
namespace {

constexpr int HD = 128;
constexpr int BN = 128;                       // keys per tile
constexpr uint32_t TILE_BYTES = BN * HD * 2;  // 32 KB
constexpr uint32_t HALF_BYTES = TILE_BYTES / 2;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_O = 256;
constexpr float LAZY_RESCALE_LOG2 = 16.0f;  // keep a stale max while it is within 2^16
constexpr uint32_t IDESC_QK = ptx::idesc_bf16_f32(128, BN, 0, 0);  // Q, K both K-major
constexpr uint32_t IDESC_PV = ptx::idesc_bf16_f32(128, HD, 0, 1);  // P in tensor memory, V MN-major
constexpr int METAS = 4;

// What the softmax needs to know of a tile's keys.
struct TileMeta {
    const __nv_bfloat16 *v[BN];  // V rows, for the elements that `odd` takes out
    int val[BN];
    uint32_t kind[BN / 4];       // a byte per key
    uint32_t masked[4];          // per producer warp: some key has kind != 0
    uint32_t odd[4];             // bit per key: V holds an infinity or NaN that not every row sees
};

template <int HALVES>
struct Layout {
    // ring slots: what 227 KB leave next to the queries and the bookkeeping
    static constexpr int NS = HALVES == 2 ? 4 : 5;
    static constexpr int THREADS = (HALVES + 2) * 128;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_RING = HALVES * TILE_BYTES;
    static constexpr uint32_t OFF_META = OFF_RING + NS * TILE_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_META + METAS * sizeof(TileMeta);
    static constexpr int B_FULL = 0;                 // NS
    static constexpr int B_EMPTY = B_FULL + NS;      // NS
    static constexpr int B_QFULL = B_EMPTY + NS;     // HALVES
    static constexpr int B_SFULL = B_QFULL + HALVES; // 2: per half, or per score buffer
    static constexpr int B_PFULL = B_SFULL + 2;      // HALVES
    static constexpr int B_PVDONE = B_PFULL + HALVES;// HALVES: two halves per list, one half per tile
    static constexpr int B_OFREE = B_PVDONE + HALVES;// HALVES
    static constexpr int B_DRAIN = B_OFREE + HALVES;
    static constexpr int NUM_BARS = B_DRAIN + 1;
    static constexpr uint32_t OFF_TMEMPTR = OFF_BAR + NUM_BARS * 8;
    static constexpr uint32_t OFF_ABORT = OFF_TMEMPTR + 4;
    static constexpr uint32_t OFF_FIRST = (OFF_ABORT + 4 + 15) / 16 * 16;
    // then: tiles before each sequence [B], 16 warp sums, per half parents [T] and a bit row per
    // query row [128][words]
    static uint32_t bytes(int B, int T) {
        return OFF_FIRST + 8 * (B + 16) + HALVES * (2 * ((T + 1) / 2 * 2) + 128 * 4 * ((T + 31) / 32)) + 1024;
    }
};

template <int HALVES>
__global__ void __launch_bounds__((HALVES + 2) * 128, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmKc, const __grid_constant__ CUtensorMap tmVc, const TreeArgs a,
                   const unsigned long long lim, const int skip_loads) {
    using L = Layout<HALVES>;
    constexpr int NS = L::NS;
    constexpr int BM = HALVES * 128;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    auto bar = [&](int idx) -> uint32_t { return base + L::OFF_BAR + 8u * idx; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + L::OFF_ABORT);
    TileMeta *metas = reinterpret_cast<TileMeta *>(gbase + L::OFF_META);
    int64_t *sm_first = reinterpret_cast<int64_t *>(gbase + L::OFF_FIRST);
    int64_t *sm_warp = sm_first + a.B;
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
        ptx::mbar_init(bar(L::B_SFULL), 1);
        ptx::mbar_init(bar(L::B_SFULL + 1), 1);
        ptx::mbar_init(bar(L::B_DRAIN), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc(base + L::OFF_TMEMPTR, TMEM_COLS);
        ptx::tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<uint32_t *>(gbase + L::OFF_TMEMPTR);

    const int mt = blockIdx.x % a.n_mt, group = blockIdx.x / a.n_mt;
    const Split split = make_split(a, scan_tiles(a, sm_first, sm_warp));
    const int64_t x0 = group < split.groups ? split.begin(group) : 0;
    const int64_t x1 = group < split.groups ? split.begin(group + 1) : 0;
    const bool half_used[2] = {true, HALVES == 2 && mt * BM + 128 < a.R};

    if (wg == HALVES) {
        // ------------------------------------------------------------ producers
        if constexpr (HALVES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        const int pw = warp & 3;
        const int sub = lane >> 4, chunk = lane & 15;
        bool ok = x0 < x1 && !skip_loads;
        Item it = {};
        const char *kp = nullptr, *vp = nullptr;
        int kind = 4, val = 0;
        int box_y = 0;         // of a tile of runs: this lane's box, as a row of its pool
        bool runs = false, box_core = false;
        const int per_warp = a.box_log2 > 0 ? 32 >> a.box_log2 : 0;  // boxes of a warp
        auto look_up = [&](int64_t x) {
            const int tile = static_cast<int>(x - it.first);
            runs = tile < it.k.run_tiles;
            if (runs) {
                kind = 0;
                if (lane < per_warp) {
                    const int64_t row = find_box(a, it.k, it.b, it.kv, (tile * 4 + pw) * per_warp + lane, box_core);
                    // no page: past the pool's end, where the copy fills in zeros
                    box_y = static_cast<int>(row >= 0 ? row : static_cast<int64_t>(box_core ? a.n_cpages : a.n_pages) * a.Hkv * (box_core ? a.crows : a.rows));
                    kind = row >= 0 ? 0 : 4;
                }
                // each lane: the kind of its key, which its box's lane knows
                kind = __shfl_sync(kFull, kind, lane >> a.box_log2);
                return;
            }
            const Key key = find_key(a, it.k, it.b, it.kv, (tile - it.k.run_tiles) * BN + pw * 32 + lane);
            const int64_t off = key.row * (HD * 2);
            kp = key.row < 0 ? nullptr : static_cast<const char *>(key.core ? a.Kc : a.K) + off;
            vp = key.row < 0 ? nullptr : static_cast<const char *>(key.core ? a.Vc : a.V) + off;
            kind = key.kind;
            val = key.val;
        };
        // The tile whose copies are in flight behind the one being issued.
        int prev_slot = -1;
        uint32_t prev_mixed = 0;  // lanes' keys that only some rows see
        int prev_meta = 0;
        int64_t last_run = -1;    // last tile of runs that was issued
        auto land = [&]() {       // that tile's copies (of this thread) have arrived
            if (prev_slot < 0) return;
            const int vslot = (prev_slot + 1) % NS;
            if (prev_mixed != 0) {
                // infinities and NaN in the V of such keys would reach the other rows as 0 * NaN:
                // they leave the tile, and the rows that see them add them back themselves
                for (int j = 0; j < 16; ++j) {
                    const int r = 2 * j + sub;
                    if (!((prev_mixed >> r) & 1u)) continue;
                    const int row = pw * 32 + r;
                    uint4 *p = reinterpret_cast<uint4 *>(gbase + L::OFF_RING + vslot * TILE_BYTES + (chunk >> 3) * HALF_BYTES +
                                                         row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
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
                        atomicOr(&metas[prev_meta].odd[row >> 5], 1u << (row & 31));
                    }
                }
            }
            ptx::fence_proxy_async_smem();  // the MMAs read what this thread has written
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(bar(L::B_FULL + prev_slot));
                ptx::mbar_arrive(bar(L::B_FULL + vslot));
            }
        };
        if (ok) {
            it = item_of(a, sm_first, x0);
            look_up(x0);
        }
        for (int64_t x = x0; ok && x < x1; ++x) {
            const uint32_t u = static_cast<uint32_t>(x - x0) * 2;
            const int ks = u % NS, vs = (u + 1) % NS;
            // Before it waits for room, the tile in flight is handed over: with a ring of two tiles
            // the room may depend on it (the first half's next scores come before the second
            // half's product, which frees the slot).
            if (prev_slot >= 0 && !__all_sync(kFull, ptx::mbar_try_wait(bar(L::B_EMPTY + ks), ((u / NS) & 1) ^ 1) &&
                                                         ptx::mbar_try_wait(bar(L::B_EMPTY + vs), (((u + 1) / NS) & 1) ^ 1))) {
                cp_wait<0>();
                land();
                prev_slot = -1;
            }
            if (!__all_sync(kFull, ptx::wait_bounded(bar(L::B_EMPTY + ks), ((u / NS) & 1) ^ 1, abort_flag, lim) &&
                                       ptx::wait_bounded(bar(L::B_EMPTY + vs), (((u + 1) / NS) & 1) ^ 1, abort_flag, lim))) {
                ok = false;
                break;
            }
            // A slot of METAS tiles ago: its softmax is over, as the scores of a later tile, which
            // freed this K slot, were issued after it.
            TileMeta &m = metas[(x - x0) & (METAS - 1)];
            if (runs) {
                const uint32_t gone = __ballot_sync(kFull, kind != 0);
                if (gone != 0) {
                    reinterpret_cast<uint8_t *>(m.kind)[pw * 32 + lane] = static_cast<uint8_t>(kind);
                    m.val[pw * 32 + lane] = 0;
                } else if (lane < 8) {
                    m.kind[pw * 8 + lane] = 0;  // a neighbour's missing page may make the tile masked
                }
                if (lane == 0) {
                    m.masked[pw] = gone;
                    m.odd[pw] = 0;
                }
                if (prev_slot >= 0) {
                    cp_wait<0>();
                    land();
                    prev_slot = -1;
                }
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(L::B_FULL + ks), 32 * HD * 2);
                    ptx::mbar_arrive_expect_tx(bar(L::B_FULL + vs), 32 * HD * 2);
                }
                __syncwarp();
                if (lane < per_warp) {
                    const uint32_t at = base + L::OFF_RING + (pw * 32 + (lane << a.box_log2)) * 128;
                    const void *mk = box_core ? static_cast<const void *>(&tmKc) : static_cast<const void *>(&tmK);
                    const void *mv = box_core ? static_cast<const void *>(&tmVc) : static_cast<const void *>(&tmV);
                    ptx::tma_load_2d(mk, bar(L::B_FULL + ks), at + ks * TILE_BYTES, 0, box_y);
                    ptx::tma_load_2d(mk, bar(L::B_FULL + ks), at + ks * TILE_BYTES + HALF_BYTES, 64, box_y);
                    ptx::tma_load_2d(mv, bar(L::B_FULL + vs), at + vs * TILE_BYTES, 0, box_y);
                    ptx::tma_load_2d(mv, bar(L::B_FULL + vs), at + vs * TILE_BYTES + HALF_BYTES, 64, box_y);
                }
                last_run = x - x0;
                __syncwarp();
                if (x + 1 < x1) {
                    if (x + 1 >= it.first + it.k.tiles) next_item(a, it);
                    look_up(x + 1);
                }
                continue;
            }
            const int at = pw * 32 + lane;
            m.v[at] = reinterpret_cast<const __nv_bfloat16 *>(vp);
            m.val[at] = val;
            reinterpret_cast<uint8_t *>(m.kind)[at] = static_cast<uint8_t>(kind);
            const uint32_t some = __ballot_sync(kFull, kind != 0);
            const uint32_t mixed = __ballot_sync(kFull, kind != 0 && kind != 4);
            if (lane == 0) {
                m.masked[pw] = some;
                m.odd[pw] = 0;
            }
            __syncwarp();
            const uint32_t kdst = base + L::OFF_RING + ks * TILE_BYTES + (chunk >> 3) * HALF_BYTES;
            const uint32_t vdst = base + L::OFF_RING + vs * TILE_BYTES + (chunk >> 3) * HALF_BYTES;
#pragma unroll 4
            for (int j = 0; j < 16; ++j) {
                const int row = pw * 32 + 2 * j + sub;
                const char *p = reinterpret_cast<const char *>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(kp), 2 * j + sub));
                cp16(kdst + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), p == nullptr ? static_cast<const char *>(a.K) : p + chunk * 16, p != nullptr);
            }
#pragma unroll 4
            for (int j = 0; j < 16; ++j) {
                const int row = pw * 32 + 2 * j + sub;
                const char *p = reinterpret_cast<const char *>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(vp), 2 * j + sub));
                cp16(vdst + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), p == nullptr ? static_cast<const char *>(a.V) : p + chunk * 16, p != nullptr);
            }
            cp_commit();
            if (x + 1 < x1) {
                if (x + 1 >= it.first + it.k.tiles) next_item(a, it);
                look_up(x + 1);
            }
            cp_wait<1>();
            land();
            prev_slot = ks;
            prev_mixed = mixed;
            prev_meta = static_cast<int>((x - x0) & (METAS - 1));
        }
        cp_wait<0>();
        if (ok) land();
        if (*abort_flag && lane == 0) {
            // bulk copies already issued land before the CTA's memory is given back
            volatile int never = 0;
            for (int64_t t = last_run > NS ? last_run - NS : 0; t <= last_run; ++t) {
                const uint32_t u = static_cast<uint32_t>(t) * 2;
                ptx::wait_bounded(bar(L::B_FULL + u % NS), (u / NS) & 1, &never, lim);
                ptx::wait_bounded(bar(L::B_FULL + (u + 1) % NS), ((u + 1) / NS) & 1, &never, lim);
            }
        }
        __syncwarp();
    } else if (wg == HALVES + 1) {
        // ------------------------------------------------------------ MMA issuer
        if constexpr (HALVES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        if ((warp & 3) == 0) {
            auto wwait = [&](int b, uint32_t parity) -> bool {
                return __all_sync(kFull, ptx::wait_bounded(bar(b), parity, abort_flag, lim));
            };
            const uint64_t dq = ptx::smem_desc_sw128(base + L::OFF_Q, 16, 1024);
            const uint64_t dk = ptx::smem_desc_sw128(base + L::OFF_RING, 16, 1024);
            const uint64_t dv = ptx::smem_desc_sw128(base + L::OFF_RING, HALF_BYTES, 1024);
            constexpr uint64_t STEP = TILE_BYTES >> 4;
            bool ok = true;
            uint32_t seg = 0;
            uint32_t pcount = 0;  // tiles whose P was waited for (a used half each)
            Item it = {};
            if (x0 < x1) it = item_of(a, sm_first, x0);
            int64_t x = x0;
            while (ok && x < x1) {
                const int64_t end = it.first + it.k.tiles < x1 ? it.first + it.k.tiles : x1;
                if constexpr (HALVES == 2) {
                    auto scores = [&](int h, int64_t t) {
                        const uint32_t slot = (static_cast<uint32_t>(t - x0) * 2) % NS;
                        ptx::tc_fence_after();
                        ptx::mma_ss_k128_warp(tmem + h * 128, dq + h * STEP, dk + slot * STEP, IDESC_QK, 0u);
                        ptx::tc_commit_warp(bar(L::B_SFULL + h));
                    };
                    {
                        const uint32_t u = static_cast<uint32_t>(x - x0) * 2;
                        for (int h = 0; ok && h < 2; ++h) {
                            if (!half_used[h]) continue;
                            if (!wwait(L::B_QFULL + h, seg & 1) || !wwait(L::B_FULL + u % NS, (u / NS) & 1)) {
                                ok = false;
                                break;
                            }
                            scores(h, x);
                        }
                        if (!ok) break;
                        ptx::tc_commit_warp(bar(L::B_EMPTY + u % NS));
                    }
                    for (int64_t t = x; ok && t < end; ++t) {
                        const uint32_t u = static_cast<uint32_t>(t - x0) * 2 + 1;
                        if (!wwait(L::B_FULL + u % NS, (u / NS) & 1)) {
                            ok = false;
                            break;
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!half_used[h]) continue;
                            if (!wwait(L::B_PFULL + h, pcount & 1) || (t == x && !wwait(L::B_OFREE + h, (seg & 1) ^ 1))) {
                                ok = false;
                                break;
                            }
                            ptx::tc_fence_after();
                            ptx::mma_ts_k128_warp(tmem + TM_O + h * 128, tmem + h * 128, dv + (u % NS) * STEP, IDESC_PV, t == x ? 0u : 1u);
                            if (t + 1 < end) {
                                if (!wwait(L::B_FULL + (u + 1) % NS, ((u + 1) / NS) & 1)) {
                                    ok = false;
                                    break;
                                }
                                scores(h, t + 1);
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
                    auto scores = [&](int64_t t) -> bool {
                        const uint32_t u = static_cast<uint32_t>(t - x0) * 2;
                        if (!wwait(L::B_FULL + u % NS, (u / NS) & 1)) return false;
                        const uint32_t buf = static_cast<uint32_t>(t - x0) & 1;
                        ptx::tc_fence_after();
                        ptx::mma_ss_k128_warp(tmem + buf * 128, dq, dk + (u % NS) * STEP, IDESC_QK, 0u);
                        ptx::tc_commit_warp(bar(L::B_SFULL + buf));
                        ptx::tc_commit_warp(bar(L::B_EMPTY + u % NS));
                        return true;
                    };
                    if (!wwait(L::B_QFULL, seg & 1) || !scores(x)) {
                        ok = false;
                        break;
                    }
                    for (int64_t t = x; ok && t < end; ++t) {
                        if (t + 1 < end && !scores(t + 1)) {
                            ok = false;
                            break;
                        }
                        const uint32_t u = static_cast<uint32_t>(t - x0) * 2 + 1;
                        if (!wwait(L::B_FULL + u % NS, (u / NS) & 1) || !wwait(L::B_PFULL, pcount & 1) ||
                            (t == x && !wwait(L::B_OFREE, (seg & 1) ^ 1))) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        ptx::mma_ts_k128_warp(tmem + TM_O, tmem + (static_cast<uint32_t>(t - x0) & 1) * 128, dv + (u % NS) * STEP, IDESC_PV,
                                              t == x ? 0u : 1u);
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
        if constexpr (HALVES == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int h = HALVES == 2 ? wg : 0;
        const int quarter = warp & 3;
        const int in = h * 128 + quarter * 32 + lane;  // row of the CTA
        const int row = mt * BM + in;                  // row of the KV head
        const bool live = row < a.R;
        const bool idle = mt * BM + h * 128 + quarter * 32 >= a.R;  // no row of this warp
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tO = tmem + lane_addr + TM_O + h * 128;
        int16_t *const up = reinterpret_cast<int16_t *>(sm_warp + 16) + h * ((a.T + 1) / 2 * 2);
        uint32_t *const sees = reinterpret_cast<uint32_t *>(reinterpret_cast<int16_t *>(sm_warp + 16) + HALVES * ((a.T + 1) / 2 * 2)) +
                               (h * 128 + quarter * 32 + lane) * words;
        const int node = live ? row % a.T : 0;
        bool ok = true;
        uint32_t seg = 0, n_s = 0;  // lists and tiles of this half so far
        Item it = {};
        int start = 0, cores = -1;  // this row's first raw token; its visible cores, -1: empty node
        int tree_of = -1;
        auto sees_key = [&](const TileMeta &tm, int col) {
            const int kind = reinterpret_cast<const uint8_t *>(tm.kind)[col], val = tm.val[col];
            if (kind == 3) return ((sees[val >> 5] >> (val & 31)) & 1u) != 0;
            return kind == 0 || (kind == 1 && val < cores) || (kind == 2 && val >= start);
        };
        auto begin_list = [&]() {
            // the queries, 16 chunks of a row, swizzled like the keys; S of the last tile is done,
            // so nothing reads the old ones
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.Q) +
                             ((static_cast<int64_t>(it.b) * a.Hq + static_cast<int64_t>(it.kv) * (a.Hq / a.Hkv)) * a.T + row) * HD);
            uint8_t *dst = gbase + L::OFF_Q + h * TILE_BYTES + (quarter * 32 + lane) * 128;
#pragma unroll
            for (int c = 0; c < 16; ++c)
                *reinterpret_cast<uint4 *>(dst + (c >> 3) * HALF_BYTES + (((c & 7) ^ (lane & 7)) << 4)) = live ? q[c] : make_uint4(0, 0, 0, 0);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(L::B_QFULL + h));
        };
        auto begin_tree = [&]() {
            if (it.b == tree_of) return;
            tree_of = it.b;
            const int tid = quarter * 32 + lane;
            ptx::named_bar_sync(1 + h, 128);  // the old parents have been used
            for (int t = tid; t < a.T; t += 128) {
                int p = t - 1;
                if (a.parents != nullptr) {
                    p = a.parents[static_cast<int64_t>(it.b) * a.T + t];
                    if (p != -1 && (p < 0 || p >= t)) p = -2;
                }
                up[t] = static_cast<int16_t>(p);
            }
            ptx::named_bar_sync(1 + h, 128);
            for (int i = 0; i < words; ++i) sees[i] = 0;
            int depth = -1, n = node;
            while (n >= 0) {  // parents lie below their children, so this ends
                sees[n >> 5] |= 1u << (n & 31);
                ++depth;
                n = up[n];
            }
            const int pos = it.k.len + depth;
            cores = live && n == -1 && it.k.n > 0 ? visible_cores(pos, a.w, a.g) : -1;
            start = window_start(pos, a.w, a.g, a.window_mode);
        };
        if (x0 < x1) {
            it = item_of(a, sm_first, x0);
            begin_list();
            begin_tree();
        }
        int64_t x = x0;
        while (ok && x < x1) {
            const int64_t end = it.first + it.k.tiles < x1 ? it.first + it.k.tiles : x1;
            float m = -INFINITY, l = 0.f;
            bool has_odd = false;
            float *const part = part_at(a, group, mt, x0 >= it.first ? 0 : 1, BM, HD);
            if (it.k.n == 0 && threadIdx.x == 0 && a.status != nullptr) *a.status = CCA_ERR_INVALID_ARG;
            for (int64_t t = x; t < end; ++t, ++n_s) {
                const uint32_t buf = HALVES == 2 ? h : static_cast<uint32_t>(t - x0) & 1;
                const uint32_t s_parity = HALVES == 2 ? n_s & 1 : (n_s >> 1) & 1;
                const uint32_t uv = static_cast<uint32_t>(t - x0) * 2 + 1;
                // V(t)'s barrier: what the producers wrote about the tile is visible after it, and its
                // slot is not filled again before this softmax is over
                if (!__all_sync(kFull, ptx::wait_bounded(bar(L::B_SFULL + buf), s_parity, abort_flag, lim) &&
                                           ptx::wait_bounded(bar(L::B_FULL + uv % NS), (uv / NS) & 1, abort_flag, lim))) {
                    ok = false;
                    break;
                }
                const uint32_t tS = tmem + lane_addr + buf * 128;
                const TileMeta &tm = metas[(t - x0) & (METAS - 1)];
                if (!idle) {
                    ptx::tc_fence_after();
                    uint32_t s[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) ptx::tmem_ld32(tS + c * 32, s[c]);
                    ptx::tmem_wait_ld(s[0]);
                    ptx::reg_touch(s[1]);
                    ptx::reg_touch(s[2]);
                    ptx::reg_touch(s[3]);
                    if ((tm.masked[0] | tm.masked[1] | tm.masked[2] | tm.masked[3]) != 0) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t see = 0;
#pragma unroll 1
                            for (int kk = 0; kk < 32; ++kk) see |= static_cast<uint32_t>(sees_key(tm, c * 32 + kk)) << kk;
#pragma unroll
                            for (int kk = 0; kk < 32; ++kk)
                                if (!((see >> kk) & 1u)) s[c][kk] = __float_as_uint(-INFINITY);
                        }
                    }
                    float mp[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        mp[q] = fmaxf(__uint_as_float(s[q >> 1][(q & 1) * 16]), __uint_as_float(s[q >> 1][(q & 1) * 16 + 1]));
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
#pragma unroll
                        for (int kk = 2; kk < 16; kk += 2)
                            mp[q] = ptx::max3(mp[q], __uint_as_float(s[q >> 1][(q & 1) * 16 + kk]),
                                              __uint_as_float(s[q >> 1][(q & 1) * 16 + kk + 1]));
                    }
                    const float mx = ptx::max3(ptx::max3(mp[0], mp[1], mp[2]), ptx::max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
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
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[16];
                            ptx::tmem_ld16(tO + c * 16, o);
                            ptx::tmem_wait_ld16(o);
#pragma unroll
                            for (int kk = 0; kk < 16; ++kk) o[kk] = __float_as_uint(__uint_as_float(o[kk]) * f);
                            ptx::tmem_st16(tO + c * 16, o);
                        }
                        if (rescale) {
                            l *= f;
                            m = m_new;
                        }
                    }
                    const float mu = m == -INFINITY ? 0.f : m;
                    if ((tm.odd[0] | tm.odd[1] | tm.odd[2] | tm.odd[3]) != 0) {
                        // what the producers took out of V, for the rows that see it: the sums of
                        // infinities and NaN go to this row of the CTA's partial until the output
                        float *const sum = part + static_cast<int64_t>(in) * HD;
#pragma unroll 1
                        for (int col = 0; col < BN; ++col) {
                            if (!((tm.odd[col >> 5] >> (col & 31)) & 1u)) continue;
                            __syncwarp();
                            uint32_t sc;  // the raw score is still in tensor memory
                            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(sc) : "r"(tS + col));
                            if (!live || !sees_key(tm, col)) continue;
                            const float p = ptx::ex2(fmaf(__uint_as_float(sc), a.scale_log2, -mu));
                            for (int e = 0; e < HD; ++e) {
                                const float f = __bfloat162float(tm.v[col][e]);
                                const float before = has_odd ? sum[e] : 0.f;
                                sum[e] = f - f != 0.f ? before + p * f : before;
                            }
                            has_odd = true;
                        }
                    }
                    // p = 2^(s*scale - mu), two columns per packed FMA; P rounds to bf16, the sum does not
                    const uint64_t sc2 = ptx::f2(a.scale_log2, a.scale_log2);
                    const uint64_t nm2 = ptx::f2(-mu, -mu);
                    uint64_t lp[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t pk[8];
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const int col = (c & 1) * 16 + 2 * kk;
                            const uint64_t x2 = ptx::fma2(ptx::f2(__uint_as_float(s[c >> 1][col]), __uint_as_float(s[c >> 1][col + 1])), sc2, nm2);
                            float y0, y1;
                            ptx::f2_split(x2, y0, y1);
                            const float p0 = ptx::ex2(y0);
                            const float p1 = ptx::ex2(y1);
                            lp[kk & 1] = ptx::add2(lp[kk & 1], ptx::f2(p0, p1));
                            pk[kk] = ptx::pack_bf16x2(p0, p1);
                        }
                        ptx::tmem_st8(tS + c * 8, pk);  // P over the consumed scores
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
            // the next list's queries, while the last product runs
            const Item old = it;
            const bool empty = cores < 0;
            if (end < x1) {
                next_item(a, it);
                begin_list();
            }
            const uint32_t done_parity = HALVES == 2 ? seg & 1 : (n_s & 1) ^ 1;
            if (!__all_sync(kFull, ptx::wait_bounded(bar(L::B_PVDONE + h), done_parity, abort_flag, lim))) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            if (__any_sync(kFull, has_odd)) {
                const float *const sum = part + static_cast<int64_t>(in) * HD;
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t v[16];
                    ptx::tmem_ld16(tO + c * 16, v);
                    ptx::tmem_wait_ld16(v);
#pragma unroll
                    for (int kk = 0; kk < 16; ++kk) v[kk] = __float_as_uint(__uint_as_float(v[kk]) + (has_odd ? sum[c * 16 + kk] : 0.f));
                    ptx::tmem_st16(tO + c * 16, v);
                }
                ptx::tmem_wait_st();
            }
            if (empty) {
                m = -INFINITY;
                l = 0.f;
            }
            const bool nothing = l == 0.f;  // no visible key in this part (or an empty node)
            const bool whole = x0 <= old.first && old.first + old.k.tiles <= x1;
            const float scale = nothing ? 0.f : whole ? 1.f / l : 1.f;
            const int64_t out = (static_cast<int64_t>(old.b) * a.Hq + static_cast<int64_t>(old.kv) * (a.Hq / a.Hkv)) * a.T + row;
            if (!idle) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    __syncwarp();
                    uint32_t o[32];
                    ptx::tmem_ld32(tO + c * 32, o);
                    ptx::tmem_wait_ld(o);
                    if (!live) continue;
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = nothing ? 0u : __float_as_uint(__uint_as_float(o[k]) * scale);
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.O) + out * HD + c * 32);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                v[k] = ptx::pack_bf16x2(__uint_as_float(o[8 * q + 2 * k]), __uint_as_float(o[8 * q + 2 * k + 1]));
                            dst[q] = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(part + static_cast<int64_t>(in) * HD + c * 32);
#pragma unroll
                        for (int q = 0; q < 8; ++q) dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(L::B_OFREE + h));
            if (live) {
                if (whole) {
                    a.LSE[out] = nothing ? -INFINITY : (m + log2f(l)) * kLn2;
                } else {
                    part[BM * HD + in] = m;
                    part[BM * HD + BM + in] = l;
                }
            }
            ++seg;
            x = end;
            if (x < x1) begin_tree();
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0 && a.status != nullptr) atomicCAS(a.status, 0, static_cast<int32_t>(CCA_ERR_TIMEOUT));
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int HALVES>
cudaError_t launch_halves(const CUtensorMap (&map)[4], const TreeArgs &a, unsigned long long lim, int skip_loads, cudaStream_t stream) {
    static std::atomic<int> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev].load(std::memory_order_relaxed) == 0) {
        e = cudaFuncSetAttribute(tree_tc_kernel<HALVES>, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(1, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.groups) * a.n_mt);
    cfg.blockDim = dim3(Layout<HALVES>::THREADS);
    cfg.dynamicSmemBytes = Layout<HALVES>::bytes(a.B, a.T);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_tc_kernel<HALVES>, map[0], map[1], map[2], map[3], a, lim, skip_loads);
}

}  // namespace

int tc_rows(int R) { return R <= 128 ? 128 : 256; }

cudaError_t launch_tc(TreeArgs a, unsigned long long wait_limit_ns, int skip_loads, cudaStream_t stream) {
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
    if (!encode_rows_bf16_d128(enc, &map[0], a.K, n, box) || !encode_rows_bf16_d128(enc, &map[1], a.V, n, box) ||
        !encode_rows_bf16_d128(enc, &map[2], a.Kc, nc, box) || !encode_rows_bf16_d128(enc, &map[3], a.Vc, nc, box))
        return cudaErrorInvalidValue;
    return tc_rows(a.R) == 128 ? launch_halves<1>(map, a, wait_limit_ns, skip_loads, stream)
                               : launch_halves<2>(map, a, wait_limit_ns, skip_loads, stream);
}

}  // namespace tree
}  // namespace cca
