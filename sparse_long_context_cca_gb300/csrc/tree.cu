// CCA attention of a tree of drafted tokens over paged caches (fusion equation of the
// Method section, one row per node): node t at position p = len + depth(t) takes one
// softmax over the cores j < lo(p)/g, the committed raw tokens of its window, its
// ancestors and itself.  One node per sequence is plain decoding.
//
// Three kernels walk the lists: tree_tc.cu (bf16 on tcgen05), tree_bf16_kernel (bf16, d = 64, up
// to 16 rows per KV head, mma.sync) and tree_f32_kernel (fp32 on CUDA cores).
//
// What bounds it.  The r query heads of a KV head times T nodes are R = r*T rows that share
// one list of keys: K and V rows are read once per (b, KV head) and meet R rows, so few rows
// are bound by HBM and many by the matrix units.
//
// The key list of a sequence puts the keys that every node sees first (cores before the
// shallowest node's window, raw tokens from the deepest one's window on), the few that only
// some see last (at most T/g + 1 cores, T + g raw tokens, the T nodes).  Only tiles that
// reach those, or that hold keys without a page, look at masks at all.
//
// Work split.  Lengths live on the device, so the split is made there: the tiles of all
// (b, KV head) lists, one after the other, are dealt to the groups of the grid in contiguous
// runs of equal cost, whatever the lengths are.  A group finishes lists that lie wholly in its
// run and writes a partial (max, sum, output) for its first and last list otherwise; a
// second kernel joins the partials of a list in the order of the groups.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/cca.h"
#include "internal.h"
#include "paged.cuh"
#include "sm100_ptx.cuh"
#include "tree.cuh"

namespace cca {
extern unsigned long long g_wait_limit_ns;
extern int g_skip_q_load;

namespace {

using namespace tree;

constexpr int TILE = 64;  // keys per tile of the kernels in this file
constexpr int TREE_THREADS = 128;

// ---------------------------------------------------------------- bf16: matrix units

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int STAGES = 3;
constexpr int METAS = 4;  // addresses and kinds of the tiles from the one in work to the next to load

struct Meta {
    const char *k[TILE], *v[TILE];  // null: not there
    int val[TILE];
    uint32_t masked[2];  // bit per key: kind != 0
    uint32_t odd[2];     // bit per key: V holds an infinity or NaN, and not every row sees it
    uint8_t kind[TILE];
};

constexpr int MMA_D = 64, MMA_ROWS = 16;  // head dimension and rows of the mma.sync kernel

struct TreeSmem {
    static constexpr int ROW = MMA_D * 2;                  // bytes of a key row
    static constexpr int TILE_BYTES = TILE * ROW;      // K or V
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int META_OFF = STAGES * STAGE_BYTES;
    static constexpr int START_OFF = META_OFF + METAS * static_cast<int>(sizeof(Meta));
    static constexpr int NODE_OFF = START_OFF + static_cast<int>(sizeof(Start));
    // then: node starts [T], cores [T], bits [T][words], parents [T]
    static __host__ __device__ int bytes(int T) { return NODE_OFF + 8 * T + 4 * T * ((T + 31) / 32) + 2 * T + 16; }
};

// Byte offset of 16-byte chunk c of row `row` in a tile: chunks are permuted inside a row, so
// that the eight rows of an ldmatrix fall into different banks.
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
    return static_cast<uint32_t>(row * TreeSmem::ROW + ((c ^ (row & 7)) << 4));
}

// bf16 with d = 64 and up to 16 rows: the four warps share them and take a quarter of a tile's
// keys each.  One CTA walks its group's run of tiles: cp.async keeps two tiles in flight behind
// the one in work, and the page look-ups of the tile after those are done a step ahead, under the
// matrix work.
__global__ void __launch_bounds__(TREE_THREADS) tree_bf16_kernel(const TreeArgs a) {
    using S = TreeSmem;
    constexpr int D = MMA_D;
    constexpr int BM = MMA_ROWS;
    constexpr int WK = 4;          // warps over the keys
    constexpr int KW = TILE / WK;  // keys of a warp
    constexpr int NT = KW / 8;
    constexpr int DT = D / 8;
    constexpr int CPR = D / 8;     // 16-byte chunks per row
    extern __shared__ __align__(128) unsigned char smem[];
    Meta *meta = reinterpret_cast<Meta *>(smem + S::META_OFF);
    Start &st = *reinterpret_cast<Start *>(smem + S::START_OFF);
    Nodes nodes;
    nodes.words = (a.T + 31) >> 5;
    nodes.start = reinterpret_cast<int *>(smem + S::NODE_OFF);
    nodes.cores = nodes.start + a.T;
    nodes.sees = reinterpret_cast<uint32_t *>(nodes.cores + a.T);
    nodes.up = reinterpret_cast<int16_t *>(nodes.sees + a.T * nodes.words);
    const uint32_t stage0 = ptx::smem_addr(smem);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wk = warp;
    const int mt = blockIdx.x % a.n_mt, group = blockIdx.x / a.n_mt;
    const Run run = find_run(a, group, st);
    const int x0 = run.x0, x1 = run.x1;
    if (x0 >= x1) return;

    // ---- loading
    Item ld = run.item;  // list of the tile whose addresses come next
    auto look_up = [&](int x, Key &key) {  // threads 0 .. 63, one key each
        if (x >= x1) return;
        if (x >= ld.first + ld.k.tiles) next_item(a, ld);
        if (tid < TILE) key = settled(a, ld.b, find_key(a, ld.k, ld.b, ld.kv, (x - ld.first) * TILE + tid));
    };
    auto put = [&](int x, const Key &key) {
        if (x >= x1 || tid >= TILE) return;
        Meta &m = meta[(x - x0) & (METAS - 1)];
        const int64_t off = key.row * S::ROW;
        m.k[tid] = key.row < 0 ? nullptr : static_cast<const char *>(key.core ? a.Kc : a.K) + off;
        m.v[tid] = key.row < 0 ? nullptr : static_cast<const char *>(key.core ? a.Vc : a.V) + off;
        m.kind[tid] = static_cast<uint8_t>(key.kind);
        m.val[tid] = key.val;
        const unsigned some = __ballot_sync(kFull, key.kind != 0);
        if (lane == 0) {
            m.masked[warp] = some;
            m.odd[warp] = 0;
        }
    };
    auto issue = [&](int x) {
        if (x < x1) {
            const Meta &m = meta[(x - x0) & (METAS - 1)];
            const uint32_t base = stage0 + static_cast<uint32_t>(x - x0) % STAGES * S::STAGE_BYTES;
            constexpr int PER = TILE * CPR / TREE_THREADS;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = i * TREE_THREADS + tid, row = e / CPR, c = e % CPR;
                const char *p = m.k[row];
                cp16(base + chunk_at(row, c), p == nullptr ? a.K : p + c * 16, p != nullptr);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = i * TREE_THREADS + tid, row = e / CPR, c = e % CPR;
                const char *p = m.v[row];
                cp16(base + S::TILE_BYTES + chunk_at(row, c), p == nullptr ? a.V : p + c * 16, p != nullptr);
            }
        }
        cp_commit();
    };
    Key key = {};
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {  // the first STAGES tiles' addresses, all but one of them loaded
        look_up(x0 + i, key);
        put(x0 + i, key);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue(x0 + i);

    // ---- the rows
    Item it = run.item;
    if (it.k.n == 0 && tid == 0) report(a.status, CCA_ERR_INVALID_ARG);
    uint32_t qf[D / 16][4];
    float o[DT][4], m[2], l[2];
    int node[2];  // node of this thread's two rows, -1 past the last row
    const int row0 = mt * BM + (lane >> 2);
    auto begin_item = [&]() {
        read_tree(a, nodes, it.k, it.b);
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.Q) +
                                 (static_cast<int64_t>(it.b) * a.Hq + static_cast<int64_t>(it.kv) * (a.Hq / a.Hkv)) * a.T * D;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = row0 + 8 * i;
            node[i] = row < a.R ? row % a.T : -1;
            m[i] = -INFINITY;
            l[i] = 0.f;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(q + static_cast<int64_t>(row) * D) + (lane & 3);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qf[kk][i] = node[i] >= 0 ? src[kk * 8] : 0u;
                qf[kk][2 + i] = node[i] >= 0 ? src[kk * 8 + 4] : 0u;
            }
        }
#pragma unroll
        for (int n = 0; n < DT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    };
    begin_item();

    for (int x = x0; x < x1; ++x) {
        cp_wait<STAGES - 2>();
        __syncthreads();
        issue(x + STAGES - 1);
        look_up(x + STAGES, key);

        const Meta &mt_ = meta[(x - x0) & (METAS - 1)];
        const uint32_t kbase = stage0 + static_cast<uint32_t>(x - x0) % STAGES * S::STAGE_BYTES;
        const uint32_t vbase = kbase + S::TILE_BYTES;
        const bool masked = (mt_.masked[0] | mt_.masked[1]) != 0;
        // S = Q K^T over this warp's keys
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t f[4];
                ldsm4(kbase + chunk_at(wk * KW + n * 8 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)), f);
                mma16816(s[n], qf[kk], f[0], f[1]);
                mma16816(s[n + 1], qf[kk], f[2], f[3]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] *= a.scale_log2;
        }
        if (masked) {
            // An infinity or NaN in the V of a key that only some rows see would reach the
            // others as 0 * NaN: such elements leave the tile and are added back by hand below.
            Meta &mw = meta[(x - x0) & (METAS - 1)];
            {
                const int row = tid >> 1;
                if (mw.kind[row] != 0 && mw.kind[row] != 4) {
                    bool odd = false;
                    for (int c = (tid & 1) * (CPR / 2); c < (tid & 1) * (CPR / 2) + CPR / 2; ++c) {
                        uint4 *p = reinterpret_cast<uint4 *>(smem + (vbase - stage0) + chunk_at(row, c));
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
                        if (hit) *p = make_uint4(v[0], v[1], v[2], v[3]);
                        odd |= hit;
                    }
                    if (odd) atomicOr(&mw.odd[row >> 5], 1u << (row & 31));
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = wk * KW + n * 8 + (lane & 3) * 2 + e;
                    const int kind = mw.kind[c], val = mw.val[c];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (node[i] < 0 || !row_sees(nodes, node[i], kind, val)) s[n][2 * i + e] = -INFINITY;
                }
            }
            __syncthreads();
        }
        // one step of the running softmax for this thread's two rows
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mx = s[0][2 * i];
#pragma unroll
            for (int n = 0; n < NT; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            mx = fmaxf(mx, m[i]);
            const float base = mx == -INFINITY ? 0.f : mx;  // nothing visible yet: every p is 0
            const float corr = ptx::ex2(m[i] - base);
            m[i] = mx;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                s[n][2 * i] = ptx::ex2(s[n][2 * i] - base);
                s[n][2 * i + 1] = ptx::ex2(s[n][2 * i + 1] - base);
                sum += s[n][2 * i] + s[n][2 * i + 1];
            }
            l[i] = l[i] * corr + sum;  // this thread's columns; the quad adds up at the end
#pragma unroll
            for (int n = 0; n < DT; ++n) {
                o[n][2 * i] *= corr;
                o[n][2 * i + 1] *= corr;
            }
        }
        // O += P V, each weight as two bf16 parts (the sum above has it whole)
#pragma unroll
        for (int kk = 0; kk < NT / 2; ++kk) {
            uint32_t high[4], low[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float p0 = s[2 * kk + (i >> 1)][(i & 1) * 2], p1 = s[2 * kk + (i >> 1)][(i & 1) * 2 + 1];
                high[i] = ptx::cut_bf16x2(p0, p1);
                low_parts(p0, p1, 0xffff0000u, LOW_MORE);
                low[i] = ptx::cut_bf16x2(p0, p1);
            }
#pragma unroll
            for (int n = 0; n < DT; n += 2) {
                uint32_t f[4];
                ldsm4_t(vbase + chunk_at(wk * KW + kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), n + (lane >> 4)), f);
                mma16816(o[n], high, f[0], f[1]);
                mma16816(o[n + 1], high, f[2], f[3]);
                mma16816(o[n], low, f[0], f[1]);
                mma16816(o[n + 1], low, f[2], f[3]);
            }
        }
        if (masked && (mt_.odd[0] | mt_.odd[1]) != 0) {
            // p * v for the elements that were taken out, row by row
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                for (int c8 = 0; c8 < 8; ++c8) {
                    const int c = wk * KW + n * 8 + c8;
                    if (!((mt_.odd[c >> 5] >> (c & 31)) & 1u)) continue;
                    const int owner = (lane & ~3) | (c8 >> 1);
                    float p[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float even = __shfl_sync(kFull, s[n][2 * i], owner), odd = __shfl_sync(kFull, s[n][2 * i + 1], owner);
                        p[i] = (c8 & 1) ? odd : even;
                    }
                    const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(mt_.v[c]);
#pragma unroll
                    for (int nn = 0; nn < DT; ++nn) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float f = __bfloat162float(v[nn * 8 + (lane & 3) * 2 + e]);
                            if (f - f == 0.f) continue;  // finite
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (node[i] >= 0 && row_sees(nodes, node[i], mt_.kind[c], mt_.val[c])) o[nn][2 * i + e] += p[i] * f;
                        }
                    }
                }
            }
        }
        put(x + STAGES, key);

        const int end = it.first + it.k.tiles;
        if (x + 1 != end && x + 1 != x1) continue;
        // ---- the end of this list, or of this group's part of it
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(kFull, l[i], 1);
            l[i] += __shfl_xor_sync(kFull, l[i], 2);
        }
        {
            // the warps over the keys join: through the tile that was read last, which the
            // next load reaches only after the barrier at the top
            __syncthreads();
            float *mine = reinterpret_cast<float *>(smem + (kbase - stage0)) + (wk - 1) * 16 * (D + 2);
            if (wk > 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float *dst = mine + ((lane >> 2) + 8 * i) * (D + 2);
#pragma unroll
                    for (int n = 0; n < DT; ++n) {
                        dst[n * 8 + (lane & 3) * 2] = o[n][2 * i];
                        dst[n * 8 + (lane & 3) * 2 + 1] = o[n][2 * i + 1];
                    }
                    if ((lane & 3) == 0) {
                        dst[D] = m[i];
                        dst[D + 1] = l[i];
                    }
                }
            }
            __syncthreads();
            if (wk == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float *src[WK];
                    float mx = m[i];
#pragma unroll
                    for (int q = 1; q < WK; ++q) {
                        src[q] = reinterpret_cast<float *>(smem + (kbase - stage0)) +
                                 ((q - 1) * 16 + (lane >> 2) + 8 * i) * (D + 2);
                        mx = fmaxf(mx, src[q][D]);
                    }
                    const float base = mx == -INFINITY ? 0.f : mx;
                    const float own = ptx::ex2(m[i] - base);
                    l[i] *= own;
#pragma unroll
                    for (int n = 0; n < DT; ++n) {
                        o[n][2 * i] *= own;
                        o[n][2 * i + 1] *= own;
                    }
#pragma unroll
                    for (int q = 1; q < WK; ++q) {
                        const float f = ptx::ex2(src[q][D] - base);
                        l[i] += src[q][D + 1] * f;
#pragma unroll
                        for (int n = 0; n < DT; ++n) {
                            o[n][2 * i] += src[q][n * 8 + (lane & 3) * 2] * f;
                            o[n][2 * i + 1] += src[q][n * 8 + (lane & 3) * 2 + 1] * f;
                        }
                    }
                    m[i] = mx;
                }
            }
        }
        if (wk == 0) {
            const bool whole = x0 <= it.first && end <= x1;
            const int slot = x0 >= it.first ? 0 : 1;
            float *part = part_at(a, group, mt, slot, BM, D);
            const int64_t out0 = (static_cast<int64_t>(it.b) * a.Hq + static_cast<int64_t>(it.kv) * (a.Hq / a.Hkv)) * a.T;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = row0 + 8 * i, in = (lane >> 2) + 8 * i;
                if (node[i] < 0) continue;
                if (nodes.cores[node[i]] < 0) {  // an empty node
                    m[i] = -INFINITY;
                    l[i] = 0.f;
#pragma unroll
                    for (int n = 0; n < DT; ++n) o[n][2 * i] = o[n][2 * i + 1] = 0.f;
                }
                if (whole) {
                    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
                    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.O) + (out0 + row) * D) + (lane & 3);
#pragma unroll
                    for (int n = 0; n < DT; ++n) dst[n * 4] = ptx::pack_bf16x2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
                    if ((lane & 3) == 0) a.LSE[out0 + row] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
                } else {
#pragma unroll
                    for (int n = 0; n < DT; ++n)
                        *reinterpret_cast<float2 *>(part + part_col(BM, in, n * 8 + (lane & 3) * 2)) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
                    if ((lane & 3) == 0) {
                        part[BM * D + in] = m[i];
                        part[BM * D + BM + in] = l[i];
                    }
                }
            }
        }
        if (tid == 0 && mt == 0) note_span(a, it, group, x0, x1);
        if (x + 1 < x1) {
            next_item(a, it);
            if (it.k.n == 0 && tid == 0) report(a.status, CCA_ERR_INVALID_ARG);
            __syncthreads();  // the nodes of the old list have been used
            begin_item();
        }
    }
    cp_wait<0>();
}

// ---------------------------------------------------------------- fp32: CUDA cores

constexpr int F32_BM = 16;

template <int D>
struct TreeF32Smem {
    static constexpr int LD = D + 4;  // padded row: eight lanes' 16-byte reads of eight rows miss each other
    static constexpr int V_OFF = TILE * LD;
    static constexpr int Q_OFF = V_OFF + TILE * LD;
    static constexpr int P_OFF = Q_OFF + F32_BM * D;
    static constexpr int ML_OFF = P_OFF + F32_BM * TILE;  // max, sum, correction per row
    static constexpr int KEY_OFF = ML_OFF + 3 * F32_BM;   // kind, value per key
    static constexpr int START_OFF = ((KEY_OFF + 2 * TILE) * 4 + 15) / 16 * 16;
    static constexpr int NODE_OFF = START_OFF + static_cast<int>(sizeof(Start));
    static __host__ __device__ int bytes(int T) { return NODE_OFF + 8 * T + 4 * T * ((T + 31) / 32) + 2 * T + 16; }
};

// The same walk with one tile in shared memory at a time; scores and sums in fp32.  Three sequences
// of 1.5 K, seven nodes, four heads over two (0.8 MB): 15 us, a chain of one tile per CTA and the
// join; with two tiles per CTA at least it was 23 us.
template <int D>
__global__ void __launch_bounds__(TREE_THREADS) tree_f32_kernel(const TreeArgs a) {
    using S = TreeF32Smem<D>;
    constexpr int BM = F32_BM;
    constexpr int LD = S::LD;
    constexpr int GROUPS = TREE_THREADS / D;  // row groups of the product with V
    constexpr int RPT = BM / GROUPS;
    extern __shared__ __align__(128) unsigned char smem[];
    float *sk = reinterpret_cast<float *>(smem), *sv = sk + S::V_OFF, *sq = sk + S::Q_OFF, *sp = sk + S::P_OFF;
    float *sm_m = sk + S::ML_OFF, *sm_l = sm_m + BM, *sm_c = sm_l + BM;
    int *sm_kind = reinterpret_cast<int *>(sk + S::KEY_OFF), *sm_val = sm_kind + TILE;
    Start &st = *reinterpret_cast<Start *>(smem + S::START_OFF);
    Nodes nodes;
    nodes.words = (a.T + 31) >> 5;
    nodes.start = reinterpret_cast<int *>(smem + S::NODE_OFF);
    nodes.cores = nodes.start + a.T;
    nodes.sees = reinterpret_cast<uint32_t *>(nodes.cores + a.T);
    nodes.up = reinterpret_cast<int16_t *>(nodes.sees + a.T * nodes.words);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mt = blockIdx.x % a.n_mt, group = blockIdx.x / a.n_mt;
    const Run run = find_run(a, group, st);
    const int x0 = run.x0, x1 = run.x1;
    if (x0 >= x1) return;
    Item it = run.item;
    const int col = tid % D, rg = tid / D;
    float o[RPT];
    int64_t out0 = 0;
    bool fresh = true;
    for (int x = x0; x < x1; ++x) {
        if (fresh) {
            if (it.k.n == 0 && tid == 0) report(a.status, CCA_ERR_INVALID_ARG);
            read_tree(a, nodes, it.k, it.b);
            out0 = (static_cast<int64_t>(it.b) * a.Hq + static_cast<int64_t>(it.kv) * (a.Hq / a.Hkv)) * a.T;
            for (int e = tid; e < BM * D; e += TREE_THREADS) {
                const int row = mt * BM + e / D;
                sq[e] = row < a.R ? static_cast<const float *>(a.Q)[(out0 + row) * D + e % D] : 0.f;
            }
            if (tid < BM) {
                sm_m[tid] = -INFINITY;
                sm_l[tid] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) o[i] = 0.f;
            fresh = false;
        }
        // two threads per key bring its K and V row
        {
            const int row = tid >> 1, half = tid & 1;
            const Key key = find_key(a, it.k, it.b, it.kv, (x - it.first) * TILE + row);
            if (half == 0) {
                sm_kind[row] = key.kind;
                sm_val[row] = key.val;
            }
            const float4 *k = reinterpret_cast<const float4 *>(static_cast<const float *>(key.core ? a.Kc : a.K) + key.row * D);
            const float4 *v = reinterpret_cast<const float4 *>(static_cast<const float *>(key.core ? a.Vc : a.V) + key.row * D);
            constexpr int STEP = 8;  // 16-byte loads of K, and of V, in flight together
            for (int c0 = half * (D / 8); c0 < (half + 1) * (D / 8); c0 += STEP) {
                float4 kx[STEP], vx[STEP];
#pragma unroll
                for (int i = 0; i < STEP; ++i) {
                    kx[i] = vx[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (key.row >= 0) {
                        kx[i] = k[c0 + i];
                        vx[i] = v[c0 + i];
                    }
                }
#pragma unroll
                for (int i = 0; i < STEP; ++i) {
                    *reinterpret_cast<float4 *>(sk + row * LD + (c0 + i) * 4) = kx[i];
                    *reinterpret_cast<float4 *>(sv + row * LD + (c0 + i) * 4) = vx[i];
                }
            }
        }
        __syncthreads();
        if (tid < TILE && sm_kind[tid] == 5 && nodes.cores[sm_val[tid]] >= 0) report(a.status, CCA_ERR_INVALID_ARG);
        {
            // thread: one key, eight rows
            const int key = tid & (TILE - 1), r0 = (tid / TILE) * (BM / 2);
            float s[BM / 2];
#pragma unroll
            for (int i = 0; i < BM / 2; ++i) s[i] = 0.f;
            for (int c = 0; c < D; c += 4) {
                const float4 k = *reinterpret_cast<const float4 *>(sk + key * LD + c);
#pragma unroll
                for (int i = 0; i < BM / 2; ++i) {
                    const float4 q = *reinterpret_cast<const float4 *>(sq + (r0 + i) * D + c);
                    s[i] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[i]))));
                }
            }
#pragma unroll
            for (int i = 0; i < BM / 2; ++i) {
                const int row = mt * BM + r0 + i;
                const bool sees = row < a.R && row_sees(nodes, row % a.T, sm_kind[key], sm_val[key]);
                sp[(r0 + i) * TILE + key] = sees ? s[i] * a.scale_log2 : -INFINITY;
            }
        }
        __syncthreads();
        // a warp: four rows, two keys per lane
#pragma unroll
        for (int i = 0; i < BM / 4; ++i) {
            const int row = warp * (BM / 4) + i;
            const float s0 = sp[row * TILE + lane], s1 = sp[row * TILE + lane + 32];
            float mx = fmaxf(s0, s1);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
            mx = fmaxf(mx, sm_m[row]);
            const float base = mx == -INFINITY ? 0.f : mx;
            const float p0 = exp2f(s0 - base), p1 = exp2f(s1 - base);
            float sum = p0 + p1;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
            // -1 marks a key that the row does not see: its V is left out whatever it holds
            sp[row * TILE + lane] = s0 == -INFINITY ? -1.f : p0;
            sp[row * TILE + lane + 32] = s1 == -INFINITY ? -1.f : p1;
            if (lane == 0) {
                const float corr = exp2f(sm_m[row] - base);
                sm_c[row] = corr;
                sm_l[row] = sm_l[row] * corr + sum;
                sm_m[row] = mx;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RPT; ++i) o[i] *= sm_c[rg * RPT + i];
        for (int key = 0; key < TILE; ++key) {
            const float v = sv[key * LD + col];
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float p = sp[(rg * RPT + i) * TILE + key];
                if (!(p < 0.f)) o[i] = fmaf(p, v, o[i]);
            }
        }
        const int end = it.first + it.k.tiles;
        if (x + 1 == end || x + 1 == x1) {
            const bool whole = x0 <= it.first && end <= x1;
            float *part = part_at(a, group, mt, x0 >= it.first ? 0 : 1, BM, D);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int in = rg * RPT + i, row = mt * BM + in;
                if (row >= a.R) continue;
                const bool empty = nodes.cores[row % a.T] < 0;
                const float l = empty ? 0.f : sm_l[in], mx = empty ? -INFINITY : sm_m[in], acc = empty ? 0.f : o[i];
                if (whole) {
                    static_cast<float *>(a.O)[(out0 + row) * D + col] = l == 0.f ? 0.f : acc / l;
                    if (col == 0) a.LSE[out0 + row] = l == 0.f ? -INFINITY : (mx + log2f(l)) * kLn2;
                } else {
                    part[part_col(BM, in, col)] = acc;
                    if (col == 0) {
                        part[BM * D + in] = mx;
                        part[BM * D + BM + in] = l;
                    }
                }
            }
            if (threadIdx.x == 0 && mt == 0) note_span(a, it, group, x0, x1);
            if (x + 1 < x1) {
                next_item(a, it);
                fresh = true;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- joining the partials

constexpr int JOIN_ROWS = 32;
constexpr int JOIN_RESIDENT = 8;  // blocks per SM

// A warp joins 4C columns of up to 32 rows of one list.  The time is that of three dependent steps
// (the list's span, its parts, the stores), so blocks are small.  Where the lists are few, C is
// least, for the most blocks; many lists take twice that, which makes a row's store a whole sector
// of the output (16 sequences of 64 nodes, 128 lists of 256 rows: 15.3 -> 9.6 us).  A lane takes a
// row; where there are fewer rows, the lanes left over take parts: lane group i the parts i,
// i + groups, .. of the list, in the order of the groups that wrote them, and the lane groups
// are added up in a fixed order.  Lists that one group finished are already written.
template <typename T, int D, int C>
__global__ void __launch_bounds__(128, JOIN_RESIDENT) tree_join_kernel(const TreeArgs a, int BM) {
    constexpr int AHEAD = 8 / C;  // parts whose loads are in flight together
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lanes = 32;  // a power of two that holds the rows
    while (lanes / 2 >= a.R) lanes /= 2;
    const int row = blockIdx.y * JOIN_ROWS + (lane & (lanes - 1)), step = 32 / lanes;
    const bool live = row < a.R;
    const int mt = live ? row / BM : 0, in = live ? row - mt * BM : 0;
    const int col0 = (blockIdx.z * 4 + warp) * C;  // in float4
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int2 span = a.spans[blockIdx.x];
    const int y0 = span.x >> 1, y1 = span.y;
    if (y0 < 0 || y0 >= y1 || y1 >= a.groups) return;  // no parts (or a call that gave up)
    float mx = -INFINITY, l = 0.f;
    float4 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll AHEAD
    for (int y = y0 + lane / lanes; y <= y1; y += step) {
        const float *p = part_at(a, y, mt, y == y0 ? span.x & 1 : 0, BM, D);
        const float4 *q = reinterpret_cast<const float4 *>(p) + col0 * BM + in;
        const float m = p[BM * D + in], s = p[BM * D + BM + in];
        float4 v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = q[c * BM];
        const float top = fmaxf(mx, m), base = top == -INFINITY ? 0.f : top;
        const float f0 = exp2f(mx - base), f = exp2f(m - base);
        mx = top;
        l = fmaf(s, f, l * f0);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            acc[c].x = fmaf(v[c].x, f, acc[c].x * f0);
            acc[c].y = fmaf(v[c].y, f, acc[c].y * f0);
            acc[c].z = fmaf(v[c].z, f, acc[c].z * f0);
            acc[c].w = fmaf(v[c].w, f, acc[c].w * f0);
        }
    }
    if (step > 1) {
        float top = mx;
        for (int off = 16; off >= lanes; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        const float f = exp2f(mx - (top == -INFINITY ? 0.f : top));
        mx = top;
        l *= f;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = make_float4(acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f);
        for (int off = 16; off >= lanes; off >>= 1) {
            l += __shfl_xor_sync(kFull, l, off);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                acc[c].x += __shfl_xor_sync(kFull, acc[c].x, off);
                acc[c].y += __shfl_xor_sync(kFull, acc[c].y, off);
                acc[c].z += __shfl_xor_sync(kFull, acc[c].z, off);
                acc[c].w += __shfl_xor_sync(kFull, acc[c].w, off);
            }
        }
    }
    if (!live || lane >= lanes) return;
    const int b = blockIdx.x / a.Hkv, kv = blockIdx.x - b * a.Hkv;
    const int64_t at = (static_cast<int64_t>(b) * a.Hq + static_cast<int64_t>(kv) * (a.Hq / a.Hkv)) * a.T + row;
    const bool none = l == 0.f;
    const float by = none ? 0.f : 1.f / l;
    const int64_t to = at * D + col0 * 4;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc[c].x * by, acc[c].y * by, acc[c].z * by, acc[c].w * by);
    if constexpr (sizeof(T) == 2) {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.O) + to;
        uint2 r[C];
#pragma unroll
        for (int c = 0; c < C; ++c) r[c] = make_uint2(ptx::pack_bf16x2(acc[c].x, acc[c].y), ptx::pack_bf16x2(acc[c].z, acc[c].w));
        if constexpr (C == 1) {
            *reinterpret_cast<uint2 *>(o) = r[0];
        } else {
#pragma unroll
            for (int c = 0; c < C; c += 2) reinterpret_cast<uint4 *>(o)[c / 2] = make_uint4(r[c].x, r[c].y, r[c + 1].x, r[c + 1].y);
        }
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.O) + to);
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = acc[c];
    }
    if (col0 == 0) a.LSE[at] = none ? -INFINITY : (mx + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- launch


// Resident CTAs per SM of a kernel with `smem` bytes.  The answer depends on the kernel, the
// device and the bytes alone; the last one of each kernel and device is kept.
template <auto kernel>
cudaError_t resident(int smem, int &per_sm) {
    static std::atomic<uint64_t> kept[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool room = dev >= 0 && dev < 64;
    const uint64_t k = room ? kept[dev].load(std::memory_order_relaxed) : 0;
    if (k != 0 && static_cast<int>(k >> 32) == smem) {
        per_sm = static_cast<int>(k & 0xffffffffu);
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, TREE_THREADS, smem);
    if (e == cudaSuccess && room) kept[dev].store(static_cast<uint64_t>(smem) << 32 | static_cast<uint32_t>(per_sm));
    return e;
}

constexpr int MAX_CTAS_PER_SM = 4;

// bf16 runs on tcgen05, but for up to 16 rows at d = 64, where a tile's softmax takes longer than
// its copy and mma.sync spreads it over four warps.  tcgen05 and mma.sync, us from HBM: d = 128, one
// row of 32 heads at 32 K 29.4 and 31.6, 64 such sequences of 8 K 264 and 274; d = 64, one row of 32
// heads at 32 K 18.2 and 16.3, 32 sequences of 16 rows 50.6 and 46.8, of 24 rows 41.2 and 40.8, eight
// of 24 rows 23.4 and 25.1, of 96 rows 23.7 and 38.4, one of 20 rows at 2 K 14.9 and 19.6.
bool on_tensor_cores(int dtype, int R, int d) { return dtype == CCA_BF16 && (d == 128 || R > MMA_ROWS); }

int rows_per_cta(int dtype, int R, int d) {
    if (dtype == CCA_F32) return F32_BM;
    if (on_tensor_cores(dtype, R, d)) return tc_rows(R);
    return MMA_ROWS;
}

// The spans of the lists come first, then the partials.
int64_t span_bytes(int Hkv) { return static_cast<int64_t>(TREE_MAX_BATCH) * Hkv * sizeof(int2); }

uint64_t workspace_bytes_for(int dtype, int R, int Hkv, int d, int sms) {
    // CTAs times two slots; a grid holds one CTA per SM on the tensor cores, MAX_CTAS_PER_SM at most
    // elsewhere, and one group of row tiles at least
    const int BM = rows_per_cta(dtype, R, d);
    const int64_t n_mt = (R + BM - 1) / BM;
    int64_t ctas = static_cast<int64_t>(sms) * (on_tensor_cores(dtype, R, d) ? 1 : MAX_CTAS_PER_SM);
    if (ctas < n_mt) ctas = n_mt;
    return static_cast<uint64_t>(span_bytes(Hkv) + ctas * 2 * part_floats(BM, d) * 4);
}

template <typename T, int D>
cudaError_t run_join(const TreeArgs &a, int BM, int sms, cudaStream_t stream) {
    dim3 grid(static_cast<unsigned>(a.B) * a.Hkv, (a.R + JOIN_ROWS - 1) / JOIN_ROWS, 4);
    if (static_cast<int64_t>(grid.x) * grid.y * grid.z <= static_cast<int64_t>(JOIN_RESIDENT) * sms)
        return start_dependent(tree_join_kernel<T, D, D / 64>, grid, 128, 0, stream, a, BM);
    grid.z = 2;
    return start_dependent(tree_join_kernel<T, D, D / 32>, grid, 128, 0, stream, a, BM);
}

template <auto kernel, typename T, int D>
cudaError_t run_tree(TreeArgs a, int BM, int smem, int sms, cudaStream_t stream) {
    int per_sm = 0;
    cudaError_t e = resident<kernel>(smem, per_sm);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    if (per_sm > MAX_CTAS_PER_SM) per_sm = MAX_CTAS_PER_SM;
    a.n_mt = (a.R + BM - 1) / BM;
    a.groups = per_sm * sms / a.n_mt;
    if (a.groups < 1) a.groups = 1;
    e = start_dependent(kernel, dim3(static_cast<unsigned>(a.groups) * a.n_mt), TREE_THREADS, smem, stream, a);
    if (e != cudaSuccess) return e;
    return run_join<T, D>(a, BM, sms, stream);
}

cudaError_t run_tc(TreeArgs a, int d, int sms, cudaStream_t stream) {
    const int BM = tc_rows(a.R);
    a.n_mt = (a.R + BM - 1) / BM;
    a.groups = sms / a.n_mt;
    if (a.groups < 1) a.groups = 1;
    a.tile_log2 = 7;
    const cudaError_t e = launch_tc(a, d, g_wait_limit_ns, g_skip_q_load, stream);
    if (e != cudaSuccess) return e;
    return d == 64 ? run_join<__nv_bfloat16, 64>(a, BM, sms, stream) : run_join<__nv_bfloat16, 128>(a, BM, sms, stream);
}

int check_tree(const cca_params_t *p, int T) {
    const int st = check_paged(p, true);
    if (st != CCA_OK) return st;
    if (T < 1 || p->B > 0x7fffffff / p->Hkv) return CCA_ERR_INVALID_ARG;
    if (T > TREE_MAX_NODES || T > p->w || p->B > TREE_MAX_BATCH) return CCA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(p->Hq / p->Hkv) * T > JOIN_ROWS * 65535) return CCA_ERR_UNSUPPORTED;
    return CCA_OK;
}

}  // namespace
}  // namespace cca

extern "C" {

uint64_t cca_tree_workspace_size(const cca_params_t *params, int T) {
    using namespace cca;
    if (check_tree(params, T) != CCA_OK) return 0;
    int sms = device_sms();
    if (sms < 1) sms = 152;  // no device here: the size a GB300 needs
    return workspace_bytes_for(params->dtype, params->Hq / params->Hkv * T, params->Hkv, params->d, sms);
}

int cca_tree_fwd(const void *Q, const cca_pages_t *raw, const cca_pages_t *core, const int32_t *lens,
                 const int32_t *parents, int T, void *O, float *LSE, const cca_params_t *params, void *workspace,
                 uint64_t workspace_bytes, void *stream) {
    using namespace cca;
    int st = check_tree(params, T);
    if (st != CCA_OK) return st;
    if (!pages_ok(raw, 1) || !pages_ok(core, 1)) return CCA_ERR_INVALID_ARG;
    const void *ptrs[4] = {Q, O, LSE, workspace};
    for (const void *p : ptrs)
        if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) != 0) return CCA_ERR_INVALID_ARG;
    if (!word_ptr(lens, true) || !word_ptr(parents, false)) return CCA_ERR_INVALID_ARG;
    if (workspace_bytes < cca_tree_workspace_size(params, T)) return CCA_ERR_INVALID_ARG;
    // tiles of all lists are counted in 32 bits: the cores before a window and the window, or all
    // rows of the table where that is less, and the nodes
    const double rows = static_cast<double>(raw->rows) * raw->cols;
    const double keys = fmin(rows / params->g + params->w + params->g, rows) + 3.0 * T + params->g;
    if ((keys / TILE + LIST_COST) * params->B * params->Hkv > 2.0e9) return CCA_ERR_UNSUPPORTED;
    const uint64_t es = params->dtype == CCA_BF16 ? 2 : 4;
    const uint64_t out = static_cast<uint64_t>(params->B) * params->Hq * T * params->d * es;
    if (bytes_meet(O, out, Q, out)) return CCA_ERR_INVALID_ARG;  // row tiles of other CTAs may still read Q
    if ((st = check_device()) != CCA_OK) return st;
    const int sms = device_sms();
    if (sms < 1) return CCA_ERR_CUDA;
    TreeArgs a;
    a.Q = Q;
    a.K = raw->K;
    a.V = raw->V;
    a.Kc = core->K;
    a.Vc = core->V;
    a.table = raw->table;
    a.ctable = core->table;
    a.lens = lens;
    a.parents = parents;
    a.n_pages = raw->n_pages;
    a.rows = raw->rows;
    a.cols = raw->cols;
    a.n_cpages = core->n_pages;
    a.crows = core->rows;
    a.ccols = core->cols;
    a.B = params->B;
    a.Hq = params->Hq;
    a.Hkv = params->Hkv;
    a.T = T;
    a.most = static_cast<int>(fmin(rows, 0x7fffffff - 2 * TREE_MAX_NODES));
    a.g = params->g;
    a.w = params->w;
    a.window_mode = params->window_mode;
    a.R = params->Hq / params->Hkv * T;
    a.n_mt = 1;
    a.groups = 1;
    a.by_g = fast_div(a.g);
    a.by_rows = fast_div(a.rows);
    a.by_crows = fast_div(a.crows);
    a.tile_log2 = 6;
    a.box_log2 = 0;
    a.scale_log2 = resolve_scale(params) * 1.4426950408889634f;
    a.O = O;
    a.LSE = LSE;
    a.spans = static_cast<int2 *>(workspace);
    a.ws = reinterpret_cast<float *>(static_cast<char *>(workspace) + span_bytes(a.Hkv));
    a.status = params->dev_status;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    if (on_tensor_cores(params->dtype, a.R, params->d)) return from_cuda(run_tc(a, params->d, sms, strm));
    if (params->dtype == CCA_BF16)
        return from_cuda(run_tree<tree_bf16_kernel, __nv_bfloat16, MMA_D>(a, MMA_ROWS, TreeSmem::bytes(T), sms, strm));
    if (params->d == 128)
        return from_cuda(run_tree<tree_f32_kernel<128>, float, 128>(a, F32_BM, TreeF32Smem<128>::bytes(T), sms, strm));
    return from_cuda(run_tree<tree_f32_kernel<64>, float, 64>(a, F32_BM, TreeF32Smem<64>::bytes(T), sms, strm));
}

}  // extern "C"
