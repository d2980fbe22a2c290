// What the kernels of tree attention share: the arguments, the key list of a sequence, the
// split of all lists over the groups of a grid, the nodes' visibility, the partials.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace cca {
namespace tree {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
    const void *Q, *K, *V, *Kc, *Vc;
    const int32_t *table, *ctable, *lens, *parents;
    int n_pages, rows, cols, n_cpages, crows, ccols;
    int B, Hq, Hkv, T, g, w, window_mode;
    int most;  // the longest length that lies in the table
    int R;       // query rows of a KV head: Hq / Hkv * T
    int n_mt;    // row tiles
    int tile_log2;  // keys per tile
    int box_log2;   // rows of a box that one copy can bring (0: no runs)
    int groups;  // groups of n_mt CTAs
    FastDiv by_g, by_rows, by_crows;
    float scale_log2;
    void *O;
    float *LSE;
    int2 *spans;  // per list: the group it begins in, times two, plus its slot there; the group it ends in
    float *ws;  // partials
    int32_t *status;
};

// Keys of one sequence, in the order in which they are dealt to tiles:
//   runs   with a.box > 0: whole boxes of a.box consecutive rows of one page that every node
//          sees, cores first, then raw tokens; as many as fill whole tiles
//   rest   the other keys that every node sees, then those that only some see: cores, raw
//          tokens, the nodes themselves
struct KeyList {
    int len;
    int cores_all, raw_all;   // cores [0, cores_all) and raw [raw_all, len) are seen by every node
    int cores_some;           // cores [cores_all, cores_some) by some
    int raw_some;             // raw [raw_some, raw_all) by some
    int run_tiles, run_cores; // tiles made of runs; cores in them
    int gap0, gap1;           // raw tokens [gap0, gap1) lie in runs
    int n_all, n;             // of the rest: keys seen by every node; keys in all (0: no list)
    int tiles;
};

__device__ __forceinline__ KeyList key_list_of(const TreeArgs &a, int len) {
    KeyList k = {};
    k.tiles = 1;
    // A length outside the table: an empty list, and one tile in which its rows are written.  Nodes
    // past the table's end are keys that are not there (padding may lie there).
    if (len < 0 || len > a.most) return k;
    const int last = len + a.T - 1;  // T <= w, so no window of a node begins after len
    k.len = len;
    k.cores_all = a.by_g.div(window_lo(len, a.w));
    k.cores_some = a.by_g.div(window_lo(last, a.w));
    k.raw_some = a.window_mode ? k.cores_all * a.g : window_lo(len, a.w);
    k.raw_all = a.window_mode ? k.cores_some * a.g : window_lo(last, a.w);
    k.gap0 = k.gap1 = len;
    if (a.box_log2 > 0) {
        const int lg = a.box_log2;
        const int cb = k.cores_all >> lg, r0 = (k.raw_all + (1 << lg) - 1) >> lg, r1 = len >> lg;
        const int boxes = cb + (r1 > r0 ? r1 - r0 : 0);
        k.run_tiles = boxes >> (a.tile_log2 - lg);
        const int used = k.run_tiles << (a.tile_log2 - lg);
        k.run_cores = (used < cb ? used : cb) << lg;
        if (used > cb) {
            k.gap0 = r0 << lg;
            k.gap1 = (r0 + used - cb) << lg;
        }
    }
    k.n_all = (k.cores_all - k.run_cores) + (k.gap0 - k.raw_all) + (len - k.gap1);
    k.n = k.n_all + (k.cores_some - k.cores_all) + (k.raw_all - k.raw_some) + a.T;
    k.tiles = k.run_tiles + ((k.n + (1 << a.tile_log2) - 1) >> a.tile_log2);
    return k;
}

__device__ __forceinline__ KeyList key_list(const TreeArgs &a, int b) { return key_list_of(a, a.lens[b]); }

// A node's parent: an earlier node, -1 for the root, -2 for none.
__device__ __forceinline__ int parent_in(const int32_t *parents, int t) {
    const int p = parents[t];
    return p >= -1 && p < t ? p : -2;
}
__device__ __forceinline__ int parent_of(const TreeArgs &a, int b, int t) {
    return a.parents == nullptr ? t - 1 : parent_in(a.parents + static_cast<int64_t>(b) * a.T, t);
}

// The row of its pool that row `at` of a sequence lies in, -1 where no page is.  That is reported but
// for the row of a node, which may be padding.
__device__ __forceinline__ int64_t pool_row(const TreeArgs &a, int b, int kv, bool core, int at, bool node = false) {
    const int per = core ? a.crows : a.rows;
    const int c = core ? a.by_crows.div(at) : a.by_rows.div(at);
    int page = -1;
    if (c < (core ? a.ccols : a.cols))
        page = (core ? a.ctable + static_cast<int64_t>(b) * a.ccols : a.table + static_cast<int64_t>(b) * a.cols)[c];
    if (page < 0 || page >= (core ? a.n_cpages : a.n_pages)) {
        if (!node) report(a.status, CCA_ERR_INVALID_ARG);
        return -1;
    }
    return (static_cast<int64_t>(page) * a.Hkv + kv) * per + (at - c * per);
}

// What a key is: 0 seen by every node, 1 core `val`, 2 raw token `val`, 3 node `val`, 4 not there,
// 5 node `val`, which has no page.
struct Key {
    int kind, val;
    int64_t row;  // row of its pool
    bool core;
};

// Key x of the rest.
__device__ __forceinline__ Key find_key(const TreeArgs &a, const KeyList &k, int b, int kv, int x) {
    Key r;
    r.kind = 0;
    r.core = false;
    r.row = -1;
    int at;
    if (x < k.n_all) {
        const int nc = k.cores_all - k.run_cores;
        r.core = x < nc;
        at = r.core ? k.run_cores + x : k.raw_all + (x - nc);
        if (!r.core && at >= k.gap0) at += k.gap1 - k.gap0;
    } else if (x >= k.n) {
        r.kind = 4;
        r.val = 0;
        return r;
    } else {
        x -= k.n_all;
        const int nc = k.cores_some - k.cores_all, nr = k.raw_all - k.raw_some;
        if (x < nc) {
            r.kind = 1;
            r.core = true;
            at = k.cores_all + x;
        } else if (x < nc + nr) {
            r.kind = 2;
            at = k.raw_some + (x - nc);
        } else {
            r.kind = 3;
            at = k.len + (x - nc - nr);
        }
    }
    r.val = r.kind == 3 ? at - k.len : at;
    r.row = pool_row(a, b, kv, r.core, at, r.kind == 3);
    if (r.row < 0) r.kind = r.kind == 3 ? 5 : 4;
    return r;
}

// For kernels that look keys up before they know the tree: a node without a page is reported if its
// chain reaches the root (others are padding) and becomes a key that is not there.  Not inlined, as it
// is rare.
static __device__ __noinline__ void report_node(int32_t *status, const int32_t *parents, int t) {
    if (parents == nullptr) t = -1;
    while (t >= 0) t = parent_in(parents, t);
    if (t == -1) report(status, CCA_ERR_INVALID_ARG);
}
__device__ __forceinline__ Key settled(const TreeArgs &a, int b, Key key) {
    if (key.kind == 5) {
        if (a.status != nullptr) report_node(a.status, a.parents == nullptr ? nullptr : a.parents + static_cast<int64_t>(b) * a.T, key.val);
        key.kind = 4;
    }
    return key;
}

// Pool row at which box i of the runs begins, -1 where no page is.
__device__ __forceinline__ int64_t find_box(const TreeArgs &a, const KeyList &k, int b, int kv, int i, bool &core) {
    const int at = i << a.box_log2;
    core = at < k.run_cores;
    return pool_row(a, b, kv, core, core ? at : k.gap0 + (at - k.run_cores));
}

// ---------------------------------------------------------------- the split

// All W units in equal runs: the first W mod groups groups take one more.  W < 2^31.
struct Split {
    int groups, each, more;
    __device__ __forceinline__ int begin(int y) const { return y * each + min(y, more); }
};

__device__ __forceinline__ Split make_split(const TreeArgs &a, int W) {
    Split s;
    s.groups = W < a.groups ? W : a.groups;
    s.each = W / s.groups;
    s.more = W - s.each * s.groups;
    return s;
}

// What a list's end costs its CTA (masks, output, the next list's start), in tiles: a list counts
// as its tiles and so many units behind them, and runs with a list's end in them take fewer tiles.
// 8 x 24 nodes, 64 lists over 152 CTAs: 28.3 us at 0, 26.8 at 2 and at 3; one token of 32 heads 18.5,
// 17.6, 17.7; d = 64, one token 18.4, 16.9, 16.3.  No more tiles than groups: a tile each.
constexpr int LIST_COST = 3;
__device__ __forceinline__ int unit_cost(const TreeArgs &a, int tiles) { return tiles <= a.groups ? 0 : LIST_COST; }

// Where unit u of a sequence's lists lies: list `kv`, tile `off` of it, `tiles` where it is behind them.
struct Unit {
    int kv, off;
};
__device__ __forceinline__ Unit find_unit(int u, int tiles, int cost) {
    const int kv = u / (tiles + cost);
    return Unit{kv, min(u - kv * (tiles + cost), tiles)};
}

// One (b, KV head) list.
struct Item {
    int b, kv;
    int first;  // its first tile
    KeyList k;
};

// A CTA's run of tiles and the list that it begins in.
struct Run {
    Item item;
    int x0, x1;
};

// What a larger batch needs of shared memory to find it.
struct Start {
    Run run;
    int warp_sum[16];
};

// Lengths to tiles to runs: every CTA adds up the tiles of all lists for itself, a thread per
// sequence.  Up to 32 sequences each warp does it alone, in registers; more go through shared
// memory and two barriers.
__device__ __forceinline__ Run find_run(const TreeArgs &a, int group, Start &st) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
    if (a.B <= 32) {
        KeyList k = {};
        if (lane < a.B) k = key_list(a, lane);
        const int own = k.tiles * a.Hkv;
        int x = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(kFull, x, off);
            if (lane >= off) x += y;
        }
        const int total = __shfl_sync(kFull, x, 31);
        const int cost = unit_cost(a, total), step = cost * a.Hkv;  // units behind a sequence's lists
        const Split s = make_split(a, total + step * a.B);
        Run r = {};
        if (group >= s.groups) return r;
        const int u0 = s.begin(group), u1 = s.begin(group + 1);
        // the sequences that hold units u0 and u1
        const int top = x + step * min(lane + 1, a.B);
        int src = __ffs(__ballot_sync(kFull, top > u0)) - 1;
        const int src1 = __ffs(__ballot_sync(kFull, top > u1)) - 1;
        const int tiles = __shfl_sync(kFull, k.tiles, src), tiles1 = __shfl_sync(kFull, k.tiles, src1 & 31);
        const int before = __shfl_sync(kFull, x - own, src), before1 = __shfl_sync(kFull, x - own, src1 & 31);
        Unit at = find_unit(u0 - before - step * src, tiles, cost);
        r.x0 = before + at.kv * tiles + at.off;
        r.x1 = total;
        if (src1 >= 0) {
            const Unit e = find_unit(u1 - before1 - step * src1, tiles1, cost);
            r.x1 = before1 + e.kv * tiles1 + e.off;
        }
        if (at.off == tiles) {  // behind a list: the next one
            at.off = 0;
            if (++at.kv == a.Hkv) {
                at.kv = 0;
                ++src;
            }
        }
        int *out = reinterpret_cast<int *>(&r.item.k);
        const int *in = reinterpret_cast<const int *>(&k);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(KeyList) / 4); ++i) out[i] = __shfl_sync(kFull, in[i], src & 31);
        r.item.b = src;
        r.item.kv = at.kv;
        r.item.first = r.x0 - at.off;
        return r;
    }
    const int per = (a.B + nt - 1) / nt;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int own = 0;
    KeyList k = {};
    for (int b = b0; b < b1; ++b) {
        k = key_list(a, b);
        own += k.tiles * a.Hkv;
    }
    int x = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) st.warp_sum[warp] = x;
    __syncthreads();
    int before = x - own, total = 0;
    for (int i = 0; i < nw; ++i) {
        if (i < warp) before += st.warp_sum[i];
        total += st.warp_sum[i];
    }
    const int cost = unit_cost(a, total), step = cost * a.Hkv;
    const Split s = make_split(a, total + step * a.B);
    const int u0 = s.begin(group), u1 = s.begin(group + 1);
    if (tid == 0) {
        if (group >= s.groups) st.run.x0 = st.run.x1 = 0;
        else if (group == s.groups - 1) st.run.x1 = total;
    }
    if (group < s.groups) {
        for (int b = b0; b < b1; ++b) {
            if (per > 1) k = key_list(a, b);
            const int lo = before + step * b, hi = lo + (k.tiles + cost) * a.Hkv;
            if (u0 >= lo && u0 < hi) {
                Unit at = find_unit(u0 - lo, k.tiles, cost);
                st.run.x0 = before + at.kv * k.tiles + at.off;
                st.run.item.first = st.run.x0 - at.off;
                st.run.item.b = b;
                st.run.item.kv = at.kv;
                st.run.item.k = k;
                if (at.off == k.tiles) {  // behind a list: the next one
                    st.run.item.first = st.run.x0;
                    if (++st.run.item.kv == a.Hkv) {
                        st.run.item.kv = 0;
                        if (++st.run.item.b < a.B) st.run.item.k = key_list(a, b + 1);
                    }
                }
            }
            if (u1 >= lo && u1 < hi) {
                const Unit e = find_unit(u1 - lo, k.tiles, cost);
                st.run.x1 = before + e.kv * k.tiles + e.off;
            }
            before += k.tiles * a.Hkv;
        }
    }
    __syncthreads();
    return st.run;
}

__device__ __forceinline__ void next_item(const TreeArgs &a, Item &it) {
    it.first += it.k.tiles;
    if (++it.kv == a.Hkv) {
        it.kv = 0;
        if (++it.b < a.B) it.k = key_list(a, it.b);
    }
}

// ---------------------------------------------------------------- the nodes

// Per node: its first raw token, its visible cores (-1 for an empty node), its ancestors and
// itself as bits.  All threads call; `up` holds the parents meanwhile.
struct Nodes {
    int *start, *cores;
    uint32_t *sees;  // [T][words]
    int16_t *up;
    int words;
};

// A node's chain to the root: how deep it is, whether it gets there.  Its bits are added to
// `bits`; parents lie below their children, so it ends and its words fall.
struct Chain {
    int depth;
    bool whole;
};
__device__ __forceinline__ Chain walk_chain(const int16_t *up, uint32_t *bits, int n) {
    int depth = -1, at = n >> 5;
    uint32_t word = 0;
    while (n >= 0) {
        if ((n >> 5) != at) {
            bits[at] = word;
            word = 0;
            at = n >> 5;
        }
        word |= 1u << (n & 31);
        ++depth;
        n = up[n];
    }
    bits[at] = word;
    return Chain{depth, n == -1};
}

__device__ __forceinline__ void read_tree(const TreeArgs &a, const Nodes &n, const KeyList &k, int b) {
    const int tid = threadIdx.x;
    for (int t = tid; t < a.T; t += blockDim.x) {
        n.up[t] = static_cast<int16_t>(parent_of(a, b, t));
    }
    __syncthreads();
    for (int t = tid; t < a.T; t += blockDim.x) {
        for (int i = 0; i < n.words; ++i) n.sees[t * n.words + i] = 0;
        const Chain c = walk_chain(n.up, n.sees + t * n.words, t);
        const int lo = window_lo(k.len + c.depth, a.w), cores = a.by_g.div(lo);
        n.cores[t] = c.whole && k.n > 0 ? cores : -1;
        n.start[t] = a.window_mode ? cores * a.g : lo;
    }
    __syncthreads();
}

__device__ __forceinline__ bool row_sees(const Nodes &n, int t, int kind, int val) {
    if (kind == 0) return true;
    if (kind == 1) return val < n.cores[t];
    if (kind == 2) return val >= n.start[t];
    if (kind == 3) return (n.sees[t * n.words + (val >> 5)] >> (val & 31)) & 1u;
    return false;
}

// Partials of a (group, row tile, slot): O as [D / 4][BM][4], so that the rows of a warp lie
// side by side for those who write and read a row per lane; then max [BM] and sum [BM] (log2
// domain).
__host__ __device__ __forceinline__ int64_t part_floats(int BM, int D) { return static_cast<int64_t>(BM) * (D + 2); }
__device__ __forceinline__ int part_col(int BM, int row, int col) { return (col >> 2) * BM * 4 + row * 4 + (col & 3); }

// Slot 0: the list that the group's run begins in; 1: the one it ends in.
__device__ __forceinline__ float *part_at(const TreeArgs &a, int group, int mt, int slot, int BM, int D) {
    return a.ws + ((static_cast<int64_t>(group) * a.n_mt + mt) * 2 + slot) * part_floats(BM, D);
}

// The groups of a run's first and last lists say so for the join, which need not find them again.
__device__ __forceinline__ void note_span(const TreeArgs &a, const Item &it, int group, int x0, int x1) {
    int2 *span = a.spans + it.b * a.Hkv + it.kv;
    if (it.first >= x0) span->x = 2 * group + (it.first == x0 ? 0 : 1);
    if (it.first + it.k.tiles <= x1) span->y = group;
}

// ---------------------------------------------------------------- the weights

// Rows per KV head up to which the softmax weights meet V in two bf16 parts, 2^-14 of a weight in
// all: one token of up to 16 heads is plain decoding, which keeps its weights in fp32 over a
// contiguous cache.  One part, 2^-8, makes an output's error 1.4 times what its own rounding to bf16
// makes; more rows, which are there for the matrix units, have that (a second product each and the
// parts' arithmetic took 8 sequences of 24 nodes from 26.5 to 28.7 us).
constexpr int TWO_PART_ROWS = 16;

// The high part is a weight cut off to bf16, so the low part is not negative; it takes 2^-23 of the
// weight along (factor `more`) and is 0 for the weight 0 alone: an infinity in V times either part is
// what it is times the weight.
constexpr float LOW_MORE = 1.00000011920928955f;
// p - cut(p) for two weights; mask 0 (and more = 1) leaves them as they are.
__device__ __forceinline__ void low_parts(float &p0, float &p1, uint32_t mask, float more) {
    const uint64_t cut = ptx::f2(__uint_as_float((__float_as_uint(p0) & mask) ^ 0x80000000u),
                                 __uint_as_float((__float_as_uint(p1) & mask) ^ 0x80000000u));
    ptx::f2_split(ptx::fma2(ptx::f2(p0, p1), ptx::f2(more, more), cut), p0, p1);
}

// ---------------------------------------------------------------- copies

// 16 bytes to shared memory, zeros where there is nothing to read.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there) {
    const int n = there ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Dynamic shared memory a CTA may have, resident CTAs that the workspace is sized for.
constexpr int MAX_SMEM = 227 * 1024;

// Tensor-core kernel (tree_tc.cu): bf16, d = 128.  Rows of a CTA for R rows per KV head.
int tc_rows(int R);
cudaError_t launch_tc(TreeArgs a, int d, unsigned long long wait_limit_ns, int skip_loads, cudaStream_t stream);

}  // namespace tree
}  // namespace cca
