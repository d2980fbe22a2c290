// What the kernels of tree attention share: the arguments, the key list of a sequence, the
// split of all lists over the groups of a grid, the nodes' visibility, the partials.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"

namespace cca {
namespace tree {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
    const void *Q, *K, *V, *Kc, *Vc;
    const int32_t *table, *ctable, *lens, *parents;
    int n_pages, rows, cols, n_cpages, crows, ccols;
    int B, Hq, Hkv, T, g, w, window_mode;
    int R;       // query rows of a KV head: Hq / Hkv * T
    int n_mt;    // row tiles
    int tile_log2;  // keys per tile
    int box_log2;   // rows of a box that one copy can bring (0: no runs)
    int groups;  // groups of n_mt CTAs
    int min_tiles;  // tiles a group takes at least
    float scale_log2;
    void *O;
    float *LSE;
    float *ws;
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

__device__ __forceinline__ KeyList key_list(const TreeArgs &a, int b) {
    KeyList k = {};
    k.tiles = 1;
    const int len = a.lens[b];
    // a length outside the table: an empty list, and one tile in which its rows are written
    if (len < 0 || len > 0x7fffffff - 2 * TREE_MAX_NODES ||
        static_cast<int64_t>(len) + a.T > static_cast<int64_t>(a.rows) * a.cols)
        return k;
    const int last = len + a.T - 1;  // T <= w, so no window of a node begins after len
    k.len = len;
    k.cores_all = visible_cores(len, a.w, a.g);
    k.cores_some = visible_cores(last, a.w, a.g);
    k.raw_some = window_start(len, a.w, a.g, a.window_mode);
    k.raw_all = window_start(last, a.w, a.g, a.window_mode);
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

// The row of its pool that row `at` of a sequence lies in, -1 where no page is.
__device__ __forceinline__ int64_t pool_row(const TreeArgs &a, int b, int kv, bool core, int at) {
    const int per = core ? a.crows : a.rows;
    const int c = at / per;
    int page = -1;
    if (c < (core ? a.ccols : a.cols))
        page = (core ? a.ctable + static_cast<int64_t>(b) * a.ccols : a.table + static_cast<int64_t>(b) * a.cols)[c];
    if (page < 0 || page >= (core ? a.n_cpages : a.n_pages)) {
        if (a.status != nullptr) *a.status = CCA_ERR_INVALID_ARG;
        return -1;
    }
    return (static_cast<int64_t>(page) * a.Hkv + kv) * per + (at - c * per);
}

// What a key is: 0 seen by every node, 1 core `val`, 2 raw token `val`, 3 node `val`, 4 not there.
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
    r.row = pool_row(a, b, kv, r.core, at);
    if (r.row < 0) r.kind = 4;
    return r;
}

// Pool row at which box i of the runs begins, -1 where no page is.
__device__ __forceinline__ int64_t find_box(const TreeArgs &a, const KeyList &k, int b, int kv, int i, bool &core) {
    const int at = i << a.box_log2;
    core = at < k.run_cores;
    return pool_row(a, b, kv, core, core ? at : k.gap0 + (at - k.run_cores));
}

// ---------------------------------------------------------------- the split

// Runs of tiles: group y takes tiles [begin(y), begin(y + 1)) of all W tiles.
struct Split {
    int64_t W;
    int groups;
    __device__ int64_t begin(int y) const { return W * y / groups; }
    __device__ int owner(int64_t tile) const { return static_cast<int>(((tile + 1) * groups - 1) / W); }
};

__device__ __forceinline__ Split make_split(const TreeArgs &a, int64_t W) {
    Split s;
    s.W = W;
    const int64_t most = W / a.min_tiles;
    s.groups = most < a.groups ? static_cast<int>(most < 1 ? 1 : most) : a.groups;
    return s;
}

// sm_first[b] = tiles of the sequences before b (times Hkv); returns all.  B <= 1024.
__device__ __forceinline__ int64_t scan_tiles(const TreeArgs &a, int64_t *sm_first, int64_t *sm_warp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
    const int per = (a.B + nt - 1) / nt;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int64_t own = 0;
    for (int b = b0; b < b1; ++b) own += static_cast<int64_t>(key_list(a, b).tiles) * a.Hkv;
    int64_t x = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) sm_warp[warp] = x;
    __syncthreads();
    int64_t before = x - own, total = 0;
    for (int i = 0; i < nw; ++i) {
        if (i < warp) before += sm_warp[i];
        total += sm_warp[i];
    }
    for (int b = b0; b < b1; ++b) {
        sm_first[b] = before;
        before += static_cast<int64_t>(key_list(a, b).tiles) * a.Hkv;
    }
    __syncthreads();
    return total;
}

// The list that a tile belongs to.
struct Item {
    int b, kv;
    int64_t first;  // its first tile
    KeyList k;
};

__device__ __forceinline__ Item item_of(const TreeArgs &a, const int64_t *sm_first, int64_t tile) {
    Item it;
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sm_first[mid] <= tile) lo = mid;
        else hi = mid - 1;
    }
    it.b = lo;
    it.k = key_list(a, lo);
    it.kv = static_cast<int>((tile - sm_first[lo]) / it.k.tiles);
    it.first = sm_first[lo] + static_cast<int64_t>(it.kv) * it.k.tiles;
    return it;
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

__device__ __forceinline__ void read_tree(const TreeArgs &a, const Nodes &n, const KeyList &k, int b) {
    const int tid = threadIdx.x;
    for (int t = tid; t < a.T; t += blockDim.x) {
        int p = t - 1;
        if (a.parents != nullptr) {
            p = a.parents[static_cast<int64_t>(b) * a.T + t];
            if (p != -1 && (p < 0 || p >= t)) p = -2;
        }
        n.up[t] = static_cast<int16_t>(p);
    }
    __syncthreads();
    for (int t = tid; t < a.T; t += blockDim.x) {
        for (int i = 0; i < n.words; ++i) n.sees[t * n.words + i] = 0;
        int depth = -1, x = t;
        while (x >= 0) {  // parents lie below their children, so this ends
            n.sees[t * n.words + (x >> 5)] |= 1u << (x & 31);
            ++depth;
            x = n.up[x];
        }
        const int pos = k.len + depth;
        const bool whole = x == -1 && k.n > 0;
        n.cores[t] = whole ? visible_cores(pos, a.w, a.g) : -1;
        n.start[t] = window_start(pos, a.w, a.g, a.window_mode);
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

// Partials of a (group, row tile, slot): O [BM][D], max [BM], sum [BM] (log2 domain).
__host__ __device__ __forceinline__ int64_t part_floats(int BM, int D) { return static_cast<int64_t>(BM) * (D + 2); }

// Slot 0: the list that the group's run begins in; 1: the one it ends in.
__device__ __forceinline__ float *part_at(const TreeArgs &a, int group, int mt, int slot, int BM, int D) {
    return a.ws + ((static_cast<int64_t>(group) * a.n_mt + mt) * 2 + slot) * part_floats(BM, D);
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
cudaError_t launch_tc(TreeArgs a, unsigned long long wait_limit_ns, int skip_loads, cudaStream_t stream);

}  // namespace tree
}  // namespace cca
