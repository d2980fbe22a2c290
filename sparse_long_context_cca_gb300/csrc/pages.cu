// Pages of a CCA cache: handing out, sharing, copying, compacting and freeing them, on the
// device, so that a serving step needs no host round trip and can be captured.
//
// A page's state is one number, refs[page], the table entries that hold it; free means 0.
// There is no free list to keep in step: cca_pages_reserve scans refs (4 bytes a page) for
// the lowest free pages.  Results depend on the inputs alone: counts change by integer
// atomics, whose order does not matter, and everything else has one writer.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/cca.h"
#include "internal.h"
#include "paged.cuh"

namespace cca {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// The page kernels of a step follow one another, so each is launched as a programmatic dependent
// of the kernel before it: its blocks may be scheduled while that one drains, wait for its
// completion before they read anything, and let their own dependents be scheduled.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

// ---------------------------------------------------------------- reserve

constexpr int RESERVE_THREADS = 1024;
constexpr int RESERVE_WARPS = RESERVE_THREADS / 32;

struct ReserveArgs {
    int32_t *refs, *table, *pairs;
    int n_pages, B, cols, rows;
    const int32_t *lens, *extra;
    int32_t *want;   // workspace [B * cols]: the places that get a page, in row order; then what they held
    int32_t *count;  // workspace [B]: how many each row gets, then where its first one stands
    int32_t *status;
};

// Sum over the block of one value per thread, exclusive; `total` is the whole sum.
__device__ int block_scan(int v, int *sm_warp, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) sm_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = sm_warp[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int z = __shfl_up_sync(kFull, y, off);
            if (lane >= off) y += z;
        }
        sm_warp[lane] = y;
    }
    __syncthreads();
    const int before = warp > 0 ? sm_warp[warp - 1] : 0;
    total = sm_warp[RESERVE_WARPS - 1];
    __syncthreads();
    return before + x - v;
}

// One block: the calls of a step touch a few entries per row, so what bounds this is the
// chain of dependent reads (lengths, table, refs, the scan), not bandwidth: 6.5 us for 8 rows,
// 9.1 us for 64 rows of which 32 share a page (42 us when a lane looked through the rows before
// its own one at a time; 12 us with the counts in memory and a second look for the free pages).
// Where the lowest free pages lie far up the pool, it reads the counts below them 4096 a step, twice:
// 58 us for 64 pages behind 118000 held ones.
__global__ void __launch_bounds__(RESERVE_THREADS) pages_reserve_kernel(const ReserveArgs a) {
    __shared__ int sm_warp[RESERVE_WARPS];
    __shared__ int32_t sm_count[RESERVE_THREADS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ int32_t sm_len[RESERVE_THREADS], sm_extra[RESERVE_THREADS];
    const bool few = a.B <= RESERVE_THREADS;  // then what is known of a row is kept here
    int32_t *const count = few ? sm_count : a.count;
    after_previous();
    if (few) {
        if (tid < a.B) {
            sm_len[tid] = a.lens[tid];
            sm_extra[tid] = a.extra[tid];
        }
        __syncthreads();
    }
    const int32_t *const lens = few ? sm_len : a.lens, *const extra = few ? sm_extra : a.extra;
    // The columns [c0, c1) of row b that its new rows lie in; an empty range for a bad row.
    auto range = [&](int b, int &c0, int &c1) {
        const int len = lens[b], ex = extra[b];
        c0 = c1 = 0;
        if (ex <= 0) return true;
        const int64_t end = static_cast<int64_t>(len) + ex;
        if (len < 0 || end > static_cast<int64_t>(a.cols) * a.rows) return false;
        c0 = len / a.rows;
        c1 = static_cast<int>((end + a.rows - 1) / a.rows);
        return true;
    };
    // Whether row o's range takes in column c.
    auto reaches = [&](int o, int c) {
        const int len = lens[o], ex = extra[o];
        const int64_t end = static_cast<int64_t>(len) + ex, at = static_cast<int64_t>(c) * a.rows;
        return ex > 0 && len >= 0 && end <= static_cast<int64_t>(a.cols) * a.rows && at + a.rows > len && at < end;
    };
    // 1. which entries need a page: empty ones, and shared ones but for the page's last
    // holder.  A page's holders stand in the same column (rows are positions), so the rows
    // above that leave it are counted down one column, 32 rows at a time.
    for (int b = warp; b < a.B; b += RESERVE_WARPS) {
        int c0, c1, n = 0;
        if (!range(b, c0, c1) && lane == 0) report(a.status, CCA_ERR_INVALID_ARG);
        for (int base = c0; base < c1; base += 32) {
            const int c = base + lane;
            int32_t e = -1;
            int held = 0;
            if (c < c1) {
                e = a.table[static_cast<int64_t>(b) * a.cols + c];
                if (e >= a.n_pages) e = -1;
                if (e >= 0) held = a.refs[e];
            }
            bool need = c < c1 && e < 0;
            for (unsigned shared = __ballot_sync(kFull, held > 1); shared != 0; shared &= shared - 1) {
                const int src = __ffs(shared) - 1;
                const int32_t es = __shfl_sync(kFull, e, src);
                int left = 0;
                for (int o = lane; o < b; o += 32)
                    if (a.table[static_cast<int64_t>(o) * a.cols + base + src] == es && reaches(o, base + src)) ++left;
                left = __reduce_add_sync(kFull, left);
                if (lane == src) need = held - left > 1;
            }
            const unsigned m = __ballot_sync(kFull, need);
            if (need) a.want[static_cast<int64_t>(b) * a.cols + n + __popc(m & ((1u << lane) - 1u))] = c;
            n += __popc(m);
        }
        if (lane == 0) count[b] = n;
    }
    __syncthreads();
    // 2. where each row's pages stand among all
    int total = 0;
    for (int base = 0; base < a.B; base += RESERVE_THREADS) {
        const int b = base + tid;
        const int v = b < a.B ? count[b] : 0;
        int sum;
        const int at = block_scan(v, sm_warp, sum) + total;
        if (b < a.B) count[b] = at;
        total += sum;
    }
    for (int b = tid; b < a.B; b += RESERVE_THREADS) {
        a.pairs[2 * b] = -1;
        a.pairs[2 * b + 1] = -1;
    }
    if (total == 0) return;
    // 3. are there enough free pages?  Stops as soon as there are; usually the first 4096 pages do,
    // and what was found in them is used below.
    constexpr int STEP = 4 * RESERVE_THREADS;
    bool free_page[4];
    auto look = [&](int64_t p0, int &sum) {  // this thread's four pages from p0 on: free pages before them
        int n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t p = p0 + 4 * tid + i;
            free_page[i] = p < a.n_pages && a.refs[p] == 0;
            n += free_page[i];
        }
        return block_scan(n, sm_warp, sum);  // ends with a barrier: refs are read before they change
    };
    int found = 0, k = 0;
    int64_t stop = 0;  // the pages below hold the first `found` free ones
    while (found < total && stop < a.n_pages) {
        int sum;
        k = look(stop, sum);
        found += sum;
        stop += STEP;
    }
    if (found < total) {
        if (tid == 0) report(a.status, CCA_ERR_NO_PAGES);
        return;
    }
    // 4. the k-th place gets the k-th free page.  A place is found by its number: the row by
    // bisection of the rows' first places.  Where refs are looked at again meanwhile, a page that loses
    // a holder is counted down behind that: should it lose its last one (its holders stand in several
    // columns, against the rule), it is free after the call and not given out by it.
    const bool later = stop > STEP;
    int k0 = 0;
    for (int64_t p0 = 0; k0 < total; p0 += STEP) {
        int sum = found;
        if (later) k = look(p0, sum) + k0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!free_page[i]) continue;
            if (k < total) {
                int lo = 0, hi = a.B - 1;  // the last row whose first place is <= k
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (count[mid] <= k) lo = mid;
                    else hi = mid - 1;
                }
                const int b = lo;
                int32_t *place = a.want + static_cast<int64_t>(b) * a.cols + (k - count[b]);
                const int c = *place;
                int32_t *entry = a.table + static_cast<int64_t>(b) * a.cols + c;
                const int32_t old = *entry;
                const int page = static_cast<int>(p0 + 4 * tid + i);
                *entry = page;
                a.refs[page] = 1;
                if (later) *place = old;
                if (old >= 0 && old < a.n_pages) {
                    if (!later) atomicSub(&a.refs[old], 1);
                    const int len = lens[b];
                    if (c == len / a.rows && len % a.rows != 0) {
                        a.pairs[2 * b] = old;
                        a.pairs[2 * b + 1] = page;
                    }
                }
            }
            ++k;
        }
        k0 += sum;
    }
    if (!later) return;
    __syncthreads();
    for (int b = warp; b < a.B; b += RESERVE_WARPS) {
        const int n = (b + 1 < a.B ? count[b + 1] : total) - count[b];
        for (int i = lane; i < n; i += 32) {
            const int old = a.want[static_cast<int64_t>(b) * a.cols + i];
            if (old >= 0 && old < a.n_pages) atomicSub(&a.refs[old], 1);
        }
    }
}

// ---------------------------------------------------------------- fork, free

// One block per pair.  Whether a pair counts depends on the call's lists alone and on the
// dst row before the call, which only this pair may write.
__global__ void __launch_bounds__(128) pages_fork_kernel(int32_t *refs, int n_pages, int32_t *table, int B, int cols,
                                                         int rows, const int32_t *src, const int32_t *dst, int n,
                                                         const int32_t *lens, int32_t *status) {
    const int i = blockIdx.x, tid = threadIdx.x;
    after_previous();
    const int s = src[i], d = dst[i];
    bool ok = s >= 0 && s < B && d >= 0 && d < B && s != d;
    int bad = !ok;
    for (int o = tid; o < n; o += blockDim.x)
        if (src[o] == d || (o < i && dst[o] == d)) bad = 1;
    if (ok) {
        if (lens[s] < 0) bad = 1;
    }
    bad = __syncthreads_or(bad);
    if (!bad) {
        for (int c = tid; c < cols; c += blockDim.x) {
            const int32_t e = table[static_cast<int64_t>(d) * cols + c];
            if (e >= 0 && e < n_pages) bad = 1;
        }
        bad = __syncthreads_or(bad);
    }
    if (bad) {
        if (tid == 0) report(status, CCA_ERR_INVALID_ARG);
        return;
    }
    const int64_t blocks = (static_cast<int64_t>(lens[s]) + rows - 1) / rows;
    const int shared = blocks < cols ? static_cast<int>(blocks) : cols;
    for (int c = tid; c < cols; c += blockDim.x) {
        int32_t e = c < shared ? table[static_cast<int64_t>(s) * cols + c] : -1;
        if (e < 0 || e >= n_pages) e = -1;
        if (e >= 0) atomicAdd(&refs[e], 1);
        table[static_cast<int64_t>(d) * cols + c] = e;
    }
}

__global__ void __launch_bounds__(128) pages_free_kernel(int32_t *refs, int n_pages, int32_t *table, int cols,
                                                         const int32_t *first, const int32_t *last, int32_t *status) {
    const int b = blockIdx.x;
    after_previous();
    const int c0 = max(first[b], 0), c1 = min(last[b], cols);
    for (int c = c0 + static_cast<int>(threadIdx.x); c < c1; c += blockDim.x) {
        int32_t *entry = table + static_cast<int64_t>(b) * cols + c;
        const int32_t e = *entry;
        if (e < 0 || e >= n_pages) continue;
        *entry = -1;
        if (atomicSub(&refs[e], 1) <= 0) {
            atomicAdd(&refs[e], 1);
            report(status, CCA_ERR_INVALID_ARG);
        }
    }
}

// ---------------------------------------------------------------- copy, compact

constexpr int COPY_THREADS = 256;
constexpr int COPY_UNROLL = 8;  // 16-byte loads in flight per thread

// Memory-bound: 32 pages of 131 KB, K and V in four layers (67 MB moved), take 11 us from HBM,
// of which 3 us are launch and drain.  grid (blocks of a page, pairs, layers * 2): a block moves its chunks of K
// or V of one page, eight loads ahead of the stores.
__global__ void __launch_bounds__(COPY_THREADS) pages_copy_kernel(uint4 *K, uint4 *V, int64_t page_vecs, int n_pages,
                                                                  const int2 *pairs, int n, int32_t *status) {
    const int i = blockIdx.y, tid = threadIdx.x;
    after_previous();
    const int2 p = pairs[i];
    if (p.x < 0 || p.y < 0) return;
    int bad = p.x >= n_pages || p.y >= n_pages;
    for (int o = tid; o < n; o += COPY_THREADS) {
        const int2 q = pairs[o];
        if (q.x < 0 || q.y < 0) continue;
        if (q.x == p.y || (o < i && q.y == p.y)) bad = 1;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) report(status, CCA_ERR_INVALID_ARG);
        return;
    }
    uint4 *pool = (blockIdx.z & 1) ? V : K;
    pool += static_cast<int64_t>(blockIdx.z >> 1) * n_pages * page_vecs;
    const uint4 *from = pool + p.x * page_vecs;
    uint4 *to = pool + p.y * page_vecs;
    constexpr int CHUNK = COPY_THREADS * COPY_UNROLL;
    for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * CHUNK + tid; v0 < page_vecs; v0 += static_cast<int64_t>(gridDim.x) * CHUNK) {
        uint4 x[COPY_UNROLL];
#pragma unroll
        for (int u = 0; u < COPY_UNROLL; ++u)
            if (v0 + u * COPY_THREADS < page_vecs) x[u] = from[v0 + u * COPY_THREADS];
#pragma unroll
        for (int u = 0; u < COPY_UNROLL; ++u)
            if (v0 + u * COPY_THREADS < page_vecs) to[v0 + u * COPY_THREADS] = x[u];
    }
}

struct CompactArgs {
    uint4 *K, *V;
    const int32_t *table, *lens, *path, *accepted;
    int n_pages, rows, cols, A, Hkv, row_vecs, layers;
    int32_t *status;
};

// Rows move towards the front (path[i] >= i), so a thread that owns one 16-byte column of
// one head and moves the rows in rising order never overwrites a row that it still needs;
// no other thread touches that column.  A batch of rows is read before any of it is
// written; what earlier batches wrote lies below the rows that this one reads.
// 32 sequences, 4.5 rows of 256 bytes on average, 8 heads, 8 layers (9 MB): 4.8 us, the chain of
// lengths, table, rows.  grid (blocks of head columns over every layer, K and V; sequences).
__global__ void __launch_bounds__(COPY_THREADS) pages_compact_kernel(const CompactArgs a) {
    __shared__ int64_t sm_from[TREE_MAX_NODES], sm_to[TREE_MAX_NODES];  // page << 32 | row inside it
    const int b = blockIdx.y, tid = threadIdx.x;
    after_previous();
    const int n = a.accepted[b], len = a.lens[b];
    int bad = n < 0 || n > a.A || (len < 0 && n > 0);
    if (!bad) {
        for (int i = tid; i < n; i += COPY_THREADS) {
            const int node = a.path[static_cast<int64_t>(b) * a.A + i];
            if (node < i || (i > 0 && a.path[static_cast<int64_t>(b) * a.A + i - 1] >= node)) {
                bad = 1;
                continue;
            }
            const int64_t from = static_cast<int64_t>(len) + node, to = static_cast<int64_t>(len) + i;
            const int64_t cf = from / a.rows, ct = to / a.rows;
            const int pf = cf < a.cols ? a.table[static_cast<int64_t>(b) * a.cols + cf] : -1;
            const int pt = ct < a.cols ? a.table[static_cast<int64_t>(b) * a.cols + ct] : -1;
            if (pf < 0 || pf >= a.n_pages || pt < 0 || pt >= a.n_pages) bad = 1;
            sm_from[i] = (static_cast<int64_t>(pf) << 32) | (from - cf * a.rows);
            sm_to[i] = (static_cast<int64_t>(pt) << 32) | (to - ct * a.rows);
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0 && blockIdx.x == 0) report(a.status, CCA_ERR_INVALID_ARG);
        return;
    }
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * COPY_THREADS + tid;
    const int per_layer = a.Hkv * a.row_vecs;
    if (idx >= static_cast<int64_t>(per_layer) * a.layers * 2) return;
    const int64_t plane = idx / per_layer;  // layer * 2 + (K or V)
    const int in = static_cast<int>(idx - plane * per_layer);
    const int head = in / a.row_vecs, vec = in - head * a.row_vecs;
    uint4 *pool = (plane & 1) ? a.V : a.K;
    pool += (plane >> 1) * (static_cast<int64_t>(a.n_pages) * a.Hkv * a.rows * a.row_vecs) + vec;
    auto at = [&](int64_t page_row) {
        const int64_t page = page_row >> 32, row = page_row & 0xffffffffll;
        return pool + ((page * a.Hkv + head) * a.rows + row) * a.row_vecs;
    };
    constexpr int STEP = 8;
    for (int i0 = 0; i0 < n; i0 += STEP) {
        uint4 x[STEP];
#pragma unroll
        for (int k = 0; k < STEP; ++k)
            if (i0 + k < n) x[k] = *at(sm_from[i0 + k]);
#pragma unroll
        for (int k = 0; k < STEP; ++k)
            if (i0 + k < n && sm_from[i0 + k] != sm_to[i0 + k]) *at(sm_to[i0 + k]) = x[k];
    }
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool good4(const void *p) { return p != nullptr && aligned4(p); }

// The parts of cca_params_t that say how wide a pool's row is.
int check_rows(const cca_params_t *p, bool batch) {
    if (p == nullptr || p->Hkv < 1 || p->d < 1 || (batch && p->B < 1)) return CCA_ERR_INVALID_ARG;
    if (p->dtype != CCA_BF16 && p->dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (!aligned4(p->dev_status)) return CCA_ERR_INVALID_ARG;
    if (p->d != 64 && p->d != 128) return CCA_ERR_UNSUPPORTED;
    return CCA_OK;
}

bool pools_apart(const cca_pages_t *p, const cca_params_t *q) {
    const uint64_t bytes = static_cast<uint64_t>(p->layers) * p->n_pages * p->rows * q->Hkv * q->d * (q->dtype == CCA_BF16 ? 2 : 4);
    const uintptr_t k = reinterpret_cast<uintptr_t>(p->K), v = reinterpret_cast<uintptr_t>(p->V);
    return k + bytes <= v || v + bytes <= k;
}

}  // namespace
}  // namespace cca

extern "C" {

uint64_t cca_pages_reserve_workspace_size(int B, int cols) {
    if (B < 1 || cols < 1) return 0;
    return 4ull * (static_cast<uint64_t>(B) * cols + B) + 16;
}

int cca_pages_reserve(int32_t *refs, int n_pages, int32_t *table, int B, int cols, int rows, const int32_t *lens,
                      const int32_t *extra, int32_t *pairs, void *workspace, uint64_t workspace_bytes,
                      int32_t *dev_status, void *stream) {
    using namespace cca;
    if (n_pages < 1 || B < 1 || cols < 1 || rows < 1) return CCA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(B) * cols > 0x7fffffff) return CCA_ERR_UNSUPPORTED;
    const void *ptrs[6] = {refs, table, lens, extra, pairs, workspace};
    for (const void *p : ptrs)
        if (!good4(p)) return CCA_ERR_INVALID_ARG;
    if (!aligned4(dev_status) || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return CCA_ERR_INVALID_ARG;
    if (workspace_bytes < cca_pages_reserve_workspace_size(B, cols)) return CCA_ERR_INVALID_ARG;
    int st;
    if ((st = check_device()) != CCA_OK) return st;
    ReserveArgs a;
    a.refs = refs;
    a.table = table;
    a.pairs = pairs;
    a.n_pages = n_pages;
    a.B = B;
    a.cols = cols;
    a.rows = rows;
    a.lens = lens;
    a.extra = extra;
    a.count = static_cast<int32_t *>(workspace);
    a.want = a.count + B;
    a.status = dev_status;
    return from_cuda(start_dependent(pages_reserve_kernel, dim3(1), RESERVE_THREADS, 0, static_cast<cudaStream_t>(stream), a));
}

int cca_pages_fork(int32_t *refs, int n_pages, int32_t *table, int B, int cols, int rows, const int32_t *src,
                   const int32_t *dst, int n, const int32_t *lens, int32_t *dev_status, void *stream) {
    using namespace cca;
    if (n_pages < 1 || B < 1 || cols < 1 || rows < 1 || n < 0) return CCA_ERR_INVALID_ARG;
    if (!good4(refs) || !good4(table) || !good4(lens) || !aligned4(dev_status)) return CCA_ERR_INVALID_ARG;
    if (n > 0 && (!good4(src) || !good4(dst))) return CCA_ERR_INVALID_ARG;
    if (n > 65536) return CCA_ERR_UNSUPPORTED;
    int st;
    if ((st = check_device()) != CCA_OK) return st;
    if (n == 0) return CCA_OK;
    return from_cuda(start_dependent(pages_fork_kernel, dim3(n), 128, 0, static_cast<cudaStream_t>(stream), refs, n_pages, table, B,
                                     cols, rows, src, dst, n, lens, dev_status));
}

int cca_pages_free(int32_t *refs, int n_pages, int32_t *table, int B, int cols, const int32_t *first,
                   const int32_t *last, int32_t *dev_status, void *stream) {
    using namespace cca;
    if (n_pages < 1 || B < 1 || cols < 1) return CCA_ERR_INVALID_ARG;
    if (!good4(refs) || !good4(table) || !good4(first) || !good4(last) || !aligned4(dev_status)) return CCA_ERR_INVALID_ARG;
    int st;
    if ((st = check_device()) != CCA_OK) return st;
    return from_cuda(start_dependent(pages_free_kernel, dim3(B), 128, 0, static_cast<cudaStream_t>(stream), refs, n_pages, table, cols,
                                     first, last, dev_status));
}

int cca_pages_copy(const cca_pages_t *pages, const int32_t *pairs, int n, const cca_params_t *params, void *stream) {
    using namespace cca;
    int st = check_rows(params, false);
    if (st != CCA_OK) return st;
    if (pages == nullptr || pages->K == nullptr || pages->V == nullptr) return CCA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(pages->K) | reinterpret_cast<uintptr_t>(pages->V)) & 15u) != 0) return CCA_ERR_INVALID_ARG;
    if (pages->n_pages < 1 || pages->rows < 1 || pages->layers < 1 || n < 0) return CCA_ERR_INVALID_ARG;
    if (!pools_apart(pages, params)) return CCA_ERR_INVALID_ARG;
    if (n > 0 && (pairs == nullptr || (reinterpret_cast<uintptr_t>(pairs) & 7u) != 0)) return CCA_ERR_INVALID_ARG;
    const int64_t vecs = static_cast<int64_t>(params->Hkv) * pages->rows * params->d * (params->dtype == CCA_BF16 ? 2 : 4) / 16;
    int64_t chunks = (vecs + COPY_THREADS * COPY_UNROLL - 1) / (COPY_THREADS * COPY_UNROLL);
    if (n > 65535 || pages->layers > 32767) return CCA_ERR_UNSUPPORTED;
    // Every block looks through all pairs for clashes, so a page gets as few blocks as still
    // leave 4096 in all (27 for each SM).
    const int64_t planes = 2ll * pages->layers * (n > 0 ? n : 1);
    if (chunks * planes > 4096) chunks = 4096 / planes > 1 ? 4096 / planes : 1;
    if ((st = check_device()) != CCA_OK) return st;
    if (n == 0) return CCA_OK;
    const dim3 grid(static_cast<unsigned>(chunks), n, 2 * pages->layers);
    return from_cuda(start_dependent(pages_copy_kernel, grid, COPY_THREADS, 0, static_cast<cudaStream_t>(stream),
                                     static_cast<uint4 *>(pages->K), static_cast<uint4 *>(pages->V), vecs, pages->n_pages,
                                     reinterpret_cast<const int2 *>(pairs), n, params->dev_status));
}

int cca_pages_compact(const cca_pages_t *pages, const int32_t *lens, const int32_t *path, int A,
                      const int32_t *accepted, const cca_params_t *params, void *stream) {
    using namespace cca;
    int st = check_rows(params, true);
    if (st != CCA_OK) return st;
    if (!pages_ok(pages, 0) || !pools_apart(pages, params)) return CCA_ERR_INVALID_ARG;
    if (!good4(lens) || !good4(path) || !good4(accepted) || A < 1) return CCA_ERR_INVALID_ARG;
    if (A > TREE_MAX_NODES || params->B > 65535) return CCA_ERR_UNSUPPORTED;
    CompactArgs a;
    a.K = static_cast<uint4 *>(pages->K);
    a.V = static_cast<uint4 *>(pages->V);
    a.table = pages->table;
    a.lens = lens;
    a.path = path;
    a.accepted = accepted;
    a.n_pages = pages->n_pages;
    a.rows = pages->rows;
    a.cols = pages->cols;
    a.A = A;
    a.Hkv = params->Hkv;
    a.row_vecs = params->d * (params->dtype == CCA_BF16 ? 2 : 4) / 16;
    a.layers = pages->layers;
    a.status = params->dev_status;
    const int64_t blocks = (static_cast<int64_t>(a.Hkv) * a.row_vecs * a.layers * 2 + COPY_THREADS - 1) / COPY_THREADS;
    if (blocks > 0x7fffffff) return CCA_ERR_UNSUPPORTED;
    if ((st = check_device()) != CCA_OK) return st;
    return from_cuda(start_dependent(pages_compact_kernel, dim3(static_cast<unsigned>(blocks), params->B), COPY_THREADS, 0,
                                     static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
