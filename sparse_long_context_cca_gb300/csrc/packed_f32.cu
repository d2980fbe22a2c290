// Attention over packed sequences and its gradient in fp32 on CUDA cores (a tf32 product would miss its
// tolerance; operands split into several bf16 or tf32 parts for the tensor cores were not tried).
//
// Tiles of 64 query rows by 64 keys, 256 threads.  A thread owns 4 x 4 scores, 16
// threads a row of them; operands lie in shared memory as fp32 rows padded by one 16-byte chunk, so
// that a product's four-column reads of eight different rows fall into different banks.  Per 16-byte
// read a thread does eight multiply-adds in the score products and 10.7 in the others.  A tile's copies
// (cp.async) run while the products that do not need them are formed: keys while weights meet values,
// values while scores are formed.
//
// 1500 tokens of four heads of 64 (few tiles): 25 us against 45 without the groups of small calls, which give
// each SM two blocks of 32 rows whose thread groups take every second key tile, and 21 since products leave out
// the keys that a list's last tile does not have; with many tiles the multiply-adds bound it: eight sequences of
// 4 K tokens in all, 8 heads of 128, causal, take 297-304 us, 31-32 TF/s of the units' 74, a training step of four sequences
// of 2 K in all (8 heads over 4) 631-659 us at d = 64, causal, and 452 at d = 128 with a window of 256 and cores.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "packed.cuh"
#include "sm100_ptx.cuh"

namespace cca {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int BS = 64;  // rows and keys of a tile
constexpr int SIMT_THREADS = 256;  // four threads to a row
constexpr int SMALL_BLOCKS = 4;    // blocks of 64 rows an SM below which a call is small
constexpr int SMALL_GROUPS = 2;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// The weight of a key that is not seen.  One that is seen may have a weight of +0, and that times an infinite value is NaN.
constexpr float MASKED = -0.f;

template <int D>
constexpr int PITCH = D + 4;
constexpr int SP = BS + 4;  // pitch of the score tile
template <int D>
constexpr int TILE_FLOATS = BS * PITCH<D>;

// Starts copying `rows` rows from y0 on of src (those below `end`; zeros behind) to dst, as one group.
template <int D, int THREADS>
__device__ __forceinline__ void copy_rows(float *dst, const float *src, int64_t row_stride, int y0, int end, int rows) {
    constexpr int LPR = D / 4, STEP = THREADS / LPR;
    const int tid = threadIdx.x % THREADS, c = tid % LPR * 4;
    const uint32_t to = ptx::smem_addr(dst);
#pragma unroll 4
    for (int row = tid / LPR; row < rows; row += STEP) {
        const bool in = y0 + row < end;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (row * PITCH<D> + c) * 4),
                     "l"(src + (in ? (y0 + row) * row_stride : 0) + c), "r"(in ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// s[i][j] = a_(4 ty + i) . b_(tx + 16 j), j < NJ
template <int D, int NJ = 4>
__device__ __forceinline__ void scores(const float *a, const float *b, int ty, float (&s)[4][4]) {
    const int tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 x[4], y[NJ];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(a + (ty * 4 + i) * PITCH<D> + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * PITCH<D> + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                s[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, s[i][j]))));
    }
}
// The same of the first `keys` rows of b: the last tile of a list of keys often holds few.
template <int D>
__device__ __forceinline__ void scores_of(const float *a, const float *b, int ty, int keys, float (&s)[4][4]) {
    if (keys > 32) scores<D, 4>(a, b, ty, s);
    else if (keys > 16) scores<D, 2>(a, b, ty, s);
    else scores<D, 1>(a, b, ty, s);
}

// acc[i][..] += sum_k p[4 ty + i][k] b_k, k < keys, over the columns 4 tx + 64 c.  GUARD: keys of weight MASKED take no part.
template <int D, bool GUARD>
__device__ __forceinline__ void add_rows(const float *p, const float *b, int ty, int keys, float (&acc)[4][D / 16]) {
    const int tx = threadIdx.x % 16;
#pragma unroll 2
    for (int k = 0; k < keys; k += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4 *>(p + (ty * 4 + i) * SP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 v = *reinterpret_cast<const float4 *>(b + (k + kk) * PITCH<D> + tx * 4 + 64 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
                    if (GUARD && __float_as_uint(x) == 0x80000000u) continue;
                    acc[i][4 * c] = fmaf(x, v.x, acc[i][4 * c]);
                    acc[i][4 * c + 1] = fmaf(x, v.y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(x, v.z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(x, v.w, acc[i][4 * c + 3]);
                }
            }
    }
}

// acc[i][..] += sum_q p[q][4 ty + i] b_q: the same with the weights' tile read by columns.
template <int D>
__device__ __forceinline__ void add_columns(const float *p, const float *b, float (&acc)[4][D / 16]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 4
    for (int q = 0; q < BS; ++q) {
        const float4 w = *reinterpret_cast<const float4 *>(p + q * SP + ty * 4);
        const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const float4 v = *reinterpret_cast<const float4 *>(b + q * PITCH<D> + tx * 4 + 64 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][4 * c] = fmaf(x[i], v.x, acc[i][4 * c]);
                acc[i][4 * c + 1] = fmaf(x[i], v.y, acc[i][4 * c + 1]);
                acc[i][4 * c + 2] = fmaf(x[i], v.z, acc[i][4 * c + 2]);
                acc[i][4 * c + 3] = fmaf(x[i], v.w, acc[i][4 * c + 3]);
            }
        }
    }
}

__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
struct SimtArgs {
    Rows<const float> Q, K, V, O, dO;
    Rows<float> out, dK, dV;  // out: O, or dQ
    const float *Kc, *Vc;
    float *LSE;
    PackedBwdSpace w;
    Plan plan;
    int Hq, Hkv, cores;
    float tau;
};

// ROWS query rows of one head.
struct Block {
    int a, n, i0, c0;  // first row of the sequence, its length, the block's first row in it, its first core row
    int h, kv;
};
template <int ROWS>
__device__ __forceinline__ bool query_block(const SimtArgs &p, Block &b) {
    constexpr int PER = PACK_TILE / ROWS;
    const int64_t item = blockIdx.x / p.Hq;
    if (item >= static_cast<int64_t>(PER) * plan_counts(p.plan).y) return false;
    const int4 e = p.plan.tiles[item / PER];
    b.a = e.x, b.n = e.y, b.c0 = e.w;
    b.i0 = e.z * PACK_TILE + (PER - 1 - static_cast<int>(item % PER)) * ROWS;
    b.h = blockIdx.x % p.Hq;
    b.kv = b.h / (p.Hq / p.Hkv);
    return b.i0 < b.n;
}

// The key tiles that `rows` query rows see: cores, then the band from the first row's window on.
struct Keys {
    int cores, lo, tiles, end;
    __device__ __forceinline__ Keys(const Plan &p, const Block &b, int rows) {
        const int last = min(b.i0 + rows, b.n) - 1;
        cores = p.cores_of(last);
        lo = p.start_of(b.i0);
        end = last + 1;
        tiles = (cores + BS - 1) / BS + (end - lo + BS - 1) / BS;
    }
    // tile t: whether of cores, its first key, and its end (behind it: not there)
    __device__ __forceinline__ bool at(int t, int &y0, int &stop) const {
        const int tc = (cores + BS - 1) / BS;
        y0 = t < tc ? t * BS : lo + (t - tc) * BS;
        stop = t < tc ? cores : end;
        return t < tc;
    }
};

// What row i sees: the cores below `cores`, and the tokens from `start` to i.
struct Sight {
    int i, cores, start;
    __device__ __forceinline__ Sight() {}
    __device__ __forceinline__ Sight(const Plan &p, int row)
        : i(row), cores(p.cores_of(row)), start(p.start_of(row)) {}
    __device__ __forceinline__ bool sees(bool core, int key) const { return core ? key < cores : key >= start && key <= i; }
};

// GROUPS: groups of threads that take the key tiles in turn, each with its own running maximum, sum and output,
// which are joined at the end (few blocks: the chain of tiles is what takes the time).
template <int D, int ROWS, int GROUPS>
__global__ void __launch_bounds__(ROWS * 4 * GROUPS) attn_packed_kernel(const SimtArgs p) {
    constexpr int THREADS = ROWS * 4;
    const int group = threadIdx.x / THREADS;
    extern __shared__ float4 smem4[];
    float *const sQ = reinterpret_cast<float *>(smem4), *const sK = sQ + ROWS * PITCH<D> + group * (2 * TILE_FLOATS<D> + ROWS * SP),
                *const sV = sK + TILE_FLOATS<D>, *const sP = sV + TILE_FLOATS<D>;
    auto sync = [&]() {
        if constexpr (GROUPS == 1) __syncthreads();
        else ptx::named_bar_sync(1 + group, THREADS);
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    Block b;
    if (!query_block<ROWS>(p, b)) return;
    const Keys keys(p.plan, b, ROWS);
    const int ty = threadIdx.x % THREADS / 16, tx = threadIdx.x % 16;
    const float *kc = p.Kc + (static_cast<int64_t>(b.kv) * p.plan.G + b.c0) * D, *vc = p.Vc + (static_cast<int64_t>(b.kv) * p.plan.G + b.c0) * D;
    auto copy_k = [&](int t) {
        int y0, stop;
        const bool core = t < keys.tiles && keys.at(t, y0, stop);
        if (t >= keys.tiles) y0 = 0, stop = 0;
        if (core) copy_rows<D, THREADS>(sK, kc, D, y0, stop, t < keys.tiles ? BS : 0);
        else copy_rows<D, THREADS>(sK, p.K.at(b.kv, b.a), p.K.row, y0, stop, t < keys.tiles ? BS : 0);
    };
    auto copy_v = [&](int t) {
        int y0, stop;
        const bool core = t < keys.tiles && keys.at(t, y0, stop);
        if (t >= keys.tiles) y0 = 0, stop = 0;
        if (core) copy_rows<D, THREADS>(sV, vc, D, y0, stop, t < keys.tiles ? BS : 0);
        else copy_rows<D, THREADS>(sV, p.V.at(b.kv, b.a), p.V.row, y0, stop, t < keys.tiles ? BS : 0);
    };
    // every group copies the queries (the same values to the same place), so that it waits for its own copies alone
    copy_rows<D, THREADS>(sQ, p.Q.at(b.h, b.a), p.Q.row, b.i0, b.n, ROWS);
    copy_k(group);
    copy_v(group);
    float m[4], l[4], o[4][D / 16];
    Sight sight[4];
    const Sight top_row(p.plan, b.i0), last_row(p.plan, min(b.i0 + ROWS, b.n) - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sight[i] = Sight(p.plan, b.i0 + ty * 4 + i);
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    const float scale = p.tau * LOG2E;
    for (int t = group; t < keys.tiles; t += GROUPS) {
        int y0, stop;
        const bool core = keys.at(t, y0, stop);
        const int here = min(stop - y0, BS);
        copies_wait<1>();  // all but the values
        sync();
        float s[4][4];
        scores_of<D>(sQ, sK, ty, here, s);
        sync();
        copy_k(t + GROUPS);
        // whether every row sees every key of the tile
        const bool whole = y0 + BS <= stop && top_row.sees(core, y0) && top_row.sees(core, y0 + BS - 1) && last_row.sees(core, y0);
        unsigned seen = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = y0 + tx + 16 * j;
                const bool in = whole || (key < stop && sight[i].sees(core, key));
                seen |= in ? 1u << (4 * i + j) : 0u;
                s[i][j] = in ? s[i][j] * scale : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
            const float mn = fmaxf(m[i], top), ref = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - ref);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - ref);
                if (!whole && !(seen & (1u << (4 * i + j)))) s[i][j] = MASKED;
                sum += s[i][j];
                sP[(ty * 4 + i) * SP + tx + 16 * j] = s[i][j];
            }
            l[i] = l[i] * f + sum;  // of this thread's columns
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= f;
        }
        copies_wait<1>();  // all but the next keys
        sync();
        if (whole) add_rows<D, false>(sP, sV, ty, BS, o);
        else add_rows<D, true>(sP, sV, ty, here, o);
        sync();
        copy_v(t + GROUPS);
    }
    if constexpr (GROUPS > 1) {
        // group 0 joins: the others leave (m, l, o) where their keys were, a thread's values together
        copies_wait<0>();
        float *const mine = sK + (threadIdx.x % THREADS) * (8 + D / 4 + 1);
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mine[i] = m[i], mine[4 + i] = l[i];
#pragma unroll
                for (int c = 0; c < D / 16; ++c) mine[8 + i * (D / 16) + c] = o[i][c];
            }
        }
        __syncthreads();
        if (group > 0) return;
        for (int k = 1; k < GROUPS; ++k) {
            const float *const other = mine + k * (2 * TILE_FLOATS<D> + ROWS * SP);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mn = fmaxf(m[i], other[i]), ref = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[i] - ref), g = exp2f(other[i] - ref);
                m[i] = mn;
                l[i] = l[i] * f + other[4 + i] * g;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) o[i][c] = o[i][c] * f + other[8 + i * (D / 16) + c] * g;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = b.i0 + ty * 4 + i;
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(kFull, l[i], x);
        if (row >= b.n) continue;
        const float inv = 1.f / l[i];
        float *out = p.out.at(b.h, b.a + row);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            store4(out + tx * 4 + 64 * c, o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv);
        if (tx == 0) p.LSE[static_cast<int64_t>(b.h) * p.plan.T + b.a + row] = (m[i] + log2f(l[i])) * LN2;
    }
}

// dQ of ROWS query rows: dQ = tau sum dS k (+ the pooling's share of a group-last row).
template <int D, int ROWS, int GROUPS>
__global__ void __launch_bounds__(ROWS * 4 * GROUPS) packed_dq_kernel(const SimtArgs p) {
    constexpr int THREADS = ROWS * 4;
    const int group = threadIdx.x / THREADS;
    auto sync = [&]() {
        if constexpr (GROUPS == 1) __syncthreads();
        else ptx::named_bar_sync(1 + group, THREADS);
    };
    extern __shared__ float4 smem4[];
    float *const sQ = reinterpret_cast<float *>(smem4), *const sO = sQ + ROWS * PITCH<D>,
                *const sK = sO + ROWS * PITCH<D> + group * (2 * TILE_FLOATS<D> + ROWS * SP),
                *const sV = sK + TILE_FLOATS<D>, *const sP = sV + TILE_FLOATS<D>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    Block b;
    if (!query_block<ROWS>(p, b)) return;
    const Keys keys(p.plan, b, ROWS);
    const int ty = threadIdx.x % THREADS / 16, tx = threadIdx.x % 16;
    const int64_t core0 = (static_cast<int64_t>(b.kv) * p.plan.G + b.c0) * D;
    auto copy_keys = [&](float *dst, const float *cores, const Rows<const float> &raw, int t) {
        int y0 = 0, stop = 0;
        const bool core = t < keys.tiles && keys.at(t, y0, stop);
        if (core) copy_rows<D, THREADS>(dst, cores + core0, D, y0, stop, BS);
        else copy_rows<D, THREADS>(dst, raw.at(b.kv, b.a), raw.row, y0, stop, t < keys.tiles ? BS : 0);
    };
    copy_rows<D, THREADS>(sQ, p.Q.at(b.h, b.a), p.Q.row, b.i0, b.n, ROWS);
    copy_rows<D, THREADS>(sO, p.dO.at(b.h, b.a), p.dO.row, b.i0, b.n, ROWS);
    copy_keys(sV, p.Vc, p.V, group);
    copy_keys(sK, p.Kc, p.K, group);
    float lse[4], d[4], dq[4][D / 16];
    Sight sight[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = b.i0 + ty * 4 + i;
        sight[i] = Sight(p.plan, row);
        const int64_t at = static_cast<int64_t>(b.h) * p.plan.T + b.a + row;
        lse[i] = row < b.n ? p.LSE[at] * LOG2E : 0.f;
        d[i] = row < b.n ? p.w.D[at] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dq[i][c] = 0.f;
    }
    const float scale = p.tau * LOG2E;
    for (int t = group; t < keys.tiles; t += GROUPS) {
        int y0, stop;
        const bool core = keys.at(t, y0, stop);
        const int here = min(stop - y0, BS);
        copies_wait<1>();  // all but the keys
        sync();
        float s[4][4], g[4][4];
        scores_of<D>(sO, sV, ty, here, g);
        sync();
        copy_keys(sV, p.Vc, p.V, t + GROUPS);
        copies_wait<1>();  // all but the next values
        sync();
        scores_of<D>(sQ, sK, ty, here, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = b.i0 + ty * 4 + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = y0 + tx + 16 * j;
                const bool seen = row < b.n && key < stop && sight[i].sees(core, key);
                sP[(ty * 4 + i) * SP + tx + 16 * j] = seen ? exp2f(fmaf(s[i][j], scale, -lse[i])) * (g[i][j] - d[i]) : 0.f;
            }
        }
        sync();
        add_rows<D, false>(sP, sK, ty, here, dq);
        sync();
        copy_keys(sK, p.Kc, p.K, t + GROUPS);
    }
    if constexpr (GROUPS > 1) {
        copies_wait<0>();
        float *const mine = sK + (threadIdx.x % THREADS) * (D / 4 + 1);
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < D / 16; ++c) mine[i * (D / 16) + c] = dq[i][c];
        }
        __syncthreads();
        if (group > 0) return;
        for (int k = 1; k < GROUPS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < D / 16; ++c) dq[i][c] += mine[k * (2 * TILE_FLOATS<D> + ROWS * SP) + i * (D / 16) + c];
    }
    const int seen = p.cores ? seen_cores(b.n, p.plan.w, p.plan.g) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = b.i0 + ty * 4 + i;
        if (row >= b.n) continue;
        float *out = p.out.at(b.h, b.a + row);
        const int j = row / p.plan.g;
        const bool last = j < seen && row - j * p.plan.g == p.plan.g - 1;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const int col = tx * 4 + 64 * c;
            float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
            if (last) add = *reinterpret_cast<const float4 *>(p.w.dqs + core0 + static_cast<int64_t>(j) * D + col);
            store4(out + col, fmaf(dq[i][4 * c], p.tau, add.x), fmaf(dq[i][4 * c + 1], p.tau, add.y),
                   fmaf(dq[i][4 * c + 2], p.tau, add.z), fmaf(dq[i][4 * c + 3], p.tau, add.w));
        }
    }
}

// dK and dV of 64 keys of one KV head, raw tokens or cores, over the rows of its query heads that see any.
template <int D, bool CORE>
__global__ void __launch_bounds__(SIMT_THREADS) packed_dkv_kernel(const SimtArgs p) {
    extern __shared__ float4 smem4[];
    float *const sK = reinterpret_cast<float *>(smem4), *const sV = sK + TILE_FLOATS<D>, *const sQ = sV + TILE_FLOATS<D>,
                *const sO = sQ + TILE_FLOATS<D>, *const sP = sO + TILE_FLOATS<D>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t item = blockIdx.x / p.Hkv;
    const int3 counts = plan_counts(p.plan);
    if (item >= 2ll * (CORE ? counts.z : counts.y)) return;
    const int4 e = (CORE ? p.plan.cores : p.plan.tiles)[item / 2];
    const int a = e.x, n = e.y, kv = blockIdx.x % p.Hkv, r = p.Hq / p.Hkv;
    const Plan &pl = p.plan;
    const int nk = CORE ? seen_cores(n, pl.w, pl.g) : n;  // keys of this kind
    const int tile = (nk + PACK_TILE - 1) / PACK_TILE - 1 - e.z;
    const int y0 = tile * PACK_TILE + static_cast<int>(item % 2) * BS;
    if (y0 >= nk) return;
    const int y1 = min(y0 + BS, nk) - 1;
    // the rows [r0, r1] that see a key of the block
    int64_t r0, r1;
    if (CORE) {
        r0 = static_cast<int64_t>(y0 + 1) * pl.g + pl.w - 1;
        r1 = n - 1;
    } else {
        r0 = y0;
        r1 = pl.window_mode ? static_cast<int64_t>(y1 / pl.g + 1) * pl.g + pl.w - 2 : static_cast<int64_t>(y1) + pl.w - 1;
        if (r1 > n - 1) r1 = n - 1;
    }
    int q0 = static_cast<int>(r0) / BS, q1 = static_cast<int>(r1) / BS + 1;
    if (CORE && gridDim.y > 1) {
        const int per = (q1 - q0 + gridDim.y - 1) / gridDim.y;
        q0 += per * blockIdx.y;
        q1 = min(q1, q0 + per);
    }
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int64_t core0 = (static_cast<int64_t>(kv) * pl.G + e.w) * D;
    copy_rows<D, SIMT_THREADS>(sK, CORE ? p.Kc + core0 : p.K.at(kv, a), CORE ? D : p.K.row, y0, nk, BS);
    copy_rows<D, SIMT_THREADS>(sV, CORE ? p.Vc + core0 : p.V.at(kv, a), CORE ? D : p.V.row, y0, nk, BS);
    // the query tiles of all heads, one after the other
    const int per_head = max(q1 - q0, 0), steps = per_head * r;
    auto copy_q = [&](float *dst, const Rows<const float> &src, int x) {
        const bool in = x < steps;
        const int h = kv * r + (in ? x / per_head : 0), i0 = in ? (q0 + x % per_head) * BS : 0;
        copy_rows<D, SIMT_THREADS>(dst, src.at(h, a), src.row, i0, n, in ? BS : 0);
    };
    copy_q(sO, p.dO, 0);
    copy_q(sQ, p.Q, 0);
    float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
    const float scale = p.tau * LOG2E;
    for (int x = 0; x < steps; ++x) {
        const int h = kv * r + x / per_head, i0 = (q0 + x % per_head) * BS;
        float lse[4], d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i0 + ty * 4 + i;
            const int64_t at = static_cast<int64_t>(h) * pl.T + a + row;
            lse[i] = row < n ? p.LSE[at] * LOG2E : 0.f;
            d[i] = row < n ? p.w.D[at] : 0.f;
        }
        copies_wait<1>();  // all but the queries
        __syncthreads();
        float s[4][4], g[4][4];
        scores<D>(sO, sV, ty, g);
        copies_wait<0>();
        __syncthreads();
        scores<D>(sQ, sK, ty, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i0 + ty * 4 + i;
            const Sight sight(pl, row);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = y0 + tx + 16 * j;
                const bool seen = row < n && key < nk && sight.sees(CORE, key);
                s[i][j] = seen ? exp2f(fmaf(s[i][j], scale, -lse[i])) : 0.f;
                g[i][j] = seen ? s[i][j] * (g[i][j] - d[i]) : 0.f;
                sP[(ty * 4 + i) * SP + tx + 16 * j] = s[i][j];
            }
        }
        __syncthreads();
        add_columns<D>(sP, sO, dv);
        __syncthreads();
        copy_q(sO, p.dO, x + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sP[(ty * 4 + i) * SP + tx + 16 * j] = g[i][j];
        __syncthreads();
        add_columns<D>(sP, sQ, dk);
        __syncthreads();
        copy_q(sQ, p.Q, x + 1);
    }
    copies_wait<0>();  // without query rows, keys and values are still under way
    const int seen = !CORE && p.cores ? seen_cores(n, pl.w, pl.g) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = y0 + ty * 4 + i;
        if (key >= nk) continue;
        if (CORE) {
            const int64_t at = blockIdx.y * static_cast<int64_t>(p.Hkv) * pl.G * D + core0 + static_cast<int64_t>(key) * D;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int col = tx * 4 + 64 * c;
                store4(p.w.dKc + at + col, dk[i][4 * c] * p.tau, dk[i][4 * c + 1] * p.tau, dk[i][4 * c + 2] * p.tau, dk[i][4 * c + 3] * p.tau);
                store4(p.w.dVc + at + col, dv[i][4 * c], dv[i][4 * c + 1], dv[i][4 * c + 2], dv[i][4 * c + 3]);
            }
            continue;
        }
        const int j = key / pl.g;
        const bool pooled = j < seen;
        const int64_t tok = static_cast<int64_t>(kv) * pl.T + a + key, cj = core0 + static_cast<int64_t>(j) * D;
        const float w = pooled ? p.w.a[tok] : 0.f, cds = pooled ? p.w.cds[tok] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const int col = tx * 4 + 64 * c;
            float4 xk = make_float4(0.f, 0.f, 0.f, 0.f), xv = xk, xq = xk;
            if (pooled) {
                xk = *reinterpret_cast<const float4 *>(p.w.dKc + cj + col);
                xv = *reinterpret_cast<const float4 *>(p.w.dVc + cj + col);
                xq = *reinterpret_cast<const float4 *>(p.w.qsum + cj + col);
            }
            store4(p.dK.at(kv, a + key) + col, fmaf(cds, xq.x, fmaf(w, xk.x, dk[i][4 * c] * p.tau)),
                   fmaf(cds, xq.y, fmaf(w, xk.y, dk[i][4 * c + 1] * p.tau)), fmaf(cds, xq.z, fmaf(w, xk.z, dk[i][4 * c + 2] * p.tau)),
                   fmaf(cds, xq.w, fmaf(w, xk.w, dk[i][4 * c + 3] * p.tau)));
            store4(p.dV.at(kv, a + key) + col, fmaf(w, xv.x, dv[i][4 * c]), fmaf(w, xv.y, dv[i][4 * c + 1]),
                   fmaf(w, xv.z, dv[i][4 * c + 2]), fmaf(w, xv.w, dv[i][4 * c + 3]));
        }
    }
}

template <typename K>
cudaError_t start(K kernel, int64_t blocks, int splits, int threads, int floats, cudaStream_t stream, const SimtArgs &a) {
    if (blocks > 0x7fffffff) return cudaErrorNotSupported;
    const int smem = floats * 4;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return start_dependent(kernel, dim3(static_cast<unsigned>(blocks), splits), threads, smem, stream, a);
}

template <int D>
cudaError_t launch(const PackedArgs &p, const PackedBwdSpace *w, int part, cudaStream_t stream) {
    SimtArgs a = {};
    a.Q = rows_of<const float>(p.Q);
    a.K = rows_of<const float>(p.K);
    a.V = rows_of<const float>(p.V);
    a.Kc = static_cast<const float *>(p.Kc);
    a.Vc = static_cast<const float *>(p.Vc);
    a.LSE = p.LSE;
    a.plan = p.plan;
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.cores = p.Kc != nullptr;
    a.tau = p.scale;
    constexpr int F = TILE_FLOATS<D>, S = BS * SP;
    // Few blocks: of 32 query rows, in two groups.  fp32, us, 64 rows against 32 in two groups: 1500 tokens of 4 heads
    // 32 and 25, 1024 of 8 heads 58 and 43, a training step of 2048 of 8 heads 846 and 702.
    const int64_t heads64 = static_cast<int64_t>(PACK_TILE / 64) * p.plan.max_tiles * p.Hq;
    const bool small = heads64 < SMALL_BLOCKS * device_sms();
    if (w == nullptr) {
        a.out = rows_of<float>(p.O);
        if (small) return start(attn_packed_kernel<D, 32, SMALL_GROUPS>, 2 * heads64, 1, 128 * SMALL_GROUPS, F / 2 + SMALL_GROUPS * (2 * F + S / 2), stream, a);
        return start(attn_packed_kernel<D, 64, 1>, heads64, 1, 256, 3 * F + S, stream, a);
    }
    a.w = *w;
    a.dO = rows_of<const float>(p.dO);
    a.out = rows_of<float>(p.dQ);
    a.dK = rows_of<float>(p.dK);
    a.dV = rows_of<float>(p.dV);
    if (part == 0) return start(packed_dkv_kernel<D, true>, 2ll * p.plan.max_cores * p.Hkv, w->splits, SIMT_THREADS, 4 * F + S, stream, a);
    if (part == 1) {
        if (small) return start(packed_dq_kernel<D, 32, SMALL_GROUPS>, 2 * heads64, 1, 128 * SMALL_GROUPS, F + SMALL_GROUPS * (2 * F + S / 2), stream, a);
        return start(packed_dq_kernel<D, 64, 1>, heads64, 1, 256, 4 * F + S, stream, a);
    }
    return start(packed_dkv_kernel<D, false>, 2ll * p.plan.max_tiles * p.Hkv, 1, SIMT_THREADS, 4 * F + S, stream, a);
}

}  // namespace

cudaError_t launch_attn_packed_f32(const PackedArgs &a, cudaStream_t stream) {
    return a.d == 128 ? launch<128>(a, nullptr, 0, stream) : launch<64>(a, nullptr, 0, stream);
}
cudaError_t launch_packed_bwd_f32(const PackedArgs &a, const PackedBwdSpace &w, int part, cudaStream_t stream) {
    return a.d == 128 ? launch<128>(a, &w, part, stream) : launch<64>(a, &w, part, stream);
}

}  // namespace cca
