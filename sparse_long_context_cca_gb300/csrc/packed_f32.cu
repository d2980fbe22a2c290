// Attention over packed sequences and its gradient in fp32 on CUDA cores (tf32 products would miss its
// tolerance).
//
// Tiles of 64 query rows by 64 keys, 256 threads.  A thread owns 4 x 4 scores, 16
// threads a row of them; operands lie in shared memory as fp32 rows padded by one 16-byte chunk, so
// that a product's four-column reads of eight different rows fall into different banks.  Per 16-byte
// read a thread does eight multiply-adds in the score products and 10.7 in the others.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "packed.cuh"

namespace cca {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int BS = 64;  // rows and keys of a tile
constexpr int SIMT_THREADS = 256;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <int D>
constexpr int PITCH = D + 4;
constexpr int SP = BS + 4;  // pitch of the score tile
template <int D>
constexpr int TILE_FLOATS = BS * PITCH<D>;

// rows [y0, y0 + 64) of src, those below `end`; zeros behind
template <int D>
__device__ __forceinline__ void load_rows(float *dst, const float *src, int64_t row_stride, int y0, int end) {
    constexpr int LPR = D / 4, STEP = SIMT_THREADS / LPR;
#pragma unroll
    for (int r = 0; r < BS; r += STEP) {
        const int row = r + threadIdx.x / LPR, c = threadIdx.x % LPR * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (y0 + row < end) v = *reinterpret_cast<const float4 *>(src + (y0 + row) * row_stride + c);
        *reinterpret_cast<float4 *>(dst + row * PITCH<D> + c) = v;
    }
}

// s[i][j] = a_(4 ty + i) . b_(tx + 16 j)
template <int D>
__device__ __forceinline__ void scores(const float *a, const float *b, float (&s)[4][4]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = *reinterpret_cast<const float4 *>(a + (ty * 4 + i) * PITCH<D> + k);
            y[i] = *reinterpret_cast<const float4 *>(b + (tx + 16 * i) * PITCH<D> + k);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, s[i][j]))));
    }
}

// acc[i][..] += sum_k p[4 ty + i][k] b_k over the columns 4 tx + 64 c.  GUARD: keys of weight zero take no part.
template <int D, bool GUARD>
__device__ __forceinline__ void add_rows(const float *p, const float *b, float (&acc)[4][D / 16]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 2
    for (int k = 0; k < BS; k += 4) {
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
                    if (GUARD && x == 0.f) continue;
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

// 64 query rows of one head.
struct Block {
    int a, n, i0, c0;  // first row of the sequence, its length, the block's first row in it, its first core row
    int h, kv;
};
__device__ __forceinline__ bool query_block(const SimtArgs &p, Block &b) {
    const int64_t item = blockIdx.x / p.Hq;
    if (item >= 2ll * plan_counts(p.plan).y) return false;
    const int4 e = p.plan.tiles[item / 2];
    b.a = e.x, b.n = e.y, b.c0 = e.w;
    b.i0 = e.z * PACK_TILE + (1 - static_cast<int>(item % 2)) * BS;
    b.h = blockIdx.x % p.Hq;
    b.kv = b.h / (p.Hq / p.Hkv);
    return b.i0 < b.n;
}

// The key tiles that 64 query rows see: cores, then the band from the first row's window on.
struct Keys {
    int cores, lo, tiles, end;
    __device__ __forceinline__ Keys(const Plan &p, const Block &b) {
        const int last = min(b.i0 + BS, b.n) - 1;
        cores = visible_cores(last, p.w, p.g);
        lo = window_start(b.i0, p.w, p.g, p.window_mode);
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

__device__ __forceinline__ bool sees(const Plan &p, int i, bool core, int key) {
    return core ? key < visible_cores(i, p.w, p.g) : key >= window_start(i, p.w, p.g, p.window_mode) && key <= i;
}

template <int D>
__global__ void __launch_bounds__(SIMT_THREADS) attn_packed_kernel(const SimtArgs p) {
    extern __shared__ float4 smem4[];
    float *const sQ = reinterpret_cast<float *>(smem4), *const sK = sQ + TILE_FLOATS<D>, *const sP = sK + TILE_FLOATS<D>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    Block b;
    if (!query_block(p, b)) return;
    const Keys keys(p.plan, b);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    load_rows<D>(sQ, p.Q.at(b.h, b.a), p.Q.row, b.i0, b.n);
    const float *kc = p.Kc + (static_cast<int64_t>(b.kv) * p.plan.G + b.c0) * D, *vc = p.Vc + (static_cast<int64_t>(b.kv) * p.plan.G + b.c0) * D;
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    const float scale = p.tau * LOG2E;
    for (int t = 0; t < keys.tiles; ++t) {
        int y0, stop;
        const bool core = keys.at(t, y0, stop);
        __syncthreads();
        if (core) load_rows<D>(sK, kc, D, y0, stop);
        else load_rows<D>(sK, p.K.at(b.kv, b.a), p.K.row, y0, stop);
        __syncthreads();
        float s[4][4];
        scores<D>(sQ, sK, s);
        // whether every row sees every key of the tile
        const bool whole = y0 + BS <= stop && sees(p.plan, b.i0, core, y0) && sees(p.plan, b.i0, core, y0 + BS - 1) &&
                           sees(p.plan, min(b.i0 + BS, b.n) - 1, core, y0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = b.i0 + ty * 4 + i;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = y0 + tx + 16 * j;
                s[i][j] = whole || (key < stop && sees(p.plan, row, core, key)) ? s[i][j] * scale : -INFINITY;
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
                sum += s[i][j];
                sP[(ty * 4 + i) * SP + tx + 16 * j] = s[i][j];
            }
            l[i] = l[i] * f + sum;  // of this thread's columns
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= f;
        }
        __syncthreads();
        if (core) load_rows<D>(sK, vc, D, y0, stop);
        else load_rows<D>(sK, p.V.at(b.kv, b.a), p.V.row, y0, stop);
        __syncthreads();
        if (whole) add_rows<D, false>(sP, sK, o);
        else add_rows<D, true>(sP, sK, o);
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

// dQ of 64 query rows: dQ = tau sum dS k (+ the pooling's share of a group-last row).
template <int D>
__global__ void __launch_bounds__(SIMT_THREADS) packed_dq_kernel(const SimtArgs p) {
    extern __shared__ float4 smem4[];
    float *const sQ = reinterpret_cast<float *>(smem4), *const sO = sQ + TILE_FLOATS<D>, *const sK = sO + TILE_FLOATS<D>,
                *const sV = sK + TILE_FLOATS<D>, *const sP = sV + TILE_FLOATS<D>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    Block b;
    if (!query_block(p, b)) return;
    const Keys keys(p.plan, b);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    load_rows<D>(sQ, p.Q.at(b.h, b.a), p.Q.row, b.i0, b.n);
    load_rows<D>(sO, p.dO.at(b.h, b.a), p.dO.row, b.i0, b.n);
    const int64_t core0 = (static_cast<int64_t>(b.kv) * p.plan.G + b.c0) * D;
    float lse[4], d[4], dq[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = b.i0 + ty * 4 + i;
        const int64_t at = static_cast<int64_t>(b.h) * p.plan.T + b.a + row;
        lse[i] = row < b.n ? p.LSE[at] * LOG2E : 0.f;
        d[i] = row < b.n ? p.w.D[at] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dq[i][c] = 0.f;
    }
    const float scale = p.tau * LOG2E;
    for (int t = 0; t < keys.tiles; ++t) {
        int y0, stop;
        const bool core = keys.at(t, y0, stop);
        __syncthreads();
        if (core) {
            load_rows<D>(sK, p.Kc + core0, D, y0, stop);
            load_rows<D>(sV, p.Vc + core0, D, y0, stop);
        } else {
            load_rows<D>(sK, p.K.at(b.kv, b.a), p.K.row, y0, stop);
            load_rows<D>(sV, p.V.at(b.kv, b.a), p.V.row, y0, stop);
        }
        __syncthreads();
        float s[4][4], g[4][4];
        scores<D>(sQ, sK, s);
        scores<D>(sO, sV, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = b.i0 + ty * 4 + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = y0 + tx + 16 * j;
                const bool seen = row < b.n && key < stop && sees(p.plan, row, core, key);
                sP[(ty * 4 + i) * SP + tx + 16 * j] = seen ? exp2f(fmaf(s[i][j], scale, -lse[i])) * (g[i][j] - d[i]) : 0.f;
            }
        }
        __syncthreads();
        add_rows<D, false>(sP, sK, dq);
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
    if (CORE) {
        load_rows<D>(sK, p.Kc + core0, D, y0, nk);
        load_rows<D>(sV, p.Vc + core0, D, y0, nk);
    } else {
        load_rows<D>(sK, p.K.at(kv, a), p.K.row, y0, nk);
        load_rows<D>(sV, p.V.at(kv, a), p.V.row, y0, nk);
    }
    float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
    const float scale = p.tau * LOG2E;
    for (int h = kv * r; h < (kv + 1) * r; ++h) {
        for (int q = q0; q < q1; ++q) {
            const int i0 = q * BS;
            __syncthreads();
            load_rows<D>(sQ, p.Q.at(h, a), p.Q.row, i0, n);
            load_rows<D>(sO, p.dO.at(h, a), p.dO.row, i0, n);
            __syncthreads();
            float s[4][4], g[4][4];
            scores<D>(sQ, sK, s);
            scores<D>(sO, sV, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i0 + ty * 4 + i;
                const int64_t at = static_cast<int64_t>(h) * pl.T + a + row;
                const float lse = row < n ? p.LSE[at] * LOG2E : 0.f, d = row < n ? p.w.D[at] : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = y0 + tx + 16 * j;
                    const bool seen = row < n && key < nk && sees(pl, row, CORE, key);
                    s[i][j] = seen ? exp2f(fmaf(s[i][j], scale, -lse)) : 0.f;
                    g[i][j] = seen ? s[i][j] * (g[i][j] - d) : 0.f;
                    sP[(ty * 4 + i) * SP + tx + 16 * j] = s[i][j];
                }
            }
            __syncthreads();
            add_columns<D>(sP, sO, dv);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sP[(ty * 4 + i) * SP + tx + 16 * j] = g[i][j];
            __syncthreads();
            add_columns<D>(sP, sQ, dk);
        }
    }
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
cudaError_t start(K kernel, int64_t blocks, int splits, int floats, cudaStream_t stream, const SimtArgs &a) {
    if (blocks > 0x7fffffff) return cudaErrorNotSupported;
    const int smem = floats * 4;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return start_dependent(kernel, dim3(static_cast<unsigned>(blocks), splits), SIMT_THREADS, smem, stream, a);
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
    const int64_t rows = 2ll * p.plan.max_tiles;
    if (w == nullptr) {
        a.out = rows_of<float>(p.O);
        return start(attn_packed_kernel<D>, rows * p.Hq, 1, 2 * F + S, stream, a);
    }
    a.w = *w;
    a.dO = rows_of<const float>(p.dO);
    a.out = rows_of<float>(p.dQ);
    a.dK = rows_of<float>(p.dK);
    a.dV = rows_of<float>(p.dV);
    if (part == 0) return start(packed_dkv_kernel<D, true>, 2ll * p.plan.max_cores * p.Hkv, w->splits, 4 * F + S, stream, a);
    if (part == 1) return start(packed_dq_kernel<D>, rows * p.Hq, 1, 4 * F + S, stream, a);
    return start(packed_dkv_kernel<D, false>, rows * p.Hkv, 1, 4 * F + S, stream, a);
}

}  // namespace

cudaError_t launch_attn_packed_f32(const PackedArgs &a, cudaStream_t stream) {
    return a.d == 128 ? launch<128>(a, nullptr, 0, stream) : launch<64>(a, nullptr, 0, stream);
}
cudaError_t launch_packed_bwd_f32(const PackedArgs &a, const PackedBwdSpace &w, int part, cudaStream_t stream) {
    return a.d == 128 ? launch<128>(a, &w, part, stream) : launch<64>(a, &w, part, stream);
}

}  // namespace cca
