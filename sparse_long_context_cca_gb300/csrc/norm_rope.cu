// Norms of queries and keys for each head with their rotation in the same pass, its gradient, and
// the serving form that stores the new tokens of a step into paged caches.  With r the inverse root
// mean square of a row x and w its weights,
//   y_a = f r (x_a w_a cos t - x_b w_b sin t),   y_b = f r (x_b w_b cos t + x_a w_a sin t),
// so a row is one sum of squares and, per element, its own value and its partner's with two
// coefficients that do not depend on the row's values: A = f w cos t and B = -/+ f w' sin t, made
// once per position and used for every head.  Backward, with dn the rotation back of dy and
// t = dn w:  dx = r (t - x r^2 mean(t x)),  dw = sum dn x r; both sums of a row are formed in one go.
//
// Memory-bound: a row is read once and written once (backward: x and dy read, dx written).  Lanes
// hold a row in 16-byte chunks, 8 to 32 lanes to a row, so that sums are shuffles and loads whole
// sectors; a partner lies in another lane's chunk at the same place (rotation by halves, one shuffle
// per word), in the same chunk (interleaved pairs), or anywhere (a rotated part whose half is no
// whole number of chunks: through shared memory).
//
// What bounds them: 32 K tokens of 32 + 8 heads of 128 (bf16, 671 MB) take 130 us, 5.2 TB/s; half the issue slots
// go to unpacking, sums and packing (2.6 instructions a cycle), so waiting loads are not all of it: rings of
// cp.async in shared memory, two chunks a lane and paired arithmetic gave 130-141 us.  Four heads in flight a thread
// (two with weights for each head, whose coefficients take the registers) were best of 1 to 8.  The gradient of
// 2 x 4099 tokens of 16 + 4 heads: 37 us with dw's partial sums, and 4 to add them; forward there 30.  A step's 64
// tokens are stored in 4.5 us, 8 x 24 drafted ones in 8.1: the chain from the table to the page, not bytes.  fp32: 16 K tokens
// of 32 + 8 heads 113 us (671 MB, 5.9 TB/s).  That training size is 2.8 TB/s forward, not 5.2, by its launches (counted,
// not taken apart): 1539 blocks of seven heads in 2.5 waves, each with its angles and barriers for two batches of
// loads, and backward 513 row tiles on 304 blocks, two rounds for 1.7 of work.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/cca.h"
#include "internal.h"
#include "paged.cuh"
#include "rope.cuh"

namespace cca {
namespace {

constexpr int NORM_THREADS = 256;
constexpr int NORM_WARPS = NORM_THREADS / 32;
constexpr int NORM_BATCH = 4;      // heads whose loads are in flight together
constexpr int NORM_BWD_BATCH = 4;  // the same backward
constexpr int NORM_BWD_BLOCKS = 2; // resident
constexpr int HEAD_SUMS = 2;       // heads of a block whose dw it keeps apart
constexpr int DW_THREADS = 1024;

enum Turn { TURN_HALF, TURN_PAIRS, TURN_ANY };  // where a column's partner lies (above)

struct NormSrc {
    const char *x;
    char *y;
    const char *dy, *w;
    float *part;                  // backward: partial sums of dw, or nullptr
    int64_t xs[3], ys[3], gs[3];  // bytes, of (b, h, n)
    int64_t w_step;               // bytes from one head's weights to the next one's (0: shared)
    int H;
    int plain, paged;             // plain: copied only
};

struct NormArgs {
    NormSrc t[3];
    int n_t, heads;       // tensors, and their heads added up
    int heads_per_block;  // heads one thread walks through
    int rows_per_block;   // a power of two; the rest of a block's row slots take other heads
    int B, N, rot;
    int w_f32;
    float factor, eps, offset;
    const double *inv_freq;
    const int32_t *positions;
    int64_t pos_stride, start;
    // serving form
    const int32_t *lens, *parents, *counts;
    const int32_t *table;
    int n_pages, rows, cols;
    int32_t *status;
};

template <typename T>
struct Vec {
    static constexpr int E = 16 / sizeof(T);
    uint4 raw;
    __device__ __forceinline__ void floats(float (&f)[E]) const {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (E == 8) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                f[i] = __uint_as_float(w[i]);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[E]) {
        Chunk<T, E> c;
#pragma unroll
        for (int i = 0; i < E; ++i) from_f(f[i], c.e[i]);
        raw = c.raw;
    }
};

// The lane's row group: its chunk's columns and their partners'.
template <typename T, int D, int TURN>
struct Lane {
    static constexpr int E = Vec<T>::E;
    static constexpr int LPR = D / E;  // lanes of a row
    int lane, col, half, rot;
    unsigned mask;  // the row's lanes
    uint4 *sm;      // the warp's 32 chunks (TURN_ANY)

    __device__ __forceinline__ Lane(int rot_, uint4 *rows) : lane(threadIdx.x & 31), half(rot_ / 2), rot(rot_) {
        col = (lane % LPR) * E;
        mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1) << (lane / LPR * LPR);
        sm = TURN == TURN_ANY ? rows + (threadIdx.x & ~31) : nullptr;
    }
    __device__ __forceinline__ int pair(int e) const { return TURN == TURN_PAIRS ? (col + e) / 2 : col + e < half ? col + e : col + e - half; }
    __device__ __forceinline__ bool first(int e) const { return TURN == TURN_PAIRS ? (e & 1) == 0 : col + e < half; }
    __device__ __forceinline__ int partner(int e) const {
        if (col + e >= rot) return col + e;
        return TURN == TURN_PAIRS ? (col + e) ^ 1 : first(e) ? col + e + half : col + e - half;
    }
    __device__ __forceinline__ float sum(float v) const {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
        return v;
    }
    // the partners' values of this lane's elements
    __device__ __forceinline__ void partners(const Vec<T> &v, const float (&own)[E], float (&f)[E]) const {
        if constexpr (TURN == TURN_PAIRS) {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = own[e ^ 1];
        } else if constexpr (TURN == TURN_HALF) {
            const int src = col >= rot ? lane : col < half ? lane + half / E : lane - half / E;
            Vec<T> p;
            p.raw.x = __shfl_sync(mask, v.raw.x, src);
            p.raw.y = __shfl_sync(mask, v.raw.y, src);
            p.raw.z = __shfl_sync(mask, v.raw.z, src);
            p.raw.w = __shfl_sync(mask, v.raw.w, src);
            p.floats(f);
        } else {
            __syncwarp(mask);
            sm[lane] = v.raw;
            __syncwarp(mask);
            const T *row = reinterpret_cast<const T *>(sm + lane / LPR * LPR);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = to_f(row[partner(e)]);
        }
    }
    // offset + weight of this lane's columns (own) or of their partners
    __device__ __forceinline__ void weights(const NormArgs &a, const char *w, bool own, float (&f)[E]) const {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = own ? col + e : partner(e);
            f[e] = w == nullptr ? 1.f
                                : a.offset + (a.w_f32 ? reinterpret_cast<const float *>(w)[c]
                                                      : to_f(reinterpret_cast<const __nv_bfloat16 *>(w)[c]));
        }
    }
    // factor * cos and factor * sin of the columns' angles (1 and 0 behind the rotated part), from the row's
    // line of the block's table
    __device__ __forceinline__ void angles(const float2 *line, float (&c)[E], float (&s)[E]) const {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 v = col + e < rot ? line[pair(e)] : make_float2(1.f, 0.f);
            c[e] = v.x, s[e] = v.y;
        }
    }
};

__device__ __forceinline__ void load_freq(const NormArgs &a, uint64_t *freq) {
    for (int i = threadIdx.x; i < a.rot / 2; i += NORM_THREADS) {
        double f = a.inv_freq[i] * 0.15915494309189535;  // turns per position
        f -= floor(f);
        freq[i] = static_cast<uint64_t>(f * 18446744073709551616.0);
    }
}

// The angles of `rows` rows at positions pos[..], made by the whole block: table[row][pair].
template <int D>
__device__ __forceinline__ void make_angles(const NormArgs &a, const uint64_t *freq, const int64_t *pos, int rows, float2 *table) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < rows * (D / 2); i += NORM_THREADS) {
        const int row = i / (D / 2), pair = i % (D / 2);
        if (pair >= half) continue;
        float2 v;
        turn_cos_sin(static_cast<uint64_t>(pos[row]) * freq[pair], a.factor, v.x, v.y);
        table[i] = v;
    }
}

// PER_HEAD: a tensor has weights for each head, so they are no part of the coefficients.
// PAGED: the serving form, one block row per sequence.
template <typename T, int D, int TURN, bool PER_HEAD, bool PAGED>
__global__ void __launch_bounds__(NORM_THREADS, 4) norm_rope_kernel(const NormArgs a) {
    using L = Lane<T, D, TURN>;
    constexpr int E = L::E;
    constexpr int SLOTS = NORM_THREADS / L::LPR;
    constexpr int BATCH = PER_HEAD ? NORM_BATCH / 2 : NORM_BATCH;
    __shared__ uint64_t sm_freq[D / 2];
    __shared__ int64_t sm_pos[SLOTS];
    __shared__ float2 sm_angle[SLOTS * (D / 2)];
    __shared__ int16_t sm_parent[PAGED ? TREE_MAX_NODES : 1];
    __shared__ uint4 sm_rows[TURN == TURN_ANY ? NORM_THREADS : 1];
    const L ln(a.rot, sm_rows);
    const int slot_of_block = threadIdx.x / L::LPR;
    const int64_t total = PAGED ? a.N : static_cast<int64_t>(a.B) * a.N;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * a.rows_per_block + (slot_of_block & (a.rows_per_block - 1));
    const int sub = slot_of_block / a.rows_per_block, subs = SLOTS / a.rows_per_block;
    const int h0 = (blockIdx.y * subs + sub) * a.heads_per_block, h1 = min(h0 + a.heads_per_block, a.heads);
    const bool work = row < total && h0 < h1;
    const int b = PAGED ? static_cast<int>(blockIdx.z) : static_cast<int>(row / a.N);
    const int64_t n = PAGED ? row : row - static_cast<int64_t>(b) * a.N;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    int which = 0, first = 0;  // the tensor of the head walk, heads before it
    while (work && h0 - first >= a.t[which].H) first += a.t[which++].H;
    Vec<T> x[BATCH];
    auto load = [&](int h, int count) {
        const NormSrc &t = a.t[which];
        const char *p = t.x + b * t.xs[0] + (h - first) * t.xs[1] + n * t.xs[2] + ln.col * static_cast<int64_t>(sizeof(T));
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (k < count) x[k].raw = *reinterpret_cast<const uint4 *>(p + k * t.xs[1]);
    };
    auto batch_heads = [&](int h) { return min(min(BATCH, h1 - h), first + a.t[which].H - h); };
    if (work) load(h0, batch_heads(h0));
    int len = 0, count_b = 0;
    if constexpr (PAGED) {
        len = a.lens[b];
        count_b = a.counts != nullptr ? a.counts[b] : a.N;
        if (a.parents != nullptr)
            for (int i = threadIdx.x; i < a.N; i += NORM_THREADS) {
                const int p = a.parents[static_cast<int64_t>(b) * a.N + i];
                sm_parent[i] = static_cast<int16_t>(p >= -1 && p < i ? p : -2);
            }
    }
    load_freq(a, sm_freq);
    if (PAGED && a.parents != nullptr) __syncthreads();
    int64_t pos = 0, page = -1;
    int page_off = 0;
    bool real = row < total;
    if constexpr (PAGED) {
        if (len < 0) {
            report(a.status, CCA_ERR_INVALID_ARG);
            real = false;
            len = 0;
        }
        pos = static_cast<int64_t>(len) + n;
        if (n >= count_b) real = false;
        if (real) {
            const uint32_t slot = static_cast<uint32_t>(len) + static_cast<uint32_t>(n);  // below 2^32
            const uint32_t c = slot / static_cast<uint32_t>(a.rows);
            page = c < static_cast<uint32_t>(a.cols) ? a.table[static_cast<int64_t>(b) * a.cols + c] : -1;
            page_off = static_cast<int>(slot - c * a.rows);
        }
        if (a.parents != nullptr) {
            int depth = 0, k = row < total ? sm_parent[n] : -1;
            while (k >= 0) {  // parents are below their children, so this ends
                ++depth;
                k = sm_parent[k];
            }
            if (k != -1) real = false;
            pos = static_cast<int64_t>(len) + depth;
        }
        if (real && (page < 0 || page >= a.n_pages)) report(a.status, CCA_ERR_INVALID_ARG);
        if (!real || page >= a.n_pages) page = -1;
    } else if (row < total) {
        pos = a.positions != nullptr ? a.positions[b * a.pos_stride + n] : a.start + n;
    }
    if (sub == 0 && ln.col == 0) sm_pos[slot_of_block] = pos;
    __syncthreads();
    make_angles<D>(a, sm_freq, sm_pos, a.rows_per_block, sm_angle);
    __syncthreads();
    if (!work) return;  // whole row groups leave together
    const float2 *const line = sm_angle + (slot_of_block & (a.rows_per_block - 1)) * (D / 2);

    for (int h = h0; h < h1;) {
        // one tensor's heads
        const NormSrc &t = a.t[which];
        const int end = min(h1, first + t.H);
        float A[E], B[E];
        if (!t.plain) {
            ln.angles(line, A, B);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (ln.first(e)) B[e] = -B[e];
            if (!PER_HEAD) {
                float w[E];
                ln.weights(a, t.w, true, w);
#pragma unroll
                for (int e = 0; e < E; ++e) A[e] *= w[e];
                ln.weights(a, t.w, false, w);
#pragma unroll
                for (int e = 0; e < E; ++e) B[e] *= w[e];
            }
        }
        for (; h < end;) {
            const int count = batch_heads(h);
            if (h > h0) load(h, count);
            char *y;
            int64_t step;
            bool store = true;
            if (PAGED && t.paged) {
                step = static_cast<int64_t>(a.rows) * D * sizeof(T);
                y = t.y + ((page * t.H + (h - first)) * a.rows + page_off) * D * static_cast<int64_t>(sizeof(T));
                store = page >= 0;
            } else {
                step = t.ys[1];
                y = t.y + b * t.ys[0] + (h - first) * step + n * t.ys[2];
            }
            y += ln.col * static_cast<int64_t>(sizeof(T));
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (k >= count) continue;  // the same for all lanes of a row
                if (!t.plain) {
                    float f[E], p[E];
                    x[k].floats(f);
                    ln.partners(x[k], f, p);
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) ss = fmaf(f[e], f[e], ss);
                    const float r = rsqrtf(fmaf(ln.sum(ss), 1.f / D, a.eps));
                    if (PER_HEAD) {
                        float w[E], wp[E];
                        const char *wr = t.w != nullptr ? t.w + (h - first + k) * t.w_step : nullptr;
                        ln.weights(a, wr, true, w);
                        ln.weights(a, wr, false, wp);
#pragma unroll
                        for (int e = 0; e < E; ++e) f[e] *= w[e], p[e] *= wp[e];
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e) f[e] = r * fmaf(p[e], B[e], f[e] * A[e]);
                    x[k].set(f);
                }
                if (PAGED && !real) x[k].raw = make_uint4(0u, 0u, 0u, 0u);
                if (store) *reinterpret_cast<uint4 *>(y + k * step) = x[k].raw;
            }
            h += count;
        }
        if (h < h1) {
            first += t.H;
            ++which;
        }
    }
}

// A block walks over row tiles, tensor by tensor, so that a thread's share of dw stays in registers;
// the block's sums go to `part` ([blocks, D] for shared weights, [gridDim.x, H, D] for those of each
// head), and norm_dw_kernel adds them up in order.
template <typename T, int D, int TURN, bool PER_HEAD>
__global__ void __launch_bounds__(NORM_THREADS, NORM_BWD_BLOCKS) norm_rope_bwd_kernel(const NormArgs a) {
    using L = Lane<T, D, TURN>;
    constexpr int E = L::E;
    constexpr int SLOTS = NORM_THREADS / L::LPR;
    constexpr int NB = PER_HEAD ? HEAD_SUMS : NORM_BWD_BATCH;
    __shared__ uint64_t sm_freq[D / 2];
    __shared__ int64_t sm_pos[SLOTS];
    __shared__ float2 sm_angle[SLOTS * (D / 2)];
    __shared__ uint4 sm_rows[TURN == TURN_ANY ? NORM_THREADS : 1];
    __shared__ float sm_dw[NORM_WARPS][D];
    const L ln(a.rot, sm_rows);
    const int64_t total = static_cast<int64_t>(a.B) * a.N;
    const int64_t tiles = (total + SLOTS - 1) / SLOTS;
    const int h0 = blockIdx.y * a.heads_per_block, h1 = min(h0 + a.heads_per_block, a.heads);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    load_freq(a, sm_freq);
    int first = 0;
    for (int which = 0; which < a.n_t; first += a.t[which++].H) {
        const NormSrc &t = a.t[which];
        const int hs = max(h0, first), he = min(h1, first + t.H);
        if (hs >= he && (PER_HEAD || t.part == nullptr)) continue;  // the same for the whole block
        float dw[PER_HEAD ? NB : 1][E], w[E];
#pragma unroll
        for (int k = 0; k < (PER_HEAD ? NB : 1); ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) dw[k][e] = 0.f;
        if (!PER_HEAD) ln.weights(a, t.w, true, w);
        for (int64_t tile = blockIdx.x; hs < he && tile < tiles; tile += gridDim.x) {
            const int64_t row = tile * SLOTS + threadIdx.x / L::LPR;
            const int64_t b = row / a.N, n = row - b * a.N;
            if (ln.col == 0)
                sm_pos[threadIdx.x / L::LPR] = row >= total ? 0 : a.positions != nullptr ? a.positions[b * a.pos_stride + n] : a.start + n;
            __syncthreads();  // also: the tile before is done with its angles
            make_angles<D>(a, sm_freq, sm_pos, SLOTS, sm_angle);
            __syncthreads();
            if (row >= total) continue;  // whole row groups
            float C[E], S[E];
            ln.angles(sm_angle + threadIdx.x / L::LPR * (D / 2), C, S);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (!ln.first(e)) S[e] = -S[e];  // the rotation back
            const int64_t at = ln.col * static_cast<int64_t>(sizeof(T));
            const char *px = t.x + b * t.xs[0] + n * t.xs[2] + at, *pg = t.dy + b * t.gs[0] + n * t.gs[2] + at;
            char *py = t.y + b * t.ys[0] + n * t.ys[2] + at;
            for (int h = hs; h < he; h += NB) {
                Vec<T> x[NB], g[NB];
#pragma unroll
                for (int k = 0; k < NB; ++k)
                    if (h + k < he) {
                        x[k].raw = *reinterpret_cast<const uint4 *>(px + (h + k - first) * t.xs[1]);
                        g[k].raw = *reinterpret_cast<const uint4 *>(pg + (h + k - first) * t.gs[1]);
                    }
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    if (h + k >= he) continue;
                    float f[E], dn[E], p[E];
                    x[k].floats(f);
                    g[k].floats(dn);
                    ln.partners(g[k], dn, p);
                    if (PER_HEAD) ln.weights(a, t.w != nullptr ? t.w + (h + k - first) * t.w_step : nullptr, true, w);
                    float ss = 0.f, tx = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        dn[e] = fmaf(p[e], S[e], dn[e] * C[e]);
                        ss = fmaf(f[e], f[e], ss);
                        tx = fmaf(dn[e] * w[e], f[e], tx);
                    }
                    const float r = rsqrtf(fmaf(ln.sum(ss), 1.f / D, a.eps));
                    const float c = ln.sum(tx) * (1.f / D) * r * r;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float xr = f[e] * r;
                        dw[PER_HEAD ? k : 0][e] = fmaf(dn[e], xr, dw[PER_HEAD ? k : 0][e]);
                        f[e] = r * fmaf(dn[e], w[e], -f[e] * c);
                    }
                    x[k].set(f);
                    *reinterpret_cast<uint4 *>(py + (h + k - first) * t.ys[1]) = x[k].raw;
                }
            }
        }
        if (t.part == nullptr) continue;
#pragma unroll
        for (int k = 0; k < (PER_HEAD ? NB : 1); ++k) {
            if (PER_HEAD && hs + k >= he) continue;  // the same for the whole block
            __syncwarp();
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float v = dw[k][e];
#pragma unroll
                for (int o = L::LPR; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (ln.lane < L::LPR) sm_dw[threadIdx.x / 32][ln.col + e] = v;
            }
            __syncthreads();
            if (threadIdx.x < D) {
                float v = 0.f;
#pragma unroll
                for (int i = 0; i < NORM_WARPS; ++i) v += sm_dw[i][threadIdx.x];
                const int64_t at = PER_HEAD ? static_cast<int64_t>(blockIdx.x) * t.H + (hs + k - first)
                                            : static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
                t.part[at * D + threadIdx.x] = v;
            }
            __syncthreads();
        }
    }
}

struct DwArgs {
    const float *part[2];
    void *dw[2];
    int heads[2];  // rows of dw
    int parts[2];  // partial sums of a row, heads[i] rows apart
    int w_f32;
};

// 32 columns of dw of one head (or of all that share it): a block adds their partial sums, in a fixed order.
template <int D>
__global__ void __launch_bounds__(DW_THREADS) norm_dw_kernel(const DwArgs a) {
    constexpr int SLICES = DW_THREADS / 32;
    __shared__ float sm[SLICES][32];
    const int which = static_cast<int>(blockIdx.x) < a.heads[0] ? 0 : 1;
    const int head = blockIdx.x - (which ? a.heads[0] : 0);
    const float *part = which ? a.part[1] : a.part[0];
    const int heads = which ? a.heads[1] : a.heads[0], parts = which ? a.parts[1] : a.parts[0];
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32, col = blockIdx.y * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    float v = 0.f;
#pragma unroll 16
    for (int i = slice; i < parts; i += SLICES) v += part[(static_cast<int64_t>(i) * heads + head) * D + col];
    sm[slice][lane] = v;
    __syncthreads();
    if (slice != 0) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < SLICES; ++i) v += sm[i][lane];
    const int64_t at = static_cast<int64_t>(head) * D + col;
    void *dw = which ? a.dw[1] : a.dw[0];
    if (a.w_f32) static_cast<float *>(dw)[at] = v;
    else static_cast<__nv_bfloat16 *>(dw)[at] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------- launches

int turn_of(const cca_rope_params_t &p) {
    if (p.rot == 0 || p.layout == 1) return TURN_PAIRS;
    return p.rot / 2 % (p.dtype == CCA_BF16 ? 8 : 4) == 0 ? TURN_HALF : TURN_ANY;
}

template <typename T, int D, int TURN, bool PAGED>
cudaError_t launch_fwd(const NormArgs &a, bool per_head, dim3 grid, cudaStream_t stream) {
    if (per_head) return start_dependent(norm_rope_kernel<T, D, TURN, true, PAGED>, grid, NORM_THREADS, 0, stream, a);
    return start_dependent(norm_rope_kernel<T, D, TURN, false, PAGED>, grid, NORM_THREADS, 0, stream, a);
}

template <typename T, int D, bool PAGED>
cudaError_t launch_fwd_turn(NormArgs &a, int turn, bool per_head, cudaStream_t stream) {
    const int slots = NORM_THREADS / (D / Vec<T>::E);
    const int64_t total = PAGED ? a.N : static_cast<int64_t>(a.B) * a.N;
    a.rows_per_block = 1;
    while (a.rows_per_block < slots && a.rows_per_block < total) a.rows_per_block *= 2;
    const int64_t blocks = (total + a.rows_per_block - 1) / a.rows_per_block;
    if (blocks > 0x7fffffff) return cudaErrorNotSupported;
    const int sms = device_sms();
    if (sms < 1) return cudaErrorNoDevice;
    // Angles are shared by the heads of a group: as many heads per thread as still leave eight blocks
    // for every SM, but a batch of loads at least.
    const int subs = slots / a.rows_per_block;
    const int64_t all = blocks * (PAGED ? a.B : 1) * subs;
    const int most = (a.heads + NORM_BATCH - 1) / NORM_BATCH;
    int groups = static_cast<int>((8ll * sms * subs + all - 1) / all);
    if (groups > most) groups = most;
    a.heads_per_block = (a.heads + groups - 1) / groups;
    groups = (a.heads + a.heads_per_block * subs - 1) / (a.heads_per_block * subs);
    if (groups > 65535) return cudaErrorNotSupported;
    const dim3 grid(static_cast<unsigned>(blocks), groups, PAGED ? a.B : 1);
    switch (turn) {
        case TURN_HALF: return launch_fwd<T, D, TURN_HALF, PAGED>(a, per_head, grid, stream);
        case TURN_PAIRS: return launch_fwd<T, D, TURN_PAIRS, PAGED>(a, per_head, grid, stream);
        default: return launch_fwd<T, D, TURN_ANY, PAGED>(a, per_head, grid, stream);
    }
}

template <bool PAGED>
cudaError_t launch_norm(int dtype, int d, NormArgs &a, int turn, bool per_head, cudaStream_t stream) {
    if (dtype == CCA_BF16)
        return d == 128 ? launch_fwd_turn<__nv_bfloat16, 128, PAGED>(a, turn, per_head, stream)
                        : launch_fwd_turn<__nv_bfloat16, 64, PAGED>(a, turn, per_head, stream);
    return d == 128 ? launch_fwd_turn<float, 128, PAGED>(a, turn, per_head, stream)
                    : launch_fwd_turn<float, 64, PAGED>(a, turn, per_head, stream);
}

// The backward launch: blocks over the row tiles and over head groups, and the heads of a group.
struct BwdGrid {
    int x, y, heads_per_block;
};
BwdGrid bwd_grid(const cca_rope_params_t &p, int heads, bool per_head, int sms) {
    const int e = p.dtype == CCA_BF16 ? 8 : 4, slots = NORM_THREADS / (p.d / e);
    const int64_t tiles = (static_cast<int64_t>(p.B) * p.N + slots - 1) / slots;
    const int want = NORM_BWD_BLOCKS * sms;
    BwdGrid g;
    if (per_head) {
        // one batch of heads to a block, whose sums it keeps apart
        g.heads_per_block = HEAD_SUMS;
    } else {
        const int most = (heads + NORM_BWD_BATCH - 1) / NORM_BWD_BATCH;
        int64_t groups = (want + tiles - 1) / tiles;
        if (groups > most) groups = most;
        g.heads_per_block = static_cast<int>((heads + groups - 1) / groups);
    }
    g.y = (heads + g.heads_per_block - 1) / g.heads_per_block;
    const int64_t x = (want + g.y - 1) / g.y;
    g.x = static_cast<int>(x < tiles ? x : tiles);
    return g;
}

template <typename T, int D>
cudaError_t launch_bwd(const NormArgs &a, int turn, bool per_head, dim3 grid, cudaStream_t stream) {
    auto go = [&](auto kernel) { return start_dependent(kernel, grid, NORM_THREADS, 0, stream, a); };
    if (per_head) {
        switch (turn) {
            case TURN_HALF: return go(norm_rope_bwd_kernel<T, D, TURN_HALF, true>);
            case TURN_PAIRS: return go(norm_rope_bwd_kernel<T, D, TURN_PAIRS, true>);
            default: return go(norm_rope_bwd_kernel<T, D, TURN_ANY, true>);
        }
    }
    switch (turn) {
        case TURN_HALF: return go(norm_rope_bwd_kernel<T, D, TURN_HALF, false>);
        case TURN_PAIRS: return go(norm_rope_bwd_kernel<T, D, TURN_PAIRS, false>);
        default: return go(norm_rope_bwd_kernel<T, D, TURN_ANY, false>);
    }
}

// ---------------------------------------------------------------- arguments

int check_norm(const cca_norm_params_t *p) {
    int st;
    if (p == nullptr) return CCA_ERR_INVALID_ARG;
    if (!params_ok(&p->rope, st)) return st;
    if (p->rope.inverse != 0 || !(p->eps >= 0.f) || isinf(p->eps) || !(p->offset == p->offset)) return CCA_ERR_INVALID_ARG;
    if (p->weight_dtype != CCA_BF16 && p->weight_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    return CCA_OK;
}

bool weight_ok(const cca_norm_tensor_t &t, const cca_norm_params_t &p) {
    const uintptr_t align = p.weight_dtype == CCA_BF16 ? 1u : 3u;
    if (((reinterpret_cast<uintptr_t>(t.weight) | reinterpret_cast<uintptr_t>(t.dweight)) & align) != 0) return false;
    if (t.weight == nullptr) return t.dweight == nullptr;
    return t.weight_heads == 1 || t.weight_heads == t.H;
}

bool has_head_weights(const cca_norm_tensor_t &t) { return t.weight != nullptr && t.weight_heads > 1; }

Span weight_span(const void *w, const cca_norm_tensor_t &t, const cca_norm_params_t &p) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(w);
    return {b, b + (w == nullptr ? 0 : static_cast<uintptr_t>(t.weight_heads) * p.rope.d * (p.weight_dtype == CCA_BF16 ? 2 : 4))};
}

NormArgs norm_args(const cca_norm_params_t &p) {
    NormArgs a = {};
    a.B = p.rope.B;
    a.N = p.rope.N;
    a.rot = p.rope.rot;
    a.factor = p.rope.factor;
    a.eps = p.eps;
    a.offset = p.offset;
    a.w_f32 = p.weight_dtype == CCA_F32;
    a.inv_freq = p.rope.inv_freq;
    a.positions = p.rope.positions;
    a.pos_stride = p.rope.pos_stride;
    a.start = p.rope.start;
    return a;
}

NormSrc norm_src(const cca_norm_tensor_t &t, const cca_norm_params_t &p) {
    const int es = p.rope.dtype == CCA_BF16 ? 2 : 4, ws = p.weight_dtype == CCA_BF16 ? 2 : 4;
    NormSrc r = {};
    r.x = static_cast<const char *>(t.x);
    r.y = static_cast<char *>(t.y);
    r.dy = static_cast<const char *>(t.dy);
    r.w = static_cast<const char *>(t.weight);
    for (int i = 0; i < 3; ++i) {
        r.xs[i] = t.x_stride[i] * es;
        r.ys[i] = t.y_stride[i] * es;
        r.gs[i] = t.dy_stride[i] * es;
    }
    r.w_step = has_head_weights(t) ? static_cast<int64_t>(p.rope.d) * ws : 0;
    r.H = t.H;
    return r;
}

cca_rope_tensor_t rope_view(const cca_norm_tensor_t &t) {
    cca_rope_tensor_t r = {t.x, t.y, t.H, {}, {}};
    for (int i = 0; i < 3; ++i) {
        r.x_stride[i] = t.x_stride[i];
        r.y_stride[i] = t.y_stride[i];
    }
    return r;
}

uint64_t bwd_floats(const cca_norm_tensor_t *t, int n, const cca_norm_params_t &p, const BwdGrid &g, bool per_head,
                    uint64_t (&at)[2]) {
    uint64_t floats = 0;
    for (int i = 0; i < n; ++i) {
        at[i] = floats;
        if (t[i].dweight != nullptr) floats += static_cast<uint64_t>(g.x) * (per_head ? t[i].H : g.y) * p.rope.d;
    }
    return floats;
}

int check_bwd(const cca_norm_tensor_t *t, int n, const cca_norm_params_t *p) {
    int st = check_norm(p);
    if (st != CCA_OK) return st;
    if (t == nullptr || n < 1 || n > 2) return CCA_ERR_INVALID_ARG;
    const int es = p->rope.dtype == CCA_BF16 ? 2 : 4;
    Span in[6], out[4];
    int n_in = 0, n_out = 0;
    for (int i = 0; i < n; ++i) {
        if (t[i].H < 1 || t[i].H > (1 << 20) || !weight_ok(t[i], *p)) return CCA_ERR_INVALID_ARG;
        const int64_t size[3] = {p->rope.B, t[i].H, p->rope.N};
        if (!span_of(t[i].x, t[i].x_stride, size, p->rope.d, es, in[n_in++]) ||
            !span_of(t[i].dy, t[i].dy_stride, size, p->rope.d, es, in[n_in++]) ||
            !span_of(t[i].y, t[i].y_stride, size, p->rope.d, es, out[n_out++]) || !rows_apart(t[i].y_stride, size, p->rope.d))
            return CCA_ERR_INVALID_ARG;
        in[n_in++] = weight_span(t[i].weight, t[i], *p);
        out[n_out++] = weight_span(t[i].dweight, t[i], *p);
    }
    for (int i = 0; i < n_out; ++i) {
        for (int k = 0; k < n_in; ++k)
            if (spans_meet(out[i], in[k])) return CCA_ERR_INVALID_ARG;
        for (int k = i + 1; k < n_out; ++k)
            if (spans_meet(out[i], out[k])) return CCA_ERR_INVALID_ARG;
    }
    return CCA_OK;
}

}  // namespace
}  // namespace cca

extern "C" {

int cca_norm_rope(const cca_norm_tensor_t *tensors, int n_tensors, const cca_norm_params_t *params, void *stream) {
    using namespace cca;
    int st = check_norm(params);
    if (st != CCA_OK) return st;
    if (tensors == nullptr || n_tensors < 1 || n_tensors > 2) return CCA_ERR_INVALID_ARG;
    cca_rope_tensor_t view[2];
    NormArgs a = norm_args(*params);
    a.n_t = n_tensors;
    bool per_head = false;
    for (int i = 0; i < n_tensors; ++i) {
        view[i] = rope_view(tensors[i]);
        if (tensors[i].H < 1 || tensors[i].H > (1 << 20) || !weight_ok(tensors[i], *params)) return CCA_ERR_INVALID_ARG;
        a.t[i] = norm_src(tensors[i], *params);
        a.heads += tensors[i].H;
        per_head = per_head || has_head_weights(tensors[i]);
    }
    if ((st = check_rope_tensors(view, n_tensors, params->rope)) != CCA_OK) return st;
    const int es = params->rope.dtype == CCA_BF16 ? 2 : 4;
    for (int i = 0; i < n_tensors; ++i) {
        Span y;
        const int64_t size[3] = {params->rope.B, tensors[i].H, params->rope.N};
        span_of(tensors[i].y, tensors[i].y_stride, size, params->rope.d, es, y);
        for (int k = 0; k < n_tensors; ++k)
            if (spans_meet(y, weight_span(tensors[k].weight, tensors[k], *params))) return CCA_ERR_INVALID_ARG;
    }
    if ((st = check_device()) != CCA_OK) return st;
    return from_cuda(launch_norm<false>(params->rope.dtype, params->rope.d, a, turn_of(params->rope), per_head,
                                        static_cast<cudaStream_t>(stream)));
}

uint64_t cca_norm_rope_bwd_workspace_size(const cca_norm_tensor_t *tensors, int n_tensors, const cca_norm_params_t *params) {
    using namespace cca;
    if (check_bwd(tensors, n_tensors, params) != CCA_OK) return 0;
    const int sms = device_sms();
    if (sms < 1) return 0;
    int heads = 0;
    bool per_head = false;
    for (int i = 0; i < n_tensors; ++i) heads += tensors[i].H, per_head = per_head || has_head_weights(tensors[i]);
    uint64_t at[2];
    return 4 * bwd_floats(tensors, n_tensors, *params, bwd_grid(params->rope, heads, per_head, sms), per_head, at);
}

int cca_norm_rope_bwd(const cca_norm_tensor_t *tensors, int n_tensors, const cca_norm_params_t *params, void *workspace,
                      uint64_t workspace_bytes, void *stream) {
    using namespace cca;
    int st = check_bwd(tensors, n_tensors, params);
    if (st != CCA_OK) return st;
    if ((st = check_device()) != CCA_OK) return st;
    const int sms = device_sms();
    if (sms < 1) return CCA_ERR_CUDA;
    NormArgs a = norm_args(*params);
    a.n_t = n_tensors;
    bool per_head = false;
    for (int i = 0; i < n_tensors; ++i) {
        a.t[i] = norm_src(tensors[i], *params);
        a.heads += tensors[i].H;
        per_head = per_head || has_head_weights(tensors[i]);
    }
    const BwdGrid g = bwd_grid(params->rope, a.heads, per_head, sms);
    if (g.y > 65535) return CCA_ERR_UNSUPPORTED;
    a.heads_per_block = g.heads_per_block;
    uint64_t at[2];
    const uint64_t need = 4 * bwd_floats(tensors, n_tensors, *params, g, per_head, at);
    if (need > 0) {
        if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0 || workspace_bytes < need)
            return CCA_ERR_INVALID_ARG;
        const Span ws = {reinterpret_cast<uintptr_t>(workspace), reinterpret_cast<uintptr_t>(workspace) + need};
        const int es = params->rope.dtype == CCA_BF16 ? 2 : 4;
        for (int i = 0; i < n_tensors; ++i) {
            const int64_t size[3] = {params->rope.B, tensors[i].H, params->rope.N};
            Span s[5];
            span_of(tensors[i].x, tensors[i].x_stride, size, params->rope.d, es, s[0]);
            span_of(tensors[i].dy, tensors[i].dy_stride, size, params->rope.d, es, s[1]);
            span_of(tensors[i].y, tensors[i].y_stride, size, params->rope.d, es, s[2]);
            s[3] = weight_span(tensors[i].weight, tensors[i], *params);
            s[4] = weight_span(tensors[i].dweight, tensors[i], *params);
            for (const Span &x : s)
                if (spans_meet(ws, x)) return CCA_ERR_INVALID_ARG;
        }
    }
    DwArgs d = {};
    int rows = 0;
    for (int i = 0, k = 0; i < n_tensors; ++i) {
        if (tensors[i].dweight == nullptr) continue;
        // shared weights next to another tensor's own for each head: the heads' partial sums are added up
        a.t[i].part = static_cast<float *>(workspace) + at[i];
        d.part[k] = a.t[i].part;
        d.dw[k] = tensors[i].dweight;
        d.heads[k] = has_head_weights(tensors[i]) ? tensors[i].H : 1;
        d.parts[k] = per_head ? (has_head_weights(tensors[i]) ? g.x : g.x * tensors[i].H) : g.x * g.y;
        rows += d.heads[k++];
    }
    d.w_f32 = params->weight_dtype == CCA_F32;
    const dim3 grid(g.x, g.y);
    const int turn = turn_of(params->rope);
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (params->rope.dtype == CCA_BF16)
        e = params->rope.d == 128 ? launch_bwd<__nv_bfloat16, 128>(a, turn, per_head, grid, strm)
                                  : launch_bwd<__nv_bfloat16, 64>(a, turn, per_head, grid, strm);
    else
        e = params->rope.d == 128 ? launch_bwd<float, 128>(a, turn, per_head, grid, strm)
                                  : launch_bwd<float, 64>(a, turn, per_head, grid, strm);
    if (e != cudaSuccess || rows == 0) return from_cuda(e);
    return from_cuda(params->rope.d == 128 ? start_dependent(norm_dw_kernel<128>, dim3(rows, 4), DW_THREADS, 0, strm, d)
                                           : start_dependent(norm_dw_kernel<64>, dim3(rows, 2), DW_THREADS, 0, strm, d));
}

int cca_norm_rope_append(const cca_norm_tensor_t *q, const cca_norm_tensor_t *k, const cca_rope_tensor_t *v,
                         const cca_pages_t *raw, const int32_t *lens, const int32_t *parents, const int32_t *counts,
                         int32_t *dev_status, const cca_norm_params_t *params, void *stream) {
    using namespace cca;
    int st = check_norm(params);
    if (st != CCA_OK) return st;
    if (k == nullptr) return CCA_ERR_INVALID_ARG;
    cca_rope_tensor_t qv, kv = rope_view(*k);
    if (q != nullptr) qv = rope_view(*q);
    if ((st = check_append(q != nullptr ? &qv : nullptr, &kv, v, raw, lens, parents, counts, dev_status, params->rope)) != CCA_OK)
        return st;
    NormArgs a = norm_args(*params);
    bool per_head = false;
    Span written[3] = {};
    const cca_norm_tensor_t *in[2] = {q, k};
    for (const cca_norm_tensor_t *t : in) {
        if (t == nullptr) continue;
        if (!weight_ok(*t, *params)) return CCA_ERR_INVALID_ARG;
        a.t[a.n_t] = norm_src(*t, *params);
        if (t == k) a.t[a.n_t].paged = 1, a.t[a.n_t].y = static_cast<char *>(raw->K);
        ++a.n_t;
        a.heads += t->H;
        per_head = per_head || has_head_weights(*t);
    }
    const int es = params->rope.dtype == CCA_BF16 ? 2 : 4;
    if (q != nullptr) {
        const int64_t size[3] = {params->rope.B, q->H, params->rope.N};
        span_of(q->y, q->y_stride, size, params->rope.d, es, written[0]);
    }
    const uint64_t pool = static_cast<uint64_t>(raw->n_pages) * raw->rows * k->H * params->rope.d * es;
    written[1] = {reinterpret_cast<uintptr_t>(raw->K), reinterpret_cast<uintptr_t>(raw->K) + pool};
    written[2] = {reinterpret_cast<uintptr_t>(raw->V), reinterpret_cast<uintptr_t>(raw->V) + pool};
    for (const cca_norm_tensor_t *t : in)
        for (const Span &s : written)
            if (t != nullptr && spans_meet(s, weight_span(t->weight, *t, *params))) return CCA_ERR_INVALID_ARG;
    NormSrc &values = a.t[a.n_t++];
    values.x = static_cast<const char *>(v->x);
    for (int i = 0; i < 3; ++i) values.xs[i] = v->x_stride[i] * es;
    values.y = static_cast<char *>(raw->V);
    values.H = v->H;
    values.plain = values.paged = 1;
    a.heads += v->H;
    a.lens = lens;
    a.parents = parents;
    a.counts = counts;
    a.table = raw->table;
    a.n_pages = raw->n_pages;
    a.rows = raw->rows;
    a.cols = raw->cols;
    a.status = dev_status;
    if ((st = check_device()) != CCA_OK) return st;
    return from_cuda(launch_norm<true>(params->rope.dtype, params->rope.d, a, turn_of(params->rope), per_head,
                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
