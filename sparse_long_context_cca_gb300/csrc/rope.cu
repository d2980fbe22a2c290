// Rotary positions of queries and keys, and their serving form that stores the new
// tokens of a step into paged caches.  Pair i of a head at position p turns by
// t = p * inv_freq[i]:  y_a = f (x_a cos t - x_b sin t),  y_b = f (x_b cos t + x_a sin t);
// the gradient is the same kernel with -t.
//
// Angles.  inv_freq / (2 pi) is kept as a 64-bit fraction of a turn, F / 2^64, so that
// p * F modulo 2^64 (one integer multiplication that wraps) is the angle modulo one turn,
// exactly reduced for every p: the only error is F's rounding, at most p * 2^-53 turns of
// the double that came in.  The top two bits (rounded) are the quadrant, and the rest is
// at most 1/8 turn either way, which a float holds to 2^-25 of its size.
//
// Memory-bound: every row is read once and written once.  A thread owns V columns and
// their V partners at one position, makes its V sines and cosines once and uses them
// for every head of its head group, so the angles cost little next to the rows.  Two
// heads' loads are in flight per thread (the first two from before the angles are made), and
// 48 registers a thread keep 1280 threads on an SM.  Queries and keys of a 32 K prompt (32 + 8
// heads of 128, bf16, read from a projection's layout): 107 us, 6.26 TB/s of the 6.70 that a
// copy reaches; with four heads at 80 registers 118 us, at 100 registers 167 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/cca.h"
#include "internal.h"
#include "paged.cuh"
#include "rope.cuh"

namespace cca {
namespace {

constexpr int ROPE_THREADS = 256;

struct RopeSrc {
    const char *x;
    char *y;
    int64_t xs[3], ys[3];  // bytes, of (b, h, n); ys unused for a paged store
    int H;
    int rotate, paged;
};

struct RopeArgs {
    RopeSrc t[3];
    int n_t, heads;       // tensors, and their heads added up
    int heads_per_block;  // heads one thread walks through
    uint64_t by_units;    // 2^64 over the units of a row, rounded up
    int B, N, d, rot, layout, inverse;
    float factor;
    const double *inv_freq;
    const int32_t *positions;
    int64_t pos_stride, start;
    // serving form
    const int32_t *lens, *parents, *counts;
    const int32_t *table;
    int n_pages, rows, cols;
    int32_t *status;
};

constexpr int ROPE_BATCH = 2;  // heads whose loads are in flight together
template <int V, bool HALF>
__host__ __device__ constexpr int angles() { return HALF ? V : V / 2 > 0 ? V / 2 : 1; }  // of a thread
__host__ __device__ constexpr int share(int n) { return n < 4 ? n : 4; }                 // threads that make them
// Heads per thread up to which they are shared.  Each thread its own against shared, us: 32 + 8 heads
// of 128, bf16, 16 tokens 3.2 and 2.5, 512 (2 heads) 5.0 and 3.6, 2048 (3) 10.4 and 9.0, 4096 (4)
// 16.6 and 17.7; fp32, 1024 (3) 7.5 and 7.6, 2048 (4) 13.0 and 15.7; storing 16 x 32 tokens of 48
// heads (2) 8.0 and 4.8.
constexpr int SHARE_MAX = 3;

// V: columns per access.  HALF: pairs (i, i + rot/2), a thread owns V pairs in two chunks;
// otherwise pairs (2i, 2i + 1), a thread owns the V/2 pairs of one chunk.
// PAGED: the serving form, one block row per sequence.
// SHARED: few heads per thread, so that the angles would be most of the work: a block takes fewer
// rows and `share` times the heads, and its threads make the angles together.
template <typename T, int V, bool HALF, bool PAGED, bool SHARED>
__global__ void __launch_bounds__(ROPE_THREADS, SHARED ? 3 : 5) rope_kernel(const RopeArgs a) {
    using R = typename Raw<sizeof(T) * V>::type;
    __shared__ uint64_t sm_freq[64];
    __shared__ int16_t sm_parent[PAGED ? TREE_MAX_NODES : 1];
    constexpr int NA = angles<V, HALF>();
    constexpr int S = SHARED ? share(NA) : 1;
    constexpr int PER = ROPE_THREADS / S;  // row units of a block
    __shared__ float2 sm_angle[SHARED ? NA * PER : 1];
    const int half = a.rot / 2;
    // units of a row: the rotated chunks (or chunk pairs), then the copied ones
    const int turned = (HALF ? half : a.rot) / V;
    const int units = turned + (a.d - a.rot) / V;
    const int local = SHARED ? threadIdx.x % PER : threadIdx.x, sub = SHARED ? threadIdx.x / PER : 0;
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * PER + local;
    const int64_t row = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(idx), a.by_units));
    const int u = static_cast<int>(idx - row * units);
    const bool inside = row < (PAGED ? a.N : static_cast<int64_t>(a.B) * a.N);
    const int b = PAGED ? static_cast<int>(blockIdx.z) : static_cast<int>(row / a.N);
    const int64_t n = PAGED ? row : row - static_cast<int64_t>(b) * a.N;
    const bool turn = u < turned;
    const int col = turn ? u * V : a.rot + (u - turned) * V;
    const int64_t other = HALF ? half * static_cast<int64_t>(sizeof(T)) : 0;

    // The head walk: tensors one after the other, ROPE_BATCH heads at a time.
    const int h0 = (blockIdx.y * S + sub) * a.heads_per_block, h1 = min(h0 + a.heads_per_block, a.heads);
    const bool work = inside && (!SHARED || h0 < h1);
    int which = 0, first = 0;  // tensor of the batch, heads before it
    while ((!SHARED || work) && h0 - first >= a.t[which].H) first += a.t[which++].H;
    Chunk<T, V> lo[ROPE_BATCH], hi[ROPE_BATCH];
    auto batch_heads = [&](int h) { return min(min(ROPE_BATCH, h1 - h), first + a.t[which].H - h); };
    auto load = [&](int h, int count) {
        const RopeSrc &t = a.t[which];
        const char *x = t.x + b * t.xs[0] + (h - first) * t.xs[1] + n * t.xs[2] + col * static_cast<int64_t>(sizeof(T));
#pragma unroll
        for (int k = 0; k < ROPE_BATCH; ++k)
            if (k < count) {
                lo[k].raw = *reinterpret_cast<const R *>(x + k * t.xs[1]);
                if (HALF && turn) hi[k].raw = *reinterpret_cast<const R *>(x + k * t.xs[1] + other);
            }
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (work) load(h0, batch_heads(h0));
    int len = 0, count_b = 0;
    if constexpr (PAGED) {  // asked for with the rest: what follows is a chain
        len = a.lens[b];
        count_b = a.counts != nullptr ? a.counts[b] : a.N;
    }

    for (int i = threadIdx.x; i < half; i += ROPE_THREADS) {
        double f = a.inv_freq[i] * 0.15915494309189535;  // turns per position
        f -= floor(f);
        sm_freq[i] = static_cast<uint64_t>(f * 18446744073709551616.0);
    }
    if constexpr (PAGED) {
        if (a.parents != nullptr)
            for (int i = threadIdx.x; i < a.N; i += ROPE_THREADS) {
                const int p = a.parents[static_cast<int64_t>(b) * a.N + i];
                sm_parent[i] = static_cast<int16_t>(p >= -1 && p < i ? p : -2);
            }
    }
    __syncthreads();
    if (!SHARED && !work) return;
    int64_t pos = 0;
    bool real = true;
    int64_t page = -1;  // of the row's slot, and the row inside it
    int page_off = 0;
    if constexpr (PAGED) {
        if (len < 0) {
            report(a.status, CCA_ERR_INVALID_ARG);
            real = false;
            len = 0;
        }
        pos = static_cast<int64_t>(len) + n;
        if (n >= count_b) real = false;
        if (real && inside) {
            const uint32_t slot = static_cast<uint32_t>(len) + static_cast<uint32_t>(n);  // below 2^32
            const uint32_t c = slot / static_cast<uint32_t>(a.rows);
            page = c < static_cast<uint32_t>(a.cols) ? a.table[static_cast<int64_t>(b) * a.cols + c] : -1;
            page_off = static_cast<int>(slot - c * a.rows);
        }
        if (a.parents != nullptr) {
            int depth = 0, k = inside ? sm_parent[n] : -1;
            while (k >= 0) {  // parents are below their children, so this ends
                ++depth;
                k = sm_parent[k];
            }
            if (k != -1) real = false;
            pos = static_cast<int64_t>(len) + depth;
        }
        if (real && inside && (page < 0 || page >= a.n_pages)) report(a.status, CCA_ERR_INVALID_ARG);
        if (!real || page >= a.n_pages) page = -1;
    } else if (inside) {
        pos = a.positions != nullptr ? a.positions[b * a.pos_stride + n] : a.start + n;
    }
    // this thread's cosines and sines
    float c[NA], s[NA];
    if (turn) {
#pragma unroll
        for (int i = 0; i < NA / S; ++i) {
            const int k = sub * (NA / S) + i, pair = HALF ? col + k : col / 2 + k;
            turn_cos_sin(static_cast<uint64_t>(pos) * sm_freq[pair], a.factor, c[i], s[i]);
            if (a.inverse) s[i] = -s[i];
            if (SHARED) sm_angle[k * PER + local] = make_float2(c[i], s[i]);
        }
    }
    if constexpr (SHARED) {
        __syncthreads();
        if (!work) return;
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const float2 cs = sm_angle[i * PER + local];
            c[i] = cs.x;
            s[i] = cs.y;
        }
    }
    for (int h = h0; h < h1;) {
        const int count = batch_heads(h);
        if (h > h0) load(h, count);
        const RopeSrc &t = a.t[which];
        char *y;
        int64_t step;
        bool store = true;
        if (PAGED && t.paged) {
            step = static_cast<int64_t>(a.rows) * a.d * sizeof(T);
            y = t.y + ((page * t.H + (h - first)) * a.rows + page_off) * a.d * static_cast<int64_t>(sizeof(T));
            store = page >= 0;
        } else {
            step = t.ys[1];
            y = t.y + b * t.ys[0] + (h - first) * step + n * t.ys[2];
        }
        y += col * static_cast<int64_t>(sizeof(T));
        const bool rotate = turn && t.rotate;
#pragma unroll
        for (int k = 0; k < ROPE_BATCH; ++k) {
            if (k >= count || !store) continue;
            if (rotate) {
                if constexpr (HALF) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float xa = to_f(lo[k].e[i]), xb = to_f(hi[k].e[i]);
                        from_f(xa * c[i] - xb * s[i], lo[k].e[i]);
                        from_f(xb * c[i] + xa * s[i], hi[k].e[i]);
                    }
                } else if constexpr (V >= 2) {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float xa = to_f(lo[k].e[2 * i]), xb = to_f(lo[k].e[2 * i + 1]);
                        from_f(xa * c[i] - xb * s[i], lo[k].e[2 * i]);
                        from_f(xb * c[i] + xa * s[i], lo[k].e[2 * i + 1]);
                    }
                }
            }
            if (PAGED && !real) lo[k].raw = hi[k].raw = R{};
            *reinterpret_cast<R *>(y + k * step) = lo[k].raw;
            if (HALF && turn) *reinterpret_cast<R *>(y + k * step + other) = hi[k].raw;
        }
        h += count;
        if (h < h1 && h - first >= a.t[which].H) first += a.t[which++].H;
    }
}

template <typename T, int V, bool PAGED, bool SHARED>
cudaError_t launch_one(const RopeArgs &a, dim3 grid, cudaStream_t stream) {
    if (a.layout == 0) return start_dependent(rope_kernel<T, V, true, PAGED, SHARED>, grid, ROPE_THREADS, 0, stream, a);
    // an interleaved chunk holds whole pairs
    constexpr int VI = V < 2 ? 2 : V;
    return start_dependent(rope_kernel<T, VI, false, PAGED, SHARED>, grid, ROPE_THREADS, 0, stream, a);
}

// The widest access that every chunk boundary allows: rows are 16-byte aligned, so it is
// the largest power of two that divides the pairs' offset (rot/2, or rot when pairs are
// interleaved) and the copied columns.
int access_width(const RopeArgs &a, int max_v) {
    const int step = a.layout == 0 ? a.rot / 2 : a.rot;
    int v = max_v;
    while (v > 1 && (step % v != 0 || (a.d - a.rot) % v != 0)) v /= 2;
    return v;
}

template <bool PAGED>
cudaError_t launch_rope_any(int dtype, RopeArgs a, cudaStream_t stream) {
    const int v = access_width(a, dtype == CCA_BF16 ? 8 : 4);
    const int vv = a.layout == 1 && v < 2 ? 2 : v;
    const int units = (a.layout == 0 ? a.rot / 2 : a.rot) / vv + (a.d - a.rot) / vv;
    a.by_units = ~uint64_t{0} / units + 1;  // units >= 4; exact below 2^57
    const int64_t rows = PAGED ? a.N : static_cast<int64_t>(a.B) * a.N;
    const int64_t blocks = (rows * units + ROPE_THREADS - 1) / ROPE_THREADS;
    if (blocks > 0x7fffffff) return cudaErrorNotSupported;
    const int sms = device_sms();
    if (sms < 1) return cudaErrorNoDevice;
    // Angles are shared by the heads of a group: as many heads per thread as still leave
    // eight blocks for every SM, but a batch of loads at least.
    const int64_t all = blocks * (PAGED ? a.B : 1);
    const int most = (a.heads + ROPE_BATCH - 1) / ROPE_BATCH;
    int groups = static_cast<int>((8ll * sms + all - 1) / all);
    if (groups > most) groups = most;
    a.heads_per_block = (a.heads + groups - 1) / groups;
    groups = (a.heads + a.heads_per_block - 1) / a.heads_per_block;
    if (groups > 65535) return cudaErrorNotSupported;
    dim3 grid(static_cast<unsigned>(blocks), groups, PAGED ? a.B : 1);
    if (a.heads_per_block <= SHARE_MAX && v == (dtype == CCA_BF16 ? 8 : 4)) {
        const int s = share(a.layout == 0 ? v : v / 2), per = ROPE_THREADS / s;
        grid.x = static_cast<unsigned>((rows * units + per - 1) / per);
        grid.y = (a.heads + s * a.heads_per_block - 1) / (s * a.heads_per_block);
        return dtype == CCA_BF16 ? launch_one<__nv_bfloat16, 8, PAGED, true>(a, grid, stream)
                                 : launch_one<float, 4, PAGED, true>(a, grid, stream);
    }
    if (dtype == CCA_BF16) {
        switch (v) {
            case 8: return launch_one<__nv_bfloat16, 8, PAGED, false>(a, grid, stream);
            case 4: return launch_one<__nv_bfloat16, 4, PAGED, false>(a, grid, stream);
            case 2: return launch_one<__nv_bfloat16, 2, PAGED, false>(a, grid, stream);
            default: return launch_one<__nv_bfloat16, 1, PAGED, false>(a, grid, stream);
        }
    }
    switch (v) {
        case 4: return launch_one<float, 4, PAGED, false>(a, grid, stream);
        case 2: return launch_one<float, 2, PAGED, false>(a, grid, stream);
        default: return launch_one<float, 1, PAGED, false>(a, grid, stream);
    }
}

// ---------------------------------------------------------------- arguments

RopeArgs base_args(const cca_rope_params_t *p) {
    RopeArgs a = {};
    a.B = p->B;
    a.N = p->N;
    a.d = p->d;
    a.rot = p->rot;
    a.layout = p->layout;
    a.inverse = p->inverse;
    a.factor = p->factor;
    a.inv_freq = p->inv_freq;
    a.positions = p->positions;
    a.pos_stride = p->pos_stride;
    a.start = p->start;
    return a;
}

RopeSrc to_src(const cca_rope_tensor_t &t, int es) {
    RopeSrc r = {};
    r.x = static_cast<const char *>(t.x);
    r.y = static_cast<char *>(t.y);
    for (int i = 0; i < 3; ++i) {
        r.xs[i] = t.x_stride[i] * es;
        r.ys[i] = t.y_stride[i] * es;
    }
    r.H = t.H;
    r.rotate = 1;
    return r;
}

}  // namespace
}  // namespace cca

extern "C" {

int cca_rope(const cca_rope_tensor_t *tensors, int n_tensors, const cca_rope_params_t *params, void *stream) {
    using namespace cca;
    int st;
    if (!params_ok(params, st)) return st;
    if (tensors == nullptr || n_tensors < 1 || n_tensors > 2) return CCA_ERR_INVALID_ARG;
    const int es = params->dtype == CCA_BF16 ? 2 : 4;
    RopeArgs a = base_args(params);
    a.n_t = n_tensors;
    for (int i = 0; i < n_tensors; ++i) {
        if (tensors[i].H < 1 || tensors[i].H > (1 << 20)) return CCA_ERR_INVALID_ARG;
        a.t[i] = to_src(tensors[i], es);
        a.heads += tensors[i].H;
    }
    if ((st = check_rope_tensors(tensors, n_tensors, *params)) != CCA_OK) return st;
    if ((st = check_device()) != CCA_OK) return st;
    return from_cuda(launch_rope_any<false>(params->dtype, a, static_cast<cudaStream_t>(stream)));
}

int cca_rope_append(const cca_rope_tensor_t *q, const cca_rope_tensor_t *k, const cca_rope_tensor_t *v,
                    const cca_pages_t *raw, const int32_t *lens, const int32_t *parents, const int32_t *counts,
                    int32_t *dev_status, const cca_rope_params_t *params, void *stream) {
    using namespace cca;
    int st;
    if (!params_ok(params, st)) return st;
    if ((st = check_append(q, k, v, raw, lens, parents, counts, dev_status, *params)) != CCA_OK) return st;
    const int es = params->dtype == CCA_BF16 ? 2 : 4;
    RopeArgs a = base_args(params);
    const cca_rope_tensor_t *in[3] = {q, k, v};
    for (int i = 0; i < 3; ++i) {
        if (in[i] == nullptr) continue;
        RopeSrc &t = a.t[a.n_t++];
        t = to_src(*in[i], es);
        t.rotate = i < 2;
        t.paged = i > 0;
        if (i > 0) t.y = static_cast<char *>(i == 1 ? raw->K : raw->V);
        a.heads += in[i]->H;
    }
    a.lens = lens;
    a.parents = parents;
    a.counts = counts;
    a.table = raw->table;
    a.n_pages = raw->n_pages;
    a.rows = raw->rows;
    a.cols = raw->cols;
    a.status = dev_status;
    if ((st = check_device()) != CCA_OK) return st;
    return from_cuda(launch_rope_any<true>(params->dtype, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
