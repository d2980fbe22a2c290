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

template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

template <typename T, int V>
struct Chunk {
    union {
        typename Raw<sizeof(T) * V>::type raw;
        T e[V];
    };
    __device__ Chunk() {}
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float &x) { x = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 &x) { x = __float2bfloat16_rn(v); }

// factor * (cos, sin) of the angle `turn` / 2^64 turns
__device__ __forceinline__ void turn_cos_sin(uint64_t turn, float factor, float &c, float &s) {
    const uint32_t hi = static_cast<uint32_t>(turn >> 32);
    const uint32_t quadrant = (hi + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(hi - (quadrant << 30));  // [-2^29, 2^29) / 2^32 turns
    float sn, cs;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &sn, &cs);  // half turns: 2 / 2^32
    c = (quadrant & 1) ? sn : cs;
    s = (quadrant & 1) ? cs : sn;
    // quadrant q turns (cos, sin) of the rest by q * 90 degrees
    if (quadrant == 1 || quadrant == 2) c = -c;
    if (quadrant == 2 || quadrant == 3) s = -s;
    c *= factor;
    s *= factor;
}

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

// ---------------------------------------------------------------- argument checks

struct Span {
    uintptr_t lo, hi;  // bytes [lo, hi)
};

bool spans_meet(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }

// The bytes that a strided [B, H, N, d] tensor touches; false when a row is misaligned.
bool span_of(const void *p, const int64_t (&stride)[3], const int64_t (&size)[3], int d, int es, Span &out) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(p);
    if (p == nullptr || (base & 15u) != 0) return false;
    int64_t lo = 0, hi = 0;
    for (int i = 0; i < 3; ++i) {
        if (size[i] <= 1) continue;
        // keeps every product below inside 64 bits
        if (stride[i] > (int64_t{1} << 58) / size[i] || stride[i] < -((int64_t{1} << 58) / size[i])) return false;
        if ((stride[i] * es) % 16 != 0) return false;
        const int64_t far = (size[i] - 1) * stride[i];
        (far < 0 ? lo : hi) += far;
    }
    out.lo = base + lo * es;
    out.hi = base + (hi + d) * es;
    return true;
}

// Whether no two rows of a strided [B, H, N, d] output share memory: each dimension steps
// over everything that the smaller ones cover.
bool rows_apart(const int64_t (&stride)[3], const int64_t (&size)[3], int d) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (stride[order[j]] < stride[order[i]]) {
                const int k = order[i];
                order[i] = order[j];
                order[j] = k;
            }
    int64_t covered = d;
    for (int k : order) {
        if (size[k] <= 1) continue;
        if (stride[k] < covered) return false;
        covered += (size[k] - 1) * stride[k];
    }
    return true;
}

bool params_ok(const cca_rope_params_t *p, int &st) {
    st = CCA_ERR_INVALID_ARG;
    if (p == nullptr || p->B < 1 || p->N < 1 || p->d < 1) return false;
    if (p->rot < 0 || p->rot % 2 != 0 || p->rot > p->d || (p->layout != 0 && p->layout != 1)) return false;
    if ((p->inverse != 0 && p->inverse != 1) || !(p->factor == p->factor)) return false;
    if (p->dtype != CCA_BF16 && p->dtype != CCA_F32) return false;
    if (p->rot > 0 && (p->inv_freq == nullptr || (reinterpret_cast<uintptr_t>(p->inv_freq) & 7u) != 0)) return false;
    if ((reinterpret_cast<uintptr_t>(p->positions) & 3u) != 0 || p->pos_stride < 0) return false;
    if (p->d != 64 && p->d != 128) {
        st = CCA_ERR_UNSUPPORTED;
        return false;
    }
    st = CCA_OK;
    return true;
}

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
    Span x[2], y[2];
    bool in_place[2];
    RopeArgs a = base_args(params);
    a.n_t = n_tensors;
    for (int i = 0; i < n_tensors; ++i) {
        const cca_rope_tensor_t &t = tensors[i];
        if (t.H < 1 || t.H > (1 << 20)) return CCA_ERR_INVALID_ARG;
        const int64_t size[3] = {params->B, t.H, params->N};
        if (!span_of(t.x, t.x_stride, size, params->d, es, x[i]) || !span_of(t.y, t.y_stride, size, params->d, es, y[i]))
            return CCA_ERR_INVALID_ARG;
        if (!rows_apart(t.y_stride, size, params->d)) return CCA_ERR_INVALID_ARG;
        in_place[i] = t.x == t.y;
        for (int k = 0; k < 3; ++k)
            if (size[k] > 1 && t.x_stride[k] != t.y_stride[k]) in_place[i] = false;
        if (!in_place[i] && spans_meet(x[i], y[i])) return CCA_ERR_INVALID_ARG;
        a.t[i] = to_src(t, es);
        a.heads += t.H;
    }
    if (n_tensors == 2) {
        // Two tensors may interleave (queries and keys of one packed projection): rows of the
        // same strides, the one's heads wholly before the other's inside each token.
        bool apart = !spans_meet(y[0], y[1]) && !spans_meet(y[0], x[1]) && !spans_meet(x[0], y[1]);
        if (!apart && in_place[0] && in_place[1]) {
            const cca_rope_tensor_t *f = &tensors[0], *g = &tensors[1];
            if (reinterpret_cast<uintptr_t>(f->x) > reinterpret_cast<uintptr_t>(g->x)) {
                f = &tensors[1];
                g = &tensors[0];
            }
            const int64_t gap = static_cast<int64_t>(reinterpret_cast<uintptr_t>(g->x) - reinterpret_cast<uintptr_t>(f->x)) / es;
            const int inner = params->N > 1 ? 2 : 0;  // the dimension that steps from token to token
            const int64_t token = f->x_stride[inner];
            apart = token == g->x_stride[inner] &&
                    (params->N == 1 || params->B == 1 ||
                     (f->x_stride[0] == g->x_stride[0] && f->x_stride[0] >= token * params->N)) &&
                    gap >= (f->H - 1) * f->x_stride[1] + params->d &&
                    gap + (g->H - 1) * g->x_stride[1] + params->d <= token;
        }
        if (!apart) return CCA_ERR_INVALID_ARG;
    }
    if ((st = check_device()) != CCA_OK) return st;
    return from_cuda(launch_rope_any<false>(params->dtype, a, static_cast<cudaStream_t>(stream)));
}

int cca_rope_append(const cca_rope_tensor_t *q, const cca_rope_tensor_t *k, const cca_rope_tensor_t *v,
                    const cca_pages_t *raw, const int32_t *lens, const int32_t *parents, const int32_t *counts,
                    int32_t *dev_status, const cca_rope_params_t *params, void *stream) {
    using namespace cca;
    int st;
    if (!params_ok(params, st)) return st;
    if (params->positions != nullptr || params->pos_stride != 0 || params->start != 0 || params->inverse != 0)
        return CCA_ERR_INVALID_ARG;
    if (k == nullptr || v == nullptr || k->H < 1 || k->H > (1 << 20) || v->H != k->H) return CCA_ERR_INVALID_ARG;
    if (!pages_ok(raw, 1) || lens == nullptr || params->B > 65535) return CCA_ERR_INVALID_ARG;
    const void *words[4] = {lens, parents, counts, dev_status};
    for (const void *p : words)
        if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return CCA_ERR_INVALID_ARG;
    if (parents != nullptr && params->N > TREE_MAX_NODES) return CCA_ERR_UNSUPPORTED;
    const int es = params->dtype == CCA_BF16 ? 2 : 4;
    const uint64_t pool = static_cast<uint64_t>(raw->n_pages) * raw->rows * k->H * params->d * es;
    const Span kp = {reinterpret_cast<uintptr_t>(raw->K), reinterpret_cast<uintptr_t>(raw->K) + pool};
    const Span vp = {reinterpret_cast<uintptr_t>(raw->V), reinterpret_cast<uintptr_t>(raw->V) + pool};
    if (spans_meet(kp, vp)) return CCA_ERR_INVALID_ARG;
    RopeArgs a = base_args(params);
    Span y = {};
    const cca_rope_tensor_t *in[3] = {q, k, v};
    for (int i = 0; i < 3; ++i) {
        if (in[i] == nullptr) continue;
        Span x;
        const int64_t size[3] = {params->B, in[i]->H, params->N};
        if (in[i]->H < 1 || in[i]->H > (1 << 20) || !span_of(in[i]->x, in[i]->x_stride, size, params->d, es, x)) return CCA_ERR_INVALID_ARG;
        if (i == 0) {
            if (!span_of(q->y, q->y_stride, size, params->d, es, y) || !rows_apart(q->y_stride, size, params->d))
                return CCA_ERR_INVALID_ARG;
            bool same = q->x == q->y;
            for (int s = 0; s < 3; ++s)
                if (size[s] > 1 && q->x_stride[s] != q->y_stride[s]) same = false;
            if ((!same && spans_meet(x, y)) || spans_meet(y, kp) || spans_meet(y, vp)) return CCA_ERR_INVALID_ARG;
        } else if (q != nullptr && spans_meet(x, y)) {
            return CCA_ERR_INVALID_ARG;
        }
        if (spans_meet(x, kp) || spans_meet(x, vp)) return CCA_ERR_INVALID_ARG;
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
