// Packed sequences: the plan of a batch, the pooling of all its groups, the pooling's gradient, and the
// entry points of the calls over packed tensors.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "packed.cuh"
#include "rope.cuh"
#include "sm100_ptx.cuh"

namespace cca {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int PACK_THREADS = 256;

// ---------------------------------------------------------------- the plan

// (a + b may pass 2^31: so may a loop's index plus its step, which is why those are unsigned)
__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0 ? 1 : 0); }

// One block column per sequence.  Entry (s, p) of a list stands behind every entry of a higher tile number
// and behind those of the same number of longer sequences (of equal ones, the earlier first): its place is
// the sum over all sequences s' of max(0, tiles(s') - p - 1), and the rank of s by length.  So a block needs no
// other block's result, and nothing is sorted; an entry costs a walk over the lengths, which a warp shares.
__global__ void __launch_bounds__(PACK_THREADS) pack_kernel(const int32_t *cu, char *plan, const PlanLayout l, int S, int T, int g,
                                                            int w, int window_mode, int32_t *status) {
    const int s = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int a = cu[s], n = cu[s + 1] - a;
    bool good = true;
    int longer = 0;
    for (int i = threadIdx.x; i < S; i += PACK_THREADS) {
        const int x = cu[i], y = cu[i + 1];
        good = good && x >= 0 && x <= y && y <= T;
        longer += y - x > n || (y - x == n && i < s) ? 1 : 0;
    }
    __shared__ int sm_longer;
    if (threadIdx.x == 0) sm_longer = 0;
    good = __syncthreads_and(good);
    int32_t *header = reinterpret_cast<int32_t *>(plan);
    if (!good) {
        if (s == 0 && blockIdx.y == 0 && threadIdx.x < PACK_HEADER) header[threadIdx.x] = 0;
        if (s == 0 && blockIdx.y == 0 && threadIdx.x == 0) report(status, CCA_ERR_INVALID_ARG);
        return;
    }
    atomicAdd(&sm_longer, longer);
    __syncthreads();
    const int rank = sm_longer;
    const int tid = blockIdx.y * PACK_THREADS + threadIdx.x, step = gridDim.y * PACK_THREADS;
    auto tiles_of = [&](int list, int m) {
        return list == 0 ? ceil_div(m, PACK_PAIR) : list == 1 ? ceil_div(m, PACK_TILE) : ceil_div(seen_cores(m, w, g), PACK_TILE);
    };
    const uint64_t at[3] = {l.pairs, l.tiles, l.cores};
#pragma unroll
    for (int list = 0; list < 3; ++list) {
        const int mine = tiles_of(list, n);
        int4 *out = reinterpret_cast<int4 *>(plan + at[list]);
        for (int p = tid / 32; p < mine; p += step / 32) {
            int place = 0;
            for (int i = tid % 32; i < S; i += 32) place += max(0, tiles_of(list, cu[i + 1] - cu[i]) - p - 1);
            place = __reduce_add_sync(kFull, place) + rank;
            if (tid % 32 == 0) out[place] = make_int4(a, n, p, a / g);
        }
    }
    int32_t *positions = reinterpret_cast<int32_t *>(plan + l.positions), *first = reinterpret_cast<int32_t *>(plan + l.first);
    auto each = [&](int from, int to, auto f) {
        for (unsigned i = static_cast<unsigned>(from) + tid; i < static_cast<unsigned>(to); i += step) f(static_cast<int>(i));
    };
    each(0, n, [&](int i) { positions[a + i] = i; });
    const int c0 = a / g, c1 = (a + n) / g, groups = n / g;
    each(c0, c1, [&](int c) { first[c] = c - c0 < groups ? a + (c - c0) * g : -1; });
    if (s == 0) {  // tokens and core rows of no sequence
        auto clear = [&](int i) { positions[i] = 0; };
        auto none = [&](int c) { first[c] = -1; };
        each(0, a, clear);
        each(0, c0, none);
        const int end = cu[S];
        each(end, T, clear);
        each(end / g, T / g, none);
        if (blockIdx.y == 0 && threadIdx.x < 32) {
            int count[6] = {0, 0, 0, 0, 0, 0};  // tiles of each list; sequences of 1 to 128, 64, 32 tokens
            for (int i = threadIdx.x; i < S; i += 32) {
                const int m = cu[i + 1] - cu[i];
#pragma unroll
                for (int list = 0; list < 3; ++list) count[list] += tiles_of(list, m);
#pragma unroll
                for (int c = 0; c < 3; ++c) count[3 + c] += m > 0 && m <= 128 >> c ? 1 : 0;
            }
#pragma unroll
            for (int c = 0; c < 6; ++c)
                for (int o = 16; o > 0; o >>= 1) count[c] += __shfl_xor_sync(kFull, count[c], o);
            if (threadIdx.x == 0) {
                const int32_t h[PACK_HEADER] = {PACK_MAGIC, T, g, w, window_mode, S, cu[0], end, count[0], count[1], count[2], 0,
                                                count[0] - count[3], count[0] - count[4], count[0] - count[5], 0};
                for (int i = 0; i < PACK_HEADER; ++i) header[i] = h[i];
            }
        }
    }
}

// ---------------------------------------------------------------- pooling

template <typename T>
struct Row16;
template <>
struct Row16<__nv_bfloat16> {
    static constexpr int E = 8;
    __device__ static void unpack(const uint4 &v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 pack(const float (&f)[8]) {
        return make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                          ptx::pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Row16<float> {
    static constexpr int E = 4;
    __device__ static void unpack(const uint4 &v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    __device__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

struct PoolPackedArgs {
    Rows<const char> Q, K, V;  // strides in bytes
    char *Kc, *Vc;
    Plan plan;
    int Hq, Hkv, mode, heads_first;
    float scale_log2;
};

constexpr int POOL_WARPS = 4;
constexpr int POOL_BLOCKS = 4;  // resident
constexpr int POOL_PASSES = 4;  // steps of a chunk: all its rows are asked for before any is used

// One warp per core row and KV head.  D * sizeof(T) / 16 lanes hold a row, so a step takes 32 over that
// many rows; a chunk of POOL_PASSES steps (8 rows of 128 bf16 columns) goes through one running
// (maximum, sum).  12 prompts of 32 K tokens in all, 8 heads, g = 16: chunks of 8 steps 44 us at 12 warps an
// SM (51 at 16, with spills), of 4 steps 38 us at 16 warps (47 at 24): 159 MB at 4.2 TB/s.  Rows under way are held in
// registers, eight a warp, so 16 warps an SM are all that fit; a ring of copies in shared memory, with which the pooling of
// contiguous tensors reads 5.8 TB/s, was not built for packed ones.
template <typename T, int D>
__global__ void __launch_bounds__(POOL_WARPS * 32, POOL_BLOCKS) pool_packed_kernel(const PoolPackedArgs a) {
    using RT = Row16<T>;
    constexpr int E = RT::E, LPR = D / E, RPP = 32 / LPR;
    const int lane = threadIdx.x & 31, sub = lane / LPR, cl = lane % LPR;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t item = static_cast<int64_t>(blockIdx.x) * POOL_WARPS + (threadIdx.x >> 5);
    if (plan_counts(a.plan).y < 0 || item >= static_cast<int64_t>(a.plan.G) * a.Hkv) return;
    const int c = static_cast<int>(a.heads_first ? item / a.Hkv : item % a.plan.G);
    const int kv = static_cast<int>(a.heads_first ? item % a.Hkv : item / a.plan.G);
    const int64_t t0 = a.plan.first[c];
    char *out = (sub == 0 ? a.Kc : a.Vc) + ((static_cast<int64_t>(kv) * a.plan.G + c) * D + cl * E) * sizeof(T);
    char *const vout = a.Vc + ((static_cast<int64_t>(kv) * a.plan.G + c) * D + cl * E) * sizeof(T);
    if (t0 < 0) {  // of no group
        if (sub == 0) {
            *reinterpret_cast<uint4 *>(out) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(vout) = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int g = a.plan.g, r = a.Hq / a.Hkv;
    // a chunk's keys and values; those of the first are asked for before the queries
    uint4 k[POOL_PASSES], v[POOL_PASSES];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < POOL_PASSES; ++i) {
            const int t = base + i * RPP + sub;
            k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (t < g) {
                k[i] = *reinterpret_cast<const uint4 *>(a.K.at(kv, t0 + t) + cl * 16);
                v[i] = *reinterpret_cast<const uint4 *>(a.V.at(kv, t0 + t) + cl * 16);
            }
        }
    };
    load(0);
    float q[E], ak[E], av[E];
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = ak[e] = av[e] = 0.f;
    const float scale = a.scale_log2 / r;
    if (a.mode == 0) {
        for (int h = 0; h < r; h += 4) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (h + i < r) x[i] = *reinterpret_cast<const uint4 *>(a.Q.at(kv * r + h + i, t0 + g - 1) + cl * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (h + i >= r) continue;
                float f[E];
                RT::unpack(x[i], f);
#pragma unroll
                for (int e = 0; e < E; ++e) q[e] += f[e];
            }
        }
    }
    float m = -INFINITY, l = 0.f;
    for (int base = 0; base < g; base += POOL_PASSES * RPP) {
        if (base > 0) load(base);
        float s[POOL_PASSES], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < POOL_PASSES; ++i) {
            float f[E], x = 0.f;
            RT::unpack(k[i], f);
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(q[e], f[e], x);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
            if (a.mode == 1) x = 0.f;  // a mean has no scores, whatever the keys hold
            s[i] = base + i * RPP + sub < g ? x * scale : -INFINITY;
            top = fmaxf(top, s[i]);
        }
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
        const float f0 = exp2f(m - ref);
        m = mn;
        l *= f0;
#pragma unroll
        for (int e = 0; e < E; ++e) ak[e] *= f0, av[e] *= f0;
#pragma unroll
        for (int i = 0; i < POOL_PASSES; ++i) {
            if (base + i * RPP + sub >= g) continue;
            const float p = exp2f(s[i] - ref);
            float f[E];
            l += p;
            RT::unpack(k[i], f);
#pragma unroll
            for (int e = 0; e < E; ++e) ak[e] = fmaf(p, f[e], ak[e]);
            RT::unpack(v[i], f);
#pragma unroll
            for (int e = 0; e < E; ++e) av[e] = fmaf(p, f[e], av[e]);
        }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
        l += __shfl_xor_sync(kFull, l, o);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            ak[e] += __shfl_xor_sync(kFull, ak[e], o);
            av[e] += __shfl_xor_sync(kFull, av[e], o);
        }
    }
    if (sub != 0) return;
    const float inv = 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) ak[e] *= inv, av[e] *= inv;
    *reinterpret_cast<uint4 *>(out) = RT::pack(ak);
    *reinterpret_cast<uint4 *>(vout) = RT::pack(av);
}

// ---------------------------------------------------------------- backward: D, and the pooling's gradient

// D_i = dO_i . O_i, a row per LPR lanes (and zeros for the counters of the kernels behind it): bound by memory (16 K rows of 32 heads of 128, 268 MB, 45 us, 6.0 TB/s).
constexpr int D_ROWS = 4;
template <typename T, int D>
__global__ void __launch_bounds__(256) packed_d_kernel(Rows<const char> O, Rows<const char> dO, float *out, Plan plan, int Hq, int heads_first,
                                                       int32_t *zero, int n_zero) {
    using RT = Row16<T>;
    constexpr int E = RT::E, LPR = D / E;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n_zero; i += gridDim.x * 256ll) zero[i] = 0;
    const int64_t n = static_cast<int64_t>(plan.T) * Hq;
    uint4 a[D_ROWS], b[D_ROWS];
    int64_t at[D_ROWS];  // the row's place in `out`; -1: none
#pragma unroll
    for (int k = 0; k < D_ROWS; ++k) {
        const int64_t item = (static_cast<int64_t>(blockIdx.x) * D_ROWS + k) * (256 / LPR) + threadIdx.x / LPR;
        const int64_t row = heads_first ? item / Hq : item % plan.T;
        const int h = static_cast<int>(heads_first ? item % Hq : item / plan.T);
        at[k] = item < n ? static_cast<int64_t>(h) * plan.T + row : -1;
        a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
        if (item < n) {
            a[k] = *reinterpret_cast<const uint4 *>(O.at(h, row) + threadIdx.x % LPR * 16);
            b[k] = *reinterpret_cast<const uint4 *>(dO.at(h, row) + threadIdx.x % LPR * 16);
        }
    }
#pragma unroll
    for (int k = 0; k < D_ROWS; ++k) {
        float f[E], g[E], x = 0.f;
        RT::unpack(a[k], f);
        RT::unpack(b[k], g);
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(f[e], g[e], x);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
        if (at[k] >= 0 && threadIdx.x % LPR == 0) out[at[k]] = x;
    }
}

struct ClearArgs {
    Rows<char> t[4];  // strides in bytes
    int heads[4], n, chunks;  // chunks: 16-byte pieces of a row
    Plan plan;
};
__global__ void __launch_bounds__(256) packed_clear_kernel(ClearArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    a.plan.status = nullptr;
    const bool good = plan_counts(a.plan).y >= 0;
    const int begin = good ? a.plan.header[6] : a.plan.T, end = good ? a.plan.header[7] : a.plan.T;
    const int64_t rows = static_cast<int64_t>(begin) + a.plan.T - end;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= a.n) break;
        const int64_t all = rows * a.heads[i] * a.chunks;
        for (int64_t x = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; x < all; x += static_cast<int64_t>(gridDim.x) * 256) {
            const int64_t row = x / a.chunks % rows;
            *reinterpret_cast<uint4 *>(a.t[i].at(static_cast<int>(x / a.chunks / rows), row < begin ? row : row - begin + end) +
                                       x % a.chunks * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

struct PoolBwdArgs {
    Rows<const char> Q, K, V;
    PackedBwdSpace w;
    Plan plan;
    int Hq, Hkv, heads_first;
    float c;  // tau / r
};

// The pooling's gradient for one group that some row sees (its core tile was visited), reduced to what
// the raw tokens' kernels add to their rows: a_t and c ds_t per token, the queries' sum, and the
// gradient of each group-last query, c sum_t ds_t k_t; ds_t = a_t (da_t - sum_u a_u da_u),
// da_t = dKc . k_t + dVc . v_t.  One warp per group and KV head, two walks over its rows: 832 groups of 8 KV
// heads with the partial sums of their cores 28 us, bound by the walks' latency.
template <typename T, int D>
__global__ void __launch_bounds__(POOL_WARPS * 32) pool_packed_bwd_kernel(const PoolBwdArgs a) {
    using RT = Row16<T>;
    constexpr int E = RT::E, LPR = D / E, RPP = 32 / LPR;
    const int lane = threadIdx.x & 31, sub = lane / LPR, cl = lane % LPR;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t item = static_cast<int64_t>(blockIdx.x) * POOL_WARPS + (threadIdx.x >> 5);
    const int3 counts = plan_counts(a.plan);
    // items run through the core tiles of the plan, 128 cores to a tile
    const int64_t cores = static_cast<int64_t>(counts.z) * PACK_TILE;
    if (item >= cores * a.Hkv) return;
    const int64_t x = a.heads_first ? item / a.Hkv : item % cores;
    const int kv = static_cast<int>(a.heads_first ? item % a.Hkv : item / cores);
    const int4 e4 = a.plan.cores[x / PACK_TILE];
    const int g = a.plan.g, r = a.Hq / a.Hkv;
    const int j = e4.z * PACK_TILE + static_cast<int>(x % PACK_TILE);
    if (j >= seen_cores(e4.y, a.plan.w, g)) return;
    const int64_t t0 = e4.x + static_cast<int64_t>(j) * g;
    const int64_t core = (static_cast<int64_t>(kv) * a.plan.G + e4.w + j) * D + cl * E;
    const int64_t split = static_cast<int64_t>(a.Hkv) * a.plan.G * D;
    float q[E], dk[E], dv[E], dq[E];
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = dk[e] = dv[e] = dq[e] = 0.f;
    for (int s = 0; s < a.w.splits; ++s)
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(a.w.dKc + s * split + core + e);
            const float4 z = *reinterpret_cast<const float4 *>(a.w.dVc + s * split + core + e);
            dk[e] += y.x, dk[e + 1] += y.y, dk[e + 2] += y.z, dk[e + 3] += y.w;
            dv[e] += z.x, dv[e + 1] += z.y, dv[e + 2] += z.z, dv[e + 3] += z.w;
        }
    for (int h = 0; h < r; ++h) {
        float f[E];
        RT::unpack(*reinterpret_cast<const uint4 *>(a.Q.at(kv * r + h, t0 + g - 1) + cl * 16), f);
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] += f[e];
    }
    constexpr int P = POOL_PASSES;
    uint4 k[P], v[P];
    float s[P], da[P];
    auto chunk = [&](int base) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int t = base + i * RPP + sub;
            k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (t < g) {
                k[i] = *reinterpret_cast<const uint4 *>(a.K.at(kv, t0 + t) + cl * 16);
                v[i] = *reinterpret_cast<const uint4 *>(a.V.at(kv, t0 + t) + cl * 16);
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float f[E];
            RT::unpack(k[i], f);
            s[i] = da[i] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s[i] = fmaf(q[e], f[e], s[i]), da[i] = fmaf(dk[e], f[e], da[i]);
            RT::unpack(v[i], f);
#pragma unroll
            for (int e = 0; e < E; ++e) da[i] = fmaf(dv[e], f[e], da[i]);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
                s[i] += __shfl_xor_sync(kFull, s[i], o);
                da[i] += __shfl_xor_sync(kFull, da[i], o);
            }
            s[i] = base + i * RPP + sub < g ? s[i] * a.c : -INFINITY;
        }
    };
    float m = -INFINITY, den = 0.f, num = 0.f;
    for (int base = 0; base < g; base += P * RPP) {
        chunk(base);
        float top = m;
#pragma unroll
        for (int i = 0; i < P; ++i) top = fmaxf(top, s[i]);
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        const float f0 = m == -INFINITY ? 0.f : expf(m - top);
        den *= f0, num *= f0;
        m = top;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float p = s[i] == -INFINITY ? 0.f : expf(s[i] - m);
            den += p;
            num += p != 0.f ? p * da[i] : 0.f;
        }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
        den += __shfl_xor_sync(kFull, den, o);
        num += __shfl_xor_sync(kFull, num, o);
    }
    const float mean = num / den, inv = 1.f / den;
    for (int base = 0; base < g; base += P * RPP) {
        if (g > P * RPP) chunk(base);  // else the one chunk is still there
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int t = base + i * RPP + sub;
            if (t >= g) continue;
            const float at = expf(s[i] - m) * inv, cds = a.c * at * (da[i] - mean);
            float f[E];
            RT::unpack(k[i], f);
#pragma unroll
            for (int e = 0; e < E; ++e) dq[e] = fmaf(cds, f[e], dq[e]);
            if (cl == 0) {
                a.w.a[static_cast<int64_t>(kv) * a.plan.T + t0 + t] = at;
                a.w.cds[static_cast<int64_t>(kv) * a.plan.T + t0 + t] = cds;
            }
        }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < E; ++e) dq[e] += __shfl_xor_sync(kFull, dq[e], o);
    if (sub != 0) return;
    // the first split's sums become the whole ones
#pragma unroll
    for (int e = 0; e < E; e += 4) {
        *reinterpret_cast<float4 *>(a.w.qsum + core + e) = make_float4(q[e], q[e + 1], q[e + 2], q[e + 3]);
        *reinterpret_cast<float4 *>(a.w.dqs + core + e) = make_float4(dq[e], dq[e + 1], dq[e + 2], dq[e + 3]);
        if (a.w.splits > 1) {
            *reinterpret_cast<float4 *>(a.w.dKc + core + e) = make_float4(dk[e], dk[e + 1], dk[e + 2], dk[e + 3]);
            *reinterpret_cast<float4 *>(a.w.dVc + core + e) = make_float4(dv[e], dv[e + 1], dv[e + 2], dv[e + 3]);
        }
    }
}

// Mean pooling: a_t = 1/g and no gradient through the weights.
__global__ void __launch_bounds__(256) pool_packed_mean_bwd_kernel(const PoolBwdArgs a, int d) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t n = static_cast<int64_t>(a.Hkv) * a.plan.G * d, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) {
        a.w.qsum[i] = a.w.dqs[i] = 0.f;
        if (a.w.splits > 1) {
            float x = 0.f, y = 0.f;
            for (int s = 0; s < a.w.splits; ++s) x += a.w.dKc[s * n + i], y += a.w.dVc[s * n + i];
            a.w.dKc[i] = x, a.w.dVc[i] = y;
        }
    }
    const int64_t tokens = static_cast<int64_t>(a.Hkv) * a.plan.T;
    for (int64_t t = i; t < tokens; t += static_cast<int64_t>(gridDim.x) * 256) {
        a.w.a[t] = 1.f / a.plan.g;
        a.w.cds[t] = 0.f;
    }
}

// ---------------------------------------------------------------- arguments

bool packed_ok(const cca_packed_t *p) {
    if (p == nullptr || p->S < 1 || p->S > 65535 || p->T < 1 || p->g < 1 || p->w < 1) return false;
    if (p->window_mode < 0 || p->window_mode > 1) return false;
    return p->plan != nullptr && (reinterpret_cast<uintptr_t>(p->plan) & 15u) == 0 &&
           p->plan_bytes >= plan_layout(p->S, p->T, p->g).bytes;
}

int params_packed(const cca_params_t *p) {
    if (p == nullptr || p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv != 0 || p->Hq > 65535) return CCA_ERR_INVALID_ARG;
    if (p->dtype != CCA_BF16 && p->dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (!(p->scale == p->scale) || isinf(p->scale) || p->pool_mode < 0 || p->pool_mode > 3) return CCA_ERR_INVALID_ARG;
    if (!word_ptr(p->dev_status, false)) return CCA_ERR_INVALID_ARG;
    if (p->d != 64 && p->d != 128) return CCA_ERR_UNSUPPORTED;
    if (p->pool_mode > 1) return CCA_ERR_UNSUPPORTED;
    return CCA_OK;
}

// Where a tensor lies: from its first byte to its last, and, where all heads of a token stand within one
// row of `row` bytes, how much of that row they take.
struct Place {
    Span span;
    uint64_t row, inner;  // row 0: not of that kind
};

bool rows_ok(const cca_packed_rows_t *r, int H, int T, const cca_params_t &p, bool written, Place &out) {
    if (r == nullptr) return false;
    const int es = p.dtype == CCA_BF16 ? 2 : 4;
    const int64_t size[3] = {1, H, T}, stride[3] = {0, r->head_stride, r->row_stride};
    if (!span_of(r->p, stride, size, p.d, es, out.span)) return false;
    // the copy engine's strides lie between a row's bytes and 2^40
    if (H > 1 && (r->head_stride < p.d || r->head_stride * es >= (int64_t{1} << 40))) return false;
    if (T > 1 && (r->row_stride < p.d || r->row_stride * es >= (int64_t{1} << 40))) return false;
    out.inner = (static_cast<uint64_t>(H - 1) * (H > 1 ? r->head_stride : 0) + p.d) * es;
    out.row = T > 1 && out.inner <= static_cast<uint64_t>(r->row_stride) * es ? r->row_stride * es : 0;
    return !written || rows_apart(stride, size, p.d);
}

Place bytes_at(const void *p, uint64_t n) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return {{b, b + (p == nullptr ? 0 : n)}, 0, 0};
}

// Slices of one wider row, as queries, keys and values of a single projection are, lie between one another
// without sharing memory.
bool meet(const Place &a, const Place &b) {
    if (!spans_meet(a.span, b.span)) return false;
    if (a.row == 0 || a.row != b.row) return true;
    const uint64_t to_b = ((b.span.lo % a.row) + a.row - a.span.lo % a.row) % a.row;  // b's place in the row that begins with a
    return !(a.inner <= to_b && to_b + b.inner <= a.row);
}

// Whether any of what is written meets what is read or something else that is written.
bool apart(const Place *out, int n_out, const Place *in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int k = 0; k < n_in; ++k)
            if (meet(out[i], in[k])) return false;
        for (int k = i + 1; k < n_out; ++k)
            if (meet(out[i], out[k])) return false;
    }
    return true;
}

Rows<const char> in_bytes(const cca_packed_rows_t &r, int dtype) {
    const int es = dtype == CCA_BF16 ? 2 : 4;
    return {static_cast<const char *>(r.p), r.head_stride * es, r.row_stride * es};
}

// Whether heads lie closer than rows (tensors laid out token by token): neighbours then share DRAM pages.
int heads_inside(const cca_packed_rows_t &r) { return r.head_stride < r.row_stride; }

cca_packed_rows_t or_dense(const cca_packed_rows_t &r, int d, int T, int H) {
    // strides of dimensions of one element are never used, but reach the tensor maps: give them room
    cca_packed_rows_t x = r;
    if (T == 1) x.row_stride = d;
    if (H == 1) x.head_stride = static_cast<int64_t>(d) * 8;
    return x;
}

PackedArgs packed_args(const cca_packed_t &pk, const cca_params_t &p) {
    PackedArgs a = {};
    a.plan = plan_of(pk, p.dev_status);
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.d = p.d;
    a.scale = resolve_scale(&p);
    a.pool_mode = p.pool_mode;
    return a;
}

// Tiles of tokens (of all KV heads) an SM up to which long ones are dealt out in halves: the longest item is longer
// than a CTA's mean then.  One sequence of 4 K tokens, 16 heads over 4 (0.9 an SM) 193 -> 132 us, three of 4 K over one
// (0.2) 147 -> 86, six of 8 K over 4 (1.8) 128 -> 115; with 3.5 an SM six of 16 K gain 4% and six of 8 K with 8 heads
// over 8 lose 7%.
constexpr int HALVED_TILES = 2;

inline uint64_t round256(uint64_t n) { return (n + 255) / 256 * 256; }

uint64_t bwd_space(const cca_packed_t &pk, const cca_params_t &p, int sms, char *base, PackedBwdSpace *w) {
    const uint64_t G = pk.T / pk.g, core = 4ull * p.Hkv * G * p.d, tok = 4ull * p.Hkv * pk.T;
    const bool cores = pk.w < pk.T && G > 0;
    uint64_t at = 0;
    auto take = [&](uint64_t n) {
        float *r = base != nullptr ? reinterpret_cast<float *>(base + at) : nullptr;
        at += round256(n);
        return r;
    };
    // The query rows of a core tile are split so that there is an item for every SM (a tile's rows are a serial
    // chain, and its items go to whoever comes); 8 parts at most.  Four items an SM were no faster, and the
    // pooling's gradient adds more parts up (29 us instead of 24 for 16 K tokens).
    int splits = 1;
    if (cores) {
        const int64_t tiles = (static_cast<int64_t>(G) / PACK_TILE + 1) * p.Hkv;
        while (splits < 8 && tiles * splits < sms) splits *= 2;
    }
    PackedBwdSpace s = {};
    s.splits = splits;
    s.D = take(4ull * p.Hq * pk.T);
    s.token_splits = 1;
    if (p.dtype == CCA_BF16) {
        const PlanLayout l = plan_layout(pk.S, pk.T, pk.g);
        const int64_t tiles = static_cast<int64_t>(l.max_tiles) * p.Hkv;
        if (tiles <= HALVED_TILES * sms) s.token_splits = 2;
        s.n_zero = 2 + (s.token_splits == 2 ? static_cast<int>(tiles) * 8 : 0);
        s.taken = reinterpret_cast<int32_t *>(take(4ull * s.n_zero));
        s.there = s.taken + 2;
        if (s.token_splits == 2) s.parts = take(tiles * 2 * 2ull * PACK_TILE * p.d * 4);
    }
    if (cores) {
        s.dKc = take(core * splits);
        s.dVc = take(core * splits);
        s.a = take(tok);
        s.cds = take(tok);
        s.qsum = take(core);
        s.dqs = take(core);
    }
    if (w != nullptr) *w = s;
    return at;
}

}  // namespace
}  // namespace cca

extern "C" {

uint64_t cca_pack_size(int S, int T, int g) {
    if (S < 1 || S > 65535 || T < 1 || g < 1) return 0;
    return cca::plan_layout(S, T, g).bytes;
}

uint64_t cca_pack_positions_offset(int S, int T, int g) {
    if (S < 1 || S > 65535 || T < 1 || g < 1) return 0;
    return cca::plan_layout(S, T, g).positions;
}

int cca_pack(const int32_t *cu_seqlens, const cca_packed_t *packed, int32_t *dev_status, void *stream) {
    using namespace cca;
    if (!packed_ok(packed) || !word_ptr(cu_seqlens, true) || !word_ptr(dev_status, false)) return CCA_ERR_INVALID_ARG;
    const PlanLayout l = plan_layout(packed->S, packed->T, packed->g);
    if (bytes_meet(cu_seqlens, 4ull * (packed->S + 1), packed->plan, l.bytes)) return CCA_ERR_INVALID_ARG;
    if (dev_status != nullptr && bytes_meet(dev_status, 4, packed->plan, l.bytes)) return CCA_ERR_INVALID_ARG;
    const int st = check_device();
    if (st != CCA_OK) return st;
    // blocks of one sequence: a few thousand tokens each
    int y = packed->T / packed->S / 2048 + 1;
    if (packed->S < 64 && y < packed->T / 8192) y = packed->T / 8192;
    if (y > 64) y = 64;
    return from_cuda(start_dependent(pack_kernel, dim3(packed->S, y), PACK_THREADS, 0, static_cast<cudaStream_t>(stream), cu_seqlens,
                                     static_cast<char *>(packed->plan), l, packed->S, packed->T, packed->g, packed->w,
                                     packed->window_mode, dev_status));
}

int cca_pool_packed(const cca_packed_rows_t *Q, const cca_packed_rows_t *K, const cca_packed_rows_t *V, void *Kc, void *Vc,
                    const cca_packed_t *packed, const cca_params_t *params, void *stream) {
    using namespace cca;
    int st = params_packed(params);
    if (st != CCA_OK) return st;
    if (!packed_ok(packed)) return CCA_ERR_INVALID_ARG;
    const cca_params_t &p = *params;
    const int G = packed->T / packed->g;
    Place in[4], out[2];
    if (!rows_ok(Q, p.Hq, packed->T, p, false, in[0]) || !rows_ok(K, p.Hkv, packed->T, p, false, in[1]) ||
        !rows_ok(V, p.Hkv, packed->T, p, false, in[2]))
        return CCA_ERR_INVALID_ARG;
    if (G == 0) return CCA_OK;  // no group fits: nothing to write
    if (Kc == nullptr || Vc == nullptr || ((reinterpret_cast<uintptr_t>(Kc) | reinterpret_cast<uintptr_t>(Vc)) & 15u) != 0)
        return CCA_ERR_INVALID_ARG;
    const uint64_t bytes = static_cast<uint64_t>(p.Hkv) * G * p.d * (p.dtype == CCA_BF16 ? 2 : 4);
    in[3] = bytes_at(packed->plan, packed->plan_bytes);
    out[0] = bytes_at(Kc, bytes);
    out[1] = bytes_at(Vc, bytes);
    if (!apart(out, 2, in, 4)) return CCA_ERR_INVALID_ARG;
    if ((st = check_device()) != CCA_OK) return st;
    PoolPackedArgs a;
    a.Q = in_bytes(*Q, p.dtype);
    a.K = in_bytes(*K, p.dtype);
    a.V = in_bytes(*V, p.dtype);
    a.Kc = static_cast<char *>(Kc);
    a.Vc = static_cast<char *>(Vc);
    a.plan = plan_of(*packed, p.dev_status);
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.mode = p.pool_mode;
    a.heads_first = heads_inside(*K);
    a.scale_log2 = resolve_scale(&p) * 1.4426950408889634f;
    const int64_t blocks = (static_cast<int64_t>(G) * p.Hkv + POOL_WARPS - 1) / POOL_WARPS;
    if (blocks > 0x7fffffff) return CCA_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) { return from_cuda(start_dependent(kernel, grid, POOL_WARPS * 32, 0, s, a)); };
    if (p.dtype == CCA_BF16) return p.d == 128 ? go(pool_packed_kernel<__nv_bfloat16, 128>) : go(pool_packed_kernel<__nv_bfloat16, 64>);
    return p.d == 128 ? go(pool_packed_kernel<float, 128>) : go(pool_packed_kernel<float, 64>);
}

int cca_attn_packed(const cca_packed_rows_t *Q, const cca_packed_rows_t *K, const cca_packed_rows_t *V, const void *Kc,
                    const void *Vc, const cca_packed_rows_t *O, float *LSE, const cca_packed_t *packed,
                    const cca_params_t *params, void *stream) {
    using namespace cca;
    int st = params_packed(params);
    if (st != CCA_OK) return st;
    if (!packed_ok(packed) || !word_ptr(LSE, true)) return CCA_ERR_INVALID_ARG;
    const cca_params_t &p = *params;
    const int T = packed->T, G = T / packed->g;
    Place in[6], out[2];
    if (!rows_ok(Q, p.Hq, T, p, false, in[0]) || !rows_ok(K, p.Hkv, T, p, false, in[1]) || !rows_ok(V, p.Hkv, T, p, false, in[2]) ||
        !rows_ok(O, p.Hq, T, p, true, out[0]))
        return CCA_ERR_INVALID_ARG;
    const uint64_t bytes = static_cast<uint64_t>(p.Hkv) * G * p.d * (p.dtype == CCA_BF16 ? 2 : 4);
    const bool cores = packed->w < T && G > 0;
    if (cores && (Kc == nullptr || Vc == nullptr || ((reinterpret_cast<uintptr_t>(Kc) | reinterpret_cast<uintptr_t>(Vc)) & 15u) != 0))
        return CCA_ERR_INVALID_ARG;
    in[3] = bytes_at(cores ? Kc : nullptr, bytes);
    in[4] = bytes_at(cores ? Vc : nullptr, bytes);
    in[5] = bytes_at(packed->plan, packed->plan_bytes);
    out[1] = bytes_at(LSE, 4ull * p.Hq * T);
    if (!apart(out, 2, in, 6)) return CCA_ERR_INVALID_ARG;
    if ((st = check_device()) != CCA_OK) return st;
    PackedArgs a = packed_args(*packed, p);
    a.Q = or_dense(*Q, p.d, T, p.Hq);
    a.K = or_dense(*K, p.d, T, p.Hkv);
    a.V = or_dense(*V, p.d, T, p.Hkv);
    a.O = or_dense(*O, p.d, T, p.Hq);
    a.Kc = cores ? Kc : nullptr;
    a.Vc = cores ? Vc : nullptr;
    a.LSE = LSE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.dtype == CCA_BF16) return from_cuda(launch_attn_packed_tc(a, s));
    return from_cuda(launch_attn_packed_f32(a, s));
}

int cca_packed_clear(const cca_packed_rows_t *tensors, const int32_t *heads, int n, const cca_packed_t *packed,
                     const cca_params_t *params, void *stream) {
    using namespace cca;
    if (params == nullptr || (params->dtype != CCA_BF16 && params->dtype != CCA_F32)) return CCA_ERR_INVALID_ARG;
    if (!packed_ok(packed) || tensors == nullptr || heads == nullptr || n < 1 || n > 4) return CCA_ERR_INVALID_ARG;
    if (params->d != 64 && params->d != 128) return CCA_ERR_UNSUPPORTED;
    ClearArgs a = {};
    const int es = params->dtype == CCA_BF16 ? 2 : 4;
    Place out[4];
    for (int i = 0; i < n; ++i) {
        if (heads[i] < 1 || heads[i] > 65535 || !rows_ok(&tensors[i], heads[i], packed->T, *params, true, out[i])) return CCA_ERR_INVALID_ARG;
        a.t[i] = {static_cast<char *>(tensors[i].p), tensors[i].head_stride * es, tensors[i].row_stride * es};
        a.heads[i] = heads[i];
    }
    const Place plan = bytes_at(packed->plan, packed->plan_bytes);
    if (!apart(out, n, &plan, 1)) return CCA_ERR_INVALID_ARG;
    const int st = check_device();
    if (st != CCA_OK) return st;
    a.n = n;
    a.chunks = params->d * es / 16;
    a.plan = plan_of(*packed, nullptr);
    return from_cuda(start_dependent(packed_clear_kernel, dim3(2 * device_sms()), 256, 0, static_cast<cudaStream_t>(stream), a));
}

uint64_t cca_packed_bwd_workspace_size(const cca_packed_t *packed, const cca_params_t *params) {
    using namespace cca;
    if (params_packed(params) != CCA_OK || packed == nullptr || packed->S < 1 || packed->T < 1 || packed->g < 1 || packed->w < 1) return 0;
    const int sms = device_sms();
    return sms < 1 ? 0 : bwd_space(*packed, *params, sms, nullptr, nullptr);
}

int cca_packed_bwd(const cca_packed_rows_t *Q, const cca_packed_rows_t *K, const cca_packed_rows_t *V, const void *Kc,
                   const void *Vc, const cca_packed_rows_t *O, const float *LSE, const cca_packed_rows_t *dO,
                   const cca_packed_rows_t *dQ, const cca_packed_rows_t *dK, const cca_packed_rows_t *dV,
                   const cca_packed_t *packed, const cca_params_t *params, void *workspace, uint64_t workspace_bytes,
                   void *stream) {
    using namespace cca;
    int st = params_packed(params);
    if (st != CCA_OK) return st;
    if (!packed_ok(packed) || !word_ptr(LSE, true) || workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return CCA_ERR_INVALID_ARG;
    const cca_params_t &p = *params;
    const int T = packed->T, G = T / packed->g;
    Place in[9], out[4];
    if (!rows_ok(Q, p.Hq, T, p, false, in[0]) || !rows_ok(K, p.Hkv, T, p, false, in[1]) || !rows_ok(V, p.Hkv, T, p, false, in[2]) ||
        !rows_ok(O, p.Hq, T, p, false, in[3]) || !rows_ok(dO, p.Hq, T, p, false, in[4]) || !rows_ok(dQ, p.Hq, T, p, true, out[0]) ||
        !rows_ok(dK, p.Hkv, T, p, true, out[1]) || !rows_ok(dV, p.Hkv, T, p, true, out[2]))
        return CCA_ERR_INVALID_ARG;
    const uint64_t bytes = static_cast<uint64_t>(p.Hkv) * G * p.d * (p.dtype == CCA_BF16 ? 2 : 4);
    const bool cores = packed->w < T && G > 0;
    if (cores && (Kc == nullptr || Vc == nullptr || ((reinterpret_cast<uintptr_t>(Kc) | reinterpret_cast<uintptr_t>(Vc)) & 15u) != 0))
        return CCA_ERR_INVALID_ARG;
    in[5] = bytes_at(cores ? Kc : nullptr, bytes);
    in[6] = bytes_at(cores ? Vc : nullptr, bytes);
    in[7] = bytes_at(packed->plan, packed->plan_bytes);
    in[8] = bytes_at(LSE, 4ull * p.Hq * T);
    if (!apart(out, 3, in, 9)) return CCA_ERR_INVALID_ARG;
    if ((st = check_device()) != CCA_OK) return st;
    const int sms = device_sms();
    if (sms < 1) return CCA_ERR_CUDA;
    PackedBwdSpace w;
    const uint64_t need = bwd_space(*packed, p, sms, static_cast<char *>(workspace), &w);
    if (workspace_bytes < need) return CCA_ERR_INVALID_ARG;
    out[3] = bytes_at(workspace, need);
    if (!apart(out, 4, in, 9)) return CCA_ERR_INVALID_ARG;
    PackedArgs a = packed_args(*packed, p);
    a.Q = or_dense(*Q, p.d, T, p.Hq);
    a.K = or_dense(*K, p.d, T, p.Hkv);
    a.V = or_dense(*V, p.d, T, p.Hkv);
    a.O = or_dense(*O, p.d, T, p.Hq);
    a.dO = or_dense(*dO, p.d, T, p.Hq);
    a.dQ = or_dense(*dQ, p.d, T, p.Hq);
    a.dK = or_dense(*dK, p.d, T, p.Hkv);
    a.dV = or_dense(*dV, p.d, T, p.Hkv);
    a.Kc = cores ? Kc : nullptr;
    a.Vc = cores ? Vc : nullptr;
    a.LSE = const_cast<float *>(LSE);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto part = [&](int k) { return p.dtype == CCA_BF16 ? launch_packed_bwd_tc(a, w, k, s) : launch_packed_bwd_f32(a, w, k, s); };
    auto by_type = [&](auto f) {
        if (p.dtype == CCA_BF16) return p.d == 128 ? f(__nv_bfloat16(), std::integral_constant<int, 128>()) : f(__nv_bfloat16(), std::integral_constant<int, 64>());
        return p.d == 128 ? f(float(), std::integral_constant<int, 128>()) : f(float(), std::integral_constant<int, 64>());
    };
    cudaError_t e = by_type([&](auto t, auto d) {
        using X = decltype(t);
        constexpr int D = decltype(d)::value;
        const int64_t per = D_ROWS * 256 / (D * sizeof(X) / 16), blocks = (static_cast<int64_t>(T) * p.Hq + per - 1) / per;
        if (blocks > 0x7fffffff) return cudaErrorNotSupported;
        return start_dependent(packed_d_kernel<X, D>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, in_bytes(*O, p.dtype),
                               in_bytes(*dO, p.dtype), w.D, a.plan, p.Hq, heads_inside(*O), w.taken, w.n_zero);
    });
    if (e == cudaSuccess && cores) {
        e = part(0);
        PoolBwdArgs b;
        b.Q = in_bytes(*Q, p.dtype);
        b.K = in_bytes(*K, p.dtype);
        b.V = in_bytes(*V, p.dtype);
        b.w = w;
        b.plan = a.plan;
        b.Hq = p.Hq;
        b.Hkv = p.Hkv;
        b.heads_first = heads_inside(*K);
        b.c = a.scale / (p.Hq / p.Hkv);
        if (e == cudaSuccess && p.pool_mode == 1) {
            const int64_t n = (static_cast<int64_t>(p.Hkv) * G * p.d + 255) / 256;
            e = start_dependent(pool_packed_mean_bwd_kernel, dim3(static_cast<unsigned>(n)), 256, 0, s, b, p.d);
        } else if (e == cudaSuccess) {
            const int64_t n = (static_cast<int64_t>(a.plan.max_cores) * PACK_TILE * p.Hkv + POOL_WARPS - 1) / POOL_WARPS;
            if (n > 0x7fffffff) return CCA_ERR_UNSUPPORTED;
            e = by_type([&](auto t, auto d) {
                return start_dependent(pool_packed_bwd_kernel<decltype(t), decltype(d)::value>, dim3(static_cast<unsigned>(n)),
                                       POOL_WARPS * 32, 0, s, b);
            });
        }
    }
    if (e == cudaSuccess) e = part(1);
    if (e == cudaSuccess) e = part(2);
    return from_cuda(e);
}

}  // extern "C"
