// Pooling of newly completed groups over paged caches (pooling equation of the Method
// section): the g raw rows of a group, wherever its pages lie, become one core row in the
// core tokens' pages, weighted by the softmax of the group-last query's logits.
//
// Memory-bound: every K and V row of the group is read once.  D*sizeof(T)/16 lanes hold one
// row's 16-byte chunks, so a warp works on 32/that rows at a time, under one running
// (max, sum) per lane group that is merged at the end.
//
// pool_pages_ring_kernel: a warp takes several groups of one (b, KV head) in turn through a
// ring of its own in shared memory, so that copies are always under way: the queries, keys and
// values of the next group, and the page entries of the one after.  A group is a chain of dots,
// shuffles and exponentials, so warps count for more than stages: a 32 K prompt of 32 heads
// (g = 16, d = 128, bf16) takes 108 us with 12 warps of two stages (5.4 TB/s; 124 us with 8 warps
// of three, 170 us from global memory).
// pool_pages_kernel: one warp per group straight from global memory, for groups that do not
// fit the ring (RING_BYTES for a group's rows of K and V and its r query rows: with r = 1 and
// d = 128 up to g = 56 in bf16, 27 in fp32) and for the pooling modes that read the rows more than
// once or no queries.  A 32 K prompt of 32 heads, d = 128: bf16, g = 64 122 us (its bytes: 82), fp32,
// g = 32 192 us (168).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/cca.h"
#include "internal.h"
#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace cca {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int PP_WARPS = 4;
constexpr int PP_UNROLL = 4;
constexpr int PP_HEADS_MAX = 8;

template <typename T>
struct Row;
template <>
struct Row<__nv_bfloat16> {
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
struct Row<float> {
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

struct PoolPagesArgs {
    const void *Q;
    const void *K, *V;  // raw pool
    void *Kc, *Vc;      // core pool
    const int32_t *table, *ctable, *lens, *accepted, *path;
    int n_pages, rows, cols, n_cpages, crows, ccols;
    int B, Hq, Hkv, T, A, g, mode, slots;  // slots: groups a sequence may complete
    FastDiv by_g, by_rows, by_crows;
    float scale_log2;
    int32_t *status;
};

template <typename T, int D>
__global__ void __launch_bounds__(PP_WARPS * 32) pool_pages_kernel(const PoolPagesArgs a) {
    using RT = Row<T>;
    constexpr int E = RT::E;
    constexpr int LPR = D / E;     // lanes per row
    constexpr int RPI = 32 / LPR;  // rows per warp-wide step
    __shared__ float2 sm_head[PP_WARPS][PP_HEADS_MAX];
    const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
    const int sub = lane / LPR, cl = lane % LPR;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * PP_WARPS + wib;
    const int64_t bk = item / a.slots;
    if (bk >= static_cast<int64_t>(a.B) * a.Hkv) return;
    const int b = static_cast<int>(bk / a.Hkv), kv = static_cast<int>(bk - static_cast<int64_t>(b) * a.Hkv);
    const int r = a.Hq / a.Hkv;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int len = a.lens[b], got = a.accepted[b];
    if (len < 0 || got < 0 || got > a.A || got > 0x7fffffff - len) {
        if (lane == 0) report(a.status, CCA_ERR_INVALID_ARG);
        return;
    }
    const int64_t j = len / a.g + (item - bk * a.slots);
    const int64_t end = (j + 1) * a.g;
    if (end > static_cast<int64_t>(len) + got) return;
    // the group-last token's query, its core row, its raw rows
    const int last = static_cast<int>(end - 1 - len);
    const int node = a.path != nullptr ? a.path[static_cast<int64_t>(b) * a.A + last] : last;
    const int64_t cc = j / a.crows;
    const int cpage = cc < a.ccols ? a.ctable[static_cast<int64_t>(b) * a.ccols + cc] : -1;
    bool ok = node >= 0 && node < a.T && cpage >= 0 && cpage < a.n_cpages;
    const int64_t first = j * a.g;
    const int64_t c0 = first / a.rows, c1 = (end - 1) / a.rows;
    for (int64_t c = c0 + lane; c <= c1; c += 32) {
        const int p = c < a.cols ? a.table[static_cast<int64_t>(b) * a.cols + c] : -1;
        if (p < 0 || p >= a.n_pages) ok = false;
    }
    if (!__all_sync(kFull, ok)) {
        if (lane == 0) report(a.status, CCA_ERR_INVALID_ARG);
        return;
    }
    const T *Kp = static_cast<const T *>(a.K) + cl * E, *Vp = static_cast<const T *>(a.V) + cl * E;
    const int64_t page0 = a.table[static_cast<int64_t>(b) * a.cols + c0];
    auto row_at = [&](int t) {  // element offset of group row t in the pool
        const int64_t x = first + t;
        const int64_t c = c0 == c1 ? c0 : x / a.rows;
        const int64_t page = c0 == c1 ? page0 : a.table[static_cast<int64_t>(b) * a.cols + c];
        return ((page * a.Hkv + kv) * a.rows + (x - c * a.rows)) * D;
    };
    auto load = [](const T *p) { return *reinterpret_cast<const uint4 *>(p); };
    const T *q = static_cast<const T *>(a.Q) + ((static_cast<int64_t>(b) * a.Hq + kv * r) * a.T + node) * D + cl * E;
    auto query = [&](int h, float (&f)[E]) { RT::unpack(load(q + static_cast<int64_t>(h) * a.T * D), f); };
    const bool by_max = a.mode == 2, by_mean = a.mode == 1, per_head = a.mode == 3;
    float qs[E];
#pragma unroll
    for (int e = 0; e < E; ++e) qs[e] = 0.f;
    if (a.mode == 0)
        for (int h = 0; h < r; ++h) {
            float f[E];
            query(h, f);
#pragma unroll
            for (int e = 0; e < E; ++e) qs[e] += f[e];
        }
    auto dot = [&](const float (&x)[E], const float (&y)[E]) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(x[e], y[e], s);
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
        return s;
    };
    if (per_head) {
        // each head's normaliser over the group: (max, sum) in the log2 domain
        for (int h = 0; h < r; ++h) {
            float qf[E], m = -INFINITY, l = 0.f;
            query(h, qf);
            for (int t0 = 0; t0 < a.g; t0 += RPI) {
                const int t = t0 + sub;
                float kf[E];
                RT::unpack(t < a.g ? load(Kp + row_at(t)) : make_uint4(0, 0, 0, 0), kf);
                const float x = dot(qf, kf) * a.scale_log2;
                if (t < a.g) {
                    const float mn = fmaxf(m, x);
                    l = l * ptx::ex2(m - mn) + ptx::ex2(x - mn);
                    m = mn;
                }
            }
#pragma unroll
            for (int off = LPR; off < 32; off <<= 1) {
                const float mo = __shfl_xor_sync(kFull, m, off), lo = __shfl_xor_sync(kFull, l, off);
                const float mn = fmaxf(m, mo);
                l = l * (m == -INFINITY ? 0.f : ptx::ex2(m - mn)) + lo * (mo == -INFINITY ? 0.f : ptx::ex2(mo - mn));
                m = mn;
            }
            if (lane == 0) sm_head[wib][h] = make_float2(m, 1.f / (l * static_cast<float>(r)));
        }
        __syncwarp();
    }
    const float init = by_max ? -INFINITY : 0.f;
    float m = -INFINITY, l = 0.f, ak[E], av[E];
#pragma unroll
    for (int e = 0; e < E; ++e) ak[e] = av[e] = init;
    for (int t0 = 0; t0 < a.g; t0 += RPI * PP_UNROLL) {
        uint4 kk[PP_UNROLL], vv[PP_UNROLL];
#pragma unroll
        for (int u = 0; u < PP_UNROLL; ++u) {
            const int t = t0 + u * RPI + sub;
            kk[u] = vv[u] = make_uint4(0, 0, 0, 0);
            if (t < a.g) {
                const int64_t at = row_at(t);
                kk[u] = load(Kp + at);
                vv[u] = load(Vp + at);
            }
        }
#pragma unroll
        for (int u = 0; u < PP_UNROLL; ++u) {
            const int t = t0 + u * RPI + sub;
            float kf[E], vf[E];
            RT::unpack(kk[u], kf);
            RT::unpack(vv[u], vf);
            if (by_max) {
                if (t < a.g) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        ak[e] = fmaxf(ak[e], kf[e]);
                        av[e] = fmaxf(av[e], vf[e]);
                    }
                }
                continue;
            }
            if (per_head) {
                float p = 0.f;
                for (int h = 0; h < r; ++h) {
                    float qf[E];
                    query(h, qf);
                    const float2 st = sm_head[wib][h];
                    p = fmaf(ptx::ex2(dot(qf, kf) * a.scale_log2 - st.x), st.y, p);
                }
                if (t < a.g) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        ak[e] = fmaf(p, kf[e], ak[e]);
                        av[e] = fmaf(p, vf[e], av[e]);
                    }
                }
                continue;
            }
            const float x = by_mean ? 0.f : dot(qs, kf) * a.scale_log2;
            if (t < a.g) {
                const float mn = fmaxf(m, x);
                const float corr = ptx::ex2(m - mn), p = ptx::ex2(x - mn);
                l = l * corr + p;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ak[e] = fmaf(p, kf[e], ak[e] * corr);
                    av[e] = fmaf(p, vf[e], av[e] * corr);
                }
                m = mn;
            }
        }
    }
    // the warp's lane groups hold every RPI-th row
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
        float ca = 1.f, cb = 1.f;
        if (!by_max && !per_head) {
            const float mo = __shfl_xor_sync(kFull, m, off), lo = __shfl_xor_sync(kFull, l, off);
            const float mn = fmaxf(m, mo);
            ca = m == -INFINITY ? 0.f : ptx::ex2(m - mn);
            cb = mo == -INFINITY ? 0.f : ptx::ex2(mo - mn);
            l = l * ca + lo * cb;
            m = mn;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float ko = __shfl_xor_sync(kFull, ak[e], off), vo = __shfl_xor_sync(kFull, av[e], off);
            ak[e] = by_max ? fmaxf(ak[e], ko) : ak[e] * ca + ko * cb;
            av[e] = by_max ? fmaxf(av[e], vo) : av[e] * ca + vo * cb;
        }
    }
    if (!by_max && !per_head) {
        const float inv = 1.f / l;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            ak[e] *= inv;
            av[e] *= inv;
        }
    }
    if (sub == 0) {
        const int64_t at = ((static_cast<int64_t>(cpage) * a.Hkv + kv) * a.crows + (j - cc * a.crows)) * D + cl * E;
        *reinterpret_cast<uint4 *>(static_cast<T *>(a.Kc) + at) = RT::pack(ak);
        *reinterpret_cast<uint4 *>(static_cast<T *>(a.Vc) + at) = RT::pack(av);
    }
}

// ---------------------------------------------------------------- softmax pooling through a ring

constexpr int RING_SMEM = 226 * 1024;
constexpr int RING_MAX_WARPS = 12, RING_MIN_WARPS = 4;
constexpr int RING_STAGES = 2;
constexpr int RING_BYTES = RING_SMEM / (RING_MIN_WARPS * RING_STAGES);  // of a stage, at most

__device__ __forceinline__ void ring_copy(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Stage: the r heads' queries, then K [g][D], then V [g][D].
template <typename T, int D>
__global__ void __launch_bounds__(RING_MAX_WARPS * 32) pool_pages_ring_kernel(const PoolPagesArgs a, const int per_warp, const int parts,
                                                                          const int stage_bytes) {
    using RT = Row<T>;
    constexpr int E = RT::E;
    constexpr int LPR = D / E;
    constexpr int RPI = 32 / LPR;
    constexpr int ROW = D * static_cast<int>(sizeof(T));
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
    const int sub = lane / LPR, cl = lane % LPR;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + wib;
    const int64_t bk = w / parts;
    if (bk >= static_cast<int64_t>(a.B) * a.Hkv) return;
    const int b = static_cast<int>(bk / a.Hkv), kv = static_cast<int>(bk - static_cast<int64_t>(b) * a.Hkv);
    const int r = a.Hq / a.Hkv;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int len = a.lens[b], got = a.accepted[b];
    if (len < 0 || got < 0 || got > a.A || got > 0x7fffffff - len) {
        if (lane == 0) report(a.status, CCA_ERR_INVALID_ARG);
        return;
    }
    const int64_t begin = a.by_g.div(len) + (w - bk * parts) * static_cast<int64_t>(per_warp);
    const int64_t end = min(static_cast<int64_t>(a.by_g.div(len + got)), begin + per_warp);
    if (begin >= end) return;
    const int j0 = static_cast<int>(begin), j1 = static_cast<int>(end);  // rows of groups below j1 fit 31 bits
    const uint32_t ring = ptx::smem_addr(smem) + static_cast<uint32_t>(wib) * RING_STAGES * stage_bytes;
    unsigned char *const mem = smem + wib * RING_STAGES * stage_bytes;
    const int32_t *table = a.table + static_cast<int64_t>(b) * a.cols;

    // What group j's copies need: the page of the lane's first row, its query's node, its core row
    // (-1: reported and skipped).  A lane copies chunk cl of rows sub, sub + RPI, ...
    struct Where {
        int page, node, cpage;
    };
    auto look_up = [&](int j) {
        Where p = {-1, -1, -1};
        if (j >= j1) return p;
        const int last = (j + 1) * a.g - 1 - len;
        p.node = a.path != nullptr ? a.path[static_cast<int64_t>(b) * a.A + last] : last;
        const int cc = a.by_crows.div(j), c = a.by_rows.div(j * a.g);
        p.cpage = cc < a.ccols ? a.ctable[static_cast<int64_t>(b) * a.ccols + cc] : -1;
        p.page = c < a.cols ? table[c] : -1;
        return p;
    };
    // Starts group j's copies; the group's core page, or -1 when something is not there.
    auto fill = [&](int j, const Where &p) {
        int core = -1;
        if (j < j1) {
            const int first = j * a.g, c0 = a.by_rows.div(first);
            bool ok = p.node >= 0 && p.node < a.T && p.cpage >= 0 && p.cpage < a.n_cpages && p.page >= 0 && p.page < a.n_pages;
            const uint32_t dst = ring + static_cast<uint32_t>(j - j0) % RING_STAGES * stage_bytes;
            const bool one_page = first + a.g <= static_cast<int64_t>(c0 + 1) * a.rows;
            // row t of the group, as an element offset of the pool; -1 where no page is
            auto at = [&](int t) -> int64_t {
                const int x = first + t, c = one_page ? c0 : a.by_rows.div(x);
                const int page = c == c0 ? p.page : c < a.cols ? table[c] : -1;
                if (page < 0 || page >= a.n_pages) return -1;
                return ((static_cast<int64_t>(page) * a.Hkv + kv) * a.rows + (x - c * a.rows)) * D;
            };
            if (!one_page)
                for (int t = sub; t < a.g; t += RPI) ok = ok && at(t) >= 0;
            ok = __all_sync(kFull, ok);
            if (ok) {
                const T *q = static_cast<const T *>(a.Q) + ((static_cast<int64_t>(b) * a.Hq + kv * r) * a.T + p.node) * D + cl * E;
                for (int h = sub; h < r; h += RPI) ring_copy(dst + h * ROW + cl * 16, q + static_cast<int64_t>(h) * a.T * D);
                const uint32_t kd = dst + r * ROW + cl * 16, vd = kd + a.g * ROW;
                const int64_t row0 = at(0);
                for (int t = sub; t < a.g; t += RPI) {
                    const int64_t row = (one_page ? row0 + static_cast<int64_t>(t) * D : at(t)) + cl * E;
                    ring_copy(kd + t * ROW, static_cast<const T *>(a.K) + row);
                    ring_copy(vd + t * ROW, static_cast<const T *>(a.V) + row);
                }
                core = p.cpage;
            } else if (lane == 0) {
                report(a.status, CCA_ERR_INVALID_ARG);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return core;
    };
    int core[RING_STAGES];
#pragma unroll
    for (int i = 0; i < RING_STAGES - 1; ++i) core[i] = fill(j0 + i, look_up(j0 + i));
    Where next = look_up(j0 + RING_STAGES - 1);
    for (int j = j0; j < j1; ++j) {
        core[RING_STAGES - 1] = fill(j + RING_STAGES - 1, next);
        next = look_up(j + RING_STAGES);
        asm volatile("cp.async.wait_group %0;" ::"n"(RING_STAGES - 1) : "memory");
        __syncwarp();
        if (core[0] >= 0) {
            const unsigned char *st = mem + static_cast<unsigned>(j - j0) % RING_STAGES * stage_bytes + cl * 16;
            auto chunk = [&](int row, float (&f)[E]) { RT::unpack(*reinterpret_cast<const uint4 *>(st + row * ROW), f); };
            float qs[E];
#pragma unroll
            for (int e = 0; e < E; ++e) qs[e] = 0.f;
            for (int h = 0; h < r; ++h) {
                float f[E];
                chunk(h, f);
#pragma unroll
                for (int e = 0; e < E; ++e) qs[e] += f[e];
            }
            float m = -INFINITY, l = 0.f, ak[E], av[E];
#pragma unroll
            for (int e = 0; e < E; ++e) ak[e] = av[e] = 0.f;
            for (int t0 = 0; t0 < a.g; t0 += RPI * PP_UNROLL) {
                float kf[PP_UNROLL][E], x[PP_UNROLL], mn = m;
#pragma unroll
                for (int u = 0; u < PP_UNROLL; ++u) {
                    const int t = t0 + u * RPI + sub;
                    chunk(r + min(t, a.g - 1), kf[u]);
                    float s = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) s = fmaf(qs[e], kf[u][e], s);
#pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
                    x[u] = t < a.g ? s * a.scale_log2 : -INFINITY;
                    mn = fmaxf(mn, x[u]);
                }
                const float base = mn == -INFINITY ? 0.f : mn;
                const float corr = ptx::ex2(m - base);
                m = mn;
                l *= corr;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ak[e] *= corr;
                    av[e] *= corr;
                }
#pragma unroll
                for (int u = 0; u < PP_UNROLL; ++u) {
                    const int t = t0 + u * RPI + sub;
                    if (t < a.g) {
                        const float p = ptx::ex2(x[u] - base);
                        float vf[E];
                        chunk(r + a.g + t, vf);
                        l += p;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            ak[e] = fmaf(p, kf[u][e], ak[e]);
                            av[e] = fmaf(p, vf[e], av[e]);
                        }
                    }
                }
            }
#pragma unroll
            for (int off = LPR; off < 32; off <<= 1) {
                const float mo = __shfl_xor_sync(kFull, m, off), lo = __shfl_xor_sync(kFull, l, off);
                const float mn = fmaxf(m, mo);
                const float ca = m == -INFINITY ? 0.f : ptx::ex2(m - mn), cb = mo == -INFINITY ? 0.f : ptx::ex2(mo - mn);
                l = l * ca + lo * cb;
                m = mn;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ak[e] = ak[e] * ca + __shfl_xor_sync(kFull, ak[e], off) * cb;
                    av[e] = av[e] * ca + __shfl_xor_sync(kFull, av[e], off) * cb;
                }
            }
            const float inv = 1.f / l;
            if (sub == 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ak[e] *= inv;
                    av[e] *= inv;
                }
                const int64_t at = ((static_cast<int64_t>(core[0]) * a.Hkv + kv) * a.crows + (j - a.by_crows.div(j) * a.crows)) * D + cl * E;
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.Kc) + at) = RT::pack(ak);
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.Vc) + at) = RT::pack(av);
            }
        }
#pragma unroll
        for (int i = 0; i + 1 < RING_STAGES; ++i) core[i] = core[i + 1];
        __syncwarp();  // the stage has been read
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, int D>
cudaError_t launch_ring(const PoolPagesArgs &a, cudaStream_t stream) {
    const int stage = (a.Hq / a.Hkv + 2 * a.g) * D * static_cast<int>(sizeof(T));
    int warps_per_block = RING_SMEM / (stage * RING_STAGES);
    if (warps_per_block > RING_MAX_WARPS) warps_per_block = RING_MAX_WARPS;
    const int smem = stage * RING_STAGES * warps_per_block;
    static std::atomic<int> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev].load(std::memory_order_relaxed) == 0) {
        e = cudaFuncSetAttribute(pool_pages_ring_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(1, std::memory_order_relaxed);
    }
    const int sms = device_sms();
    if (sms < 1) return cudaErrorNoDevice;
    // One wave: as many groups per warp as it takes for every resident warp to have one run.
    int blocks_per_sm = (227 * 1024) / (smem + 1024);
    if (blocks_per_sm > 2) blocks_per_sm = 2;
    const int64_t warps = static_cast<int64_t>(sms) * blocks_per_sm * warps_per_block, lists = static_cast<int64_t>(a.B) * a.Hkv;
    int64_t per_warp = (lists * a.slots + warps - 1) / warps;
    if (per_warp > a.slots) per_warp = a.slots;
    const int64_t parts = (a.slots + per_warp - 1) / per_warp;
    if (lists * parts < static_cast<int64_t>(sms) * warps_per_block)  // few lists: spread over the SMs
        warps_per_block = static_cast<int>((lists * parts + sms - 1) / sms);
    const int64_t blocks = (lists * parts + warps_per_block - 1) / warps_per_block;
    if (blocks > 0x7fffffff) return cudaErrorNotSupported;
    return start_dependent(pool_pages_ring_kernel<T, D>, dim3(static_cast<unsigned>(blocks)), warps_per_block * 32, smem, stream, a,
                           static_cast<int>(per_warp), static_cast<int>(parts), stage);
}

}  // namespace
}  // namespace cca

extern "C" int cca_pool_pages(const void *Q, const cca_pages_t *raw, const cca_pages_t *core, const int32_t *lens,
                              const int32_t *accepted, const int32_t *path, int A, int T, const cca_params_t *params,
                              void *stream) {
    using namespace cca;
    int st = check_paged(params, false);
    if (st != CCA_OK) return st;
    if (params->pool_mode == 3 && params->Hq / params->Hkv > PP_HEADS_MAX) return CCA_ERR_UNSUPPORTED;
    if (!pages_ok(raw, 1) || !pages_ok(core, 1) || pools_meet(raw, core, params)) return CCA_ERR_INVALID_ARG;
    if (Q == nullptr || (reinterpret_cast<uintptr_t>(Q) & 15u) != 0) return CCA_ERR_INVALID_ARG;
    if (!word_ptr(lens, true) || !word_ptr(accepted, true) || !word_ptr(path, false)) return CCA_ERR_INVALID_ARG;
    if (A < 1 || T < 1 || (path == nullptr && A != T)) return CCA_ERR_INVALID_ARG;
    PoolPagesArgs a;
    a.Q = Q;
    a.K = raw->K;
    a.V = raw->V;
    a.Kc = core->K;
    a.Vc = core->V;
    a.table = raw->table;
    a.ctable = core->table;
    a.lens = lens;
    a.accepted = accepted;
    a.path = path;
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
    a.A = A;
    a.g = params->g;
    a.mode = params->pool_mode;
    a.slots = (A - 1) / params->g + 1;
    a.by_g = fast_div(params->g);
    a.by_rows = fast_div(raw->rows);
    a.by_crows = fast_div(core->rows);
    a.status = params->dev_status;
    // mode 0 scores with the sum of the heads' queries, so the mean is in the scale
    const float heads = params->pool_mode == 0 ? static_cast<float>(params->Hq / params->Hkv) : 1.f;
    a.scale_log2 = resolve_scale(params) * 1.4426950408889634f / heads;
    const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * a.slots;
    const int64_t blocks = (items + PP_WARPS - 1) / PP_WARPS;
    if (blocks > 0x7fffffff) return CCA_ERR_UNSUPPORTED;
    if ((st = check_device()) != CCA_OK) return st;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    const int64_t stage = (static_cast<int64_t>(params->Hq / params->Hkv) + 2ll * params->g) * params->d * (params->dtype == CCA_BF16 ? 2 : 4);
    if (params->pool_mode == 0 && stage <= RING_BYTES) {
        if (params->dtype == CCA_BF16)
            return from_cuda(params->d == 128 ? launch_ring<__nv_bfloat16, 128>(a, strm) : launch_ring<__nv_bfloat16, 64>(a, strm));
        return from_cuda(params->d == 128 ? launch_ring<float, 128>(a, strm) : launch_ring<float, 64>(a, strm));
    }
    const dim3 grid(static_cast<unsigned>(blocks));
    constexpr int threads = PP_WARPS * 32;
    if (params->dtype == CCA_BF16)
        return from_cuda(params->d == 128 ? start_dependent(pool_pages_kernel<__nv_bfloat16, 128>, grid, threads, 0, strm, a)
                                          : start_dependent(pool_pages_kernel<__nv_bfloat16, 64>, grid, threads, 0, strm, a));
    return from_cuda(params->d == 128 ? start_dependent(pool_pages_kernel<float, 128>, grid, threads, 0, strm, a)
                                      : start_dependent(pool_pages_kernel<float, 64>, grid, threads, 0, strm, a));
}
