// Shared by the kernels that give queries and keys their rotary positions (rope.cu, norm_rope.cu):
// row accesses, angles, and the host-side checks of strided rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/cca.h"
#include "paged.cuh"

namespace cca {

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

struct Span {
    uintptr_t lo, hi;  // bytes [lo, hi)
};

inline bool spans_meet(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }

// The bytes that a strided [B, H, N, d] tensor touches; false when a row is misaligned.
inline bool span_of(const void *p, const int64_t (&stride)[3], const int64_t (&size)[3], int d, int es, Span &out) {
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
inline bool rows_apart(const int64_t (&stride)[3], const int64_t (&size)[3], int d) {
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

inline bool params_ok(const cca_rope_params_t *p, int &st) {
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

// What cca_rope and cca_norm_rope ask of their tensors (heads already checked): rows aligned, outputs
// whose rows are apart, nothing written that is read, but for a call in place.
inline int check_rope_tensors(const cca_rope_tensor_t *tensors, int n_tensors, const cca_rope_params_t &params) {
    const int es = params.dtype == CCA_BF16 ? 2 : 4;
    Span x[2], y[2];
    bool in_place[2];
    for (int i = 0; i < n_tensors; ++i) {
        const cca_rope_tensor_t &t = tensors[i];
        const int64_t size[3] = {params.B, t.H, params.N};
        if (!span_of(t.x, t.x_stride, size, params.d, es, x[i]) || !span_of(t.y, t.y_stride, size, params.d, es, y[i]))
            return CCA_ERR_INVALID_ARG;
        if (!rows_apart(t.y_stride, size, params.d)) return CCA_ERR_INVALID_ARG;
        in_place[i] = t.x == t.y;
        for (int k = 0; k < 3; ++k)
            if (size[k] > 1 && t.x_stride[k] != t.y_stride[k]) in_place[i] = false;
        if (!in_place[i] && spans_meet(x[i], y[i])) return CCA_ERR_INVALID_ARG;
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
            const int inner = params.N > 1 ? 2 : 0;  // the dimension that steps from token to token
            const int64_t token = f->x_stride[inner];
            apart = token == g->x_stride[inner] &&
                    (params.N == 1 || params.B == 1 ||
                     (f->x_stride[0] == g->x_stride[0] && f->x_stride[0] >= token * params.N)) &&
                    gap >= (f->H - 1) * f->x_stride[1] + params.d &&
                    gap + (g->H - 1) * g->x_stride[1] + params.d <= token;
        }
        if (!apart) return CCA_ERR_INVALID_ARG;
    }
    return CCA_OK;
}

// What cca_rope_append and cca_norm_rope_append ask of theirs (params_ok already).
inline int check_append(const cca_rope_tensor_t *q, const cca_rope_tensor_t *k, const cca_rope_tensor_t *v,
                        const cca_pages_t *raw, const int32_t *lens, const int32_t *parents, const int32_t *counts,
                        const int32_t *dev_status, const cca_rope_params_t &params) {
    if (params.positions != nullptr || params.pos_stride != 0 || params.start != 0 || params.inverse != 0)
        return CCA_ERR_INVALID_ARG;
    if (k == nullptr || v == nullptr || k->H < 1 || k->H > (1 << 20) || v->H != k->H) return CCA_ERR_INVALID_ARG;
    if (!pages_ok(raw, 1) || lens == nullptr || params.B > 65535) return CCA_ERR_INVALID_ARG;
    const void *words[4] = {lens, parents, counts, dev_status};
    for (const void *p : words)
        if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return CCA_ERR_INVALID_ARG;
    if (parents != nullptr && params.N > TREE_MAX_NODES) return CCA_ERR_UNSUPPORTED;
    const int es = params.dtype == CCA_BF16 ? 2 : 4;
    const uint64_t pool = static_cast<uint64_t>(raw->n_pages) * raw->rows * k->H * params.d * es;
    const Span kp = {reinterpret_cast<uintptr_t>(raw->K), reinterpret_cast<uintptr_t>(raw->K) + pool};
    const Span vp = {reinterpret_cast<uintptr_t>(raw->V), reinterpret_cast<uintptr_t>(raw->V) + pool};
    if (spans_meet(kp, vp)) return CCA_ERR_INVALID_ARG;
    Span y = {};
    const cca_rope_tensor_t *in[3] = {q, k, v};
    for (int i = 0; i < 3; ++i) {
        if (in[i] == nullptr) continue;
        Span x;
        const int64_t size[3] = {params.B, in[i]->H, params.N};
        if (in[i]->H < 1 || in[i]->H > (1 << 20) || !span_of(in[i]->x, in[i]->x_stride, size, params.d, es, x)) return CCA_ERR_INVALID_ARG;
        if (i == 0) {
            if (!span_of(q->y, q->y_stride, size, params.d, es, y) || !rows_apart(q->y_stride, size, params.d))
                return CCA_ERR_INVALID_ARG;
            bool same = q->x == q->y;
            for (int s = 0; s < 3; ++s)
                if (size[s] > 1 && q->x_stride[s] != q->y_stride[s]) same = false;
            if ((!same && spans_meet(x, y)) || spans_meet(y, kp) || spans_meet(y, vp)) return CCA_ERR_INVALID_ARG;
        } else if (q != nullptr && spans_meet(x, y)) {
            return CCA_ERR_INVALID_ARG;
        }
        if (spans_meet(x, kp) || spans_meet(x, vp)) return CCA_ERR_INVALID_ARG;
    }
    return CCA_OK;
}

}  // namespace cca
