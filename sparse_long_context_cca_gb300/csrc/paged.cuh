// Shared by the kernels over paged caches: limits, host-side checks, and the list of keys
// that the nodes of a drafted tree see.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/cca.h"
#include "internal.h"
#include "visibility.cuh"

namespace cca {

// Launches a kernel as a programmatic dependent of what the stream ran before it.  A kernel that allocates
// tensor memory does so before it lets dependents start: one of them could take it first, and wait for it.
template <typename... P, typename... A>
cudaError_t start_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// An error for the caller's status word.  One word may serve all calls of a step: the first error in
// it stays, but a bad argument gives way to what matters more (too few pages, of which a bad argument
// in a later call may be the consequence; a time-out, after which an output is not complete).
__device__ __forceinline__ void report(int32_t *status, int code) {
    if (status == nullptr) return;
    int held = *static_cast<volatile int32_t *>(status);  // many threads may report the same
    if (held == 0) held = atomicCAS(status, 0, code);
    if (held == CCA_ERR_INVALID_ARG && code != held) atomicCAS(status, held, code);
}

constexpr int TREE_MAX_NODES = 256;
constexpr int TREE_MAX_BATCH = 1024;

// Division by a number that the host knows: floor(n / d) for 0 <= n < 2^31 and d < 2^31 is the
// high half of 4n * ceil(2^62 / d), as n * d < 2^62 keeps the rounding of the factor below 1/d.
struct FastDiv {
    uint64_t m;
    __device__ __forceinline__ int div(int n) const { return static_cast<int>(__umul64hi(static_cast<uint64_t>(n) << 2, m)); }
};
inline FastDiv fast_div(int d) { return FastDiv{((uint64_t{1} << 62) + d - 1) / d}; }

// A pool and its table as the ABI wants them (layers 0: any number).
inline bool pages_ok(const cca_pages_t *p, int layers) {
    if (p == nullptr || p->K == nullptr || p->V == nullptr || p->table == nullptr) return false;
    if (((reinterpret_cast<uintptr_t>(p->K) | reinterpret_cast<uintptr_t>(p->V)) & 15u) != 0) return false;
    if ((reinterpret_cast<uintptr_t>(p->table) & 3u) != 0) return false;
    return p->n_pages >= 1 && p->rows >= 1 && p->cols >= 1 && p->layers >= 1 && (layers == 0 || p->layers == layers);
}

inline bool word_ptr(const void *p, bool needed) {
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0 && (p != nullptr || !needed);
}

inline uint64_t pool_bytes(const cca_pages_t *p, const cca_params_t *q) {
    return static_cast<uint64_t>(p->layers) * p->n_pages * p->rows * q->Hkv * q->d * (q->dtype == CCA_BF16 ? 2 : 4);
}

inline bool bytes_meet(const void *p, uint64_t n, const void *q, uint64_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

// Whether what is written (the core pool) lies in what is read, or its K in its V.  One pool
// for both is fine: their tables name different pages.
inline bool pools_meet(const cca_pages_t *raw, const cca_pages_t *core, const cca_params_t *q) {
    const uint64_t r = pool_bytes(raw, q), c = pool_bytes(core, q);
    if (raw->K == core->K && raw->V == core->V && raw->n_pages == core->n_pages && raw->rows == core->rows)
        return bytes_meet(core->K, c, core->V, c);
    return bytes_meet(core->K, c, core->V, c) || bytes_meet(core->K, c, raw->K, r) || bytes_meet(core->K, c, raw->V, r) ||
           bytes_meet(core->V, c, raw->K, r) || bytes_meet(core->V, c, raw->V, r);
}

// cca_params_t for the paged calls: N is not used, w only where asked.
inline int check_paged(const cca_params_t *p, bool need_w) {
    if (p == nullptr) return CCA_ERR_INVALID_ARG;
    if (p->B < 1 || p->Hq < 1 || p->Hkv < 1 || p->d < 1 || p->g < 1 || (need_w && p->w < 1)) return CCA_ERR_INVALID_ARG;
    if (p->Hq % p->Hkv != 0) return CCA_ERR_INVALID_ARG;
    if (p->dtype != CCA_BF16 && p->dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (!(p->scale == p->scale) || isinf(p->scale)) return CCA_ERR_INVALID_ARG;
    if (p->window_mode < 0 || p->window_mode > 1 || p->pool_mode < 0 || p->pool_mode > 3) return CCA_ERR_INVALID_ARG;
    if (!word_ptr(p->dev_status, false)) return CCA_ERR_INVALID_ARG;
    if (p->d != 64 && p->d != 128) return CCA_ERR_UNSUPPORTED;
    return CCA_OK;
}

inline float resolve_scale(const cca_params_t *p) {
    return p->scale > 0.f ? p->scale : 1.0f / sqrtf(static_cast<float>(p->d));
}

}  // namespace cca
