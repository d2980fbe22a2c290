// Packed sequences: the plan that cca_pack makes of a batch's lengths, as the kernels read it, and
// what the kernels over packed tensors share.
//
// A plan holds three lists of tiles, one entry {first row, length, tile of the sequence, first core row}
// each: tiles of 256 query rows, tiles of 128 rows, and tiles of 128 visible cores.  A list runs through
// the tile numbers from the highest down, and through the sequences that have such a tile from the longest
// down.  A row's cost rises with its position (more cores, more of the window), so for tiles of
// queries that is heaviest first; a key's cost rises with the rows behind it, so kernels over keys read
// the lists with the tile number counted from the sequence's end.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/cca.h"
#include "internal.h"
#include "paged.cuh"
#include "visibility.cuh"

namespace cca {

constexpr int PACK_PAIR = 256, PACK_TILE = 128;  // rows of an entry
constexpr int PACK_HEADER = 16;                  // words
constexpr int PACK_MAGIC = 0x43504b31;

struct PlanLayout {  // bytes from the plan's start
    uint64_t pairs, tiles, cores, positions, first, bytes;
    int max_pairs, max_tiles, max_cores;
};
inline PlanLayout plan_layout(int S, int T, int g) {
    PlanLayout l;
    l.max_pairs = T / PACK_PAIR + S;
    l.max_tiles = T / PACK_TILE + S;
    l.max_cores = T / g / PACK_TILE + S;
    l.pairs = 4 * PACK_HEADER;
    l.tiles = l.pairs + 16ull * l.max_pairs;
    l.cores = l.tiles + 16ull * l.max_tiles;
    l.positions = l.cores + 16ull * l.max_cores;
    l.first = l.positions + (4ull * T + 15) / 16 * 16;
    l.bytes = l.first + (4ull * (T / g) + 15) / 16 * 16;
    return l;
}

// What kernels take of a plan.
struct Plan {
    const int4 *pairs, *tiles, *cores;
    const int32_t *header, *first;
    int S, T, G, g, w, window_mode;
    int max_pairs, max_tiles, max_cores;
    int32_t *status;
    FastDiv by_g;
    // visibility.cuh's, with a division that the host has prepared
    __device__ __forceinline__ int cores_of(int i) const { return by_g.div(window_lo(i, w)); }
    __device__ __forceinline__ int start_of(int i) const {
        const int lo = window_lo(i, w);
        return window_mode ? by_g.div(lo) * g : lo;
    }
    __device__ __forceinline__ int seen_of(int n) const { return n > w ? by_g.div(n - w) : 0; }
};
inline Plan plan_of(const cca_packed_t &p, int32_t *status) {
    const PlanLayout l = plan_layout(p.S, p.T, p.g);
    const char *base = static_cast<const char *>(p.plan);
    Plan r;
    r.header = reinterpret_cast<const int32_t *>(base);
    r.pairs = reinterpret_cast<const int4 *>(base + l.pairs);
    r.tiles = reinterpret_cast<const int4 *>(base + l.tiles);
    r.cores = reinterpret_cast<const int4 *>(base + l.cores);
    r.first = reinterpret_cast<const int32_t *>(base + l.first);
    r.S = p.S;
    r.T = p.T;
    r.G = p.T / p.g;
    r.g = p.g;
    r.w = p.w;
    r.window_mode = p.window_mode;
    r.max_pairs = l.max_pairs;
    r.max_tiles = l.max_tiles;
    r.max_cores = l.max_cores;
    r.status = status;
    r.by_g = fast_div(p.g);
    return r;
}

// Entries of the lists (x: pairs, y: tiles, z: core tiles); -1 for a plan that is not the call's.
__device__ __forceinline__ int3 plan_counts(const Plan &p) {
    const int4 a = *reinterpret_cast<const int4 *>(p.header), b = *reinterpret_cast<const int4 *>(p.header + 4),
               c = *reinterpret_cast<const int4 *>(p.header + 8);
    if (a.x != PACK_MAGIC || a.y != p.T || a.z != p.g || a.w != p.w || b.x != p.window_mode || b.y != p.S) {
        if (threadIdx.x == 0) report(p.status, CCA_ERR_INVALID_ARG);
        return make_int3(-1, -1, -1);
    }
    return make_int3(min(c.x, p.max_pairs), min(c.y, p.max_tiles), min(c.z, p.max_cores));
}

// Where the entries of pairs[] of sequences of at most 128, 64 and 32 tokens begin (there are one each, and
// they come last).
__device__ __forceinline__ int3 plan_short(const Plan &p) {
    const int4 d = *reinterpret_cast<const int4 *>(p.header + 12);
    return make_int3(d.x, d.y, d.z);
}

// The item of a persistent CTA in its round-th turn (n or more: none).  Lists run from heavy to light, so the CTAs
// go through them to and fro: straight rounds would give the first CTA the heaviest item of each.  Where the third
// round is the last and does not reach every CTA, it begins at the last one: with few items their costs fall
// steeply, and the first CTA's first item outweighs the light one that it has had since (32 prompts with one of
// 648 tokens: 19.2 us instead of 22.9; with many rounds it is a loss, 466 against 461 us for 12 long prompts; a last
// fifth round, to which the same would apply, was not measured).
__device__ __forceinline__ int item_of_round(int round, int n = 0x7fffffff) {
    const bool back = (round & 1) != 0 || (round == 2 && n < 3 * static_cast<int>(gridDim.x));
    return round * gridDim.x + (back ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Cores that any row of a sequence of n tokens sees: (j + 1) * g <= n - w.
__host__ __device__ __forceinline__ int seen_cores(int n, int w, int g) { return n > w ? (n - w) / g : 0; }

// A packed tensor in a kernel: strides in elements.
template <typename T>
struct Rows {
    T *p;
    int64_t head, row;
    __device__ __forceinline__ T *at(int h, int64_t r) const { return p + h * head + r * row; }
};
template <typename T>
inline Rows<T> rows_of(const cca_packed_rows_t &r) {
    return {static_cast<T *>(r.p), r.head_stride, r.row_stride};
}

struct PackedArgs {  // of a call, checked
    cca_packed_rows_t Q, K, V, O, dO, dQ, dK, dV;
    const void *Kc, *Vc;
    float *LSE;
    Plan plan;
    int Hq, Hkv, d;
    float scale;
    int pool_mode;
};

// Workspace of the backward pass, fp32.
struct PackedBwdSpace {
    float *D;              // [Hq, T]: dO . O
    float *dKc, *dVc;      // [splits, Hkv, G, d]
    float *a, *cds;        // [Hkv, T]: a_t and (tau / r) ds_t
    float *qsum, *dqs;     // [Hkv, G, d]: sum of the group-last queries, and their gradient through the pooling
    int splits;            // parts of a core tile's query rows
    // bf16: counters of the items that CTAs have taken (cores, tokens); a token tile's rows in one or two parts, with the
    // sums of both, [tile, Hkv, 8 warps, 2], and how many of them are there
    int32_t *taken;
    int token_splits;
    float *parts;
    int32_t *there;
    int n_zero;            // words from `taken` on that start at zero
};

cudaError_t launch_attn_packed_tc(const PackedArgs &a, cudaStream_t stream);
cudaError_t launch_attn_packed_f32(const PackedArgs &a, cudaStream_t stream);
// part 0: dKc, dVc; 1: dQ; 2: dK, dV
cudaError_t launch_packed_bwd_tc(const PackedArgs &a, const PackedBwdSpace &w, int part, cudaStream_t stream);
cudaError_t launch_packed_bwd_f32(const PackedArgs &a, const PackedBwdSpace &w, int part, cudaStream_t stream);

}  // namespace cca
