// Attention over packed sequences (packed.cuh), bf16, d = 128 or 64, on the sm_103a tensor cores.
//
// The pipeline is the contiguous kernel's (attn_tc.cu, where its roles and tensor memory are described): a persistent
// CTA per SM, items of 256 query rows in two halves that share the key tiles, core tiles first, then the raw
// band; one warp copies, one issues the products, four warps for each half keep an online softmax.  What differs: an
// item's rows, its sequence's first row and its cores come from the batch's plan, rows keep their indices in their
// sequence, tensors are read and written by strides, and items are dealt to and fro.  (One template for both kernels
// made the contiguous one 3% slower.)
//
// What is masked must not reach an output, not even as 0 * NaN: the producer sets values behind a sequence's end
// (the next sequence's) to zero before it hands over the tile that holds them, and where a row's sums are not finite
// although its scores are, a later token's value may have done it: the warp looks at such rows again once its last
// item is done (mend_rows), when no bounded wait depends on it.  One sequence of 32 K tokens, causal, 8 heads over
// one: 1.3 ms; with a NaN among its first values 1.8, an infinite one 7.0 (every later row's values are looked
// through), a column of them 15, either in its last row 10.6 (the other rows of its tiles are formed again); row by row
// inside the pipeline it was 801 ms.
//
// A short sequence (n <= 256 / 2^k) fills an item with 2^k query heads of a KV head side by side, 128 / 2^k rows of
// each in a half, as far as 2^k divides the heads: an item costs 4 us at least (its plan entry, first copies, scores,
// softmax, output one after the other), 32 short prompts with 32 heads 31 us without and 22 with it (18.3-18.9 since).
//
// 12 prompts of 32 K tokens in all (32 heads over 8, window 1024) take 452-474 us on different boxes, 1.01-1.06 PF/s of
// visible pairs, the tensor pipe active 53% of the time: their tiles hold 20% more pairs than are visible (a last core
// tile is multiplied whole), 8 tiles an item leave a quarter to an item's start and end, and a tile waits for its chain as in
// the contiguous kernel.  Three of 64 K (15 tiles an item, 11% more pairs): 1.43-1.46 ms, 1.24-1.27 PF/s; d = 64, 12 prompts
// of 16 K: 192-195 us, 0.51-0.52 PF/s.  Letting a half go on with the next item by itself was slower (517 us).
//
// Every mbarrier wait is bounded in time; on a time-out the CTA stops, drains what it has in flight, frees its tensor
// memory and reports CCA_ERR_TIMEOUT.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "internal.h"
#include "packed.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.h"
#include "visibility.cuh"

namespace cca {

extern unsigned long long g_wait_limit_ns;
extern int g_skip_q_load;

namespace {

constexpr int BM = 128;                       // query rows per half
constexpr int BN = 128;                       // keys per tile
constexpr int NS = 5;                         // ring slots
constexpr uint32_t HALF_BYTES = BN * 64 * 2;  // 64 columns of a tile, as one swizzled box
constexpr int NUM_THREADS = 320;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_S = 0;    // S_h at h * 128
constexpr uint32_t TM_O = 256;  // O_h at 256 + h * 128
constexpr float LAZY_RESCALE_LOG2 = 16.0f;  // keep a stale max while it is within 2^16

constexpr uint32_t IDESC_QK = ptx::idesc_bf16_f32(BM, BN, 0, 0);  // Q, K both K-major

constexpr int B_QFULL = 0;
constexpr int B_QFREE = 1;
constexpr int B_FULL = 2;               // NS
constexpr int B_EMPTY = B_FULL + NS;    // NS
constexpr int B_SFULL = B_EMPTY + NS;   // 2 (per half)
constexpr int B_PFULL = B_SFULL + 2;    // 2
constexpr int B_PVDONE = B_PFULL + 2;   // 2
constexpr int B_OFREE = B_PVDONE + 2;   // 2
constexpr int B_DRAIN = B_OFREE + 2;
constexpr int B_CUT = B_DRAIN + 1;      // copies of a tile that ends behind its sequence
constexpr int NUM_BARS = B_CUT + 1;

// shared-memory layout for head dimension HD (offsets from a 1024-byte aligned base)
template <int HD>
struct Layout {
    static constexpr uint32_t TILE_BYTES = BN * HD * 2;  // one bf16 tile
    static constexpr uint32_t IDESC_PV = ptx::idesc_bf16_f32(BM, HD, 0, 1);  // P (TMEM), V MN-major
    static constexpr uint32_t OFF_Q = 0;  // Q_A, Q_B
    static constexpr uint32_t OFF_RING = 2 * TILE_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_RING + NS * TILE_BYTES;
    static constexpr uint32_t OFF_TMEMPTR = OFF_BAR + NUM_BARS * 8;
    static constexpr uint32_t OFF_ABORT = OFF_TMEMPTR + 4;
    static constexpr uint32_t OFF_MEND = OFF_ABORT + 4;   // some row's sums are not finite
    static constexpr uint32_t OFF_BEGIN = OFF_MEND + 4;  // begin[3] of make_item, and the number of items
    static constexpr uint32_t SMEM_BYTES = OFF_BEGIN + 16 + 1024;  // slack for manual alignment
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct Params {
    Plan plan;
    Rows<const __nv_bfloat16> Q, K, V;
    Rows<__nv_bfloat16> O;
    const __nv_bfloat16 *Kc, *Vc;
    float *LSE;
    CUtensorMap mQ[3];  // Q in boxes of 2, 4, 8 heads of 64, 32, 16 rows
    int Hq;
    int most;           // log2 of the heads that may share a half
    FastDiv by_r, by_heads[4];  // by Hq / Hkv, and by Hq >> c
    float scale_log2;
    unsigned long long wait_limit_ns;
    int skip_q_load;  // test hook: never load Q, so the pipeline waits run out
    int o_align32;    // O's rows are 32-byte aligned: the epilogue may use 32-byte stores
};
// The tile sequence of one work item and which half uses which tile.  Per-half
// fields are scalars chosen with selects (no runtime-indexed arrays, which
// would live in local memory).
struct Half {
    int a, b;     // first / last valid row
    bool valid;
    int tc;       // core tiles used: [0, tc)
    int kl, kh;   // local tiles used: [kl, kh)
};

struct Item {
    int kvz;
    Half hA, hB;
    int Tc;   // core tiles loaded (max of the halves' tc)
    int lo0;  // first key of local tile 0
    int T;    // tiles loaded
    // the sequence's first row in the tensors, its first core row, its length, the head
    int row0, core0, n, h;
    int lr;  // log2 of the rows of one head in a half (7, less where heads share it)

    __device__ __forceinline__ const Half &half(int h) const { return h ? hB : hA; }
};

__device__ __forceinline__ bool half_uses(const Half &x, int Tc, int t) {
    if (!x.valid) return false;
    if (t < Tc) return t < x.tc;
    const int k = t - Tc;
    return k >= x.kl && k < x.kh;
}
__device__ __forceinline__ int half_first(const Half &x, int Tc) { return x.tc > 0 ? 0 : Tc + x.kl; }
// next used tile after t, or -1
__device__ __forceinline__ int half_next(const Half &x, int Tc, int t) {
    if (t < Tc) return (t + 1 < x.tc) ? t + 1 : Tc + x.kl;
    return (t + 1 < Tc + x.kh) ? t + 1 : -1;
}
__device__ __forceinline__ int half_count(const Half &x) { return x.valid ? x.tc + x.kh - x.kl : 0; }

// Rows a .. a + rows - 1 of a sequence of n.
__device__ __forceinline__ Half make_half(const Plan &plan, int a, int lo0, int n, int rows) {
    Half x;
    x.a = a;
    x.valid = a < n;
    x.b = min(a + rows - 1, n - 1);
    if (!x.valid) {
        x.tc = x.kl = x.kh = 0;
        return x;
    }
    x.tc = (plan.cores_of(x.b) + BN - 1) / BN;
    x.kl = (plan.start_of(a) - lo0) / BN;
    x.kh = (x.b - lo0) / BN + 1;
    return x;
}

// Largest step between consecutive tiles of a half: only the step from its last core tile
// to its first local tile can exceed 1.
__device__ __forceinline__ int half_max_step(const Half &x, int Tc) {
    return (x.valid && x.tc > 0) ? Tc + x.kl - (x.tc - 1) : 1;
}

// begin[c - 1] is the first entry of pairs[] whose halves hold 2^c heads.
__device__ __forceinline__ Item make_item(const Params &p, int k, const int *begin) {
    Item it;
    // heaviest first, all heads of a pair side by side; short sequences, the last ones, by groups of 2^c heads
    int c = 0, at = k;
    for (; c < 3; ++c) {
        const int some = (begin[c] - (c > 0 ? begin[c - 1] : 0)) * (p.Hq >> c);
        if (at < some) break;
        at -= some;
    }
    int idx = p.by_heads[c].div(at);
    at -= idx * (p.Hq >> c);
    idx += c > 0 ? begin[c - 1] : 0;
    const int4 e = p.plan.pairs[idx];
    it.lr = 7 - c;
    it.h = at << c;
    it.kvz = p.by_r.div(it.h);
    it.row0 = e.x;
    it.core0 = e.w;
    it.n = e.y;
    const int i0 = e.z * 2 * BM;
    it.lo0 = p.plan.start_of(i0);
    it.hA = make_half(p.plan, i0, it.lo0, e.y, 1 << it.lr);
    it.hB = make_half(p.plan, i0 + (1 << it.lr), it.lo0, e.y, 1 << it.lr);
    const int last = it.hB.valid ? it.hB.b : it.hA.b;
    it.Tc = max(it.hA.tc, it.hB.tc);
    it.T = it.Tc + (last - it.lo0) / BN + 1;
    return it;
}

// Parity of the FULL barrier of the ring slot holding K for ring index u (u even).
// Only K slots complete a FULL barrier (the tile's V copy completes the same one),
// and with NS odd an even u reaches each slot once every 2*NS indices.
__device__ __forceinline__ uint32_t k_full_parity(uint32_t u) { return (u / (2 * NS)) & 1; }

// The top bits of a word's bf16 that are not finite: their exponents are all ones, and one more carries over.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// What a lane of a warp that holds whole rows has of one: E columns from E * lane on.
template <int HD>
struct Piece {
    static constexpr int E = HD / 32;
    using Raw = typename std::conditional<E == 4, uint2, uint32_t>::type;
    Raw raw;
    static __device__ __forceinline__ Piece at(const __nv_bfloat16 *row) {
        Piece x;
        x.raw = reinterpret_cast<const Raw *>(row)[threadIdx.x & 31];
        return x;
    }
    // not zero where an element is not finite
    __device__ __forceinline__ uint32_t odd_halves() const {
        if constexpr (E == 4) return cca::odd_halves(raw.x) | cca::odd_halves(raw.y);
        else return cca::odd_halves(raw);
    }
    __device__ __forceinline__ void floats(float (&f)[E]) const {
        uint32_t w[E / 2];
        if constexpr (E == 4) w[0] = raw.x, w[1] = raw.y;
        else w[0] = raw;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
__device__ __forceinline__ bool not_finite(float x) { return !(x - x == 0.f); }

// A row's keys and values: rows [0, cores) of Kc, Vc and [from, to] of K, V, of one sequence and KV head.
template <int HD>
struct RowKeys {
    const __nv_bfloat16 *kc, *vc, *k, *v;  // rows 0
    int64_t k_step, v_step;                // from a token to the next one
    int cores, from, to;
    __device__ __forceinline__ int count() const { return cores + max(to - from + 1, 0); }
    __device__ __forceinline__ Piece<HD> key(int j) const {
        return Piece<HD>::at(j < cores ? kc + static_cast<int64_t>(j) * HD : k + (from + j - cores) * k_step);
    }
    __device__ __forceinline__ Piece<HD> value(int j) const {
        return Piece<HD>::at(j < cores ? vc + static_cast<int64_t>(j) * HD : v + (from + j - cores) * v_step);
    }
    // Adds up what is not finite of the values [j0, j1), column by column: zero where nothing is, and otherwise what a
    // weighted sum becomes: an infinity, or NaN of both, of a NaN, or of one whose weight is zero.  (The row's LSE is finite, so a key that
    // is not has a score of minus infinity; a weight that is small, however small, is not zero.)  Ends early where every
    // lane's columns in `asked` are NaN.
    __device__ __forceinline__ void add_odd(int j0, int j1, unsigned asked, float (&odd)[HD / 32]) const {
        constexpr int E = HD / 32, AHEAD = 16;
        for (int j = j0; j < j1; j += AHEAD) {
            Piece<HD> x[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) x[i] = value(min(j + i, j1 - 1));
            uint32_t some = 0;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) some |= x[i].odd_halves();
            if (!__any_sync(0xffffffffu, some != 0)) continue;
            Piece<HD> y[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) y[i] = key(min(j + i, j1 - 1));
            unsigned none = 0;  // keys of weight zero
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) none |= y[i].odd_halves() != 0 ? 1u << i : 0u;
            none = __reduce_or_sync(0xffffffffu, none);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                float f[E];
                x[i].floats(f);
#pragma unroll
                for (int e = 0; e < E; ++e) odd[e] += !not_finite(f[e]) ? 0.f : none & (1u << i) ? NAN : f[e];
            }
            bool all = true;
#pragma unroll
            for (int e = 0; e < E; ++e) all = all && (!(asked & (1u << e)) || odd[e] != odd[e]);
            if (__all_sync(0xffffffffu, all)) return;
        }
    }
};

// A place of O that is to be formed again; no conversion to bf16 makes this NaN.
constexpr uint32_t FORM_AGAIN = 0x7fa5;

// Two bf16 of a word, zero where one is not finite.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) { return w & ~((odd_halves(w) >> 15) * 0xffffu); }
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The places FORM_AGAIN of those of a half's 16 rows from `base` on that `rows` names, by one warp: values that are not finite
// count as zero (no such place has one among its visible keys), and weights are 2^(s - LSE), about 1 at most, so that no sum
// passes the largest number that the result does not.  16 keys a step: S = Q K^T, P in registers, O += P V.  Which columns of the
// head a fragment's depth (S) or width (O) stands for is free as long as both sides agree, so a lane reads 16-byte pieces:
// of keys lane / 4 at columns 32 c + 8 (lane % 4), of values (lane % 4) * 2, + 1, + 8, + 9 at lane / 4 * HD / 8.
template <int HD>
__device__ __forceinline__ void form_again(const Params &p, const Item &it, const Half &x, int base, unsigned rows) {
    constexpr int C = HD / 32, NT = HD / 8;  // 16-byte pieces of a lane's share of a row; width tiles of O
    const unsigned full = 0xffffffffu;
    const int lane = threadIdx.x & 31, quad = lane >> 2, t = lane & 3, h = it.h + (base >> it.lr);
    bool in[2];
    int i[2], cores[2], from[2];
    float lse2[2], l[2] = {0.f, 0.f};
    uint4 q[2][C];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = quad + 8 * k;
        in[k] = (rows >> r) & 1;
        i[k] = min(x.a + ((base + r) & ((1 << it.lr) - 1)), x.b);
        cores[k] = in[k] ? p.plan.cores_of(i[k]) : 0;
        from[k] = in[k] ? p.plan.start_of(i[k]) : 0x7fffffff;
        lse2[k] = in[k] ? p.LSE[static_cast<int64_t>(h) * p.plan.T + it.row0 + i[k]] * 1.4426950408889634f : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) q[k][c] = *reinterpret_cast<const uint4 *>(p.Q.at(h, it.row0 + i[k]) + 32 * c + 8 * t);
    }
    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    const int64_t head = (static_cast<int64_t>(it.kvz) * p.plan.G + it.core0) * HD;
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {  // cores, then tokens
        const bool core = part == 0;
        const int k0 = core ? 0 : __reduce_min_sync(full, min(from[0], from[1]));
        const int k1 = core ? __reduce_max_sync(full, max(cores[0], cores[1])) : __reduce_max_sync(full, max(in[0] ? i[0] : 0, in[1] ? i[1] : 0)) + 1;
        const __nv_bfloat16 *const K = core ? p.Kc + head : p.K.at(it.kvz, it.row0), *const V = core ? p.Vc + head : p.V.at(it.kvz, it.row0);
        const int64_t ks = core ? HD : p.K.row, vs = core ? HD : p.V.row;
#pragma unroll 1
        for (int k = k0; k < k1; k += 16) {
            uint4 kk[2][C], vv[4][C / 2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    kk[j][c] = *reinterpret_cast<const uint4 *>(K + min(k + 8 * j + quad, k1 - 1) * ks + 32 * c + 8 * t);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < C / 2; ++c)
                    vv[j][c] = *reinterpret_cast<const uint4 *>(V + min(k + 2 * t + (j & 1) + 8 * (j >> 1), k1 - 1) * vs + quad * NT + 8 * c);
            uint32_t w[4];  // weights, as the left side of the second product
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint32_t lo[4] = {q[0][c].x, q[1][c].x, q[0][c].y, q[1][c].y}, hi[4] = {q[0][c].z, q[1][c].z, q[0][c].w, q[1][c].w};
                    mma_16x8x16(s, lo, kk[j][c].x, kk[j][c].y);
                    mma_16x8x16(s, hi, kk[j][c].z, kk[j][c].w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = e >> 1, key = k + 8 * j + 2 * t + (e & 1);
                    const bool seen = core ? key < cores[r] : key >= from[r] && key <= i[r];
                    s[e] = seen ? exp2f(fmaf(s[e], p.scale_log2, -lse2[r])) : 0.f;
                    l[r] += s[e];
                }
                w[2 * j] = ptx::pack_bf16x2(s[0], s[1]);
                w[2 * j + 1] = ptx::pack_bf16x2(s[2], s[3]);
            }
#pragma unroll
            for (int c = 0; c < C / 2; ++c) {
                uint32_t f[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[j][0] = finite_only(vv[j][c].x), f[j][1] = finite_only(vv[j][c].y);
                    f[j][2] = finite_only(vv[j][c].z), f[j][3] = finite_only(vv[j][c].w);
                }
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const unsigned half = n & 1 ? 0x7632 : 0x5410;
                    mma_16x8x16(o[8 * c + n], w, __byte_perm(f[0][n / 2], f[1][n / 2], half), __byte_perm(f[2][n / 2], f[3][n / 2], half));
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(full, l[k], 1);
        l[k] += __shfl_xor_sync(full, l[k], 2);
        if (!in[k]) continue;
        // width tile j of column n is column n * NT + j, so a lane has 2 NT columns side by side
        __nv_bfloat16 *const out = p.O.at(h, it.row0 + i[k]) + 2 * NT * t;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (__bfloat16_as_ushort(out[n * NT + j]) == FORM_AGAIN) out[n * NT + j] = __float2bfloat16_rn(o[j][2 * k + n] / l[k]);
    }
}

// Once more through the CTA's items, for the rows of this warp whose sums were not finite although their scores are
// (LSE is finite).  Such a column is what the row's visible values say if one of them is not finite; if none is, a masked
// key's value or a sum that passed the largest number has come in, and it is formed again.  The other columns stand.
template <int HD>
__device__ __noinline__ void mend_rows(const Params &p, int n_items, const int *begin, int h, int quarter) {
    constexpr int E = HD / 32;
    const unsigned full = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    __syncwarp();  // the rows that the other lanes have stored
    for (int round = 0, k; (k = item_of_round(round, n_items)) < n_items; ++round) {
        const Item it = make_item(p, k, begin);
        const Half x = h ? it.hB : it.hA;
        if (!x.valid) continue;
        auto row_of = [&](int r) { return x.a + ((quarter * 32 + r) & ((1 << it.lr) - 1)); };   // its place in the sequence
        auto head_of = [&](int r) { return it.h + ((quarter * 32 + r) >> it.lr); };
        auto odd_columns = [&](const Piece<HD> &v) {
            float f[E];
            v.floats(f);
            unsigned bits = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) bits |= not_finite(f[e]) ? 1u << e : 0u;
            return bits;
        };
        const int mine = row_of(lane);
        const float lse = mine <= x.b ? p.LSE[static_cast<int64_t>(head_of(lane)) * p.plan.T + it.row0 + mine] : INFINITY;
        unsigned rows = __ballot_sync(full, !not_finite(lse)), todo = 0, asked = 0, again = 0;
        for (; rows != 0; rows &= rows - 1) {
            const int r = __ffs(rows) - 1;
            const unsigned c = odd_columns(Piece<HD>::at(p.O.at(head_of(r), it.row0 + row_of(r))));
            if (__any_sync(full, c != 0)) todo |= 1u << r;
            asked |= c;
        }
        if (todo == 0) continue;
        // what all of them see: cores [0, shared.cores), tokens [shared.from, shared.to]
        const bool in = (todo >> lane) & 1;
        const int i0 = __reduce_min_sync(full, in ? mine : 0x7fffffff), i1 = __reduce_max_sync(full, in ? mine : 0);
        const int64_t head = (static_cast<int64_t>(it.kvz) * p.plan.G + it.core0) * HD;
        const RowKeys<HD> shared = {p.Kc + head, p.Vc + head, p.K.at(it.kvz, it.row0), p.V.at(it.kvz, it.row0), p.K.row, p.V.row,
                                    p.plan.cores_of(i0), p.plan.start_of(i1), i0};
        float seen[E];
#pragma unroll
        for (int e = 0; e < E; ++e) seen[e] = 0.f;
        shared.add_odd(0, shared.count(), asked, seen);
        for (; todo != 0; todo &= todo - 1) {
            const int r = __ffs(todo) - 1, i = row_of(r);
            __nv_bfloat16 *const out = p.O.at(head_of(r), it.row0 + i);
            const unsigned c = odd_columns(Piece<HD>::at(out));
            // ... and what this one sees besides: later cores, earlier tokens, later tokens
            RowKeys<HD> own = shared;
            own.cores = p.plan.cores_of(i), own.from = p.plan.start_of(i), own.to = i;
            float odd[E];
#pragma unroll
            for (int e = 0; e < E; ++e) odd[e] = seen[e];
            const int t0 = own.cores - own.from;  // place of token 0 among the row's keys
            own.add_odd(shared.cores, own.cores, c, odd);
            own.add_odd(t0 + own.from, t0 + min(shared.from, i + 1), c, odd);
            own.add_odd(t0 + max(shared.from, i0 + 1), t0 + i + 1, c, odd);
            bool left = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (!((c >> e) & 1)) continue;
                left = left || !not_finite(odd[e]);
                out[lane * E + e] = not_finite(odd[e]) ? __float2bfloat16_rn(odd[e]) : __ushort_as_bfloat16(FORM_AGAIN);
            }
            if (__any_sync(full, left)) again |= 1u << r;
        }
        __syncwarp();
        for (int k = 0; k < 32; k += 16)  // 16 rows are of one head: a half has 16 of each at least
            if ((again >> k) & 0xffff) form_again<HD>(p, it, x, quarter * 32 + k, (again >> k) & 0xffff);
    }
}

template <int HD>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    attn_packed_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKc,
                        const __grid_constant__ CUtensorMap tmVc,
                        const __grid_constant__ Params p) {
    using L = Layout<HD>;
    constexpr uint32_t TILE_BYTES = L::TILE_BYTES, OFF_Q = L::OFF_Q, OFF_RING = L::OFF_RING, OFF_BAR = L::OFF_BAR,
                       IDESC_PV = L::IDESC_PV;
    constexpr int HALVES = HD / 64;  // boxes of a tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    auto bar = [&](int idx) -> uint32_t { return base + OFF_BAR + 8u * idx; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + L::OFF_ABORT);
    volatile int *mend_flag = reinterpret_cast<volatile int *>(gbase + L::OFF_MEND);
    uint32_t *tmem_ptr_smem = reinterpret_cast<uint32_t *>(gbase + L::OFF_TMEMPTR);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        ptx::mbar_init(bar(B_QFULL), 1);
        ptx::mbar_init(bar(B_QFREE), 1);
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(bar(B_FULL + s), 1);
            ptx::mbar_init(bar(B_EMPTY + s), 1);
        }
        for (int h = 0; h < 2; ++h) {
            ptx::mbar_init(bar(B_SFULL + h), 1);
            ptx::mbar_init(bar(B_PFULL + h), 4);  // one arrive per softmax warp
            ptx::mbar_init(bar(B_PVDONE + h), 1);
            ptx::mbar_init(bar(B_OFREE + h), 4);
        }
        ptx::mbar_init(bar(B_DRAIN), 1);
        ptx::mbar_init(bar(B_CUT), 1);
        *abort_flag = *mend_flag = 0;
    }
    if (warp == 0) {
        ptx::tmem_alloc(base + L::OFF_TMEMPTR, TMEM_COLS);
        ptx::tmem_relinquish();
    }
    // Everything above runs while the kernel before ends.  This one does not let the next begin early: CTAs that
    // take SMs one by one lie anywhere, and 12 prompts then take 473 us instead of 462, a training step with cores
    // 1233 instead of 1209 (neighbours read the same keys).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) {
        const int pairs = max(plan_counts(p.plan).x, 0);
        const int3 s = pairs > 0 ? plan_short(p.plan) : make_int3(0, 0, 0);
        const int first[5] = {0, p.most >= 1 ? s.x : pairs, p.most >= 2 ? s.y : pairs, p.most >= 3 ? s.z : pairs, pairs};
        int *out = reinterpret_cast<int *>(gbase + L::OFF_BEGIN), items = 0;
        for (int c = 0; c < 4; ++c) items += (first[c + 1] - first[c]) * (p.Hq >> c);
        for (int c = 0; c < 3; ++c) out[c] = first[c + 1];
        out[3] = items;
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_ptr_smem;
    const uint64_t lim = p.wait_limit_ns;
    const int *const begin = reinterpret_cast<const int *>(gbase + L::OFF_BEGIN);
    const int n_items = begin[3];

    if (warp < 2) {
        if (warp == 0) {
            // ------------------------------------------------------------ producer over packed sequences: the
            // whole warp, for the tiles that end behind their sequence
            if (lane == 0) {
                ptx::prefetch_tmap(&tmQ);
                ptx::prefetch_tmap(&tmK);
                ptx::prefetch_tmap(&tmV);
                ptx::prefetch_tmap(&tmKc);
                ptx::prefetch_tmap(&tmVc);
            }
            auto wwait = [&](uint32_t b, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, ptx::wait_bounded(b, parity, abort_flag, lim));
            };
            uint32_t u = 0, cut = 0;  // ring loads issued so far, tiles cut
            int n_iter = 0;
            bool ok = true;
            for (int k; ok && (k = item_of_round(n_iter, n_items)) < n_items; ++n_iter) {
                const Item it = make_item(p, k, begin);
                const int groups = p.plan.by_g.div(it.n);
                if (!wwait(bar(B_QFREE), (n_iter & 1) ^ 1)) break;
                if (!p.skip_q_load && lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(B_QFULL), 2 * TILE_BYTES);
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t dst = base + OFF_Q + h * TILE_BYTES;
                        const int row0 = it.row0 + (h ? it.hB.a : it.hA.a);
#pragma unroll
                        for (int x = 0; x < HALVES; ++x)
                            ptx::tma_load_3d(it.lr < 7 ? (const void *)&p.mQ[6 - it.lr] : (const void *)&tmQ, bar(B_QFULL), dst + x * HALF_BYTES, 64 * x, row0, it.h);
                    }
                }
                for (int t = 0; t < it.T; ++t, u += 2) {
                    const bool core = t < it.Tc;
                    const int first = core ? t * BN : it.lo0 + (t - it.Tc) * BN;  // the tile's first key in the sequence
                    const int left = (core ? groups : it.n) - first;
                    const int y = (core ? it.core0 : it.row0) + first;
                    const int ks = u % NS, vs = (u + 1) % NS;
                    if (!(ok = wwait(bar(B_EMPTY + ks), ((u / NS) & 1) ^ 1) && wwait(bar(B_EMPTY + vs), (((u + 1) / NS) & 1) ^ 1))) break;
                    const uint32_t full = bar(B_FULL + ks), here = left < BN ? bar(B_CUT) : full;
                    const uint32_t kdst = base + OFF_RING + ks * TILE_BYTES, vdst = base + OFF_RING + vs * TILE_BYTES;
                    if (lane == 0) {
                        const void *mk = core ? (const void *)&tmKc : (const void *)&tmK;
                        const void *mv = core ? (const void *)&tmVc : (const void *)&tmV;
                        ptx::mbar_arrive_expect_tx(here, 2 * TILE_BYTES);
#pragma unroll
                        for (int x = 0; x < HALVES; ++x) ptx::tma_load_3d(mk, here, kdst + x * HALF_BYTES, 64 * x, y, it.kvz);
#pragma unroll
                        for (int x = 0; x < HALVES; ++x) ptx::tma_load_3d(mv, here, vdst + x * HALF_BYTES, 64 * x, y, it.kvz);
                    }
                    __syncwarp();
                    if (left >= BN) continue;
                    if (!(ok = wwait(bar(B_CUT), cut & 1))) {
                        volatile int never = 0;  // these copies land before the CTA exits
                        ptx::wait_bounded(bar(B_CUT), cut & 1, &never, lim);
                        break;
                    }
                    ++cut;
                    for (int i = left * 8 + lane; i < BN * 8; i += 32)
#pragma unroll
                        for (int x = 0; x < HALVES; ++x) ptx::st_shared_v4(vdst + x * HALF_BYTES + i * 16, 0.f, 0.f, 0.f, 0.f);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(full);
                }
            }
            __syncwarp();
            // The copies land before the CTA exits.  Whoever gives up later than this may leave some that nobody else
            // waits for; otherwise they have been waited for and this takes no time.
            volatile int never = 0;
            for (uint32_t v = u > 2 * NS ? u - 2 * NS : 0; v < u; v += 2)
                ptx::wait_bounded(bar(B_FULL + v % NS), k_full_parity(v), &never, lim);
            if (!p.skip_q_load && n_iter > 0) ptx::wait_bounded(bar(B_QFULL), (n_iter - 1) & 1, &never, lim);
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            // The whole warp runs the issuer with identical values in every lane; the
            // MMAs and commits are issued by one elected lane.
            auto wwait = [&](uint32_t b, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, ptx::wait_bounded(b, parity, abort_flag, lim));
            };
            uint32_t ubase = 0;
            int n_iter = 0;
            uint32_t kpend = 0;  // pending S issues per ring slot, 2 bits per slot
            uint32_t pf_cnt[2] = {0, 0};
            int n_half[2] = {0, 0};  // items each half has processed
            // Descriptors of step 0 for Q_A, Q_B and for ring slot 0; a slot adds TILE_BYTES/16.
            const uint64_t dq0 = ptx::smem_desc_sw128(base + OFF_Q, 16, 1024);
            const uint64_t dq1 = ptx::smem_desc_sw128(base + OFF_Q + TILE_BYTES, 16, 1024);
            const uint64_t dk0 = ptx::smem_desc_sw128(base + OFF_RING, 16, 1024);
            const uint64_t dv0 = ptx::smem_desc_sw128(base + OFF_RING, HALF_BYTES, 1024);
            bool ok = true;
            for (int k; ok && (k = item_of_round(n_iter, n_items)) < n_items; ++n_iter) {
                const Item it = make_item(p, k, begin);
                if (!wwait(bar(B_QFULL), n_iter & 1)) break;
                int s_left = half_count(it.hA) + half_count(it.hB);
                // S_h = Q_h K(t)^T into S_h.  The first user of a ring slot waits for the copy.
                auto issue_s = [&](int h, int t) -> bool {
                    const uint32_t uk = ubase + 2 * t;
                    const int slot = uk % NS;
                    uint32_t pend = (kpend >> (2 * slot)) & 3u;
                    if (pend == 0) {
                        // the tile's first S: wait for its K and V copies
                        if (!wwait(bar(B_FULL + slot), k_full_parity(uk))) return false;
                        pend = (half_uses(it.hA, it.Tc, t) ? 1u : 0u) + (half_uses(it.hB, it.Tc, t) ? 1u : 0u);
                    }
                    ptx::tc_fence_after();
                    if constexpr (HD == 128)
                        ptx::mma_ss_k128_warp(tmem + TM_S + h * BN, h ? dq1 : dq0, dk0 + static_cast<uint64_t>(slot) * (TILE_BYTES >> 4),
                                         IDESC_QK, 0u);
                    else
                        ptx::mma_ss_k64_warp(tmem + TM_S + h * BN, h ? dq1 : dq0, dk0 + static_cast<uint64_t>(slot) * (TILE_BYTES >> 4),
                                        IDESC_QK, 0u);
                    ptx::tc_commit_warp(bar(B_SFULL + h));
                    --pend;
                    kpend = (kpend & ~(3u << (2 * slot))) | (pend << (2 * slot));
                    if (pend == 0) ptx::tc_commit_warp(bar(B_EMPTY + slot));
                    if (--s_left == 0) ptx::tc_commit_warp(bar(B_QFREE));
                    return true;
                };
                // Prologue: first S of each half, earliest tile first, so that the issuer
                // never waits on a copy that sits behind one it has not consumed yet.
                {
                    const bool b_first = it.hB.valid && half_first(it.hB, it.Tc) < half_first(it.hA, it.Tc);
                    for (int q = 0; ok && q < 2; ++q) {
                        const int h = b_first ? 1 - q : q;
                        const Half &x = it.half(h);
                        if (x.valid) ok = issue_s(h, half_first(x, it.Tc));
                    }
                }
                // The tile loop.  After a half's PV on tile t the issuer starts S on the
                // half's next tile, which first waits for that tile's copies; with a ring of
                // two and a half tiles whose earlier slots only this loop frees, that wait can
                // end only if the next tile is at most t + 2.  With the window aligned to groups
                // of more than 128 tokens, half B's band can start further than that after its
                // last core tile, so items with such a step take the second copy of the loop,
                // which holds the S back (defer[h]) until the loop is two tiles short of it.
                // The copies are separate so that the common loop carries none of that logic.
                if (half_max_step(it.hA, it.Tc) <= 2 && half_max_step(it.hB, it.Tc) <= 2) {
                    bool first_pv[2] = {true, true};
                    for (int t = 0; ok && t < it.T; ++t) {
                        // V(t) has landed: the tile's first S waited for its K and V together
                        const uint32_t uv = ubase + 2 * t + 1;
                        const int vslot = uv % NS;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // unrolled: per-half counters stay in registers
                            const Half &x = it.half(h);
                            if (!half_uses(x, it.Tc, t)) continue;
                            if (!wwait(bar(B_PFULL + h), pf_cnt[h] & 1)) {
                                ok = false;
                                break;
                            }
                            ++pf_cnt[h];
                            if (first_pv[h]) {
                                // the epilogue of this half's previous item must have read O_h
                                if (!wwait(bar(B_OFREE + h), (n_half[h] & 1) ^ 1)) {
                                    ok = false;
                                    break;
                                }
                            }
                            ptx::tc_fence_after();
                            ptx::mma_ts_k128_warp(tmem + TM_O + h * HD, tmem + TM_S + h * BN,
                                             dv0 + static_cast<uint64_t>(vslot) * (TILE_BYTES >> 4), IDESC_PV,
                                             first_pv[h] ? 0u : 1u);
                            first_pv[h] = false;
                            const int tn = half_next(x, it.Tc, t);
                            if (tn >= 0) {
                                if (!issue_s(h, tn)) {
                                    ok = false;
                                    break;
                                }
                            } else {
                                ptx::tc_commit_warp(bar(B_PVDONE + h));
                            }
                        }
                        if (!ok) break;
                        ptx::tc_commit_warp(bar(B_EMPTY + vslot));
                    }
                } else {
                    bool first_pv[2] = {true, true};
                    int defer[2] = {-1, -1};
                    for (int t = 0; ok && t < it.T; ++t) {
                        // V(t) has landed: the tile's first S waited for its K and V together
                        const uint32_t uv = ubase + 2 * t + 1;
                        const int vslot = uv % NS;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (defer[h] >= 0 && defer[h] <= t + 2) {
                                if (!issue_s(h, defer[h])) {
                                    ok = false;
                                    break;
                                }
                                defer[h] = -1;
                            }
                        }
                        if (!ok) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // unrolled: per-half counters stay in registers
                            const Half &x = it.half(h);
                            if (!half_uses(x, it.Tc, t)) continue;
                            if (!wwait(bar(B_PFULL + h), pf_cnt[h] & 1)) {
                                ok = false;
                                break;
                            }
                            ++pf_cnt[h];
                            if (first_pv[h]) {
                                // the epilogue of this half's previous item must have read O_h
                                if (!wwait(bar(B_OFREE + h), (n_half[h] & 1) ^ 1)) {
                                    ok = false;
                                    break;
                                }
                            }
                            ptx::tc_fence_after();
                            ptx::mma_ts_k128_warp(tmem + TM_O + h * HD, tmem + TM_S + h * BN,
                                             dv0 + static_cast<uint64_t>(vslot) * (TILE_BYTES >> 4), IDESC_PV,
                                             first_pv[h] ? 0u : 1u);
                            first_pv[h] = false;
                            const int tn = half_next(x, it.Tc, t);
                            if (tn > t + 2) {
                                defer[h] = tn;
                            } else if (tn >= 0) {
                                if (!issue_s(h, tn)) {
                                    ok = false;
                                    break;
                                }
                            } else {
                                ptx::tc_commit_warp(bar(B_PVDONE + h));
                            }
                        }
                        if (!ok) break;
                        ptx::tc_commit_warp(bar(B_EMPTY + vslot));
                    }
                }
                ubase += 2 * it.T;
                n_half[0] += it.hA.valid ? 1 : 0;
                n_half[1] += it.hB.valid ? 1 : 0;
            }
            // Whatever was issued must complete before tensor memory is freed.
            ptx::tc_commit_warp(bar(B_DRAIN));
            volatile int never = 0;
            ptx::wait_bounded(bar(B_DRAIN), 0, &never, lim);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax + epilogue
        const int h = (warp - 2) >> 2;  // half
        const int quarter = warp & 3;   // TMEM lane quarter this warp may access
        const int row = quarter * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_addr + TM_S + h * BN;
        const uint32_t tO = tmem + lane_addr + TM_O + h * HD;
        uint32_t sf_cnt = 0;
        int n_done = 0;  // items of this half finished
        bool ok = true;
        for (int round = 0, k; ok && (k = item_of_round(round, n_items)) < n_items; ++round) {
            const Item it = make_item(p, k, begin);
            const Half x = h ? it.hB : it.hA;
            if (!x.valid) continue;
            const int i = x.a + (row & ((1 << it.lr) - 1));
            const int lo_i = p.plan.start_of(i);           // first raw token of this row's window
            const int nc_i = p.plan.cores_of(i);         // cores visible to this row
            const int nc_first = p.plan.cores_of(x.a);
            const int lo_last = p.plan.start_of(x.b);
            float m = -INFINITY;  // running max of the log2-scaled logits
            float l = 0.f;
            for (int t = half_first(x, it.Tc); t >= 0; t = half_next(x, it.Tc, t)) {
                if (!__all_sync(0xffffffffu, ptx::wait_bounded(bar(B_SFULL + h), sf_cnt & 1, abort_flag, lim))) {
                    ok = false;
                    break;
                }
                ++sf_cnt;
                ptx::tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) ptx::tmem_ld32(tS + c * 32, s[c]);
                ptx::tmem_wait_ld(s[0]);
                ptx::reg_touch(s[1]);
                ptx::reg_touch(s[2]);
                ptx::reg_touch(s[3]);

                // visibility window of this row within the tile: columns [c_lo, c_hi]
                int c_lo = 0, c_hi = BN - 1;
                bool masked;
                if (t < it.Tc) {
                    const int y0 = t * BN;
                    masked = y0 + BN > nc_first;
                    c_hi = min(nc_i - y0, BN) - 1;
                } else {
                    const int y0 = it.lo0 + (t - it.Tc) * BN;
                    masked = (y0 < lo_last) || (y0 + BN - 1 > x.a);
                    c_lo = max(lo_i - y0, 0);
                    c_hi = min(i - y0, BN - 1);
                }
                // row max: 3-input max over eight independent partial maxima
                float mp[8];
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        // most 32-column pieces of a masked tile lie wholly inside every row's part; in the others
                        // a column is a bit (with comparisons a masked tile took 1.8 us, three times a plain one)
                        if (__all_sync(0xffffffffu, c_lo <= c * 32 && c_hi >= c * 32 + 31)) continue;
                        const uint32_t seen = ptx::bits(c_lo - c * 32, c_hi - c * 32);
#pragma unroll
                        for (int kk = 0; kk < 32; ++kk)
                            if (!(seen & (1u << kk))) s[c][kk] = __float_as_uint(-INFINITY);
                    }
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    mp[q] = fmaxf(__uint_as_float(s[q >> 1][(q & 1) * 16]), __uint_as_float(s[q >> 1][(q & 1) * 16 + 1]));
#pragma unroll
                for (int q = 0; q < 8; ++q) {
#pragma unroll
                    for (int kk = 2; kk < 16; kk += 2)
                        mp[q] = ptx::max3(mp[q], __uint_as_float(s[q >> 1][(q & 1) * 16 + kk]),
                                          __uint_as_float(s[q >> 1][(q & 1) * 16 + kk + 1]));
                }
                const float mx = ptx::max3(ptx::max3(mp[0], mp[1], mp[2]), ptx::max3(mp[3], mp[4], mp[5]),
                                           fmaxf(mp[6], mp[7]));
                const float m_tile = mx * p.scale_log2;  // -inf stays -inf
                const float m_new = fmaxf(m, m_tile);
                bool rescale = false;
                if (m == -INFINITY) {
                    m = m_new;  // nothing accumulated yet for this row
                } else if (m_new > m + LAZY_RESCALE_LOG2) {
                    rescale = true;
                }
                if (__any_sync(0xffffffffu, rescale)) {
                    // S_h complete => every earlier PV of this half is complete: O_h is stable.
                    const float f = rescale ? ptx::ex2(m - m_new) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < HD / 16; ++c) {
                        uint32_t o[16];
                        ptx::tmem_ld16(tO + c * 16, o);
                        ptx::tmem_wait_ld16(o);
#pragma unroll
                        for (int kk = 0; kk < 16; ++kk) o[kk] = __float_as_uint(__uint_as_float(o[kk]) * f);
                        ptx::tmem_st16(tO + c * 16, o);
                    }
                    if (rescale) {
                        l *= f;
                        m = m_new;
                    }
                }
                const float mu = (m == -INFINITY) ? 0.f : m;
                // p = 2^(s*scale - mu), two columns per packed FMA; row sum in four packed partials
                const uint64_t sc2 = ptx::f2(p.scale_log2, p.scale_log2);
                const uint64_t nm2 = ptx::f2(-mu, -mu);
                uint64_t lp[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t pk[8];
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const int col = (c & 1) * 16 + 2 * kk;
                        const uint64_t x2 = ptx::fma2(
                            ptx::f2(__uint_as_float(s[c >> 1][col]), __uint_as_float(s[c >> 1][col + 1])), sc2, nm2);
                        float x0, x1;
                        ptx::f2_split(x2, x0, x1);
                        const float p0 = ptx::ex2(x0);
                        const float p1 = ptx::ex2(x1);
                        lp[kk & 1] = ptx::add2(lp[kk & 1], ptx::f2(p0, p1));
                        pk[kk] = ptx::pack_bf16x2(p0, p1);
                    }
                    ptx::tmem_st8(tS + c * 8, pk);  // P_h over the consumed columns of S_h
                }
                {
                    float a0, a1, b0, b1;
                    ptx::f2_split(lp[0], a0, a1);
                    ptx::f2_split(lp[1], b0, b1);
                    l += (a0 + a1) + (b0 + b1);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_PFULL + h));
            }
            if (!ok) break;
            // ---- epilogue: O_h / l -> bf16, LSE
            if (!__all_sync(0xffffffffu, ptx::wait_bounded(bar(B_PVDONE + h), n_done & 1, abort_flag, lim))) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const bool valid = i <= x.b;
            const int hh = it.h + (row >> it.lr);
            __nv_bfloat16 *const orow = p.O.at(hh, it.row0 + i);
            float *const lse = p.LSE + static_cast<int64_t>(hh) * p.plan.T + it.row0 + i;
            const float inv = 1.f / l;
            uint32_t o[HD / 32][32];
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) ptx::tmem_ld32(tO + c * 32, o[c]);
            ptx::tmem_wait_ld(o[0]);
#pragma unroll
            for (int c = 1; c < HD / 32; ++c) ptx::reg_touch(o[c]);
            // O_h is in registers: the issuer may start this half's next item
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_OFREE + h));
            uint64_t odd = 0;  // stays zero as long as every sum is finite
#pragma unroll
            for (int c = 0; c < HD / 32; ++c)
#pragma unroll
                for (int k = 0; k < 32; k += 2)
                    odd = ptx::fma2(ptx::f2(__uint_as_float(o[c][k]), __uint_as_float(o[c][k + 1])), 0, odd);
            float odd0, odd1;
            ptx::f2_split(odd, odd0, odd1);
            if (valid && !(odd0 + odd1 == 0.f) && l - l == 0.f) *mend_flag = 1;  // l is NaN: so is the row, by its scores
            // O / l as bf16, one 32-byte sector per store (two 16-byte stores if O is
            // only 16-byte aligned)
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = ptx::pack_bf16x2(__uint_as_float(o[c][16 * q + 2 * k]) * inv,
                                                __uint_as_float(o[c][16 * q + 2 * k + 1]) * inv);
                    if (valid) {
                        if (p.o_align32) {
                            ptx::st_global_v8(orow + c * 32 + q * 16, v);
                        } else {
                            uint4 *dst = reinterpret_cast<uint4 *>(orow + c * 32 + q * 16);
                            dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
                            dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
            }
            if (valid) *lse = (m + __log2f(l)) * 0.6931471805599453f;
            ++n_done;
        }
        // nobody waits for this warp any more
        __syncwarp();
        if (ok && __any_sync(0xffffffffu, *mend_flag)) mend_rows<HD>(p, n_items, begin, h, quarter);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) report(p.plan.status, CCA_ERR_TIMEOUT);
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ---------------------------------------------------------------- host side
struct DeviceInfo {
    bool ready = false;
    int sms = 0;
    cudaError_t err = cudaSuccess;
};

DeviceInfo &device_info(int dev) {
    static DeviceInfo info[64];
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    DeviceInfo &d = info[dev & 63];
    if (!d.ready) {
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        d.err = cudaFuncSetAttribute(attn_packed_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(Layout<128>::SMEM_BYTES));
        if (d.err == cudaSuccess)
            d.err = cudaFuncSetAttribute(attn_packed_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(Layout<64>::SMEM_BYTES));
        d.ready = true;
    }
    return d;
}

}  // namespace

cudaError_t launch_attn_packed_tc(const PackedArgs &a, cudaStream_t stream) {
    EncodeTiledFn enc = get_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const DeviceInfo &di = device_info(dev);
    if (di.err != cudaSuccess) return di.err;
    CUtensorMap mQ, mK, mV, mKc, mVc;
    Params p = {};
    while (p.most < 3 && (a.Hq / a.Hkv) % (2 << p.most) == 0) ++p.most;
    for (int c = 0; c < p.most; ++c)
        if (!encode_packed_bf16(enc, &p.mQ[c], a.Q, a.d, a.plan.T, a.Hq, 2 << c)) return cudaErrorInvalidValue;
    if (!encode_packed_bf16(enc, &mQ, a.Q, a.d, a.plan.T, a.Hq) || !encode_packed_bf16(enc, &mK, a.K, a.d, a.plan.T, a.Hkv) ||
        !encode_packed_bf16(enc, &mV, a.V, a.d, a.plan.T, a.Hkv))
        return cudaErrorInvalidValue;
    if (a.Kc != nullptr) {
        const int64_t head = static_cast<int64_t>(a.plan.G) * a.d;
        const cca_packed_rows_t kc = {const_cast<void *>(a.Kc), head, a.d}, vc = {const_cast<void *>(a.Vc), head, a.d};
        if (!encode_packed_bf16(enc, &mKc, kc, a.d, a.plan.G, a.Hkv) || !encode_packed_bf16(enc, &mVc, vc, a.d, a.plan.G, a.Hkv))
            return cudaErrorInvalidValue;
    } else {
        mKc = mK;  // no tile of cores is loaded
        mVc = mV;
    }
    p.Hq = a.Hq;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.LSE = a.LSE;
    p.wait_limit_ns = g_wait_limit_ns;
    p.skip_q_load = g_skip_q_load;
    p.plan = a.plan;
    p.by_r = fast_div(a.Hq / a.Hkv);
    for (int c = 0; c <= p.most; ++c) p.by_heads[c] = fast_div(a.Hq >> c);
    p.Q = rows_of<const __nv_bfloat16>(a.Q);
    p.K = rows_of<const __nv_bfloat16>(a.K);
    p.V = rows_of<const __nv_bfloat16>(a.V);
    p.O = rows_of<__nv_bfloat16>(a.O);
    p.Kc = static_cast<const __nv_bfloat16 *>(a.Kc);
    p.Vc = static_cast<const __nv_bfloat16 *>(a.Vc);
    p.o_align32 = ((reinterpret_cast<uintptr_t>(a.O.p) | (a.O.head_stride | a.O.row_stride) * 2) & 31u) == 0 ? 1 : 0;
    const int64_t most = static_cast<int64_t>(a.plan.max_pairs) * a.Hq;
    if (most > 0x7fffffff) return cudaErrorNotSupported;
    const unsigned grid = static_cast<unsigned>(most < di.sms ? most : di.sms);
    if (a.d == 128)
        return start_dependent(attn_packed_tc_kernel<128>, dim3(grid), NUM_THREADS, Layout<128>::SMEM_BYTES, stream, mQ, mK, mV, mKc, mVc, p);
    return start_dependent(attn_packed_tc_kernel<64>, dim3(grid), NUM_THREADS, Layout<64>::SMEM_BYTES, stream, mQ, mK, mV, mKc, mVc, p);
}

}  // namespace cca
