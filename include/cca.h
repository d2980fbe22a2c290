/*
 * cca.h - C ABI of libcca.so: prefill forward of Core Context Aware (CCA)
 * attention on an sm_103a GPU.
 *
 * The method ("Core Context Aware Transformers for Long Context Language
 * Modeling", ICML 2025) replaces self-attention over N tokens by two steps:
 *
 *  1. Global-aware pooling (Method section, pooling equation
 *     c_i = softmax(Q_{ig} K'_{I_i}^T / sqrt(d)) X^G_{I_i}): the sequence is cut
 *     into N/g non-overlapping groups of g tokens; each group becomes one core
 *     key and one core value, the softmax-weighted sum of the group's keys and
 *     values, weighted by the logits of the group's last query against the
 *     group's keys.
 *  2. Fused attention (Method section, fusion equation
 *     Att_i = softmax(Q_i [K^G_{T_i}; K^L_{U_i}]^T / sqrt(d)) [V^G_{T_i}; V^L_{U_i}]):
 *     query i takes ONE softmax over the core tokens of the groups that lie
 *     entirely before its local window, followed by the raw tokens of the
 *     window.
 *
 * Index conventions (0-indexed; the pages leave them open):
 *   lo(i)      = max(0, i - w + 1)            first token of i's window
 *   window     = tokens [lo(i), i]           (n_loc = min(w, i + 1) tokens)
 *   core j     visible to i iff (j + 1) * g <= lo(i)   (n_core = lo(i) / g)
 *   group j    = tokens [j*g, (j+1)*g - 1], scored by the query of token (j+1)*g - 1
 *   GQA        query head h reads KV head h / (Hq / Hkv); a KV head's pooling
 *              logit is the mean of the logits of its Hq/Hkv query heads,
 *              taken before the group softmax.
 *   scale      tau = 1/sqrt(d) unless params.scale > 0; the same tau is used by
 *              both steps.  LSE is the natural log-sum-exp of the tau-scaled
 *              logits over the visible set.
 *
 * Layouts (all contiguous, row-major, d innermost; element type = dtype):
 *   Q  [B, Hq,  N,   d]      K, V   [B, Hkv, N,   d]
 *   Kc [B, Hkv, N/g, d]      Vc     [B, Hkv, N/g, d]
 *   O  [B, Hq,  N,   d]      LSE    [B, Hq,  N]  (always fp32)
 *
 * Ownership and execution: the caller allocates and owns every buffer; all
 * pointers except `params` are DEVICE pointers (16-byte aligned).  The library
 * keeps no allocation and no state between calls.  Calls are asynchronous on
 * `stream` (a cudaStream_t, NULL = legacy default stream); results are
 * defined after the stream reaches the call.  Arithmetic: bf16 inputs with
 * fp32 accumulation and fp32 softmax, outputs rounded to nearest even; f32
 * inputs computed in fp32 throughout.
 *
 * Errors: the return value reports host-side checks and the launch.  Nothing
 * is launched and nothing is written when a check fails.  A device-side
 * give-up (a pipeline wait that exceeded its time limit) is reported by
 * writing CCA_ERR_TIMEOUT into *params.dev_status when that pointer is set
 * (a caller-owned device int32 that the caller zeroes); the kernel then
 * returns without hanging and its outputs are unspecified.
 */
#ifndef CCA_H_
#define CCA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CCA_ABI_VERSION 3

enum cca_status {
    CCA_OK = 0,
    CCA_ERR_INVALID_ARG = -1, /* null/misaligned pointer, bad size, N % g != 0, Hq % Hkv != 0 */
    CCA_ERR_UNSUPPORTED = -2, /* dtype/d combination not built, or the device is not sm_103 */
    CCA_ERR_CUDA = -3,        /* a CUDA runtime/driver call or the launch failed */
    CCA_ERR_TIMEOUT = -4,     /* written to dev_status by a kernel that gave up waiting */
    CCA_ERR_SCRATCH_LIMIT = -5, /* cca_decode_fwd_noalloc: shapes exceed its fixed scratch */
    CCA_ERR_NO_PAGES = -6     /* written to dev_status by cca_pages_reserve: too few free pages */
};

enum cca_dtype {
    CCA_BF16 = 0, /* bfloat16 storage, fp32 accumulation */
    CCA_F32 = 1   /* float32 storage and arithmetic */
};

typedef struct cca_params {
    int32_t B;          /* batch                                  >= 1 */
    int32_t Hq;         /* query heads                            >= 1, multiple of Hkv */
    int32_t Hkv;        /* key/value heads                        >= 1 */
    int32_t N;          /* tokens per sequence                    >= 1, multiple of g */
    int32_t d;          /* head dimension: 64 or 128 (bf16 attention: 128 only) */
    int32_t g;          /* group size                             >= 1 */
    int32_t w;          /* local window                           >= 1 (w >= N allowed) */
    int32_t dtype;      /* enum cca_dtype */
    float scale;        /* softmax scale; <= 0 selects 1/sqrt(d) */
    int32_t *dev_status;/* optional device int32, see "Errors" above */
    int32_t window_mode;/* 0: raw window [lo(i), i] (the method as read here);
                           1: raw window [g*(lo(i)/g), i], reaching back to the group boundary
                              so that cores + window cover every earlier token */
    int32_t pool_mode;  /* 0: softmax weights of the group-last query (the method; with
                              grouped-query attention the r heads' logits are averaged
                              before the softmax);
                           1: mean pooling; 2: element-wise max pooling (the pages' ablations);
                           3: grouped-query pooling averaged after the softmax: each of the
                              r = Hq/Hkv query heads takes its own softmax over the group,
                              scored by its own group-last query, and the group weights are
                              the mean of the r weight vectors (the OpenReview rebuttal's
                              GQA answer leaves this choice open).  Equals 0 when r = 1.
                              Needs r <= 8 (else CCA_ERR_UNSUPPORTED). */
} cca_params_t;

/*
 * cca_pool - global-aware pooling (pooling equation of the Method section).
 * Reads Q (only the last token of every group is used), K and V; writes
 * Kc[b, kv, j, :] = sum_t a_t K[b, kv, j*g + t, :] and the same for Vc, with
 * a = softmax_t(tau * mean_{h in kv} Q[b, h, (j+1)*g - 1, :] . K[b, kv, j*g + t, :]).
 * Supported: dtype bf16 or f32, d in {64, 128}, any g >= 1.
 */
int cca_pool(const void *Q, const void *K, const void *V, void *Kc, void *Vc,
             const cca_params_t *params, void *stream);

/*
 * cca_attn_fwd - fused core/local attention (fusion equation of the Method
 * section).  For every (b, h, i): one softmax over the logits tau*Q_i.Kc_j for
 * visible cores j < lo(i)/g followed by tau*Q_i.K_m for m in [lo(i), i];
 * O_i = the softmax-weighted sum of the matching Vc_j and V_m rows;
 * LSE_i = log-sum-exp of the same logits.  Kc/Vc are the outputs of cca_pool
 * (or any caller-supplied core tokens of that shape).
 * Supported: bf16 with d = 128 (tensor-core kernel), f32 with d in {64, 128}.
 */
int cca_attn_fwd(const void *Q, const void *K, const void *V, const void *Kc, const void *Vc,
                 void *O, float *LSE, const cca_params_t *params, void *stream);

/*
 * cca_attn_fwd_rows - cca_attn_fwd for the query rows [q_off, q_off + n_q) of a
 * sequence of params->N tokens, reading only the raw tokens [kv_off, kv_off +
 * n_kv).  This is the attention of one shard when a sequence is split across
 * ranks along its length: pooling is group-local, so each rank pools its own
 * whole groups; the ranks then share their core tokens (all N/g of them) and
 * each receives the raw rows its first windows reach back to from the ranks
 * before it.  Rows keep their indices in the whole sequence: visibility, cores
 * and windows are exactly those of cca_attn_fwd over N tokens.
 *   Q, O   [B, Hq, n_q, d]     the rows q_off .. q_off + n_q - 1
 *   LSE    [B, Hq, n_q]        fp32
 *   K, V   [B, Hkv, n_kv, d]   the raw tokens kv_off .. kv_off + n_kv - 1
 *   Kc, Vc [B, Hkv, N/g, d]    core tokens of the whole sequence; rows below
 *                              lo(q_off + n_q - 1)/g must be valid
 * Requirements (else CCA_ERR_INVALID_ARG, nothing launched): n_q >= 1,
 * 0 <= kv_off <= first raw token of row q_off's window (lo(q_off), or its
 * group boundary with window_mode 1), q_off + n_q <= kv_off + n_kv <= N.
 * Everything else (support, alignment, errors) as cca_attn_fwd; with q_off = 0,
 * kv_off = 0 and n_q = n_kv = N it is cca_attn_fwd.
 */
int cca_attn_fwd_rows(const void *Q, const void *K, const void *V, const void *Kc, const void *Vc,
                      void *O, float *LSE, int q_off, int n_q, int kv_off, int n_kv,
                      const cca_params_t *params, void *stream);

/*
 * Decoding (one new token per sequence).  The pages describe a decode step that
 * keeps only the core tokens plus the local window in the KV cache and pools a
 * group once it has filled (news write-up, efficiency and KV-cache paragraphs;
 * OpenReview rebuttal, cache-size answer).  Here a decode step at position
 * `pos` computes exactly row `pos` of cca_attn_fwd over the caches.
 *
 * cca_decode_fwd - for every (b, h): one softmax over the visible cores
 * j < lo(pos)/g followed by the window tokens [lo(pos), pos], lo(pos) =
 * max(0, pos - w + 1).
 *   Q      [B, Hq, d]          query of the token at position pos
 *   K, V   [B, Hkv, Ncap, d]   caches; rows [lo(pos), pos] must be valid
 *   Kc, Vc [B, Hkv, Ncap/g, d] core caches; rows [0, lo(pos)/g) must be valid
 *   O      [B, Hq, d]          output (dtype of Q);  LSE [B, Hq] fp32
 *   params.N = Ncap (cache capacity, a multiple of g); 0 <= pos < Ncap.
 *   workspace: caller-owned device buffer of at least
 *   cca_decode_workspace_size(params) bytes (per-split partial results); it
 *   needs no initialisation and is fully rewritten by every call.
 * The keys are split across CTAs (flash-decoding).  For long visible lists
 * with enough (b, kv) pairs to fill the GPU, the splits of each (b, kv) form a
 * thread-block cluster and merge in it: one kernel, the workspace unused.
 * Otherwise the partial results are merged by a second kernel on the same
 * stream.  The kernels are launched as programmatic dependents: the split
 * kernel of whatever the stream ran before the call, the merge of the split
 * kernel.  Each may be scheduled while the
 * grid before it drains, and waits on the device for that grid's completion
 * before it reads anything, so the stream order is kept.  The merge lets its
 * own programmatic dependents (the next decode step's split kernel, say) be
 * scheduled once the split grid has completed.
 * Supported: bf16 or f32, d in {64, 128}, Hq/Hkv <= 8.
 */
int cca_decode_fwd(const void *Q, const void *K, const void *V, const void *Kc, const void *Vc, void *O,
                   float *LSE, int pos, const cca_params_t *params, void *workspace,
                   uint64_t workspace_bytes, void *stream);

/* Kernels one cca_decode_fwd (or _noalloc) call at `pos` launches on the current
 * device: 1 when the splits of each (b, kv) merge inside a thread-block cluster
 * (long visible lists with enough (b, kv) pairs to fill the GPU), 2 for the
 * split kernel and its merge kernel; a negative status on bad arguments. */
int cca_decode_kernels(const cca_params_t *params, int pos);

/* Bytes of workspace cca_decode_fwd needs for these shapes (0 on bad params). */
uint64_t cca_decode_workspace_size(const cca_params_t *params);

/*
 * cca_decode_fwd_noalloc - cca_decode_fwd for callers that cannot allocate
 * device memory.  The pages have no counterpart: this entry point exists for
 * deployments in which this library may not obtain memory of its own, e.g. a
 * plug-in inside a host framework that owns every device allocation through
 * its own pool, a serving loop whose memory budget is fixed at start-up, or a
 * caller that must avoid cudaMalloc's implicit device-wide synchronisation in
 * its decode loop.  Such a caller can still pass its inputs and outputs, but
 * not a workspace.
 *
 * Same arguments, semantics and support as cca_decode_fwd, minus the
 * workspace: the per-split partial results live in one fixed array of
 * CCA_DECODE_NOALLOC_MAX_BYTES inside the library's device code, which every
 * GPU that loads the library holds until the process exits.  Shapes whose
 * cca_decode_workspace_size() exceeds that maximum are rejected with
 * CCA_ERR_SCRATCH_LIMIT before anything is launched.  The function calls no
 * cudaMalloc/cudaFree and no allocating library routine.
 *
 * The first call on a device (with that device current) looks up the array's
 * device address with cudaGetSymbolAddress; make that first call before any
 * stream capture.  The address is kept together with the CUDA context that was
 * current then; a call made under another context (after cudaDeviceReset, for
 * instance) looks it up again, and is then such a first call.  All calls share the one array: calls whose kernels may
 * overlap on a GPU (different streams without ordering) race on it and give
 * undefined results.  Nothing in it needs to start at zero: every call
 * rewrites each partial it later reads.
 */
#define CCA_DECODE_NOALLOC_MAX_BYTES (4ull << 20)
int cca_decode_fwd_noalloc(const void *Q, const void *K, const void *V, const void *Kc, const void *Vc,
                           void *O, float *LSE, int pos, const cca_params_t *params, void *stream);

/*
 * cca_pool_group - pool one newly completed group j of the caches (the
 * pooling equation for a single group): for every (b, kv),
 *   Kc[b, kv, j] = sum_t a_t K[b, kv, j*g + t],  Vc likewise,
 *   a = softmax_t(tau * mean_{h in kv} q[b, h] . K[b, kv, j*g + t]),
 * where q [B, Hq, d] is the query of the group's last token (j+1)*g - 1, i.e.
 * the token just decoded.  K, V [B, Hkv, Ncap, d]; Kc, Vc [B, Hkv, Ncap/g, d];
 * params.N = Ncap; 0 <= j < Ncap/g.  Same support as cca_pool.
 */
int cca_pool_group(const void *q, const void *K, const void *V, void *Kc, void *Vc, int j,
                   const cca_params_t *params, void *stream);

/*
 * cca_prefill_bwd - backward pass of CCA prefill (pooling + fused attention):
 * gradients of the loss sum(dO * O) with respect to Q, K and V.  The pages
 * fine-tune CCA models ("differentiable fusion", digest page; fine-tuning
 * settings, OpenReview rebuttal); this is the gradient of the two equations.
 *   Q, K, V, Kc, Vc  the forward's inputs and core tokens (dtype of params)
 *   O, LSE           the forward's outputs (cca_attn_fwd)
 *   dO               [B, Hq, N, d] upstream gradient (dtype of params)
 *   dQ               [B, Hq, N, d]  fp32, overwritten
 *   dK, dV           [B, Hkv, N, d] fp32, overwritten (they include the paths
 *                    through the core tokens back into the pooled groups)
 *   workspace        caller-owned device buffer of at least
 *                    cca_prefill_bwd_workspace_size(params) bytes
 * All pooling and window modes are supported, d in {64, 128}, bf16 or f32.
 * Max pooling passes each element's gradient to the first row holding the
 * maximum.  bf16 with d = 128 computes the attention gradients on the tensor
 * cores (bf16 operands, fp32 accumulation, P and dS rounded to bf16 before
 * their products); every other case, and the pooling backward, runs on CUDA
 * cores in fp32 (with softmax or mean pooling at bf16, d = 128, the pooling
 * backward's share of each raw token's row is added as the tensor-core kernel
 * writes that row).  A kernel that gives up waiting writes CCA_ERR_TIMEOUT into
 * *params.dev_status when that pointer is set (4-byte aligned); the gradients
 * are then undefined.
 */
int cca_prefill_bwd(const void *Q, const void *K, const void *V, const void *Kc, const void *Vc,
                    const void *O, const float *LSE, const void *dO, float *dQ, float *dK, float *dV,
                    const cca_params_t *params, void *workspace, uint64_t workspace_bytes, void *stream);

/* Bytes of workspace cca_prefill_bwd needs (0 on bad params). */
uint64_t cca_prefill_bwd_workspace_size(const cca_params_t *params);

/*
 * cca_prefill_host - the whole prefill step (cca_pool, then cca_attn_fwd) on
 * HOST buffers: Q, K, V are copied to the device, pooled and attended, and O
 * (plus LSE, Kc, Vc when asked for) copied back.  The (batch, KV head) pairs
 * are independent problems (the pooling equation and the fusion equation of
 * the digest page, Method section, never mix them), so the call cuts them into
 * about eight slices of consecutive pairs and pipelines the slices over three
 * streams: copies in, kernels on `stream`, copies out.  The copies of one slice
 * overlap the kernels of another.
 *   hQ, hK, hV    host (or any UVA-addressable) [B,Hq,N,d] / [B,Hkv,N,d] inputs
 *   hO            host [B,Hq,N,d] output, dtype of params
 *   hLSE          host [B,Hq,N] fp32 output, or NULL to skip it
 *   hKc, hVc      host [B,Hkv,N/g,d] outputs, or both NULL to skip them
 *   workspace     device buffer, 16-byte aligned, of at least
 *                 cca_prefill_host_workspace_size(params) bytes (three slice buffers)
 * Host buffers should be page-locked (cudaHostAlloc / cudaHostRegister): the
 * copies from and to pageable memory are correct, but the driver stages them
 * and the host may block on each, which removes the overlap.
 * The call returns once everything is enqueued.  Work is ordered after what is
 * already queued on `stream`, and `stream` resumes only after the last copy-out,
 * so synchronising `stream` makes every output valid on the host.  The internal
 * streams and events are kept per device for later calls.  Errors: as
 * cca_attn_fwd, checked before anything is enqueued; a CUDA failure after some
 * slices were enqueued returns CCA_ERR_CUDA with the outputs undefined.
 */
int cca_prefill_host(const void *hQ, const void *hK, const void *hV, void *hO, float *hLSE, void *hKc,
                     void *hVc, const cca_params_t *params, void *workspace, uint64_t workspace_bytes,
                     void *stream);

/* Device bytes of workspace cca_prefill_host needs (0 on bad params). */
uint64_t cca_prefill_host_workspace_size(const cca_params_t *params);

/*
 * Rotary positions.  CCA scores queries against keys that already carry their
 * positions; these calls give them.  A pair (x_a, x_b) of a head at position p
 * becomes
 *   y_a = factor * (x_a cos t - x_b sin t),  y_b = factor * (x_b cos t + x_a sin t),
 *   t = p * inv_freq[i],
 * pair i = 0 .. rot/2 - 1 being columns (i, i + rot/2) with layout 0 and
 * (2i, 2i + 1) with layout 1; columns rot .. d - 1 are copied.  The angle is
 * reduced exactly: p times the frequency, held as a 64-bit fraction of a turn,
 * modulo one turn in integer arithmetic, so far positions lose nothing.
 * Frequencies scaled for long contexts come in through inv_freq and factor.
 */
typedef struct cca_rope_params {
    int32_t B, N;             /* batch, rows per sequence                    >= 1 */
    int32_t d;                /* head dimension: 64 or 128 */
    int32_t rot;              /* columns rotated: even, 0 <= rot <= d (0: plain copy) */
    int32_t layout;           /* 0: halves, 1: interleaved */
    int32_t dtype;            /* enum cca_dtype */
    int32_t inverse;          /* 1: rotate by -t (the gradient of the rotation) */
    float factor;             /* scales the rotated columns (attention scaling of long contexts) */
    const double *inv_freq;   /* device [rot/2], radians per position */
    const int32_t *positions; /* device, or NULL: row n is at position start + n */
    int64_t pos_stride;       /* elements between two sequences' positions (0: shared) */
    int64_t start;
} cca_rope_params_t;

/* One tensor of a call: x and y are [B, H, N, d] by strides (elements, of b, h and n;
 * columns contiguous, every row 16-byte aligned).  y may be x with the same strides;
 * otherwise they must not overlap.  A y stride may not make two rows share memory.
 * What is refused as overlapping is told by the spans that the strides cover, with one
 * exception: cca_rope takes two tensors of one packed projection in place, where every
 * token has the one's heads before the other's and the sequences come one after the
 * other. */
typedef struct cca_rope_tensor {
    const void *x;
    void *y;
    int32_t H;
    int64_t x_stride[3], y_stride[3];
} cca_rope_tensor_t;

/* Rotates one or two tensors (queries and keys, with their own head counts) in one launch. */
int cca_rope(const cca_rope_tensor_t *tensors, int n_tensors, const cca_rope_params_t *params, void *stream);

/*
 * Norms of queries and keys for each head, with the rotation in the same pass.  A row x of a head becomes
 *   n = x * r * (offset + weight),  r = (mean of x^2 + eps)^(-1/2),  y = n rotated as by cca_rope
 * (rot 0: not rotated).  The mean goes over all d columns; the weights are [d], one for each column, or
 * [H, d] with weight_heads = H; without weights n = x * r.  Everything between the input and the result
 * is fp32.
 */
typedef struct cca_norm_tensor {
    const void *x;            /* [B, H, N, d] by strides, as in cca_rope_tensor_t */
    void *y;                  /* the result; backward: the gradient of x */
    const void *dy;           /* backward: the gradient of the result (NULL forward) */
    const void *weight;       /* device [weight_heads, d], contiguous, or NULL */
    void *dweight;            /* backward: its gradient, overwritten, or NULL */
    int32_t H;
    int32_t weight_heads;     /* 1 or H */
    int64_t x_stride[3], y_stride[3], dy_stride[3];
} cca_norm_tensor_t;

typedef struct cca_norm_params {
    cca_rope_params_t rope;   /* sizes, type, rotation; inverse must be 0 */
    float eps;                /* >= 0 */
    float offset;             /* added to the weights (1 for weights kept around zero) */
    int32_t weight_dtype;     /* enum cca_dtype, of weight and dweight */
} cca_norm_params_t;

/* One or two tensors (queries and keys) in one launch.  y may be x with the same strides; what may not
 * overlap is as in cca_rope. */
int cca_norm_rope(const cca_norm_tensor_t *tensors, int n_tensors, const cca_norm_params_t *params, void *stream);

/*
 * Its gradient: with dn the rotation back of dy and t = dn * (offset + weight),
 *   dx = r * (t - x * r^2 * mean(t x)),   dweight = sum over rows (and heads that share it) of dn * x * r.
 * The rows' statistics are formed again from x.  The sums behind dweight have a fixed order, so that
 * results repeat to the bit.  y (= dx) may not overlap x or dy.
 *   workspace: 16-byte aligned, at least cca_norm_rope_bwd_workspace_size() bytes; not needed (NULL)
 *   where no dweight is asked for.  Calls that may run at the same time need one each.
 */
int cca_norm_rope_bwd(const cca_norm_tensor_t *tensors, int n_tensors, const cca_norm_params_t *params, void *workspace,
                      uint64_t workspace_bytes, void *stream);
/* Bytes of workspace on the current device (0 where none is needed, and on bad arguments). */
uint64_t cca_norm_rope_bwd_workspace_size(const cca_norm_tensor_t *tensors, int n_tensors, const cca_norm_params_t *params);

/*
 * Paged caches.  A pool holds pages of `rows` rows of every KV head,
 *   K, V [layers, n_pages, Hkv, rows, d],
 * and table[b * cols + c] names the page that holds rows c*rows .. (c+1)*rows - 1 of
 * sequence b (any value outside [0, n_pages), by convention -1, where there is none).
 * The raw tokens and the core tokens of a cache each have a pool and a table; the two
 * may differ in page size.  Decoding reads the core tokens and the window, so the raw
 * pages behind the window can be freed.  A contiguous cache [B, Hkv, Ncap, d] is a pool
 * of B pages of Ncap rows with the table 0 .. B - 1.
 * Lengths, tables, trees and paths are device data: the host never waits, and a
 * captured call serves later lengths.  What they hold is checked on the device: an
 * entry that names no page or a length outside the table is skipped (as described at
 * each call) and reported as CCA_ERR_INVALID_ARG in *dev_status when that pointer is
 * set; nothing out of range is read or written.
 * One status word may serve all the calls of a step, from here on to cca_pages_compact:
 * the first error in it stays, but CCA_ERR_INVALID_ARG gives way to CCA_ERR_NO_PAGES and
 * CCA_ERR_TIMEOUT.  (After a reserve that found too few pages, the calls behind it find
 * none for the new tokens; the word keeps saying why.)  The caller sets it back to 0.
 */
typedef struct cca_pages {
    void *K, *V;              /* device, 16-byte aligned, contiguous */
    const int32_t *table;     /* device [B, cols] */
    int32_t n_pages, rows, cols;
    int32_t layers;           /* cca_pages_copy / cca_pages_compact move every layer; 1 elsewhere */
} cca_pages_t;

/*
 * cca_rope_append - the new tokens of a step: rotates queries and keys and stores keys
 * and values into the raw pages of their sequences, in one launch.  Token t of sequence
 * b goes to row lens[b] + t.  With parents, the tokens are the nodes of a drafted tree
 * (see cca_tree_fwd) and node t is at position lens[b] + depth(t); without, at lens[b] + t.
 *   q       x [B, Hq, N, d] -> y, or NULL;  k, v  x [B, Hkv, N, d], y unused
 *   params  B, N = tokens per sequence, d, rot, layout, dtype, factor, inv_freq as above
 *           (positions, pos_stride, start and inverse must be 0)
 *   lens    device [B];  parents  device [B, N] or NULL (then any N; with it N <= 256)
 *   counts  device [B] or NULL: only the first counts[b] tokens are real
 * Tokens that are not real (past counts, or a node whose chain of parents does not reach
 * the root) are not stored, and their rows of q's output are zero.
 * The pages written must be the sequence's own: cca_pages_reserve gives a sequence that
 * shares a page one of its own first.
 */
int cca_rope_append(const cca_rope_tensor_t *q, const cca_rope_tensor_t *k, const cca_rope_tensor_t *v,
                    const cca_pages_t *raw, const int32_t *lens, const int32_t *parents, const int32_t *counts,
                    int32_t *dev_status, const cca_rope_params_t *params, void *stream);

/*
 * cca_norm_rope_append - cca_rope_append with queries and keys normed for each head before they are
 * rotated (see cca_norm_rope); values are stored as they are.  rope.positions, pos_stride, start and
 * inverse must be 0, and rot may be 0.  Everything else as cca_rope_append.
 */
int cca_norm_rope_append(const cca_norm_tensor_t *q, const cca_norm_tensor_t *k, const cca_rope_tensor_t *v,
                         const cca_pages_t *raw, const int32_t *lens, const int32_t *parents, const int32_t *counts,
                         int32_t *dev_status, const cca_norm_params_t *params, void *stream);

/*
 * cca_tree_fwd - CCA attention of a tree of drafted tokens over paged caches (the fusion
 * equation, for several candidate continuations at once; one token with T = 1).
 * Sequence b has lens[b] committed tokens.  Its T drafted nodes sit in raw rows
 * lens[b] .. lens[b] + T - 1; parents[b*T + t] is the node before t (below t), -1 for a
 * child of the last committed token.  Node t, at depth e below the root, is at position
 * p = lens[b] + e and attends exactly as row p of cca_attn_fwd over the committed tokens
 * followed by its chain: the cores j < lo(p)/g, the committed raw tokens from the window's
 * start on, its ancestors and itself.
 *   Q       [B, Hq, T, d];  O  [B, Hq, T, d];  LSE  [B, Hq, T] fp32
 *   raw     table entries of rows [window start of lens[b], lens[b] + T) must be there, but for
 *           those of padding nodes, which may also lie past the table's end
 *   core    rows [0, lo(lens[b] + T - 1)/g) must be there
 *   parents device [B, T], or NULL for one chain (node t's parent is t - 1)
 *   params  B, Hq, Hkv, d, g, w, dtype, scale, dev_status, window_mode (N is not used)
 * A parent that is neither -1 nor an earlier node ends the chain: such a node and its
 * descendants are empty (O = 0, LSE = -inf), which is also how padding nodes are written
 * (-2).  Keys whose table entry names no page count as not there, and are reported.
 * Keys that a row does not see never reach its output, whatever they hold.
 * workspace: caller-owned, at least cca_tree_workspace_size(params, T) bytes, rewritten by
 * every call; two calls that may run at the same time need one each.
 * O, LSE and the workspace must overlap neither an input nor one another.
 * Precision: scores, sums and outputs are fp32.  In bf16 the softmax weights meet V rounded to
 * bf16, as in cca_attn_fwd; up to 16 rows per KV head (T * Hq / Hkv: plain decoding) they meet it
 * in two bf16 parts, so that an output is off by little more than its own rounding, as it is in
 * cca_decode_fwd.
 * Supported: bf16 or f32, d in {64, 128}, 1 <= T <= min(256, w), B <= 1024.
 */
int cca_tree_fwd(const void *Q, const cca_pages_t *raw, const cca_pages_t *core, const int32_t *lens,
                 const int32_t *parents, int T, void *O, float *LSE, const cca_params_t *params, void *workspace,
                 uint64_t workspace_bytes, void *stream);
/* Bytes of workspace cca_tree_fwd needs on the current device (0 on bad params). */
uint64_t cca_tree_workspace_size(const cca_params_t *params, int T);

/*
 * cca_pool_pages - pools the groups that newly committed tokens complete (the pooling
 * equation), from raw pages into core pages.  Sequence b had lens[b] tokens and gained
 * accepted[b], whose K and V rows lie at lens[b] .. lens[b] + accepted[b] - 1; every group
 * j with lens[b] < (j+1)*g <= lens[b] + accepted[b] is pooled.  The i-th new token's query
 * is Q[b, :, path[b*A + i]] (path device [B, A]: the accepted nodes of the tree), or
 * Q[b, :, i] with path NULL (then A = T).
 *   Q [B, Hq, T, d];  params  B, Hq, Hkv, d, g, dtype, scale, dev_status, pool_mode
 * accepted[b] > A is reported and pools nothing for b; a group with a row, a core page or
 * a path entry that is not there is reported and skipped.
 * Supported: bf16 or f32, d in {64, 128}.
 */
int cca_pool_pages(const void *Q, const cca_pages_t *raw, const cca_pages_t *core, const int32_t *lens,
                   const int32_t *accepted, const int32_t *path, int A, int T, const cca_params_t *params,
                   void *stream);

/*
 * The pages' book: refs[page] is the number of table entries that hold the page; a page
 * with refs 0 is free.  All four calls order their work as if one table row came after
 * the other, and results do not depend on timing.
 * A page that several rows hold stands in the same column of each of them (rows of a page
 * are positions), and at most once in a row: the calls below keep it so.  From a table that
 * breaks this, cca_pages_reserve may take a page away from all its holders; it is free
 * after the call.
 *
 * cca_pages_reserve - room for the rows [lens[b], lens[b] + extra[b]) of every sequence
 * (extra <= 0: none): table entries of that range that name no page get one, and entries
 * whose page is shared get one of their own, but for the page's last holder (copy on
 * write).  Free pages are handed out lowest number first, in row order.  pairs[b] = (old,
 * new) where the page of row lens[b] was replaced and holds committed rows, else (-1, -1):
 * the pages for cca_pages_copy to copy.  If the pool has too few free pages, nothing
 * changes, all pairs are -1 and *dev_status becomes CCA_ERR_NO_PAGES.  A row whose range
 * leaves the table or has lens < 0 is reported (CCA_ERR_INVALID_ARG) and gets nothing.
 *   workspace: 16-byte aligned, at least cca_pages_reserve_workspace_size(B, cols) bytes
 */
int cca_pages_reserve(int32_t *refs, int n_pages, int32_t *table, int B, int cols, int rows, const int32_t *lens,
                      const int32_t *extra, int32_t *pairs, void *workspace, uint64_t workspace_bytes,
                      int32_t *dev_status, void *stream);
uint64_t cca_pages_reserve_workspace_size(int B, int cols);

/*
 * cca_pages_fork - table row dst[i] becomes a second holder of the pages of row src[i]:
 * its first ceil(lens[src[i]] / rows) entries are copied (and counted in refs), the others
 * become -1.  Every entry of a dst row must be free (-1) before.  A pair is reported and
 * skipped when a row is out of range, src = dst, dst holds pages, dst is also a source of
 * the call, or an earlier pair has the same dst.
 */
int cca_pages_fork(int32_t *refs, int n_pages, int32_t *table, int B, int cols, int rows, const int32_t *src,
                   const int32_t *dst, int n, const int32_t *lens, int32_t *dev_status, void *stream);

/*
 * cca_pages_free - entries [first[b], last[b]) of every table row (clamped to the row)
 * give up their pages: refs is counted down and the entry becomes -1.  Entries that name
 * no page are left alone; a page whose refs is already 0 is reported and stays at 0.
 */
int cca_pages_free(int32_t *refs, int n_pages, int32_t *table, int B, int cols, const int32_t *first,
                   const int32_t *last, int32_t *dev_status, void *stream);

/*
 * cca_pages_copy - copies page pairs[i][0] to page pairs[i][1] of the pool, K and V, every
 * layer (the contents behind a page that cca_pages_reserve replaced).  Pairs with a
 * negative entry are skipped.  A pair is reported and skipped when a page is out of range,
 * an earlier pair has the same destination, or its destination is the source of any pair.
 *   params  Hkv, d, dtype, dev_status;  pages  K, V, n_pages, rows, layers;  n <= 65535
 */
int cca_pages_copy(const cca_pages_t *pages, const int32_t *pairs, int n, const cca_params_t *params, void *stream);

/*
 * cca_pages_compact - keeps the accepted nodes of a drafted tree: raw row lens[b] + path[b*A
 * + i] moves to row lens[b] + i for i < accepted[b], K and V, every layer.  The path names
 * nodes from the root down, so it rises: path[i] >= i and path[i] < path[i+1].  A sequence
 * whose path does not, whose accepted is outside [0, A] or whose rows are not all there is
 * reported and left as it is.  The rows lens[b] .. of a sequence lie in pages of its own.
 *   params  B, Hkv, d, dtype, dev_status;  1 <= A <= 256
 */
int cca_pages_compact(const cca_pages_t *pages, const int32_t *lens, const int32_t *path, int A,
                      const int32_t *accepted, const cca_params_t *params, void *stream);

/*
 * Packed sequences: sequences of different lengths one behind the other, [H, T, d] by strides.  Sequence
 * s holds the rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 and knows none of the others: position,
 * groups, windows and cores are counted from its own first row, with the definitions above (its last
 * n % g tokens are in no group).  Rows before cu_seqlens[0] and from cu_seqlens[S] on belong to no
 * sequence; what is written leaves them as they were.
 * The core tokens of sequence s are the rows cu_seqlens[s] / g + j of Kc, Vc [Hkv, T / g, d]
 * (contiguous), j < n / g.
 *
 * cca_pack - reads the lengths once for all the calls of a batch (every layer, forward and backward)
 * and lays out their work in `plan`: the tiles of all sequences by falling cost, every token's position,
 * every group's first token.  The lengths stay on the device: the host never waits, and a captured call
 * serves later lengths.  The calls below read the plan alone; a plan that cca_pack did not finish, or
 * made for another S, T, g, w or window_mode than the call's, is reported in *dev_status
 * (CCA_ERR_INVALID_ARG) and nothing is written.
 * cu_seqlens that fall, start below 0 or end above T are reported and make such a plan.
 */
typedef struct cca_packed {
    void *plan;               /* device, 16-byte aligned, cca_pack_size(S, T, g) bytes */
    uint64_t plan_bytes;
    int32_t S;                /* sequences, 1 .. 65535; any of them may be empty */
    int32_t T;                /* rows of the packed tensors             >= 1 */
    int32_t g;                /* group size                             >= 1 */
    int32_t w;                /* local window                           >= 1; w >= the longest sequence:
                                 full causal attention, no core is visible */
    int32_t window_mode;
} cca_packed_t;

/* Bytes of a plan (0 on bad sizes). */
uint64_t cca_pack_size(int S, int T, int g);
/* Where a plan keeps the tokens' positions: int32 [T], from this byte on (0 for tokens of no sequence). */
uint64_t cca_pack_positions_offset(int S, int T, int g);
int cca_pack(const int32_t *cu_seqlens, const cca_packed_t *packed, int32_t *dev_status, void *stream);

/* A packed tensor [H, T, d]: columns contiguous, every row 16-byte aligned, strides (elements) of head
 * and row, each at least d (where there is more than one).  A result's rows may share no memory with one
 * another nor with another tensor of the call; tensors may be slices of the columns of one wider tensor. */
typedef struct cca_packed_rows {
    void *p;
    int64_t head_stride, row_stride;
} cca_packed_rows_t;

/* params of the calls below: Hq, Hkv, d, dtype, scale, dev_status, pool_mode; the others are not used.
 * Weighted sums are formed in fp32 before they are divided by their weights' sum: values above the largest number divided by
 * the number of a row's keys (of a group's) may overflow in pooling and in fp32 attention; bf16 attention forms such rows again. */

/*
 * cca_pool_packed - the pooling equation for every whole group of every sequence.  Core rows that
 * belong to no group are set to zero.  Supported: bf16 or f32, d in {64, 128}, pool_mode 0 or 1 (the mean: queries and the
 * other tensor's values do not reach it).
 */
int cca_pool_packed(const cca_packed_rows_t *Q, const cca_packed_rows_t *K, const cca_packed_rows_t *V, void *Kc, void *Vc,
                    const cca_packed_t *packed, const cca_params_t *params, void *stream);

/*
 * cca_attn_packed - the fusion equation for every row of every sequence.  O by strides, LSE [Hq, T] fp32.
 * Kc, Vc may be NULL where w >= T.  What a row does not see (later tokens, other sequences, other
 * cores) never reaches its output, whatever it holds; what it sees and is not finite shows in its output column by
 * column (infinities of both signs, and any NaN, as NaN).
 * Supported: bf16 (on the tensor cores) or f32, d in {64, 128}.
 */
int cca_attn_packed(const cca_packed_rows_t *Q, const cca_packed_rows_t *K, const cca_packed_rows_t *V, const void *Kc,
                    const void *Vc, const cca_packed_rows_t *O, float *LSE, const cca_packed_t *packed,
                    const cca_params_t *params, void *stream);

/*
 * cca_packed_clear - sets the rows of no sequence of n <= 4 packed tensors (heads[i] heads each) to zero; all
 * their rows for a plan that cca_pack did not finish or made for other sizes.  params: d, dtype.
 */
int cca_packed_clear(const cca_packed_rows_t *tensors, const int32_t *heads, int n, const cca_packed_t *packed,
                     const cca_params_t *params, void *stream);

/*
 * cca_packed_bwd - gradients of the loss sum(dO * O) through cca_attn_packed and, where w < T,
 * cca_pool_packed, in the inputs' type (rounded once).  Kc, Vc, O, LSE are the forward's.  No sum depends
 * on what ends first: results repeat to the bit (another batch may add up a sequence's in other parts).  bf16: weights and score gradients are rounded to bf16 before the
 * products; dO . O of rows whose keys fit one tile of 128 is formed from the weights, so that the rounding
 * of O does not reach them.  The gradients of a sequence that holds infinities or NaN
 * (in any tensor) are not defined; those of the others are not touched by it.
 *   workspace: 16-byte aligned, at least cca_packed_bwd_workspace_size() bytes, rewritten by every call;
 *   calls that may run at the same time need one each.
 * Support as cca_attn_packed and cca_pool_packed.
 */
int cca_packed_bwd(const cca_packed_rows_t *Q, const cca_packed_rows_t *K, const cca_packed_rows_t *V, const void *Kc,
                   const void *Vc, const cca_packed_rows_t *O, const float *LSE, const cca_packed_rows_t *dO,
                   const cca_packed_rows_t *dQ, const cca_packed_rows_t *dK, const cca_packed_rows_t *dV,
                   const cca_packed_t *packed, const cca_params_t *params, void *workspace, uint64_t workspace_bytes,
                   void *stream);
/* Bytes of workspace cca_packed_bwd needs on the current device (0 on bad arguments). */
uint64_t cca_packed_bwd_workspace_size(const cca_packed_t *packed, const cca_params_t *params);

/* Static English text for a status code (never NULL). */
const char *cca_status_string(int status);

/* CCA_ABI_VERSION of the loaded library. */
int cca_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CCA_H_ */
