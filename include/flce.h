/*
 * flce.h -- C ABI of libflce, a fused linear cross-entropy engine for
 * NVIDIA GB300 (sm_103a).
 *
 * The operation (Liger-Kernel project overview, "Método de API de Baixo
 * Nível": loss = loss_fn(weight, input, target) followed by loss.backward();
 * "Cálculo Preciso": forward and backward are exact, not approximations):
 *
 *   S       = X W^T                 X [N, H] tokens, W [V, H] LM-head weight
 *   lse_i   = log sum_j exp(S_ij)   (natural log)
 *   valid_i = (target_i != ignore_index),  n = sum_i valid_i
 *   loss    = (1/n) sum_{valid i} (lse_i - S_{i, target_i})
 *   G_ij    = valid_i (softmax(S_i)_j - [j == target_i]) * grad_scale / n
 *   dX      = G W   [N, H],   dW = G^T X   [V, H]
 *
 * The N x V logits are never written to device memory: the kernels recompute
 * logit tiles in tensor memory and process the vocabulary in chunks, so the
 * scratch space grows with a chunk width, not with N x V (the pages' "input
 * chunking" and "fusão de kernels", Liger Kernel paper summary, 方法详解, and
 * the overview's "Princípios Técnicos").
 *
 * Conventions shared by every entry point
 *   - X, W and dX are row-major and contiguous, element type opts->dtype
 *     (bf16 by default, or fp32 computed with tf32 tensor-core products);
 *     dW is fp32; target is int64 [N] (int32 [N] when opts->target_is_int32
 *     is set; the pointer is then read as int32_t*).  All of them are device
 *     pointers owned by the caller, except in flce_fwd_bwd_host().
 *   - X, W, dX and dW must be 16-byte aligned and H * sizeof(element) must be
 *     a multiple of 16 bytes; otherwise FLCE_ERR_ALIGN.
 *   - dX and dW are overwritten, never accumulated into.
 *   - When no row is valid (n == 0, including N == 0) the loss is 0 and both
 *     gradients are 0; the call succeeds.
 *   - A target outside [0, V) that is not ignore_index makes the call return
 *     FLCE_ERR_TARGET (synchronous calls) or sets that code in
 *     opts->status_dev (asynchronous calls); outputs are then unspecified.
 *   - Every kernel-side wait is bounded; an expired wait is reported as
 *     FLCE_ERR_TIMEOUT, never as a device trap.
 *   - The library needs a compute capability 10.3 device (FLCE_ERR_ARCH).
 *   - Calls are reentrant; the only process-wide state is a per-device cache
 *     of device attributes and kernel attributes, and one stream-ordered
 *     memory pool per device for the scratch the library allocates itself
 *     (it keeps freed scratch mapped for reuse until the process exits, so
 *     it holds at most the largest scratch of the calls made so far).
 *   - An asynchronous call (opts->sync == 0, host loss NULL, no trace events)
 *     makes only stream-ordered CUDA calls: scratch allocation and release,
 *     memsets and kernel launches.  It can therefore be captured into a CUDA
 *     graph (after one call outside the capture has set up the per-device
 *     state), and replays reproduce an eager call bit for bit.
 *   - Nothing throws across this boundary; every entry returns an int status.
 */
#ifndef FLCE_H_
#define FLCE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FLCE_VERSION 2

#if defined(__GNUC__)
#define FLCE_API __attribute__((visibility("default")))
#else
#define FLCE_API
#endif

typedef enum flce_status {
  FLCE_OK = 0,
  FLCE_ERR_ARG = 1,       /* null pointer, negative or zero size, bad option */
  FLCE_ERR_ALIGN = 2,     /* pointer or row pitch not 16-byte aligned */
  FLCE_ERR_ARCH = 3,      /* device is not compute capability 10.3 */
  FLCE_ERR_TARGET = 4,    /* target outside [0, V) that is not ignore_index */
  FLCE_ERR_WORKSPACE = 5, /* caller workspace smaller than the minimum plan */
  FLCE_ERR_CUDA = 6,      /* CUDA runtime / driver error (see flce_last_error) */
  FLCE_ERR_TIMEOUT = 7    /* a bounded wait inside a kernel expired */
} flce_status;

typedef enum flce_dtype {
  FLCE_BF16 = 0, /* X, W, dX bfloat16; products on tensor cores, fp32 accumulate */
  FLCE_FP32 = 1  /* X, W, dX float32; tf32 tensor-core products, fp32 accumulate */
} flce_dtype;

/* Launch kinds reported by the optional per-launch trace. */
typedef enum flce_trace_kind {
  FLCE_TRACE_LOGITS_LSE = 1,   /* pass 1: logit tiles -> per-tile row statistics */
  FLCE_TRACE_COMBINE = 2,      /* row logsumexp, row loss, mean, n_valid */
  FLCE_TRACE_LOGITS_GRAD = 3,  /* pass 2: logit tiles -> G chunk */
  FLCE_TRACE_DW = 4,           /* dW[chunk] = G_chunk^T X */
  FLCE_TRACE_DX = 5,           /* dX += G_chunk W[chunk] */
  FLCE_TRACE_CONVERT = 6,      /* fp32 dX accumulator -> bf16 dX */
  FLCE_TRACE_CE_COUNT = 7,     /* cross-entropy on logits: valid-row count */
  FLCE_TRACE_CE_ROWS = 8       /* cross-entropy on logits: row statistics + gradient */
} flce_trace_kind;

/*
 * Options.  Initialise with flce_opts_init(); every field then has a usable
 * default.  Pointers marked "optional" may stay NULL.
 */
typedef struct flce_opts {
  int32_t dtype;            /* flce_dtype of X, W and dX (default FLCE_BF16) */
  int32_t sync;             /* 1: block until done and report kernel-side errors
                               (default 1); 0: asynchronous on `stream` */
  void* stream;             /* cudaStream_t to launch on (default NULL = legacy
                               default stream) */
  void* workspace;          /* optional device scratch; NULL = the library
                               allocates it stream-ordered and frees it before
                               returning (stream-ordered) */
  size_t workspace_bytes;   /* size of `workspace` */
  size_t workspace_budget;  /* planner budget when workspace == NULL; 0 = one
                               sixteenth of the N x V fp32 logits, but at
                               least 96 MiB */
  int64_t vocab_chunk;      /* vocabulary columns per chunk; 0 = planner;
                               otherwise a positive multiple of 256 */
  float grad_scale;         /* multiplies G, hence dX and dW (default 1) */
  int32_t target_is_int32;  /* 1: `target` points to int32 ids [N] instead of
                               int64 (default 0) */
  int64_t norm_count;       /* > 0: normalise by this count instead of the
                               local n (a data-parallel shard normalising by
                               the global count); the loss is then
                               sum(row losses) / norm_count */
  float* loss_dev;          /* optional device float: the loss */
  float* lse_out;           /* optional device float[N]: lse_i (natural log) */
  float* loss_rows_out;     /* optional device float[N]: lse_i - S_{i,t_i}, 0
                               for ignored rows */
  int64_t* n_valid_dev;     /* optional device int64: n */
  int32_t* status_dev;      /* optional device int32: flce_status of the
                               kernels (asynchronous error reporting) */
  size_t* workspace_used;   /* optional host size_t: scratch bytes used */
  int64_t* vocab_chunk_used;/* optional host int64: chunk width used */
  void** trace_events;      /* optional cudaEvent_t[trace_capacity]: event 0 is
                               recorded before the first launch and event k
                               after launch k */
  int32_t* trace_kinds;     /* optional int32[trace_capacity]: kind of launch k
                               at index k-1 */
  int32_t trace_capacity;
  int32_t* trace_count;     /* optional host int32: events recorded */
} flce_opts;

/* Fill *opts with defaults (dtype bf16, sync 1, grad_scale 1, rest 0/NULL). */
FLCE_API void flce_opts_init(flce_opts* opts);

/*
 * Loss and both gradients, synchronous, default stream, bf16 inputs.
 *   X [N, H] bf16, W [V, H] bf16, target [N] int64   (device, read only)
 *   loss  host float* (required): the mean loss
 *   dX [N, H] bf16 and dW [V, H] fp32 (device, written)
 * Argument order: input rows, LM-head weight, targets (the hidden-states-first
 * call of the Liger Kernel command sheet, 常用示例); the Python binding keeps
 * the overview's loss_fn(weight, input, target) order instead.
 */
FLCE_API int flce_fwd_bwd(const void* X, const void* W, const int64_t* target, int64_t N, int64_t H,
                 int64_t V, int64_t ignore_index, float* loss, void* dX, float* dW);

/*
 * As flce_fwd_bwd with options (NULL = defaults).  `loss` (host) may be NULL
 * when opts->sync == 0; results then appear in the optional device outputs
 * once `stream` reaches them.  A non-NULL host `loss` forces a synchronous
 * call.
 */
FLCE_API int flce_fwd_bwd_ex(const void* X, const void* W, const int64_t* target, int64_t N, int64_t H,
                    int64_t V, int64_t ignore_index, float* loss, void* dX, float* dW,
                    const flce_opts* opts);

/*
 * Loss only (pass 1 and the row combine; no gradients, no G chunk).  Same
 * arguments and options as flce_fwd_bwd_ex without dX/dW.  Per-row outputs
 * (lse_out, loss_rows_out) make it an evaluation path.
 */
FLCE_API int flce_fwd(const void* X, const void* W, const int64_t* target, int64_t N, int64_t H,
             int64_t V, int64_t ignore_index, float* loss, const flce_opts* opts);

/*
 * Cross-entropy on logits that are already materialised in device memory
 * (the overview's LigerCrossEntropyLoss, "Kernels Básicos"; in-place
 * gradient as in "Operações In-Place"): the same loss and reductions as
 * above with S given directly.
 *   logits [N, V] of element type opts->dtype (bf16 or fp32), row-major
 *   target [N] int64;   loss: host float*, or NULL when opts->sync == 0
 *   dlogits [N, V], same type: dS = valid (softmax - onehot) * grad_scale / n;
 *   it may be the logits buffer itself (the gradient overwrites the logits,
 *   each element after it has been read); NULL computes the loss only.
 * A -inf logit (a masked entry) adds nothing to lse and gets a zero
 * gradient; a row needs one finite logit.  grad_scale may be of any sign;
 * rows whose target is ignore_index get a zero gradient.
 * Optional outputs and error reporting as for flce_fwd_bwd_ex (lse_out,
 * loss_rows_out, loss_dev, n_valid_dev, status_dev, trace).  The scratch
 * space is 12 N bytes plus a few KB.  Memory traffic: one read of the logits
 * from HBM and, with a gradient, one write (the second read of each row
 * comes from shared memory for its last 96 KB, else from L2).
 */
FLCE_API int flce_ce_fwd_bwd(const void* logits, const int64_t* target, int64_t N, int64_t V,
                             int64_t ignore_index, float* loss, void* dlogits,
                             const flce_opts* opts);

/*
 * End-to-end variant on HOST buffers: copies X, W and target to the device,
 * runs the path, and copies loss, dX and dW back.  The W upload goes in
 * pieces on a second stream with pass 1 following piece by piece, and each
 * vocabulary chunk's dW rows are copied back as soon as they are final, while
 * later chunks compute.  Device buffers come from the library's memory pool
 * (stream-ordered).  Pinned host memory gives asynchronous, overlapping
 * copies; pageable memory works but serialises them.  Always synchronous.
 */
FLCE_API int flce_fwd_bwd_host(const void* X_host, const void* W_host, const int64_t* target_host,
                      int64_t N, int64_t H, int64_t V, int64_t ignore_index, float* loss,
                      void* dX_host, float* dW_host, const flce_opts* opts);

/*
 * Scratch bytes a call needs.  with_grads = 0 for flce_fwd, 1 for the
 * gradient entry points.  The plan depends on N, H, V, dtype, vocab_chunk
 * and workspace_budget from `opts` (NULL = defaults).
 */
FLCE_API size_t flce_workspace_bytes(int64_t N, int64_t H, int64_t V, int with_grads,
                            const flce_opts* opts);

/* Static text for a status code. */
FLCE_API const char* flce_status_str(int status);

/* Text of the last error on the calling thread (empty if none). */
FLCE_API const char* flce_last_error(void);

/* FLCE_VERSION of the loaded library. */
FLCE_API int flce_version(void);

/* sizeof(flce_opts) as compiled into the library (lets bindings check their
 * mirror of the struct). */
FLCE_API size_t flce_opts_sizeof(void);

/*
 * Self-test of the kernels' bounded waits (the failure-detection path of
 * every kernel in this library): one block waits on an mbarrier that nothing
 * will arrive on.  The wait must give up after limit_ns nanoseconds (at most
 * 2e9), record the expiry in the status word and let the kernel end
 * normally; the call then returns FLCE_ERR_TIMEOUT, the context stays
 * usable, and later calls work.  Returns FLCE_OK only if the wait did not
 * expire (a fault in the mechanism).  Synchronous; allocates a few bytes.
 */
FLCE_API int flce_selftest_wait_expiry(int64_t limit_ns);

/*
 * Scale and convert a gradient on the device, in one pass over memory:
 *   dst[i] = (dst type)(src[i] * *scale_dev)   (bf16: round to nearest even)
 * This is the step of `loss.backward()` after the overview's
 * loss = loss_fn(weight, input, target) ("Método de API de Baixo Nível"): the
 * gradients were computed in the forward call (dW fp32, dX in the input
 * type), and the backward multiplies them by the incoming grad_output and
 * casts dW to the weight's type.
 *   src [n] of type src_dtype and dst [n] of type dst_dtype (FLCE_BF16 or
 *   FLCE_FP32), device memory; dst may be src itself when the two types are
 *   equal (in place); any other overlap is rejected.
 *   scale_dev: device float (e.g. grad_output), or NULL for 1.
 *   stream: cudaStream_t to launch on (NULL = legacy default stream).
 * Asynchronous.  FLCE_ERR_ARG on n < 0, an unknown type, a null buffer with
 * n > 0, or a forbidden overlap.
 */
FLCE_API int flce_scale_convert(const void* src, int32_t src_dtype, void* dst,
                                int32_t dst_dtype, int64_t n, const float* scale_dev,
                                void* stream);

/*
 * Loss-only pass (the work of flce_fwd) that allocates no device memory.
 * The paper has no counterpart to this entry point; it exists for callers
 * that cannot call cudaMalloc at the point where the loss is needed: a host
 * application that plans all device memory up front in its own arena, a
 * plugin whose execute step may not allocate, or a latency-bound loop where
 * an allocation could synchronise the device or fail under fragmentation.
 *
 * Its scratch space is a static device array inside libflce of
 * 32 MiB (33554432 bytes); every device the library runs on holds it until
 * the process exits.  A problem whose loss-only plan needs more (about
 * 4 * N * ceil(V / 256) + 8 * N bytes plus a few KB; flce_workspace_bytes()
 * with with_grads = 0 gives the exact figure) is rejected with
 * FLCE_ERR_WORKSPACE before anything is launched.
 *
 *   X [N, H], W [V, H] of element type `dtype` (FLCE_BF16 or FLCE_FP32),
 *   target [N] int64: device inputs, read only.
 *   loss_dev (required), lse_out [N], n_valid_dev, status_dev: device outputs
 *   as in flce_opts (NULL skips the optional ones); status_dev receives the
 *   kernels' flce_status (bad targets, expired waits).
 *   stream: cudaStream_t to launch on (NULL = legacy default stream).
 * The call is asynchronous: results are valid once `stream` reaches them.
 *
 * The first call on a device looks up the device address of the static
 * array with cudaGetSymbolAddress (once per device, with that device
 * current); make that first call before any stream capture.  All calls share
 * the one array and each leaves its contents behind: calls that may overlap
 * on the GPU (different streams or host threads without ordering between
 * them) race on it and must be serialised by the caller.
 */
FLCE_API int flce_fwd_noalloc(const void* X, const void* W, const int64_t* target, int64_t N,
                              int64_t H, int64_t V, int64_t ignore_index, int32_t dtype,
                              float* loss_dev, float* lse_out, int64_t* n_valid_dev,
                              int32_t* status_dev, void* stream);

/* ------------------------------------------------------------------------
 * Operators around the head: what feeds X, what takes dX back, and what turns
 * a matrix's gradient into an update.  They use these fields of flce_opts
 * (NULL = defaults) and ignore the rest: dtype, sync, stream, workspace,
 * workspace_bytes, workspace_used, status_dev, target_is_int32 (for token
 * ids).  Conventions on status, scratch, streams and graph capture are those
 * at the top of this file.  A call with opts->sync == 0 and a NULL status_dev
 * reports no kernel-side error; the outputs it names for such a case stand.
 * ------------------------------------------------------------------------ */

/*
 * Embedding lookup: Y[i] = scale * W[ids[i]], scaled in fp32 and rounded once
 * to opts->dtype.
 *   W [V, H] and Y [N, H] of type opts->dtype, row-major, contiguous, 16-byte
 *   aligned, H * sizeof(element) a multiple of 16, H <= 2^20; ids [N] int64
 *   (int32 with opts->target_is_int32); scale finite.
 * A token whose id is ignore_index gets a row of zeros.  So does a token whose
 * id is outside [0, V), which also reports FLCE_ERR_TARGET.
 */
FLCE_API int flce_embed_fwd(const void* W, const void* ids, int64_t N, int64_t H, int64_t V,
                            float scale, int64_t ignore_index, void* Y, const flce_opts* opts);

/*
 * Its gradient: dW[v] = scale * sum of dY[i] over the tokens i with ids[i] == v,
 * or dW[v] += that sum when accumulate is not 0 (a weight tied to the head's:
 * dW then holds what flce_fwd_bwd() left there; rows that no token has are not
 * touched).  Equal ids are added in fp32 in a fixed order, so the result does not
 * change from run to run: in ascending token order within pieces of 32 to 64 of them,
 * then the pieces' sums, in ascending order within eighths of them.  The length of a
 * piece depends on N and H, so other tokens in the batch may change the last bits.
 * What is added to an old value is added at L2, where numbers below 2^-126 are zero.
 *   dY [N, H] of type opts->dtype; dW [V, H] fp32; alignment as above.
 * Ignored and out-of-range ids take no part (the latter report
 * FLCE_ERR_TARGET).  N == 0 clears dW, or leaves it when accumulate is set.
 * Scratch: two fp32 rows per 4 to 64 tokens and 8 bytes per token, 24 from 2049 tokens
 * on (from 4097 beside 64 MiB or more of dW that are cleared while the ids are sorted);
 * opts->workspace_used reports it.
 */
FLCE_API int flce_embed_bwd(const void* dY, const void* ids, int64_t N, int64_t H, int64_t V,
                            float scale, int64_t ignore_index, float* dW, int32_t accumulate,
                            const flce_opts* opts);

/*
 * Causal attention over packed sequences with grouped heads.  Sequence b is
 * tokens cu_seqlens[b] .. cu_seqlens[b+1]-1 of the T tokens; a token sees the
 * tokens of its own sequence up to itself.  For query head h and kv head
 * h / (heads_q / heads_kv):
 *   S = scale Q K^T,  lse_i = ln sum_{j <= i} exp S_ij,  P = exp(S - lse),  O = P V
 * and for the gradients, with delta_i = sum_d dO_id O_id:
 *   dS = P o (dO V^T - delta),  dQ = scale dS K,
 *   dK = scale dS^T Q and dV = P^T dO, summed over the query heads of the group.
 * Products are bf16 with fp32 sums; P and dS are rounded to bf16 for theirs, and
 * delta takes o as it is stored.
 *
 * Every tensor is bf16 [T, heads, head_dim] with a contiguous last axis and
 * its own token and head strides in elements (multiples of 8, not 0, so q, k
 * and v may be slices of one projection's output), 16-byte aligned; lse is
 * fp32 [heads_q, T], contiguous.  cu_seqlens: int32 [batch + 1] on the device,
 * 0 <= cu_seqlens[0] <= ... <= cu_seqlens[batch] <= T; offsets that break this
 * are reported as FLCE_ERR_ARG and count as no sequence at all.  A sequence
 * may be empty.  Tokens outside every sequence get zeros in o, dq, dk and dv
 * and -inf in lse; what their inputs hold is not used.
 * Outputs share no element with the inputs or with one another, except that a gradient
 * may take o's place; slices of one buffer that interleave share none.  Overlaps of o
 * with q, k, v, and of the gradients with q, k, v, dO and one another, are refused with
 * FLCE_ERR_ARG where address, strides and sizes tell (same first element; equal token
 * strides).
 * A NaN or infinity reaches what the formulas take it to: nothing of another
 * sequence, o, lse and dq of no token before the one whose k or v it is in, and dk and
 * dv of no token after the one whose q or dO it is in.
 */
typedef struct flce_attn {
  int64_t T;                 /* tokens, < 2^31 - 256 */
  int64_t batch;             /* sequences, >= 0 */
  const int32_t* cu_seqlens;
  int32_t heads_q, heads_kv; /* heads_kv divides heads_q */
  int32_t head_dim;          /* a multiple of 8, 8 .. 128 */
  float scale;               /* > 0, finite */
  const void* q;             /* each followed by its token and head strides */
  int64_t q_token, q_head;
  const void* k;
  int64_t k_token, k_head;
  const void* v;
  int64_t v_token, v_head;
  void* o;                   /* written by flce_attn_fwd, read by flce_attn_bwd */
  int64_t o_token, o_head;
  float* lse;                /* likewise */
  const void* dO;            /* the rest: flce_attn_bwd only */
  int64_t dO_token, dO_head;
  void* dq;
  int64_t dq_token, dq_head;
  void* dk;
  int64_t dk_token, dk_head;
  void* dv;
  int64_t dv_token, dv_head;
} flce_attn;

FLCE_API int flce_attn_fwd(const flce_attn* a, const flce_opts* opts);
FLCE_API int flce_attn_bwd(const flce_attn* a, const flce_opts* opts);

/* sizeof(flce_attn) as compiled into the library. */
FLCE_API size_t flce_attn_sizeof(void);

/*
 * Orthogonalises matrices by Newton-Schulz products (the update of a
 * projection whose singular values are to become about 1):
 *   X = G / (|G|_F + eps);  `steps` times:  A = X X^T,  X = a X + (b A + c A^2) X
 * (with X^T X on the other side when rows > cols, which gives the same X).
 *   G [batch, rows, cols] of type opts->dtype, contiguous; out bf16, same shape,
 *   may not overlap G.  rows, cols <= 2^20; empty matrices are allowed.
 *   coeffs: {a, b, c} on the host, or NULL for {3.4445, -4.7750, 2.0315}.  A
 *   polynomial s (a + b s^2 + c s^4) that takes singular values of [0, 1] out
 *   of the range of the products (|s| < 3.8, |b s^2 + c s^4| < 15) within
 *   `steps` steps (1 .. 64) is refused with FLCE_ERR_ARG.
 *   eps >= 0; a matrix of zeros gives zeros when eps > 0, and NaN when eps == 0.
 * Products take fp16 operands with fp32 sums, beside an fp32 X; the result is
 * rounded to bf16 once.  |G|_F is summed in fp32, with G scaled by a power of two
 * where fp32 would not hold the squares: any finite entries will do.
 * Scratch: about 8 bytes per element of G and 4 per element of A.
 */
FLCE_API int flce_orthogonalize(const void* G, int64_t batch, int64_t rows, int64_t cols,
                                int32_t steps, const float* coeffs, float eps, void* out,
                                const flce_opts* opts);

/*
 * The tile shapes that flce_orthogonalize takes for a step's three products (X X^T,
 * A^2, B X) on a device of `sms` SMs, so that a test can tell what it reaches:
 * 0 CTA pairs, 1 single CTAs, 2 K shared out over a cluster, 3 A^2 and B X in one
 * launch.  Host only.
 */
FLCE_API int flce_selftest_ortho_shapes(int64_t batch, int64_t rows, int64_t cols, int32_t sms,
                                        int32_t shapes[3]);

/* ------------------------------------------------------------------------
 * Between a model's blocks: the residual join with its norms, and checkpoints
 * of activations in 8 bits.  Options, status, scratch, streams and capture as
 * for the operators around the head.
 * ------------------------------------------------------------------------ */

typedef enum flce_norm {
  FLCE_NORM_RMS = 0,  /* n(x) = x / sqrt(mean(x^2) + eps) */
  FLCE_NORM_LAYER = 1 /* n(x) = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) */
} flce_norm;

typedef enum flce_gate {
  FLCE_GATE_NONE = 0,
  FLCE_GATE_SCALAR = 1,  /* one value, a parameter */
  FLCE_GATE_CHANNEL = 2, /* [H], a parameter */
  FLCE_GATE_TOKEN = 3,   /* one value per token, gate_row elements apart */
  FLCE_GATE_FULL = 4     /* [N, H], rows gate_row elements apart */
} flce_gate;

typedef enum flce_act {
  FLCE_ACT_NONE = 0,
  FLCE_ACT_SIGMOID = 1,
  FLCE_ACT_TANH = 2
} flce_act;

/*
 * Residual join: what stands between a block's output y and the next block's input z.
 *   u     = n(y) * w_post + b_post      (post_norm; else u = y)
 *   h_out = alpha h + beta act(gate) u  (without h: the second term; without gate: 1)
 *   z     = n(h_out) * w_pre + b_pre    (pre_norm; else no z)
 * with n the RMS or layer norm over the H elements of a token.  All of it is computed in
 * fp32.  A sigmoid is off by 3.5 units in its last place at most, a tanh by 2; of gates per
 * element beside a bf16 stream a sigmoid may be off by 2^-16 of itself.  Their slopes are
 * a (1 - a) and 1 - a^2 in fp32, off by up to 2^-21 of 1 where a gate is saturated.  h_out
 * is rounded to the stream's type, and z is the norm of h_out as it is stored, so that the
 * gradients, which read the stored h_out, are those of what was computed; z is rounded once.
 *
 * y and z (dy, dz and gates per token) have type opts->dtype; the stream (h, h_out, dh,
 * dh_out) has it too, or is fp32 with stream_fp32.  Parameters (weights, biases, gates of
 * kind SCALAR and CHANNEL) have type opts->dtype, or are fp32 with params_fp32.  A weight
 * or bias may be NULL; those of a norm that there is not, and their gradients, are neither
 * read nor written, whatever they point to.  H is a multiple of 8, 8 .. 16384; N < 2^31.
 * Row tensors have a contiguous last axis and a row stride in elements of their own (a
 * multiple of 8, at least H; gate_row of kind TOKEN: at least 1); tensors are 16-byte
 * aligned (gates of kind SCALAR and TOKEN to their element).
 * h_out may be h itself and z may be y; dh may be dh_out itself, and dy may be dz (same
 * address, same stride).  Any other overlap of an output with an input or another output
 * is refused with FLCE_ERR_ARG where addresses, strides and sizes tell; row tensors that
 * interleave in one buffer at equal strides share nothing.
 * A token's NaN or infinity stays in its own row of h_out, z, dh, dy and per-token gates'
 * gradients; gradients of parameters are sums over the tokens.
 *
 * Forward.  stats, fp32 [4, N], optional: mean and 1 / sqrt(variance + eps) of y, then of
 * h_out; zeros where there is no such norm, means of 0 for RMS.  h_out is optional.
 * z_ckpt, optional: flce_ckpt_bytes(N, H) bytes that receive what flce_ckpt_save() makes
 * of the stored z.
 *
 * Backward, at y, h_out (read with pre_norm) and stats as the forward pass left them, and
 * the gradients dz (pre_norm) and dh_out (optional: what arrives on the stream besides):
 *   dy; dh, optional; dgate of the gate's shape (per token: opts->dtype, dgate_row apart;
 *   SCALAR and CHANNEL: fp32); dw_post, db_post, dw_pre, db_pre, fp32 [H], each optional.
 * dgate is required with a gate.  Sums over tokens are fp32: the same call gives the same
 * bits.  Their order goes by N, H, the types, the form of the join (norms, the gate's kind,
 * whether a bias is given or its gradient wanted) and the device: its number of SMs and, for
 * rows that several of them share, how many clusters of them run at once.
 * N == 0 makes the parameters' gradients 0.
 * Scratch: forward none; backward up to 32 KB per SM and gradient of a parameter.
 */
typedef struct flce_resnorm {
  int64_t N, H;
  int32_t norm;               /* flce_norm */
  int32_t post_norm, pre_norm;
  int32_t stream_fp32, params_fp32;
  int32_t gate_kind;          /* flce_gate */
  int32_t gate_act;           /* flce_act */
  float alpha, beta;          /* finite */
  float eps;                  /* >= 0, finite */
  const void* y;              /* each row tensor followed by its row stride */
  int64_t y_row;
  const void* h;              /* forward; NULL: none */
  int64_t h_row;
  const void* gate;
  int64_t gate_row;
  const void* w_post;
  const void* b_post;
  const void* w_pre;
  const void* b_pre;
  void* h_out;                /* written by flce_resnorm_fwd, read by flce_resnorm_bwd */
  int64_t h_out_row;
  float* stats;               /* likewise */
  void* z;                    /* forward */
  int64_t z_row;
  void* z_ckpt;
  const void* dz;             /* the rest: backward */
  int64_t dz_row;
  const void* dh_out;
  int64_t dh_out_row;
  void* dy;
  int64_t dy_row;
  void* dh;
  int64_t dh_row;
  void* dgate;
  int64_t dgate_row;
  float* dw_post;
  float* db_post;
  float* dw_pre;
  float* db_pre;
} flce_resnorm;

FLCE_API int flce_resnorm_fwd(const flce_resnorm* a, const flce_opts* opts);
FLCE_API int flce_resnorm_bwd(const flce_resnorm* a, const flce_opts* opts);

/* sizeof(flce_resnorm) as compiled into the library. */
FLCE_API size_t flce_resnorm_sizeof(void);

/*
 * Activation checkpoints in 8 bits.  32 consecutive values of a row share a scale 2^e:
 * e is the smallest with |value| <= 448 2^e for all of them, but within -117 .. 119, and
 * a value is stored as the e4m3 number next to value * 2^-e (ties to even).  So a value
 * is off by at most 2^-4 of itself or 2^(e-10), whichever is more (values above
 * 1.75 2^127 come back as that).  What is stored is exact in bf16.  A group that holds a
 * NaN or an infinity comes back as NaN, all of it.
 *
 * A checkpoint of [N, H] is one buffer of flce_ckpt_bytes(N, H) bytes, 16-byte aligned:
 * codes [N, P] with P = 32 ceil(H / 32), zeros from column H on, then scale bytes
 * [N, 4 ceil(P / 128)], e + 127 each, or 255 for a group of NaN, zeros behind the last.
 * Calls that read one take only what flce_ckpt_save() or flce_resnorm_fwd() can write.
 */

/* N (P + 4 ceil(P / 128)); 0 where N or H is out of range (0 .. 2^31 - 1, 1 .. 2^20). */
FLCE_API size_t flce_ckpt_bytes(int64_t N, int64_t H);

/*
 * ckpt = x, for x [N, H] of type opts->dtype, rows x_row elements apart; and x = ckpt.
 * H a multiple of 8, up to 2^20; x_row a multiple of 8, at least H; x 16-byte aligned.
 */
FLCE_API int flce_ckpt_save(const void* x, int64_t x_row, int64_t N, int64_t H, void* ckpt,
                            const flce_opts* opts);
FLCE_API int flce_ckpt_load(const void* ckpt, int64_t N, int64_t H, void* x, int64_t x_row,
                            const flce_opts* opts);

/*
 * Weight gradient of a projection Y = X W^T (W [O, I]) from X's checkpoint:
 *   dW = dY^T X, or dW += dY^T X when accumulate is not 0
 *   dY [N, O] bf16, rows dY_row elements apart (a multiple of 8, at least O), 16-byte
 *   aligned; ckpt of [N, I]; dW [O, I] fp32, contiguous, 16-byte aligned.  O and I are
 *   multiples of 8, up to 2^20; N < 2^31.  opts->dtype must be FLCE_BF16.
 * Products are bf16, exact for the stored X.  Sums are fp32, in an order that N, O, I and the
 * device's number of SMs fix; where they pass through the tensor core's accumulators, 2048
 * tokens at most, each 16 tokens' sum is cut off, not rounded: 6e-7 to 8e-7 of dW by norm for
 * inputs of random sign, 2.4e-6 for those of one sign, whatever N.  N == 0 makes dW 0, or
 * leaves it when accumulate is set.
 * Scratch: X in bf16, 2 N I bytes; and 256 KB per SM where the last tiles are shared out
 * along the tokens (opts->workspace_used tells).
 */
FLCE_API int flce_ckpt_wgrad(const void* dY, int64_t dY_row, const void* ckpt, int64_t N,
                             int64_t O, int64_t I, float* dW, int32_t accumulate,
                             const flce_opts* opts);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_H_ */
