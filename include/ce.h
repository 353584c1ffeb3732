/*
 * ce.h -- C ABI of the GB300 (sm_103a) softmax cross-entropy library (libce.so).
 *
 * The operation: for a [n_rows, vocab] logits matrix X (row stride ld
 * elements), targets t, optional class weights w, label smoothing eps and a
 * reduction, compute the cross-entropy loss and its gradient with respect to
 * X, writing the gradient over X. Per valid row i (t_i != ignore_index and
 * 0 <= t_i < vocab):
 *
 *   loss_i = (1-eps) * w_{t_i} * (LSE_i - x_{i,t_i})
 *          + (eps/V) * sum_c w_c * (LSE_i - x_ic),   LSE_i = log sum_c exp(x_ic)
 *   dX_ic  = s_i * [ (1-eps) * w_{t_i} * (p_ic - [c == t_i])
 *                    + (eps/V) * (p_ic * W_all - w_c) ],  p = softmax(x_i)
 *
 * with W_all = sum_c w_c, W_y = sum over valid rows of w_{t_i} (the
 * non-ignored count when unweighted), s_i = g / W_y for mean, g for sum and
 * g_i for none. Rows that are not valid contribute loss 0 and gradient 0.
 * Unweighted this is (softmax - (1-eps) onehot - eps/V) * g / N.
 *
 * Sources: Liger-Kernel PR "perf(ce): single-shot dx_y gradient correction
 * - #1268" (review diff: the eps/V term and the weighted true-class term;
 * the #1329 commit message quoted there: dx_y recomputed once in fp32 and
 * stored once, the logits buffer holding the gradient; the #1290 commit
 * message: gradient scaled in place, peak memory one logits tensor);
 * Liger-Kernel PR "perf(flce): drop host syncs that do not feed the
 * computation - #1622" (Summary: normalisers, reductions, device-side
 * grad_output == 1 skip, no host syncs); TransformerEngine PR #2325 "change
 * fused cross entropy backward grad to fp32 and reduce one read/write"
 * (forward saves per-row m, d, X_y and the smoothing sum; backward forms the
 * gradient in fp32 from them).
 *
 * Conventions for every entry point:
 *  - Pointers marked "device" are CUDA device (or managed) memory owned by
 *    the caller. The library allocates nothing and keeps no pointer after a
 *    call returns.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream). Every call
 *    only enqueues work on it and returns; nothing waits for the GPU, except
 *    ce_get_status, which synchronises `stream` explicitly.
 *  - The return code reports host-side argument checks and launch errors.
 *    On an error nothing has been enqueued (argument errors) or the CUDA
 *    error of the failed launch is reported (CE_ERR_CUDA, see
 *    ce_last_cuda_error). Data errors found on the device (a target outside
 *    [0, vocab) that is not ignore_index) set bits in the workspace status
 *    word; such rows are treated as ignored.
 *  - The workspace is scratch owned by the caller, at least
 *    ce_workspace_size() bytes, 256-byte aligned. Calls that share a
 *    workspace must be ordered on one stream (or otherwise serialised).
 *    Its contents need no initialisation.
 */
#ifndef CE_H
#define CE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CE_OK = 0,
    CE_ERR_INVALID_ARG = 1,   /* a pointer, size, stride or enum is invalid */
    CE_ERR_UNSUPPORTED = 2,   /* valid but not supported (e.g. misaligned for the asked variant) */
    CE_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
    CE_ERR_WORKSPACE = 4      /* workspace missing, too small or misaligned */
} ce_status;

typedef enum { CE_RED_NONE = 0, CE_RED_MEAN = 1, CE_RED_SUM = 2 } ce_reduction;

/* storage type of the logits / gradient buffer */
typedef enum { CE_DT_F32 = 0, CE_DT_BF16 = 1, CE_DT_F16 = 2 } ce_dtype;

/* bits of the device status word (ce_get_status) */
#define CE_FLAG_TARGET_OUT_OF_RANGE 0x1u /* some target was neither ignore_index nor in [0, vocab) */
#define CE_FLAG_NO_VALID_ROWS 0x2u       /* mean over zero valid rows: loss and gradient set to 0 */
#define CE_FLAG_WAIT_TIMEOUT 0x4u        /* a device-side wait gave up (results invalid) */
#define CE_FLAG_BAD_OFFSETS 0x8u         /* sequence offsets that fall or leave [0, n_rows] */

/* ce_params.variant: which kernels ce_fwd_bwd uses */
#define CE_VARIANT_AUTO 0   /* the library picks (ce_select_variant) */
#define CE_VARIANT_SPLIT 1  /* ce_forward then ce_backward kernels (row read twice) */
#define CE_VARIANT_FUSED 2  /* fused kernel; CE_ERR_UNSUPPORTED if the rows do not allow it */
#define CE_VARIANT_ROWPASS 3 /* one kernel, each row read twice, the second read from L2 */
#define CE_VARIANT_STREAM 4  /* as ROWPASS, the two passes streamed through a shared-memory
                                ring by bulk copies (any row alignment: the part of a row
                                before its first and after its last 16-byte boundary goes
                                through plain accesses) */
/* bits 8..15 of variant: fused-kernel cluster size override, or CTAs per SM
 * of the row-pass and stream kernels (0 = automatic) */
#define CE_VARIANT_CLUSTER_SHIFT 8
/* the workspace already holds this batch's normalisers from ce_prepare (same
 * target, weights, n_rows and reduction): ce_forward / ce_backward /
 * ce_fwd_bwd skip their own normaliser kernel */
#define CE_VARIANT_PREPARED 0x10000
/* bits 20..30 of variant: stream-kernel tuning (0 = the library's choice):
 * 1 = 16 consumer warps and one CTA per SM, 2 = second pass over each row's
 * chunks in reverse order, 4 = first pass without the L2 evict-last policy,
 * 8 = a cluster of two CTAs per row (each streams half the row),
 * 16 = three CTAs per SM with a smaller ring, 32 = with 16: a cluster of four
 * CTAs per row (each streams a quarter), 64 = with 16, for class-weighted
 * label smoothing on bf16 / f16 rows: the class weights of the second pass
 * bulk-copied into a shared-memory ring (other rows ignore the bit);
 * bits 7..9 of the tuning value (128 x k, k = 0..7): the first k/8 of the
 * first-pass chunks of each row part carry an L2 evict-first hint (useful
 * with 2, where the rows waiting for their second pass exceed the L2);
 * 1024 = with 64 and one CTA per row: the weight ring at two CTAs per SM
 * with a deeper logits ring */
#define CE_VARIANT_TUNE_SHIFT 20

typedef struct ce_params {
    int64_t n_rows;             /* BT >= 0 */
    int64_t vocab;              /* V >= 1 */
    int64_t ld;                 /* row stride of logits in elements, >= vocab; the logits
                                   pointer is aligned to its element size, else
                                   CE_ERR_INVALID_ARG (rows need no other alignment) */
    int64_t ignore_index;       /* targets equal to this are ignored (torch default -100) */
    const float *class_weight;  /* device [vocab] fp32, or NULL for all ones */
    float label_smoothing;      /* eps in [0, 1] */
    int32_t dtype;              /* ce_dtype of the logits buffer */
    int32_t reduction;          /* ce_reduction */
    int32_t target_is_int32;    /* 0: int64 targets, 1: int32 targets */
    int32_t variant;            /* CE_VARIANT_* (ce_fwd_bwd only) */
    int32_t reserved;           /* must be 0 */
    /* Options named next to the method on the Liger-Kernel #1268 page (its CE
     * suite: "class weights, softcap, label smoothing, z-loss"; its dx_y
     * correction keeps the "softcap factors") without a definition there;
     * this library takes the plain ones. Supported by ce_forward /
     * ce_backward and ce_fwd_bwd's stream, row-pass and split paths, and by
     * flce_fwd_bwd (softcap applied to the GEMM's logits); the cluster
     * variants (CE_VARIANT_FUSED, CE_FLCE_CE_CLUSTER) and
     * ce_fwd_bwd_from_host return CE_ERR_UNSUPPORTED with an option set. */
    float softcap;              /* c > 0: every logit becomes c*tanh(x/c); 0 = off */
    float z_loss;               /* lambda >= 0: loss_i += lambda*LSE_i^2 on valid rows */
    float *accuracy;            /* device fp32 [1] or NULL: share of valid rows whose argmax
                                   (first column of the row maximum) is the target */
} ce_params; /* 80 bytes */

/* Library version string, e.g. "ce-gb300 1.0". */
const char *ce_version(void);

/* Human-readable name of a status code. */
const char *ce_status_string(ce_status status);

/* Text of the last CUDA error seen by this thread's calls ("" if none). */
const char *ce_last_cuda_error(void);

/*
 * Bytes of workspace the calls below need for these parameters: O(n_rows),
 * independent of vocab (20 bytes per row plus at most 512 bytes).
 */
ce_status ce_workspace_size(const ce_params *p, size_t *bytes);

/*
 * Batch normalisers into the workspace: the number of valid rows, W_y (the
 * target-weight sum, the mean's divisor), W_all (the class-weight sum, used
 * with label smoothing), and the target check (CE_FLAG_TARGET_OUT_OF_RANGE).
 * Every other call runs this itself unless p->variant has
 * CE_VARIANT_PREPARED. One single-block kernel; no host synchronisation
 * (Liger-Kernel #1622: the count and weight sums stay on the device).
 *   target device [n_rows] int64 / int32.
 */
ce_status ce_prepare(const ce_params *p, const void *target, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * Forward: one online-softmax pass over each row (TransformerEngine #2325's
 * forward; the row statistics it saves are the pages' m_d_X_y).
 *   logits    device [n_rows, ld] of p->dtype, read only.
 *   target    device [n_rows] int64 (or int32 with target_is_int32).
 *   loss      device fp32: [1] for mean/sum, [n_rows] for none (written).
 *   stats     device fp32 [n_rows][4] or NULL. Row i gets
 *             {m_i, s_i, x_{i,t_i}, r_i}: m_i = max_c x_ic;
 *             s_i = sum_{c != t_i} exp(x_ic - m_i) (all c on invalid rows),
 *             so that d_i = s_i + exp(x_{i,t_i} - m_i); x_{i,t_i} (0 on invalid
 *             rows); r_i = sum_c w_c (x_ic - m_i). The target term is kept out
 *             of s_i so that the backward forms 1 - p_y = s/d without
 *             cancellation.
 */
ce_status ce_forward(const ce_params *p, const void *logits, const void *target, float *loss,
                     float *stats, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward from saved statistics: reads each row once more and writes the
 * fp32 gradient, rounded once to p->dtype, over it (TransformerEngine
 * #2325's backward; dx_y recomputed once in fp32 and stored once, as in
 * Liger-Kernel #1329).
 *   logits_inout device [n_rows, ld]: logits in, gradient out (columns >= vocab untouched).
 *   stats        device fp32 [n_rows][4] from ce_forward on the same logits.
 *   grad_output  device fp32 [1] for mean/sum, [n_rows] for none, or NULL for 1.0.
 * The logits are consumed: call it once per forward.
 */
ce_status ce_backward(const ce_params *p, void *logits_inout, const void *target,
                      const float *stats, const float *grad_output, void *workspace,
                      size_t workspace_bytes, void *stream);

/*
 * Forward and backward in one call: loss as ce_forward, gradient as
 * ce_backward, written over the logits. With the fused variant each row is
 * read from HBM once and written once (the row is held in the shared memory
 * of a thread-block cluster); the split variant reads it twice. Peak memory
 * is the logits buffer plus the workspace.
 *   grad_output device fp32 ([1] or [n_rows] for none) or NULL for 1.0. It is
 *               applied inside the gradient pass (single rounding).
 */
ce_status ce_fwd_bwd(const ce_params *p, void *logits_inout, const void *target, float *loss,
                     const float *grad_output, void *workspace, size_t workspace_bytes,
                     void *stream);

/* Largest n_rows ce_fwd_bwd_noalloc accepts (its fixed scratch, about
 * 1.3 MB, is sized for this many rows). */
#define CE_NOALLOC_MAX_ROWS 65536

/*
 * ce_fwd_bwd without a workspace argument, for callers that cannot allocate
 * device memory: hosts that give their extensions no allocator, such as a
 * runtime that reserves all device memory for its own pool up front, or a
 * plugin interface that hands an entry point only its inputs and outputs.
 * The pages this library follows have no counterpart to this entry point.
 * Same arguments, results and error behaviour as ce_fwd_bwd; the caller
 * still passes every input and output buffer.
 *  - Scratch: a fixed array of about 1.3 MB in the library's own device
 *    memory, present on every GPU that loads the library until the process
 *    exits. Nothing is allocated by this call.
 *  - n_rows above CE_NOALLOC_MAX_ROWS returns CE_ERR_WORKSPACE with nothing
 *    enqueued.
 *  - p->variant with CE_VARIANT_PREPARED returns CE_ERR_INVALID_ARG: the
 *    normalisers must be computed by this call, since no caller can run
 *    ce_prepare on the library's scratch.
 *  - The first call on a device looks up the array's device address (a
 *    runtime query with that device current; with lazy module loading the
 *    driver places the array in device memory at that moment), and so does
 *    the first call after the device's context was replaced
 *    (cudaDeviceReset); make those calls before any stream capture. Later
 *    calls change no device memory in use.
 *  - Every call on a device shares the one array, and the array keeps the
 *    last call's contents (each call runs its own normaliser kernel first,
 *    which resets every counter and sum that the later kernels read).
 *    Calls whose GPU work overlaps (different streams, or different host
 *    threads without ordering) race on it: serialise them, e.g. on one
 *    stream. Status bits are read with ce_get_status only through a
 *    caller-provided workspace, so this variant offers none.
 */
ce_status ce_fwd_bwd_noalloc(const ce_params *p, void *logits_inout, const void *target, float *loss,
                             const float *grad_output, void *stream);

/*
 * ce_fwd_bwd for logits that start in host memory: the rows are copied to
 * logits_dev in n_parts blocks on copy_stream, and each block's forward +
 * backward (the stream kernel, with the whole batch's normalisers computed
 * first on `stream`) runs on `stream` as soon as its copy has landed, so the
 * transfer and the kernels overlap (Liger-Kernel #1622 counts the
 * host-device traffic around the loss; this call hides the kernels under
 * it). Same results as ce_fwd_bwd on the device copy.
 *   logits_host  host [n_rows, ld] of p->dtype, page-locked (cudaHostAlloc
 *                or registered) for the copies to be asynchronous; it must
 *                stay valid and unchanged until `stream` has passed this call.
 *   logits_dev   device [n_rows, ld]: receives the logits, then the gradient.
 *   target, loss, grad_output, workspace: as in ce_fwd_bwd.
 *   copy_stream  a stream other than `stream` (not the legacy default
 *                stream, which would serialise the two); it first waits for
 *                the work already queued on `stream`.
 *   n_parts      >= 1 blocks of rows (clamped to n_rows); 8 is a good choice.
 * p->variant must be 0; softcap, z-loss and accuracy give
 * CE_ERR_UNSUPPORTED. Allocates no device memory; creates and releases CUDA
 * events.
 */
ce_status ce_fwd_bwd_from_host(const ce_params *p, const void *logits_host, void *logits_dev, const void *target,
                               float *loss, const float *grad_output, void *workspace, size_t workspace_bytes,
                               void *stream, void *copy_stream, int32_t n_parts);

/*
 * Scale a gradient already written with grad_output = 1 (ce_fwd_bwd with
 * grad_output NULL) by the grad_output that arrives later: row i is
 * multiplied by g ([1]) or g_i ([n_rows], reduction none). With a [1]
 * grad_output equal to 1.0 every block returns after reading it (the
 * device-side skip of Liger-Kernel #1622). The product is rounded again to
 * the buffer dtype; callers that know grad_output before the gradient pass
 * should pass it to ce_fwd_bwd / ce_backward instead (one rounding).
 *   grad_inout device [n_rows, ld] of p->dtype (columns < vocab are scaled).
 */
ce_status ce_scale_grad(const ce_params *p, void *grad_inout, const float *grad_output,
                        void *stream);

/*
 * The fused-kernel launch the library picks for these parameters (host
 * query, no GPU work): cluster size, CTAs per cluster row slice, clusters
 * in the grid and slice bytes per CTA. Returns CE_ERR_UNSUPPORTED when the
 * fused kernel cannot take these rows (ce_fwd_bwd then runs split).
 */
ce_status ce_fused_plan(const ce_params *p, int32_t *cluster_size, int32_t *n_clusters,
                        int32_t *ctas_per_sm, int64_t *slice_bytes);

/*
 * The kernel path ce_fwd_bwd takes for p->variant == CE_VARIANT_AUTO (host
 * query, no GPU work): one of the CE_VARIANT_* paths in *variant. `logits`
 * is only inspected for alignment.
 */
ce_status ce_select_variant(const ce_params *p, const void *logits, int32_t *variant);

/*
 * Self-test of the device-side bounded wait every kernel of this library
 * uses on its mbarriers: one block waits on an mbarrier that nothing ever
 * arrives on, gives up after about limit_ns nanoseconds, and writes
 * CE_FLAG_WAIT_TIMEOUT to *device_flags (device uint32). Lets a caller
 * check that a failed wait ends with a status instead of a hang, and that
 * the context stays usable. limit_ns in [1e6, 5e9].
 */
ce_status ce_selftest_wait_timeout(uint64_t limit_ns, uint32_t *device_flags, void *stream);

/*
 * Synchronises `stream`, then copies the workspace status word (CE_FLAG_*
 * bits of the most recent call that used this workspace) to *flags. The
 * only call that waits for the GPU.
 */
ce_status ce_get_status(const void *workspace, uint32_t *flags, void *stream);

/* ------------------------------------------------------------------------
 * Fused-linear cross-entropy (Liger-Kernel PR "perf(flce): drop host syncs
 * that do not feed the computation - #1622": logits = hidden x weight^T
 * formed chunk by chunk, cross-entropy forward and backward on each chunk,
 * then the gradient GEMMs; the full logits are never materialised and the
 * host never waits).
 * ------------------------------------------------------------------------ */

/* CE_GEMM_* output modes of ce_gemm_bf16 */
#define CE_GEMM_F32_STORE 0   /* D = A B (+ bias[n]) in fp32 */
#define CE_GEMM_F32_ACCUM 1   /* D += A B in fp32 */
#define CE_GEMM_BF16_STORE 2  /* D = A B rounded once to bf16 */

/*
 * D[M,N] = A[M,K] x B[K,N] on the tcgen05 tensor cores: bf16 operands,
 * fp32 accumulation in tensor memory, 128 x 256 tiles fed by TMA. The GEMM
 * the fused-linear path is built from, exposed for direct use and testing.
 *   A  device bf16. a_mn_major = 0: stored [M, K] row-major (row stride
 *      lda >= K); 1: stored [K, M] (lda >= M).
 *   B  device bf16. b_mn_major = 0: stored [N, K] (ldb >= K); 1: stored
 *      [K, N] (ldb >= N).
 *   D  device fp32 or bf16 (out_kind) [M, N], row stride ldd elements.
 *   bias device fp32 [N] added in CE_GEMM_F32_STORE mode, or NULL.
 * Base pointers (A, B and bias) 16-byte aligned and lda/ldb multiples of 8
 * (TMA rules), else CE_ERR_INVALID_ARG.
 */
ce_status ce_gemm_bf16(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int32_t a_mn_major,
                       const void *B, int64_t ldb, int32_t b_mn_major, int32_t out_kind, void *D,
                       int64_t ldd, const float *bias, void *stream);

/* ce_params.variant of flce_fwd_bwd (bits, 0 = the defaults):
 * CE_FLCE_DENSE runs every row through every GEMM instead of compacting the
 * valid rows first; CE_FLCE_CE_CLUSTER runs each chunk's cross-entropy with
 * the cluster kernel (row held in shared memory) instead of the default:
 * row statistics formed in the logits GEMM's epilogue, then one streaming
 * map from the fp32 logits to dZ. */
#define CE_FLCE_DENSE 1
#define CE_FLCE_CE_CLUSTER 2

/* Workspace bytes of flce_fwd_bwd for these sizes (the fp32 logits chunk,
 * the bf16 logits-gradient chunk and the cross-entropy workspace; with
 * compaction also a compacted copy of hidden, BT x H bf16, and 24 bytes per
 * row of maps, targets and grad_output). */
ce_status flce_workspace_size(const ce_params *p, int64_t hidden_dim, int64_t chunk_rows, size_t *bytes);

/*
 * Fused-linear cross-entropy forward and backward.
 *   p            n_rows = BT, vocab = V, dtype = CE_DT_BF16 (hidden and
 *                weight), ignore_index, class_weight, label_smoothing,
 *                reduction; variant a combination of the CE_FLCE_*
 *                bits (else CE_ERR_INVALID_ARG); ld is ignored.
 *   hidden       device bf16 [BT, H] row-major.
 *   weight       device bf16 [V, H] row-major (the lm head).
 *   bias         device fp32 [V] (16-byte aligned) or NULL.
 *   target       device [BT] int64 / int32.
 *   loss         device fp32 [1] (mean/sum) or [BT] (none).
 *   grad_output  device fp32 [1] / [BT] or NULL for 1.0, applied to dZ.
 *   grad_hidden  device bf16 [BT, H] (written).
 *   grad_weight  device fp32 [V, H] (written: the sum over all chunks).
 *   grad_bias    device fp32 [V] or NULL (written when bias is given).
 *   chunk_rows   rows per chunk (> 0); the logits of one chunk,
 *                chunk_rows x V fp32, are the largest intermediate.
 * Per chunk: Z = hidden_c W^T (+ b) in fp32; the fused cross-entropy kernel
 * turns Z into dZ (bf16, one rounding) with the batch's normalisers;
 * grad_hidden_c = dZ W; grad_weight (+)= dZ^T hidden_c. H and V multiples
 * of 8.
 * Ignored rows (target == ignore_index, or out of range: status bit) add
 * nothing to the loss or grad_weight and get zero grad_hidden rows. By
 * default they are also skipped, without a host sync (the device-side form
 * of Liger-Kernel PR #1554's ignored-row skip): one kernel gathers the valid
 * rows of hidden and their targets to the front of the workspace, and the
 * GEMMs and the chunk kernels read the valid-row count from device memory,
 * so chunks and tiles past it do no work. The host still launches every
 * chunk. Results equal the dense path's up to the order of fp32 sums.
 */
ce_status flce_fwd_bwd(const ce_params *p, int64_t hidden_dim, const void *hidden, const void *weight,
                       const float *bias, const void *target, float *loss, const float *grad_output,
                       void *grad_hidden, float *grad_weight, float *grad_bias, int64_t chunk_rows,
                       void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Token log-probabilities and the losses of post-training that are made of
 * them. With z = x / T (T the temperature), target t and p = softmax(z):
 *
 *   logp = z_t - LSE(z),   H = -sum_c p_c log p_c   (0 log 0 = 0)
 *   d(g logp + h H)/dx_c = (1/T) [ g (1[c = t] - p_c) - h p_c (log p_c + H) ]
 *
 * Of ce_params these calls use n_rows, vocab, ld, ignore_index, dtype,
 * target_is_int32 and, for the two losses, reduction; variant is 0
 * (CE_ERR_INVALID_ARG otherwise) and the other options are off
 * (CE_ERR_UNSUPPORTED otherwise). T is in [1e-4, 1e4]. Logits of -inf are
 * allowed (p_c = 0); a row whose logits are all -inf, or with a NaN or +inf
 * among them, comes out NaN. Rows that take no part (ignored target, or as
 * each call says) are not read and have gradient 0.
 *
 * The gradient goes to `grad`, device [n_rows, ld_grad] of p->dtype, its
 * columns < vocab: the logits buffer itself (then ld_grad = p->ld), or a
 * buffer that shares no element with it (CE_ERR_INVALID_ARG where the two
 * overlap in any other way).
 * ------------------------------------------------------------------------ */

/*
 * Log-probability and entropy of every row's target. One kernel, no workspace.
 *   logp     device fp32 [n_rows], or NULL.
 *   entropy  device fp32 [n_rows], or NULL: not formed.
 *   stats    device fp32 [n_rows][4] (16-byte aligned), or NULL: the row
 *            statistics ce_token_logprob_backward takes, {M, s, x_t, u}: M = max_c x_c,
 *            s = sum_{c != t} 2^a_c, u = sum_{c != t} 2^a_c a_c (NaN when the
 *            entropy was not asked for), a_c = (x_c - M) log2(e) / T.
 * Ignored rows: 0. Targets outside [0, vocab) other than ignore_index: NaN.
 */
ce_status ce_token_logprob(const ce_params *p, float temperature, const void *logits, const void *target, float *logp,
                           float *entropy, float *stats, void *stream);

/*
 * The gradient of sum_i g_i logp_i + h_i H_i from the statistics of
 * ce_token_logprob on the same logits. Rows without a valid target: 0.
 *   grad_logp, grad_entropy  device fp32 [n_rows], or NULL for 0 (not both).
 *   grad_entropy needs statistics formed with the entropy (else NaN).
 */
ce_status ce_token_logprob_backward(const ce_params *p, float temperature, const void *logits, const void *target,
                                    const float *stats, const float *grad_logp, const float *grad_entropy, void *grad,
                                    int64_t ld_grad, void *stream);

typedef struct ce_policy_params {
    float temperature;
    float clip_low, clip_high; /* ratio clipped to [1 - clip_low, 1 + clip_high]; clip_low in [0, 1], clip_high >= 0 */
    float kl_coef;             /* >= 0 */
    float entropy_coef;        /* finite */
    int32_t reserved;          /* must be 0 */
} ce_policy_params; /* 24 bytes */

/*
 * Clipped policy loss with a KL term and an entropy bonus, and its gradient.
 * Per row i with a valid target and weight w_i != 0 (others: loss 0):
 *   r = e^(logp_i - old_i),  kl = e^(ref_i - logp_i) - (ref_i - logp_i) - 1
 *   l_i = max(-A_i r, -A_i clip(r, 1 - clip_low, 1 + clip_high)) + kl_coef kl - entropy_coef H_i
 * and the loss is sum w_i l_i / sum w_i (mean), sum w_i l_i (sum) or the
 * vector w_i l_i (none). The gradient follows the branch that the max takes
 * (on the border of the clip range: the unclipped one).
 *   advantage   device fp32 [n_rows] (A).
 *   old_logp    device fp32 [n_rows], or NULL: old = logp, r = 1 (its gradient
 *               then is that of A logp).
 *   ref_logp    device fp32 [n_rows], or NULL (then kl_coef must be 0).
 *   row_weight  device fp32 [n_rows], or NULL for 1.
 *   grad_output device fp32 [1] ([n_rows] for none), or NULL for 1.
 *   loss        device fp32 [1] ([n_rows] for none).
 *   row_stats   device fp32 [n_rows][4] (16-byte aligned), or NULL: {logp, H, r, kl}
 *               per row (0 on rows that take no part).
 *   workspace   ce_workspace_size() bytes; status bits as for ce_fwd_bwd.
 * A mean over a weight sum of 0 gives loss and gradient 0 (CE_FLAG_NO_VALID_ROWS).
 */
ce_status ce_policy_fwd_bwd(const ce_params *p, const ce_policy_params *q, const void *logits, const void *target,
                            const float *advantage, const float *old_logp, const float *ref_logp,
                            const float *row_weight, const float *grad_output, float *loss, float *row_stats,
                            void *grad, int64_t ld_grad, void *workspace, size_t workspace_bytes, void *stream);

/* ce_preference_params.kind */
#define CE_PREF_SIGMOID 0 /* -(1-eps) log sigmoid(beta h) - eps log sigmoid(-beta h) */
#define CE_PREF_HINGE 1   /* max(0, 1 - beta h) */
#define CE_PREF_SQUARED 2 /* (h - 1 / (2 beta))^2 */

typedef struct ce_preference_params {
    int64_t n_pairs;           /* P >= 0 */
    int32_t kind;              /* CE_PREF_* */
    int32_t offsets_are_int32; /* 0: int64 offsets, 1: int32 */
    int32_t length_normalize;  /* 1: a sequence's value is the mean of its log-probabilities, 0: their sum */
    float beta;                /* > 0 */
    float label_smoothing;     /* eps in [0, 0.5], CE_PREF_SIGMOID only (0 otherwise) */
    int32_t reserved;          /* must be 0 */
} ce_preference_params; /* 32 bytes */

/* Workspace bytes of ce_preference_fwd_bwd: 20 bytes a row and 8 a pair, plus at most 1 KB. */
ce_status ce_preference_workspace_size(const ce_params *p, int64_t n_pairs, size_t *bytes);

/*
 * Paired preference loss over 2 P sequences of rows and its gradient:
 * sequence j is the rows [offsets[j], offsets[j + 1]); sequences 0..P-1 are
 * the preferred ones and P..2P-1, in the same order, the others. With v_j
 * the sum (or mean) of logp over the rows of j with a valid target,
 *   h_p = (v_p - v_{P+p}) - (ref_p - ref_{P+p}),
 * and the loss of kind applied to h_p. Pairs in which a side has no valid
 * target take no part (loss 0, not counted by the mean, which is over the
 * others). Rows outside of every sequence take no part.
 *   offsets     device [2 P + 1], never falling, within [0, n_rows]; otherwise
 *               loss and seq_logp are NaN, the gradient is 0 and
 *               CE_FLAG_BAD_OFFSETS is set.
 *   ref_logp    device fp32 [2 P] (ref_j of the same reduction over a
 *               sequence's rows), or NULL for 0.
 *   grad_output device fp32 [1] ([P] for none), or NULL for 1.
 *   loss        device fp32 [1] ([P] for none).
 *   seq_logp    device fp32 [2 P] (v_j), or NULL.
 *   workspace   ce_preference_workspace_size() bytes; status bits as for
 *               ce_fwd_bwd (CE_FLAG_NO_VALID_ROWS: no pair takes part).
 * The coefficient of a row depends on its whole pair: the logits are read
 * once for the log-probabilities and once more for the gradient.
 */
ce_status ce_preference_fwd_bwd(const ce_params *p, const ce_preference_params *q, const void *logits,
                                const void *target, const void *offsets, const float *ref_logp,
                                const float *grad_output, float *loss, float *seq_logp, void *grad, int64_t ld_grad,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * Token log-probabilities of a linear head, z = (hidden weight^T + bias) / T,
 * and their gradient. The logits are formed tile by tile on the tensor cores
 * (fp32 accumulation) and never stored.
 *   p       n_rows, vocab, ignore_index, target_is_int32; dtype = CE_DT_BF16
 *           (hidden and weight); the other fields as for ce_token_logprob,
 *           ld and reduction are ignored.
 *   hidden  device bf16 [n_rows, H], weight device bf16 [vocab, H], both
 *           row-major and 16-byte aligned; H a multiple of 8, any vocab.
 *   bias    device fp32 [vocab] (16-byte aligned) or NULL.
 *   target, logp, entropy, stats: as for ce_token_logprob.
 * Rows whose target is ignored or out of range are skipped on the device
 * (their hidden states may hold anything).
 */

/* Workspace bytes: of flce_token_logprob for chunk_rows = 0 (16 bytes per row
 * and 128 columns, and over 128 rows a compacted copy of hidden; up to 64 rows
 * at most 10 KB a row), of flce_token_logprob_backward for its chunk_rows. */
ce_status flce_token_logprob_workspace_size(const ce_params *p, int64_t hidden_dim, int64_t chunk_rows, size_t *bytes);

ce_status flce_token_logprob(const ce_params *p, int64_t hidden_dim, float temperature, const void *hidden,
                             const void *weight, const float *bias, const void *target, float *logp, float *entropy,
                             float *stats, void *workspace, size_t workspace_bytes, void *stream);

/*
 * The gradient of sum_i g_i logp_i + h_i H_i with respect to hidden, weight
 * and bias, from the statistics of flce_token_logprob on the same inputs. Per
 * chunk of chunk_rows rows the logits are formed again and their gradient dZ
 * (chunk_rows x vocab, rounded once to bf16) is kept in the workspace;
 * grad_hidden = dZ weight, grad_weight (+)= dZ^T hidden.
 *   grad_logp, grad_entropy  device fp32 [n_rows], or NULL for 0 (not both).
 *   grad_hidden  device bf16 [n_rows, H] (written; 0 on skipped rows).
 *   grad_weight  device [vocab, H] (written), fp32 or bf16 (grad_weight_dtype);
 *                bf16 with chunk_rows >= n_rows only (CE_ERR_UNSUPPORTED:
 *                several chunks add up in fp32). 16-byte aligned.
 *   grad_bias    device fp32 [vocab], or NULL.
 */
ce_status flce_token_logprob_backward(const ce_params *p, int64_t hidden_dim, float temperature, const void *hidden,
                                      const void *weight, const float *bias, const void *target, const float *stats,
                                      const float *grad_logp, const float *grad_entropy, void *grad_hidden,
                                      void *grad_weight, int32_t grad_weight_dtype, float *grad_bias,
                                      int64_t chunk_rows, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The serving head in 8 bits: norm, weights and activations in e4m3 with
 * scales, the logits product, and the verification of drafted tokens.
 *
 * 8-bit layout: e4m3 bytes [rows, cols], row-major with a row stride ld that
 * is a multiple of 16, first byte 16-byte aligned, and a scale (fp32) for every
 * block: the value is byte * scale. Blocks span 128 columns and either one row
 * (activations, scale [rows][ceil(cols / 128)]) or 128 rows (weights, scale
 * [ceil(rows / 128)][ceil(cols / 128)]); the last block of a row or column may be
 * smaller. A block's scale is max(max |y| / 448, 2^-126), its bytes the nearest
 * e4m3 of the fp32 quotient y / scale (ties to even), so zeros stay zeros. A NaN makes its block's
 * scale and bytes NaN; an infinity makes the scale infinite. Bytes between cols
 * and ld are not written and never read.
 * Inputs may have any row stride and element alignment; outputs share no memory
 * with inputs or one another (CE_ERR_INVALID_ARG otherwise) except where said.
 * ------------------------------------------------------------------------ */

typedef struct ce_norm_params {
    int64_t n_rows, cols;             /* cols in [1, 32768] (CE_ERR_UNSUPPORTED above) */
    int64_t ld_x, ld_residual, ld_residual_out, ld_q; /* row strides, elements; >= cols */
    int32_t dtype;                    /* ce_dtype of x, residual and residual_out */
    int32_t weight_dtype;             /* dtype, or CE_DT_F32 */
    float eps;                        /* >= 0 */
    int32_t reserved;                 /* must be 0 */
} ce_norm_params; /* 64 bytes */

/*
 * Root-mean-square norm with the residual's addition, in 8 bits:
 *   h = x + residual,  y = h weight / sqrt(mean_c h_c^2 + eps),
 * y quantised in blocks of 1 x 128. h and y are fp32: h is rounded once, where
 * it is stored, and the norm is that of the unrounded sum.
 *   x             device [n_rows, ld_x].
 *   residual      device [n_rows, ld_residual], or NULL for 0.
 *   weight        device [cols], 16-byte aligned.
 *   residual_out  device [n_rows, ld_residual_out], or NULL; needs residual.
 *                 May be x or residual itself (with the same row stride).
 *   q, scale      the 8-bit rows.
 * A row with a NaN comes out NaN.
 */
ce_status ce_rms_norm_fp8(const ce_norm_params *p, const void *x, const void *residual, const void *weight,
                          void *residual_out, void *q, float *scale, void *stream);

/*
 * x (device [rows, ld_x] of dtype) in 8 bits, block_rows 1 or 128.
 */
ce_status ce_quantize_fp8(int64_t rows, int64_t cols, const void *x, int64_t ld_x, int32_t dtype, int32_t block_rows,
                          void *q, int64_t ld_q, float *scale, void *stream);

/*
 * D[m, n] = sum_k A[m, k] B[n, k] (+ bias[n]) of 8-bit operands on the tcgen05
 * tensor cores: A [M, K] in blocks of 1 x 128, B [N, K] (a weight) in blocks of
 * 128 x 128. Sums of one block along K are formed by the tensor core,
 * scaled and added up in fp32, and rounded once to D.
 * Scales may be any numbers, their products below fp32's normal range or above
 * it among them, while the products for one row of A and one block of B's rows lie
 * within 2^160 of one another; terms further below may lose bits. Blocks with
 * a scale of 2^-126 count as blocks of zeros in this: what else they hold is below 5.3e-36,
 * and may lose bits.
 *   bias   device fp32 [N], or NULL.
 *   dtype  of D, device [M, ldd], ldd >= N.
 * K >= 1; M or N of 0 does nothing. Should a wait inside the kernel give up,
 * the tiles concerned come out NaN.
 */
ce_status ce_gemm_fp8(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const float *a_scale,
                      const void *B, int64_t ldb, const float *b_scale, const float *bias, int32_t dtype, void *D,
                      int64_t ldd, void *stream);

typedef struct ce_verify_params {
    int64_t n_seqs, n_drafts, vocab;  /* B, K in [0, 255], V */
    int64_t seq_stride, ld;           /* logits [B][K + 1][V]: strides of a sequence and of a row, elements */
    int64_t draft_seq_stride, ld_draft; /* draft_logits [B][K][V] */
    int32_t dtype;                    /* ce_dtype of both */
    int32_t token_is_int32;           /* draft_token and tokens: 0 int64, 1 int32 */
    float temperature;                /* T, 0 or in [1e-4, 1e4]; not used where temperatures is given */
    int32_t reserved;                 /* must be 0 */
} ce_verify_params; /* 72 bytes */

/* Workspace bytes of ce_verify_drafts: 16 for every row and part of it (2 KB, or down to
 * 512 bytes while the rows are few), plus 256. */
ce_status ce_verify_workspace_size(const ce_verify_params *p, size_t *bytes);

/*
 * Verification of drafted tokens against the target's probabilities, from given
 * random numbers. Sequence b has the drafts t_0 .. t_{K-1} and K + 1 rows of
 * target logits z_0 .. z_K (row i: the distribution of the token in place of
 * t_i). With p_i = softmax(z_i / T) and q_i = softmax(y_i / T) of the draft
 * model's logits (or, without them, 1 at t_i and 0 elsewhere):
 *   draft i stays while u_i q_i(t_i) < p_i(t_i); n drafts stay, up to the first that does not;
 *   token n is the lowest v with sum_{c <= v} w_c > r sum_c w_c, where
 *   w = max(p_n - q_n, 0) if position n has a draft, p_n otherwise (and if that sum is 0).
 * So the tokens are distributed as the target alone would have drawn them, for
 * u and r uniform in [0, 1). T = 0 (greedy): draft i stays while it is the lowest
 * index of the maximum of z_i, and token n is that index of z_n.
 *   draft_token    device [B][K]; one outside of [0, V) (say -1) ends its
 *                  sequence's drafts: shorter drafts are padded with it.
 *   accept_uniform device fp32 [B][K] (u), sample_uniform device fp32 [B] (r).
 *   temperatures   device fp32 [B] (T of every sequence), or NULL.
 *   accepted       device int32 [B] (n).
 *   tokens         device [B][K + 1], of draft_token's type: t_0 .. t_{n-1}, token n, then -1.
 *   logp           device fp32 [B][K + 1]: the target's log-probability of each
 *                  token (T = 1 where T is 0), 0 behind the last.
 * Logits of -inf have probability 0. Where a row that decides (the target's, or
 * the draft model's at a draft) is all -inf or holds a NaN or +inf, or T is not
 * as above, the sequence ends there with token -1 and log-probability NaN. Rows
 * behind a sequence's last draft are not read. K = 0 (no draft pointers needed)
 * draws one token a sequence.
 */
ce_status ce_verify_drafts(const ce_verify_params *p, const void *logits, const void *draft_logits,
                           const void *draft_token, const float *accept_uniform, const float *sample_uniform,
                           const float *temperatures, int32_t *accepted, void *tokens, float *logp, void *workspace,
                           size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CE_H */
