// lp_kernels.h -- argument blocks and launchers of the log-probability
// operators (token log-probabilities, policy loss, preference loss).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ce.h"

namespace ce {

struct WsCtl;

struct LpArgs {
    const void *x;             // logits [n_rows, ld]
    int64_t n_rows, vocab, ld;
    void *grad;                // gradient [n_rows, ld_grad], may be x
    int64_t ld_grad;
    const void *target;
    int tgt32;
    int64_t ignore_index;
    float inv_t, k;            // 1 / T and log2(e) / T
    WsCtl *ctl;
    // forward: per-row outputs (each may be NULL) and, for the preference
    // loss, the sequences' row offsets (rows outside of them are skipped)
    float *logp, *entropy;
    float4 *stats;             // {M, s, x_t, u} of lp_row_stats; read by the gradient kernel
    const void *offsets;
    int off32;
    int64_t n_seqs;
    // policy loss
    const float *adv, *old_logp, *ref_logp, *row_weight;
    float clip_lo, clip_hi, kl_coef, ent_coef;
    int reduction;
    const float *grad_output;  // NULL = 1.0
    float *loss;
    double *part;              // workspace: one loss sum per CTA (cluster); preference: one loss per pair
    int n_prep;                // blocks of the normaliser kernel
    float4 *row_stats;         // {log p, entropy, ratio, KL}
    // gradient from statistics: dL/dlogp and dL/dH (NULL: 0)
    const float *g_logp, *g_entropy;
    int row_coef;              // 1: g_logp is the workspace's row coefficients (preference): rows
                               // with coefficient 0 are not read, and the batch loss is formed
};

struct PairArgs {
    int64_t n_rows, vocab, n_pairs;
    const void *target;
    int tgt32;
    int64_t ignore_index;
    const void *offsets;
    int off32;
    float *row;                // workspace [n_rows]: in log p, out dL/dlogp
    const float *ref;          // [2 n_pairs] or NULL
    int kind, normalize, reduction;
    float beta, smoothing;
    const float *grad_output;
    float *loss;               // [1] or [n_pairs]
    float *seq_logp;           // [2 n_pairs] or NULL
    double *pair_loss;         // workspace [n_pairs]
    WsCtl *ctl;
};

enum { LP_FWD = 0, LP_POLICY = 1 };

// the normalisers of the policy loss (valid rows, their weight sum) and the target check
cudaError_t launch_lp_prep(LpArgs &a, cudaStream_t s);
// one pass over every row: log-probabilities, entropies and statistics (LP_FWD), or the policy loss and its gradient
cudaError_t launch_lp_rows(const LpArgs &a, int dtype, int mode, bool entropy, bool after_prep, cudaStream_t s);
// the same for rows that a group of warps holds in registers (launch_lp_rows picks it)
bool lp_short_takes(int64_t vocab, int dtype);
cudaError_t launch_lp_short(const LpArgs &a, int dtype, int mode, bool entropy, bool after_prep, int sms, cudaStream_t s);
// the gradient of every row from its statistics (preference: and the batch loss)
cudaError_t launch_lp_grad(const LpArgs &a, int dtype, bool entropy, bool dependent, cudaStream_t s);
// sequence sums, pair losses and row coefficients of the preference loss
cudaError_t launch_lp_pairs(const PairArgs &a, cudaStream_t s);
}  // namespace ce
