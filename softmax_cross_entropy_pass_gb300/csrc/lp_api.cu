// lp_api.cu -- C entry points of the log-probability operators: argument
// checks, workspace layout and launches. Host code only.
#include <cmath>

#include "ce_kernels.h"
#include "lp_device.cuh"
#include "lp_kernels.h"

using namespace ce;

namespace {

int64_t lp_elem_bytes(const ce_params *p) { return p->dtype == CE_DT_F32 ? 4 : 2; }

bool on(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool temperature_ok(float t) { return t >= 1e-4f && t <= 1e4f; }

ce_status lp_check(const ce_params *p, float temperature) {
    if (!p) return CE_ERR_INVALID_ARG;
    if (p->n_rows < 0 || p->vocab < 1 || p->ld < p->vocab) return CE_ERR_INVALID_ARG;
    if (p->vocab > (int64_t(1) << 31) - 1 || p->n_rows > (int64_t(1) << 31) - 1) return CE_ERR_UNSUPPORTED;
    if (p->dtype != CE_DT_F32 && p->dtype != CE_DT_BF16 && p->dtype != CE_DT_F16) return CE_ERR_INVALID_ARG;
    if (p->reduction != CE_RED_NONE && p->reduction != CE_RED_MEAN && p->reduction != CE_RED_SUM)
        return CE_ERR_INVALID_ARG;
    if (p->target_is_int32 != 0 && p->target_is_int32 != 1) return CE_ERR_INVALID_ARG;
    if (p->variant != 0 || p->reserved != 0) return CE_ERR_INVALID_ARG;
    if (p->class_weight || p->label_smoothing != 0.f || p->softcap != 0.f || p->z_loss != 0.f || p->accuracy)
        return CE_ERR_UNSUPPORTED;
    return temperature_ok(temperature) ? CE_OK : CE_ERR_INVALID_ARG;
}

ce_status lp_check_ws(const void *ws, size_t have, size_t need) {
    return ws && on(ws, 256) && have >= need ? CE_OK : CE_ERR_WORKSPACE;
}

// The gradient buffer: the logits themselves with the same row stride, or no
// element in common with them. Two views of one wider buffer, side by side,
// are told apart by their columns.
ce_status lp_check_grad(const ce_params *p, const void *x, const void *grad, int64_t ld_grad) {
    const int64_t esz = lp_elem_bytes(p);
    if (ld_grad < p->vocab || !on(grad, esz)) return CE_ERR_INVALID_ARG;
    if (p->n_rows == 0) return CE_OK;
    const bool one = p->n_rows == 1;
    if (grad == x) return one || ld_grad == p->ld ? CE_OK : CE_ERR_INVALID_ARG;
    const intptr_t a = reinterpret_cast<intptr_t>(x), b = reinterpret_cast<intptr_t>(grad);
    const int64_t a_len = ((p->n_rows - 1) * p->ld + p->vocab) * esz, b_len = ((p->n_rows - 1) * ld_grad + p->vocab) * esz;
    if (a + a_len <= b || b + b_len <= a) return CE_OK;
    if (ld_grad != p->ld || one) return CE_ERR_INVALID_ARG;
    int64_t col = ((b - a) / esz) % p->ld;
    if (col < 0) col += p->ld;
    return (b - a) % esz == 0 && col >= p->vocab && col <= p->ld - p->vocab ? CE_OK : CE_ERR_INVALID_ARG;
}

bool target_ok(const ce_params *p, const void *target) { return target && on(target, p->target_is_int32 ? 4 : 8); }

LpArgs lp_args(const ce_params *p, float temperature, const void *logits, const void *target) {
    LpArgs a{};
    a.x = logits;
    a.n_rows = p->n_rows;
    a.vocab = p->vocab;
    a.ld = p->ld;
    a.target = target;
    a.tgt32 = p->target_is_int32;
    a.ignore_index = p->ignore_index;
    a.inv_t = 1.f / temperature;
    a.k = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
    a.reduction = p->reduction;
    return a;
}

size_t preference_ws(int64_t n_rows, int64_t n_pairs) {
    return ((ws_bytes(n_rows) + 255) & ~static_cast<size_t>(255)) + static_cast<size_t>(n_pairs) * sizeof(double);
}

}  // namespace

extern "C" {

ce_status ce_token_logprob(const ce_params *p, float temperature, const void *logits, const void *target, float *logp,
                           float *entropy, float *stats, void *stream) {
    ce_status st = lp_check(p, temperature);
    if (st != CE_OK) return st;
    if (p->n_rows == 0) return CE_OK;
    if (!logp && !entropy && !stats) return CE_ERR_INVALID_ARG;
    if (!logits || !target_ok(p, target) || !on(logits, lp_elem_bytes(p))) return CE_ERR_INVALID_ARG;
    if (!on(logp, 4) || !on(entropy, 4) || !on(stats, 16)) return CE_ERR_INVALID_ARG;
    LpArgs a = lp_args(p, temperature, logits, target);
    a.logp = logp;
    a.entropy = entropy;
    a.stats = reinterpret_cast<float4 *>(stats);
    cudaError_t e = launch_lp_rows(a, p->dtype, LP_FWD, entropy != nullptr, false, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

ce_status ce_token_logprob_backward(const ce_params *p, float temperature, const void *logits, const void *target,
                                    const float *stats, const float *grad_logp, const float *grad_entropy, void *grad,
                                    int64_t ld_grad, void *stream) {
    ce_status st = lp_check(p, temperature);
    if (st != CE_OK) return st;
    if ((st = lp_check_grad(p, logits, grad, ld_grad)) != CE_OK) return st;
    if (p->n_rows == 0) return CE_OK;
    if (!grad_logp && !grad_entropy) return CE_ERR_INVALID_ARG;
    if (!logits || !target_ok(p, target) || !stats || !grad || !on(logits, lp_elem_bytes(p))) return CE_ERR_INVALID_ARG;
    if (!on(stats, 16) || !on(grad_logp, 4) || !on(grad_entropy, 4)) return CE_ERR_INVALID_ARG;
    LpArgs a = lp_args(p, temperature, logits, target);
    a.stats = reinterpret_cast<float4 *>(const_cast<float *>(stats));
    a.g_logp = grad_logp;
    a.g_entropy = grad_entropy;
    a.grad = grad;
    a.ld_grad = ld_grad;
    cudaError_t e = launch_lp_grad(a, p->dtype, grad_entropy != nullptr, false, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

ce_status ce_policy_fwd_bwd(const ce_params *p, const ce_policy_params *q, const void *logits, const void *target,
                            const float *advantage, const float *old_logp, const float *ref_logp,
                            const float *row_weight, const float *grad_output, float *loss, float *row_stats,
                            void *grad, int64_t ld_grad, void *ws, size_t ws_size, void *stream) {
    if (!q) return CE_ERR_INVALID_ARG;
    ce_status st = lp_check(p, q->temperature);
    if (st != CE_OK) return st;
    if (!(q->clip_low >= 0.f && q->clip_low <= 1.f) || !(q->clip_high >= 0.f)) return CE_ERR_INVALID_ARG;
    if (!(q->kl_coef >= 0.f && q->kl_coef < INFINITY) || !std::isfinite(q->entropy_coef) || q->reserved != 0)
        return CE_ERR_INVALID_ARG;
    if (q->kl_coef > 0.f && !ref_logp) return CE_ERR_INVALID_ARG;
    if ((st = lp_check_ws(ws, ws_size, ws_bytes(p->n_rows))) != CE_OK) return st;
    if ((st = lp_check_grad(p, logits, grad, ld_grad)) != CE_OK) return st;
    if (!loss && (p->n_rows > 0 || p->reduction != CE_RED_NONE)) return CE_ERR_INVALID_ARG;
    if (p->n_rows > 0 && (!logits || !target_ok(p, target) || !advantage || !grad || !on(logits, lp_elem_bytes(p))))
        return CE_ERR_INVALID_ARG;
    if (!on(advantage, 4) || !on(old_logp, 4) || !on(ref_logp, 4) || !on(row_weight, 4) || !on(grad_output, 4) ||
        !on(loss, 4) || !on(row_stats, 16))
        return CE_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    LpArgs a = lp_args(p, q->temperature, logits, target);
    a.grad = grad;
    a.ld_grad = ld_grad;
    a.ctl = reinterpret_cast<WsCtl *>(ws);
    a.adv = advantage;
    a.old_logp = old_logp;
    a.ref_logp = ref_logp;
    a.row_weight = row_weight;
    a.clip_lo = 1.f - q->clip_low;
    a.clip_hi = 1.f + q->clip_high;
    a.kl_coef = q->kl_coef;
    a.ent_coef = q->entropy_coef;
    a.grad_output = grad_output;
    a.loss = loss;
    a.part = reinterpret_cast<double *>(ws_stats(ws, p->n_rows));
    a.row_stats = reinterpret_cast<float4 *>(row_stats);
    cudaError_t e = launch_lp_prep(a, s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (p->n_rows == 0) {
        if (p->reduction != CE_RED_NONE && (e = cudaMemsetAsync(loss, 0, sizeof(float), s)) != cudaSuccess)
            return cuda_fail(e);
        return CE_OK;
    }
    e = launch_lp_rows(a, p->dtype, LP_POLICY, row_stats || q->entropy_coef != 0.f, true, s);
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

ce_status ce_preference_workspace_size(const ce_params *p, int64_t n_pairs, size_t *bytes) {
    ce_status st = lp_check(p, 1.f);
    if (st != CE_OK) return st;
    if (!bytes || n_pairs < 0) return CE_ERR_INVALID_ARG;
    *bytes = preference_ws(p->n_rows, n_pairs);
    return CE_OK;
}

ce_status ce_preference_fwd_bwd(const ce_params *p, const ce_preference_params *q, const void *logits,
                                const void *target, const void *offsets, const float *ref_logp,
                                const float *grad_output, float *loss, float *seq_logp, void *grad, int64_t ld_grad,
                                void *ws, size_t ws_size, void *stream) {
    ce_status st = lp_check(p, 1.f);
    if (st != CE_OK) return st;
    if (!q || q->n_pairs < 0 || q->reserved != 0) return CE_ERR_INVALID_ARG;
    if (q->n_pairs > (int64_t(1) << 30)) return CE_ERR_UNSUPPORTED;
    if (q->kind != CE_PREF_SIGMOID && q->kind != CE_PREF_HINGE && q->kind != CE_PREF_SQUARED) return CE_ERR_INVALID_ARG;
    if ((q->offsets_are_int32 != 0 && q->offsets_are_int32 != 1) || (q->length_normalize != 0 && q->length_normalize != 1))
        return CE_ERR_INVALID_ARG;
    if (!(q->beta > 0.f && q->beta < INFINITY)) return CE_ERR_INVALID_ARG;
    if (!(q->label_smoothing >= 0.f && q->label_smoothing <= 0.5f) ||
        (q->label_smoothing != 0.f && q->kind != CE_PREF_SIGMOID))
        return CE_ERR_INVALID_ARG;
    if ((st = lp_check_ws(ws, ws_size, preference_ws(p->n_rows, q->n_pairs))) != CE_OK) return st;
    if ((st = lp_check_grad(p, logits, grad, ld_grad)) != CE_OK) return st;
    if (!offsets || (!loss && (q->n_pairs > 0 || p->reduction != CE_RED_NONE))) return CE_ERR_INVALID_ARG;
    if (p->n_rows > 0 && (!logits || !target_ok(p, target) || !grad || !on(logits, lp_elem_bytes(p)))) return CE_ERR_INVALID_ARG;
    if (!on(offsets, q->offsets_are_int32 ? 4 : 8) || !on(ref_logp, 4) || !on(grad_output, 4) || !on(loss, 4) ||
        !on(seq_logp, 4))
        return CE_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t n = p->n_rows;
    LpArgs a = lp_args(p, 1.f, logits, target);
    a.ctl = reinterpret_cast<WsCtl *>(ws);
    a.offsets = offsets;
    a.off32 = q->offsets_are_int32;
    a.n_seqs = 2 * q->n_pairs;
    a.logp = ws_row_loss(ws);
    a.stats = reinterpret_cast<float4 *>(ws_stats(ws, n));
    PairArgs pa{};
    pa.n_rows = n;
    pa.vocab = p->vocab;
    pa.n_pairs = q->n_pairs;
    pa.target = target;
    pa.tgt32 = p->target_is_int32;
    pa.ignore_index = p->ignore_index;
    pa.offsets = offsets;
    pa.off32 = q->offsets_are_int32;
    pa.row = a.logp;
    pa.ref = ref_logp;
    pa.kind = q->kind;
    pa.normalize = q->length_normalize;
    pa.reduction = p->reduction;
    pa.beta = q->beta;
    pa.smoothing = q->label_smoothing;
    pa.grad_output = grad_output;
    pa.loss = loss;
    pa.seq_logp = seq_logp;
    pa.pair_loss = reinterpret_cast<double *>(reinterpret_cast<char *>(ws) + preference_ws(n, 0));
    pa.ctl = a.ctl;
    cudaError_t e = n > 0 ? launch_lp_rows(a, p->dtype, LP_FWD, false, false, s)
                          : cudaMemsetAsync(ws, 0, kWsCtlBytes, s);  // the row kernel clears the control block otherwise
    if (e == cudaSuccess) e = launch_lp_pairs(pa, s);
    if (e == cudaSuccess) {
        a.g_logp = pa.row;
        a.row_coef = 1;
        a.grad = grad;
        a.ld_grad = ld_grad;
        a.part = pa.pair_loss;
        a.loss = loss;
        a.grad_output = grad_output;
        e = launch_lp_grad(a, p->dtype, false, true, s);
    }
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

}  // extern "C"
