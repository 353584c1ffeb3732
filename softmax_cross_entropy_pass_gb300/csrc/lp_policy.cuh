// lp_policy.cuh -- the scalars of one row of the clipped policy loss, shared
// by the kernels that form it.
#pragma once

#include "lp_device.cuh"
#include "lp_kernels.h"

namespace ce {

// e^g - g - 1 >= 0, and e^g - 1 as `slope`: near 0 the former by its series (the
// subtraction would cancel) and the latter from it; elsewhere the latter from the
// exponential (from the former it would lose its digits where -g is large)
__device__ inline float kl_of_gap(float g, float &slope) {
    if (fabsf(g) < 0.25f) {
        float p = 1.f / 40320.f;  // g^8 / 8!, relative error below 2e-9 there
        p = fmaf(p, g, 1.f / 5040.f);
        p = fmaf(p, g, 1.f / 720.f);
        p = fmaf(p, g, 1.f / 120.f);
        p = fmaf(p, g, 1.f / 24.f);
        p = fmaf(p, g, 1.f / 6.f);
        p = fmaf(p, g, 0.5f);
        const float kl = p * g * g;
        slope = g + kl;
        return kl;
    }
    const float e = expf(g);
    slope = e - 1.f;
    return e - g - 1.f;
}

// What a policy row reads besides its logits, fetched before its first pass.
struct PolicyIn {
    float adv, old_logp, ref_logp, weight;
};
// a row without a usable target or with weight 0 takes no part: nothing else of it is read
__device__ inline bool policy_row_live(const LpArgs &a, int64_t row, int64_t t) {
    return target_valid(t, a.ignore_index, a.vocab) && !(a.row_weight && __ldg(a.row_weight + row) == 0.f);
}
__device__ inline PolicyIn policy_load(const LpArgs &a, int64_t row) {
    PolicyIn p;
    p.adv = __ldg(a.adv + row);
    p.old_logp = a.old_logp ? __ldg(a.old_logp + row) : 0.f;
    p.ref_logp = a.ref_logp ? __ldg(a.ref_logp + row) : 0.f;
    p.weight = a.row_weight ? __ldg(a.row_weight + row) : 1.f;
    return p;
}

struct PolicyOut {
    float loss;        // weighted, not divided by the batch's normaliser
    float g, h;        // d(weighted loss) / dlogp and / dH
    float ratio, kl;
};
// r = e^(logp - old), loss = max(-A r, -A clip(r)) + beta (e^gap - gap - 1) - eta H,
// gap = ref - logp. On the border of the clip range (the two branches equal)
// the unclipped branch's slope is taken. NaN inputs come out NaN.
__device__ inline PolicyOut policy_row(const LpArgs &a, const PolicyIn &in, const LpRow &r, float entropy) {
    PolicyOut o;
    const float log_r = a.old_logp ? r.logp - in.old_logp : 0.f;
    o.ratio = expf(log_r);
    const float clipped = fminf(fmaxf(o.ratio, a.clip_lo), a.clip_hi);
    // advantage 0 times a ratio that only fp32 takes for infinite is 0
    const bool none = in.adv == 0.f && o.ratio == INFINITY && log_r < INFINITY;
    const float u1 = none ? 0.f : -in.adv * o.ratio, u2 = -in.adv * clipped;
    float loss = u1 < u2 ? u2 : u1;
    float g = u1 < u2 ? 0.f : u1;
    o.kl = 0.f;
    if (a.ref_logp) {
        float slope;
        o.kl = kl_of_gap(in.ref_logp - r.logp, slope);
        if (a.kl_coef != 0.f) {
            loss = fmaf(a.kl_coef, o.kl, loss);
            g = fmaf(-a.kl_coef, slope, g);
        }
    }
    o.h = 0.f;
    if (a.ent_coef != 0.f) {
        loss = fmaf(-a.ent_coef, entropy, loss);
        o.h = -a.ent_coef * in.weight;
    }
    o.loss = in.weight * loss;
    o.g = in.weight * g;
    return o;
}

// What the normaliser kernel's blocks found (after a pdl_wait): the sum of the
// weights, added up in block order, and the status bits, which the first block
// of the row kernel sets.
__device__ inline float policy_weight_sum(const LpArgs &a) {
    double s = 0.0;
    for (int b = 0; b < a.n_prep; ++b) s += __ldcg(&a.ctl->prep_part[b][0]);
    return static_cast<float>(s);
}
__device__ inline void policy_flags(const LpArgs &a) {
    unsigned bad = 0;
    for (int b = 0; b < a.n_prep; ++b) bad |= __ldcg(&a.ctl->prep_bad[b]);
    const bool none = a.reduction == CE_RED_MEAN && policy_weight_sum(a) == 0.f;
    if (bad || none) atomicOr(&a.ctl->status, (bad ? CE_FLAG_TARGET_OUT_OF_RANGE : 0u) | (none ? CE_FLAG_NO_VALID_ROWS : 0u));
}

// the gradient scale of the batch: grad_output over the weight sum for mean
__device__ inline float policy_scale(const LpArgs &a, int64_t row, float w_sum) {
    const float up = a.grad_output ? __ldg(a.grad_output + (a.reduction == CE_RED_NONE ? row : 0)) : 1.f;
    if (a.reduction != CE_RED_MEAN) return up;
    return w_sum != 0.f ? up / w_sum : 0.f;
}

}  // namespace ce
