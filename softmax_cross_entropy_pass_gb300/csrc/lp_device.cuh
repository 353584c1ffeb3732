// lp_device.cuh -- the arithmetic of token log-probabilities, shared by the
// kernels that form them (from logits in memory and in the lm-head product's
// epilogue) and by those that form their gradient.
//
// With z = x / T, target t, p = softmax(z) and H = -sum_c p_c log p_c:
//   log p_t = z_t - LSE(z),
//   d(g log p_t + h H) / dx_c = (1/T) [ g (1[c = t] - p_c) - h p_c (log p_c + H) ].
// Exponents are kept in base 2: a_c = (x_c - m) k with k = log2(e) / T, so
// that x - m is exact where it matters (equal logits give exactly 0, and a
// row whose logits all lie at the type's lowest value does not overflow) and
// one multiplication takes the temperature and the base together.
#pragma once

#include "ce_device.cuh"

namespace ce {

// the exponent below which 2^a is 0 in fp32: exponents that also multiply
// something are held at it, so that a logit of -inf (a = -inf) adds 0 * (-1024)
// instead of 0 * inf. NaN passes.
constexpr float kLpMinExp = -1024.f;
__device__ inline float lp_clamp(float a) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(kLpMinExp));
    return r;
}

// Running statistics over columns: m = max x, s = sum 2^a, u = sum 2^a a
// (with the entropy only), a = (x - m) k.
struct LpState {
    float m, s, u;
};
__device__ inline LpState lp_empty() { return LpState{-INFINITY, 0.f, 0.f}; }

// move the sums from the maximum st.m to M >= st.m
template <bool ENT>
__device__ inline void lp_rebase(LpState &st, float M, float k) {
    if (st.m != -INFINITY) {
        const float d = lp_clamp((st.m - M) * k), f = ex2_hw(d);
        if (ENT) st.u = f * fmaf(st.s, d, st.u);
        st.s *= f;
    }
    st.m = M;
}

template <bool ENT>
__device__ inline LpState lp_merge(LpState a, LpState b, float k) {
    const float M = fmaxf(a.m, b.m);
    if (M != -INFINITY) {
        lp_rebase<ENT>(a, M, k);
        lp_rebase<ENT>(b, M, k);
    }
    return LpState{M, a.s + b.s, ENT ? a.u + b.u : 0.f};
}

// merge over groups of W lanes (in the same order in every group): the
// maximum first, then one move of each lane's sums to it
template <bool ENT, int W = 32>
__device__ inline LpState lp_warp_merge(LpState st, float k) {
    float M = st.m;
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (M != -INFINITY) lp_rebase<ENT>(st, M, k);
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) {
        st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
        if (ENT) st.u += __shfl_xor_sync(0xffffffffu, st.u, off);
    }
    return st;
}

// Add N values (N even) whose maximum is vmax. The sums stay empty while
// every value is -inf; a NaN among such values is kept (the maximum drops it).
template <bool ENT, int N>
__device__ inline void lp_add(LpState &st, const float *x, float vmax, float k) {
    if (vmax > st.m) lp_rebase<ENT>(st, vmax, k);
    if (st.m == -INFINITY) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (x[j] != x[j]) st.s = x[j];
        return;
    }
    const F2 mm = f2(st.m, st.m), kk = f2(k, k);
    F2 s2 = f2(0.f, 0.f), u2 = f2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < N / 2; ++p) {
        F2 a = f2_mul(f2_sub(f2(x[2 * p], x[2 * p + 1]), mm), kk);
        if (ENT) {
            float a0, a1;
            f2_split(a, a0, a1);
            a = f2(lp_clamp(a0), lp_clamp(a1));
        }
        const F2 e = f2_ex2(a);
        s2 = f2_add(s2, e);
        if (ENT) u2 = f2_fma(e, a, u2);
    }
    float lo, hi;
    f2_split(s2, lo, hi);
    st.s += lo + hi;
    if (ENT) {
        f2_split(u2, lo, hi);
        st.u += lo + hi;
    }
}
template <bool ENT>
__device__ inline void lp_add1(LpState &st, float x, float k) {
    const float v[2] = {x, -INFINITY};
    lp_add<ENT, 2>(st, v, x, k);
}

// A row's statistics as they are kept between a forward and its backward:
// M = max over all columns, s and u over the columns other than the target,
// relative to M, and the target logit. The target's own terms are kept apart
// so that 1 - p_t = s / d and log p_t near 0 form without cancellation.
__device__ inline float4 lp_row_stats(LpState off, float xy, float k) {
    const float M = fmaxf(off.m, xy);
    if (M != -INFINITY) lp_rebase<true>(off, M, k);
    return make_float4(M, off.s, xy, off.u);
}

struct LpRow {
    float logp, entropy;
    float neg_log2d;  // p_c = 2^((x_c - M) k + neg_log2d)
    float p_y, q_y;   // p_t and 1 - p_t
};
// A row without a finite maximum (all -inf, or +inf among its logits) and a
// row with a NaN come out NaN, as the formula gives them.
__device__ inline LpRow lp_row(const float4 st, float k, float inv_t) {
    const float M = st.x, s = st.y, xy = st.z, u = st.w;
    LpRow r;
    const float a_y = lp_clamp((xy - M) * k);
    const float e_y = exp2f(a_y);
    const float d = s + e_y, inv_d = 1.f / d;
    const float log2d = log2f(d);
    r.neg_log2d = -log2d;
    r.p_y = e_y * inv_d;
    r.q_y = s * inv_d;
    // -log p_t = log d + (M - x_t) / T, a sum of two parts >= 0; near p_t = 1,
    // where both are small, log(1 + s / e_y)
    const float nll = r.p_y < 0.5f ? fmaf(M - xy, inv_t, kLn2 * log2d) : log1pf(s / e_y);
    r.logp = -nll;
    // H = log d - (1/d) sum 2^a a ln 2: both terms >= 0
    r.entropy = kLn2 * (log2d - fmaf(e_y, a_y, u) * inv_d);
    return r;
}

// The gradient of one row: (A + B log2 p) p off the target, dy at it.
struct LpGrad {
    float M, neg_log2d, A, B, dy;
};
// g = dL/dlogp, h = dL/dH
__device__ inline LpGrad lp_grad(const float4 st, const LpRow &r, float inv_t, float g, float h) {
    LpGrad o;
    o.M = st.x;
    o.neg_log2d = r.neg_log2d;
    o.A = -inv_t * g;
    o.B = 0.f;
    o.dy = inv_t * g * r.q_y;
    if (h != 0.f) {
        o.A = -inv_t * fmaf(h, r.entropy, g);
        o.B = -inv_t * h * kLn2;
        if (r.p_y > 0.f) o.dy -= inv_t * h * r.p_y * (r.logp + r.entropy);
    }
    return o;
}
template <bool ENT>
__device__ inline float lp_grad_elem(const LpGrad &g, float x, float k) {
    float a = fmaf(x - g.M, k, g.neg_log2d);
    if (!ENT) return g.A * ex2_hw(a);
    a = lp_clamp(a);
    return ex2_hw(a) * fmaf(g.B, a, g.A);
}
// N values (N even) in packed pairs
template <bool ENT, int N>
__device__ inline void lp_grad_vec(const LpGrad &g, const float *x, float k, float *out) {
    const F2 mm = f2(g.M, g.M), kk = f2(k, k), nl = f2(g.neg_log2d, g.neg_log2d);
    const F2 A = f2(g.A, g.A), B = f2(g.B, g.B);
#pragma unroll
    for (int p = 0; p < N / 2; ++p) {
        F2 a = f2_fma(f2_sub(f2(x[2 * p], x[2 * p + 1]), mm), kk, nl);
        F2 c = A;
        if (ENT) {
            float a0, a1;
            f2_split(a, a0, a1);
            a = f2(lp_clamp(a0), lp_clamp(a1));
            c = f2_fma(B, a, A);
        }
        f2_split(f2_mul(f2_ex2(a), c), out[2 * p], out[2 * p + 1]);
    }
}

// The 16 bytes from byte sh on (0 < sh < 16, a multiple of the element size)
// of two consecutive vectors.
template <int KB>
__device__ inline uint4 shift16(const uint4 &a, const uint4 &b, uint32_t sh) {
    uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
    uint32_t last = b.w;
    if (sh & 8u) {
        w[0] = w[2]; w[1] = w[3]; w[2] = w[4]; w[3] = w[5]; w[4] = w[6]; w[5] = last;
    }
    if (sh & 4u) {
        w[0] = w[1]; w[1] = w[2]; w[2] = w[3]; w[3] = w[4]; w[4] = w[5];
    }
    if (KB == 2 && (sh & 2u))
        return make_uint4(__funnelshift_r(w[0], w[1], 16), __funnelshift_r(w[1], w[2], 16), __funnelshift_r(w[2], w[3], 16),
                          __funnelshift_r(w[3], w[4], 16));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Columns [c0, c1) of one row's gradient, by nt threads (whole warps; this one
// is tid): the interior in 16-byte vectors placed by the gradient's alignment.
// Where the logits lie otherwise, each lane loads the aligned vector that its
// columns start in and takes the rest from the next lane. x and grad may be the
// same row.
template <int DT, bool ENT>
__device__ inline void lp_grad_span(const char *xrow, char *grow, int64_t c0, int64_t c1, int y, const LpGrad &g, float k,
                                    int tid, int nt) {
    using F = Fmt<DT>;
    constexpr int VEC = F::kVec, KB = F::kBytes;
    const int64_t head = static_cast<int64_t>((16u - (reinterpret_cast<uintptr_t>(grow + c0 * KB) & 15u)) & 15u) / KB;
    const int64_t v0 = c0 + head < c1 ? c0 + head : c1;
    const int64_t nvec = (c1 - v0) / VEC;
    const int64_t tail = v0 + nvec * VEC;
    const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(xrow + v0 * KB)) & 15u;
    const char *const xa = xrow + v0 * KB - sh;  // 16-byte aligned; each vector read holds some of the columns
    const int lane = tid & 31;
    constexpr int U = 4;  // vectors in flight per thread
    for (int64_t vb = tid - lane; vb < nvec; vb += static_cast<int64_t>(U) * nt) {
        uint4 raw[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t v = vb + lane + static_cast<int64_t>(j) * nt;
            raw[j] = v < nvec ? ld_stream(xa + 16 * v) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (sh != 0) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t v = vb + lane + static_cast<int64_t>(j) * nt;
                uint4 next;
                next.x = __shfl_down_sync(0xffffffffu, raw[j].x, 1);
                next.y = __shfl_down_sync(0xffffffffu, raw[j].y, 1);
                next.z = __shfl_down_sync(0xffffffffu, raw[j].z, 1);
                next.w = __shfl_down_sync(0xffffffffu, raw[j].w, 1);
                if (v < nvec && (lane == 31 || v + 1 == nvec)) next = ld_stream(xa + 16 * (v + 1));
                raw[j] = shift16<KB>(raw[j], next, sh);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t v = vb + lane + static_cast<int64_t>(j) * nt;
            if (v >= nvec) continue;
            float xv[VEC], o[VEC];
            F::unpack(raw[j], xv);
            lp_grad_vec<ENT, VEC>(g, xv, k, o);
            const int64_t rel = y - (v0 + v * VEC);
            if (rel >= 0 && rel < VEC) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = e == rel ? g.dy : o[e];
            }
            st_stream(grow + (v0 + v * VEC) * KB, F::pack(o));
        }
    }
    // the columns before the first and after the last vector (fewer than VEC each)
    const int nh = static_cast<int>(v0 - c0), ne = nh + static_cast<int>(c1 - tail);
    for (int e = tid; e < ne; e += nt) {
        const int64_t c = e < nh ? c0 + e : tail + (e - nh);
        F::store1(grow, c, c == y ? g.dy : lp_grad_elem<ENT>(g, F::load1(xrow, c), k));
    }
}

// zeros over columns [c0, c1) of a gradient row
template <int DT>
__device__ inline void lp_zero_span(char *grow, int64_t c0, int64_t c1, int tid, int nt) {
    using F = Fmt<DT>;
    constexpr int VEC = F::kVec, KB = F::kBytes;
    const int64_t head = static_cast<int64_t>((16u - (reinterpret_cast<uintptr_t>(grow + c0 * KB) & 15u)) & 15u) / KB;
    const int64_t v0 = c0 + head < c1 ? c0 + head : c1;
    const int64_t nvec = (c1 - v0) / VEC;
    const int64_t tail = v0 + nvec * VEC;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t v = tid; v < nvec; v += nt) st_stream(grow + (v0 + v * VEC) * KB, z);
    const int nh = static_cast<int>(v0 - c0), ne = nh + static_cast<int>(c1 - tail);
    for (int e = tid; e < ne; e += nt) F::store1(grow, e < nh ? c0 + e : tail + (e - nh), 0.f);
}

}  // namespace ce
