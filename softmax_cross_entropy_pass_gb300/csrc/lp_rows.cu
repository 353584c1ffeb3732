// lp_rows.cu -- one kernel call per batch of rows for the log-probability
// operators: forward (log-probability, entropy, statistics) and the policy
// loss with its gradient.
#include "ce_host.h"
#include "lp_policy.cuh"

namespace ce {

constexpr int kLpThreads = 512;

template <int DT, int MODE, bool ENT>
__global__ void __launch_bounds__(kLpThreads) lp_rows_kernel(LpArgs a) {
    using F = Fmt<DT>;
    constexpr int VEC = F::kVec, KB = F::kBytes, NW = kLpThreads / 32;
    __shared__ LpState red[NW];
    __shared__ unsigned last_sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t V = a.vocab;
    double cta_sum = 0.0;
    int64_t lo = 0, hi = a.n_rows;
    if (MODE == LP_FWD && a.offsets) {
        if (blockIdx.x == 0 && tid == 0) {  // the preference loss's later kernels count and flag here
            a.ctl->status = 0u;
            a.ctl->n_correct = 0u;
        }
        lo = load_target(a.offsets, a.off32, 0);
        hi = load_target(a.offsets, a.off32, a.n_seqs);
    }
    if (MODE == LP_POLICY) pdl_wait();
    const float w_sum = MODE == LP_POLICY ? a.ctl->w_y : 0.f;
    for (int64_t row = blockIdx.x; row < a.n_rows; row += gridDim.x) {
        const int64_t t = load_target(a.target, a.tgt32, row);
        const char *xrow = reinterpret_cast<const char *>(a.x) + row * a.ld * KB;
        const bool valid = target_valid(t, a.ignore_index, V) && row >= lo && row < hi;
        const bool live = MODE == LP_POLICY ? policy_row_live(a, row, t) : valid;
        if (!live) {
            if (MODE == LP_POLICY) {
                lp_zero_span<DT>(reinterpret_cast<char *>(a.grad) + row * a.ld_grad * KB, 0, V, tid, kLpThreads);
                if (tid == 0) {
                    if (a.reduction == CE_RED_NONE) a.loss[row] = 0.f;
                    if (a.row_stats) a.row_stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            } else if (tid == 0) {
                // ignored: 0; a target outside [0, vocab): NaN (0 inside the preference loss, which flags it)
                const float none = t == a.ignore_index || a.offsets ? 0.f : NAN;
                if (a.logp) a.logp[row] = none;
                if (a.entropy) a.entropy[row] = none;
                if (a.stats) a.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            continue;
        }
        const float xy = F::load1(xrow, t);
        // the row without its target column: vectors from the row's first 16-byte boundary
        LpState st = lp_empty();
        const int64_t head = static_cast<int64_t>((16u - (reinterpret_cast<uintptr_t>(xrow) & 15u)) & 15u) / KB;
        const int64_t v0 = head < V ? head : V;
        const int64_t nvec = (V - v0) / VEC, tail = v0 + nvec * VEC;
        for (int64_t v = tid; v < nvec; v += kLpThreads) {
            float x[VEC];
            F::unpack(ld_stream(xrow + (v0 + v * VEC) * KB), x);
            const int64_t rel = t - (v0 + v * VEC);
            float vmax = -INFINITY;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                x[e] = e == rel ? -INFINITY : x[e];
                vmax = fmaxf(vmax, x[e]);
            }
            lp_add<ENT, VEC>(st, x, vmax, a.k);
        }
        const int nh = static_cast<int>(v0), ne = nh + static_cast<int>(V - tail);
        if (tid < ne) {
            const int64_t c = tid < nh ? tid : tail + (tid - nh);
            if (c != t) lp_add1<ENT>(st, F::load1(xrow, c), a.k);
        }
        st = lp_warp_merge<ENT>(st, a.k);
        __syncthreads();
        if (lane == 0) red[warp] = st;
        __syncthreads();
        st = lp_warp_merge<ENT, NW>(red[lane & (NW - 1)], a.k);
        float4 stats = lp_row_stats(st, xy, a.k);
        const LpRow r = lp_row(stats, a.k, a.inv_t);
        if (MODE == LP_FWD) {
            if (tid == 0) {
                if (a.logp) a.logp[row] = r.logp;
                if (ENT && a.entropy) a.entropy[row] = r.entropy;
                if (!ENT) stats.w = NAN;
                if (a.stats) a.stats[row] = stats;
            }
            continue;
        }
        const PolicyIn in = policy_load(a, row);
        const PolicyOut o = policy_row(a, in, r, r.entropy);
        if (tid == 0) {
            if (a.reduction == CE_RED_NONE) a.loss[row] = o.loss;
            else cta_sum += static_cast<double>(o.loss);
            if (a.row_stats) a.row_stats[row] = make_float4(r.logp, ENT ? r.entropy : 0.f, o.ratio, o.kl);
        }
        const float scale = policy_scale(a, row, w_sum);
        const LpGrad g = lp_grad(stats, r, a.inv_t, o.g * scale, o.h * scale);
        char *grow = reinterpret_cast<char *>(a.grad) + row * a.ld_grad * KB;
        lp_grad_span<DT, ENT>(xrow, grow, 0, V, static_cast<int>(t), g, a.k, tid, kLpThreads);
    }
    if (MODE == LP_POLICY && a.reduction != CE_RED_NONE) {
        if (tid == 0) {
            a.part[blockIdx.x] = cta_sum;
            __threadfence();
            last_sh = atomicAdd(&a.ctl->done, 1u) == gridDim.x - 1 ? 1u : 0u;
        }
        __syncthreads();
        if (last_sh && tid == 0) {
            __threadfence();
            double tot = 0.0;
            for (unsigned i = 0; i < gridDim.x; ++i) tot += __ldcg(a.part + i);
            if (a.reduction == CE_RED_MEAN) tot = w_sum != 0.f ? tot / static_cast<double>(w_sum) : 0.0;
            a.loss[0] = static_cast<float>(tot);
        }
    }
}

template <int DT>
static const void *rows_fn(int mode, bool ent) {
    if (mode == LP_FWD)
        return ent ? reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_FWD, true>)
                   : reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_FWD, false>);
    return ent ? reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_POLICY, true>)
               : reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_POLICY, false>);
}

cudaError_t launch_lp_rows(const LpArgs &a0, int dtype, int mode, bool entropy, bool after_prep, cudaStream_t s) {
    LpArgs a = a0;
    const void *fn = dtype == CE_DT_F32 ? rows_fn<CE_DT_F32>(mode, entropy)
                   : dtype == CE_DT_BF16 ? rows_fn<CE_DT_BF16>(mode, entropy) : rows_fn<CE_DT_F16>(mode, entropy);
    const int64_t cap = 152 * 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n_rows < cap ? a.n_rows : cap));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = after_prep ? 1 : 0;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace ce
