// lp_short.cu -- the row kernel of the log-probability operators for rows of
// up to 16 KB: a group of 1, 2 or 4 warps owns a row and holds it in registers,
// eight 16-byte vectors a thread, so that it is read once, its maximum is known
// before the exponentials, and the gradient is formed from the same registers.
// Groups go on independently of one another (a named barrier each), which keeps
// the latency of a row's merges and scalars off the other rows.
#include "ce_host.h"
#include "lp_policy.cuh"

namespace ce {

constexpr int kShortVecs = 8;
constexpr int kShortThreads = 256;
constexpr int kShortMaxWarps = 4;                  // of a group
constexpr int kShortMaxGroups = kShortThreads / 32;
constexpr int kShortCtasPerSm = 3;

__device__ inline void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// one element of a vector set to -inf
template <int DT>
__device__ inline void drop_element(uint4 &v, int e) {
    uint32_t *w = &v.x;
    constexpr uint32_t ninf = Fmt<DT>::kNegInfWord;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (Fmt<DT>::kBytes == 4) {
            if (i == e) w[i] = ninf;
        } else if (i == e / 2) {
            w[i] = (e & 1) ? (w[i] & 0xffffu) | (ninf & 0xffff0000u) : (w[i] & 0xffff0000u) | (ninf & 0xffffu);
        }
    }
}

template <int DT, int MODE, bool ENT>
__global__ void __launch_bounds__(kShortThreads, kShortCtasPerSm) lp_short_kernel(LpArgs a, int warps) {
    using F = Fmt<DT>;
    constexpr int VEC = F::kVec, KB = F::kBytes, R = kShortVecs;
    constexpr bool POLICY = MODE == LP_POLICY;
    __shared__ float red_m[kShortMaxGroups], red_s[kShortMaxGroups], red_u[kShortMaxGroups];  // of every warp
    __shared__ LpGrad grads[kShortMaxGroups];
    __shared__ double sums[kShortMaxGroups];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = warps * 32, groups = blockDim.x / G;
    const int gid = warp / warps, gw = warp - gid * warps, gt = tid - gid * G;
    const int V = static_cast<int>(a.vocab);
    const float k = a.k;
    bool have_norm = false;
    float w_sum = 0.f;
    double sum = 0.0;  // this group's row losses (its first thread)
    int64_t row_lo = 0, row_hi = a.n_rows;
    if (!POLICY && a.offsets) {
        row_lo = load_target(a.offsets, a.off32, 0);
        row_hi = load_target(a.offsets, a.off32, a.n_seqs);
        if (blockIdx.x == 0 && tid == 0) {  // the preference loss's later kernels count and flag here
            a.ctl->status = 0u;
            a.ctl->n_correct = 0u;
        }
    }
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + gid; row < a.n_rows;
         row += static_cast<int64_t>(gridDim.x) * groups) {
        const int64_t t = load_target(a.target, a.tgt32, row);
        const char *xrow = reinterpret_cast<const char *>(a.x) + row * a.ld * KB;
        char *grow = POLICY ? reinterpret_cast<char *>(a.grad) + row * a.ld_grad * KB : nullptr;
        const bool live = POLICY ? policy_row_live(a, row, t)
                                 : target_valid(t, a.ignore_index, V) && row >= row_lo && row < row_hi;
        if (!live) {
            if (POLICY) {
                lp_zero_span<DT>(grow, 0, V, gt, G);
                if (gt == 0) {
                    if (a.reduction == CE_RED_NONE) a.loss[row] = 0.f;
                    if (a.row_stats) a.row_stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            } else if (gt == 0) {
                // ignored: 0; a target outside [0, vocab): NaN (0 inside the preference loss, which flags it)
                const float none = t == a.ignore_index || a.offsets ? 0.f : NAN;
                if (a.logp) a.logp[row] = none;
                if (a.entropy) a.entropy[row] = none;
                if (a.stats) a.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            continue;
        }
        // ---------------------------------------------------- the row into registers
        const int y = static_cast<int>(t);
        const int head = min(static_cast<int>((16u - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(xrow)) & 15u)) & 15u) / KB, V);
        const int nvec = (V - head) / VEC, tail0 = head + nvec * VEC, nedge = head + V - tail0;
        const char *const xv = xrow + head * KB + 16 * gt;
        uint4 raw[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t ninf = F::kNegInfWord;
            raw[i] = gt + i * G < nvec ? ld_stream(xv + static_cast<int64_t>(16) * i * G) : make_uint4(ninf, ninf, ninf, ninf);
        }
        // the columns before the first and after the last 16-byte boundary: one a thread
        const int edge = gt < nedge ? (gt < head ? gt : tail0 + (gt - head)) : -1;
        const float xe = edge >= 0 ? F::load1(xrow, edge) : -INFINITY;
        PolicyIn in{};
        float xy = 0.f;
        if (gw == 0) {
            xy = F::load1(xrow, y);
            if (POLICY) in = policy_load(a, row);
        }
        const int yv = y >= head && y < tail0 ? (y - head) / VEC - gt : -1;  // of this thread's: a multiple of G
        const bool own = yv >= 0 && yv % G == 0;
        if (own) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (i * G == yv) drop_element<DT>(raw[i], (y - head) % VEC);
        }
        const float xs = edge == y ? -INFINITY : xe;
        // ---------------------------------------------------- maximum, then the sums relative to it
        float m = xs;
#pragma unroll
        for (int i = 0; i < R; ++i) m = fmaxf(m, F::vmax(raw[i]));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (warps > 1) {
            if (lane == 0) red_m[warp] = m;
            group_sync(1 + gid, G);
            m = red_m[gid * warps];
            for (int w = 1; w < warps; ++w) m = fmaxf(m, red_m[gid * warps + w]);
        }
        // without a finite value there is nothing to move the exponents by (NaN stays)
        const float m0 = m == -INFINITY ? 0.f : m;
        const F2 mm = f2(m0, m0), kk = f2(k, k);
        F2 s2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)}, u2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i * G >= nvec) break;
            float x[VEC];
            F::unpack(raw[i], x);
#pragma unroll
            for (int p = 0; p < VEC / 2; ++p) {
                F2 e = f2_mul(f2_sub(f2(x[2 * p], x[2 * p + 1]), mm), kk);
                if (ENT) {
                    float a0, a1;
                    f2_split(e, a0, a1);
                    e = f2(lp_clamp(a0), lp_clamp(a1));
                }
                const F2 ex = f2_ex2(e);
                s2[p & 1] = f2_add(s2[p & 1], ex);
                if (ENT) u2[p & 1] = f2_fma(ex, e, u2[p & 1]);
            }
        }
        float s0, s1, u = 0.f;
        f2_split(f2_add(s2[0], s2[1]), s0, s1);
        const float ae = lp_clamp((xs - m0) * k), ee = ex2_hw(ae);
        float s = s0 + s1 + ee;
        if (ENT) {
            f2_split(f2_add(u2[0], u2[1]), s0, s1);
            u = fmaf(ee, ae, s0 + s1);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, off);
            if (ENT) u += __shfl_xor_sync(0xffffffffu, u, off);
        }
        if (warps > 1) {
            if (lane == 0) {
                red_s[warp] = s;
                red_u[warp] = u;
            }
            group_sync(1 + gid, G);
            if (gw == 0) {
                s = lane < warps ? red_s[gid * warps + lane] : 0.f;
                u = lane < warps ? red_u[gid * warps + lane] : 0.f;
#pragma unroll
                for (int off = kShortMaxWarps / 2; off > 0; off >>= 1) {
                    s += __shfl_xor_sync(0xffffffffu, s, off);
                    u += __shfl_xor_sync(0xffffffffu, u, off);
                }
                s = __shfl_sync(0xffffffffu, s, 0);
                u = __shfl_sync(0xffffffffu, u, 0);
            }
        }
        // ---------------------------------------------------- row scalars, by the group's first warp
        LpGrad g{};
        if (gw == 0) {
            float4 stats = lp_row_stats(LpState{m, s, u}, xy, k);
            const LpRow r = lp_row(stats, k, a.inv_t);
            if (!POLICY) {
                if (lane == 0) {
                    if (a.logp) a.logp[row] = r.logp;
                    if (ENT && a.entropy) a.entropy[row] = r.entropy;
                    if (!ENT) stats.w = NAN;
                    if (a.stats) a.stats[row] = stats;
                }
            } else {
                const PolicyOut o = policy_row(a, in, r, r.entropy);
                if (!have_norm) {
                    pdl_wait();
                    w_sum = policy_weight_sum(a);
                    have_norm = true;
                }
                const float scale = policy_scale(a, row, w_sum);
                g = lp_grad(stats, r, a.inv_t, o.g * scale, o.h * scale);
                if (lane == 0) {
                    if (a.reduction == CE_RED_NONE) a.loss[row] = o.loss;
                    else sum += static_cast<double>(o.loss);
                    if (a.row_stats) a.row_stats[row] = make_float4(r.logp, ENT ? r.entropy : 0.f, o.ratio, o.kl);
                    if (warps > 1) grads[gid] = g;
                }
            }
        }
        if (!POLICY) continue;
        if (warps > 1) {
            group_sync(1 + gid, G);
            g = grads[gid];
        } else {
            __syncwarp();  // every lane has the target's logit: it may be written over
        }
        // ---------------------------------------------------- gradient
        if (((reinterpret_cast<uintptr_t>(xrow) ^ reinterpret_cast<uintptr_t>(grow)) & 15u) != 0) {
            // another alignment than the logits': read again (from L2), placed by the gradient's
            lp_grad_span<DT, ENT>(xrow, grow, 0, V, y, g, k, gt, G);
            continue;
        }
        char *const gv = grow + head * KB + 16 * gt;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (gt + i * G < nvec) {
                float x[VEC], o[VEC];
                F::unpack(raw[i], x);
                lp_grad_vec<ENT, VEC>(g, x, k, o);
                st_stream(gv + static_cast<int64_t>(16) * i * G, F::pack(o));
            }
        }
        if (own) F::store1(grow, y, g.dy);  // after the store of its vector, by the same thread
        if (edge >= 0) F::store1(grow, edge, edge == y ? g.dy : lp_grad_elem<ENT>(g, xe, k));
    }
    if (POLICY && blockIdx.x == 0 && tid == 0) {
        pdl_wait();
        policy_flags(a);
    }
    // -------------------------------------------------------- batch loss (last CTA)
    if (POLICY && a.reduction != CE_RED_NONE) {
        if (gt == 0) sums[gid] = sum;
        __syncthreads();
        if (warp == 0) {
            pdl_wait();
            unsigned last = 0;
            if (lane == 0) {
                double s = 0.0;
                for (int i = 0; i < groups; ++i) s += sums[i];
                a.part[blockIdx.x] = s;
                __threadfence();
                last = atomicAdd(&a.ctl->done, 1u) == gridDim.x - 1 ? 1u : 0u;
            }
            if (__shfl_sync(0xffffffffu, last, 0)) {
                __threadfence();
                double s = 0.0;  // in CTA order, then a fixed tree
                for (unsigned i = lane; i < gridDim.x; i += 32) s += __ldcg(a.part + i);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                if (a.reduction == CE_RED_MEAN) {
                    const float w_all = policy_weight_sum(a);
                    s = w_all != 0.f ? s / static_cast<double>(w_all) : 0.0;
                }
                if (lane == 0) a.loss[0] = static_cast<float>(s);
            }
        }
    }
}

template <int DT>
static const void *short_fn(int mode, bool ent) {
    if (mode == LP_FWD)
        return ent ? reinterpret_cast<const void *>(&lp_short_kernel<DT, LP_FWD, true>)
                   : reinterpret_cast<const void *>(&lp_short_kernel<DT, LP_FWD, false>);
    return ent ? reinterpret_cast<const void *>(&lp_short_kernel<DT, LP_POLICY, true>)
               : reinterpret_cast<const void *>(&lp_short_kernel<DT, LP_POLICY, false>);
}

bool lp_short_takes(int64_t vocab, int dtype) {
    return vocab * (dtype == CE_DT_F32 ? 4 : 2) <= static_cast<int64_t>(kShortVecs) * 16 * 32 * kShortMaxWarps;
}

cudaError_t launch_lp_short(const LpArgs &a0, int dtype, int mode, bool entropy, bool after_prep, int sms, cudaStream_t s) {
    LpArgs a = a0;
    const void *fn = dtype == CE_DT_F32 ? short_fn<CE_DT_F32>(mode, entropy)
                   : dtype == CE_DT_BF16 ? short_fn<CE_DT_BF16>(mode, entropy) : short_fn<CE_DT_F16>(mode, entropy);
    const int64_t vecs = (a.vocab * (dtype == CE_DT_F32 ? 4 : 2) + 15) / 16;
    int warps = 1;
    while (vecs > static_cast<int64_t>(warps) * 32 * kShortVecs) warps *= 2;
    const int groups = kShortThreads / (warps * 32);
    const int64_t want = (a.n_rows + groups - 1) / groups, cap = static_cast<int64_t>(sms) * kShortCtasPerSm;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < cap ? want : cap));
    cfg.blockDim = dim3(kShortThreads);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = after_prep ? 1 : 0;
    void *args[] = {&a, &warps};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace ce
