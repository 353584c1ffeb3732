// lp_rows.cu -- the row kernel of the log-probability operators: forward
// (log-probability, entropy, statistics) and the policy loss with its
// gradient.
//
// A CTA, or a cluster of 2, 4 or 8 CTAs that split the columns, owns whole
// rows. A producer warp streams them through a ring of shared-memory chunks
// with bulk copies; 8 consumer warps keep per-thread softmax statistics,
// which are merged per row (across the cluster through distributed shared
// memory). The policy loss needs the row's statistics before its gradient:
// its second pass reads the last chunks of the row where they still lie in
// the ring and the earlier ones, last first, from L2 again, so HBM sees one
// read and one write. The ring is not tied to a row, so copies go on while a
// row's statistics are merged. Every wait is bounded.
#include <mutex>

#include "ce_host.h"
#include "ce_stream.cuh"
#include "lp_policy.cuh"

namespace ce {

constexpr int kLpWarps = 8;
constexpr int kLpConsumers = kLpWarps * 32;
constexpr int kLpThreads = kLpConsumers + 32;
constexpr int kLpSlots = 4;
constexpr int kLpCtasPerSm = 3;
constexpr int kLpMaxCluster = 8;
constexpr int kLpCtlBytes = 1024;
constexpr int kLpSmemBytes = kLpSlots * kStreamChunk + kLpCtlBytes;

struct LpSmem {
    uint64_t full[kLpSlots], empty[kLpSlots];
    uint64_t xbar[2];
    // per row parity: a warp may write the next row's values while a slower
    // warp still reads this row's (never further ahead: the row's barrier
    // waits for every warp)
    float4 slot[2][kLpMaxCluster];  // each CTA's {m, s, u, target logit}
    LpState red[2][kLpWarps];
    LpGrad grad[2];                 // the row's gradient scalars, from warp 0
    float xy[2];
    int abort;
    unsigned last;
    double cta_sum;                 // this cluster's row losses (thread 0 of its first CTA)
    double sum[kLpWarps];
};
static_assert(sizeof(LpSmem) <= kLpCtlBytes, "control block too large");

__device__ inline void lp_consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kLpConsumers) : "memory"); }
__device__ inline void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// one element of a 16-byte aligned shared-memory chunk: read, and set to -inf
template <int DT>
__device__ inline float take_out(uint32_t addr) {
    if (Fmt<DT>::kBytes == 4) {
        float x;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(Fmt<DT>::kNegInfWord) : "memory");
        return x;
    }
    uint16_t b;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(addr) : "memory");
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(Fmt<DT>::kNegInfWord)) : "memory");
    return Fmt<DT>::load1(&b, 0);
}

// Add NV vectors of one thread to its statistics: one packed FMA an exponent
// pair, a' = x k - mu with mu = m k rounded. The FMA rounds a' alone, and what
// mu's rounding shifted (the same for every term) is taken out of the chunk's
// sums, so the sums are as exact as those of (x - m) k. With the entropy, a
// logit that is -inf (or so low that a' overflows) makes 0 * inf = NaN in u:
// false is returned then, and where mu is not finite, with st moved to the new
// maximum but nothing added; lp_add takes such vectors.
template <int DT, bool ENT, int NV>
__device__ inline bool add_vectors(LpState &st, const uint4 (&raw)[NV], float k) {
    using F = Fmt<DT>;
    constexpr int VEC = F::kVec;
    float cm = F::vmax(raw[0]);
#pragma unroll
    for (int i = 1; i < NV; ++i) cm = fmaxf(cm, F::vmax(raw[i]));
    if (cm > st.m) lp_rebase<ENT>(st, cm, k);
    const float mu = st.m * k;
    if (!(fabsf(mu) < 1e38f)) return false;
    const F2 kk = f2(k, k), nm = f2(-mu, -mu);
    F2 s2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)}, u2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float x[VEC];
        F::unpack(raw[i], x);
#pragma unroll
        for (int p = 0; p < VEC / 2; ++p) {
            const F2 e = f2_fma(f2(x[2 * p], x[2 * p + 1]), kk, nm);
            const F2 ex = f2_ex2(e);
            s2[p & 1] = f2_add(s2[p & 1], ex);
            if (ENT) u2[p & 1] = f2_fma(ex, e, u2[p & 1]);
        }
    }
    float s0, s1, u0 = 0.f, u1 = 0.f;
    f2_split(f2_add(s2[0], s2[1]), s0, s1);
    const float sc = s0 + s1, shift = fmaf(st.m, k, -mu), f = fmaf(-shift, kLn2, 1.f);
    if (ENT) {
        f2_split(f2_add(u2[0], u2[1]), u0, u1);
        const float uc = u0 + u1;
        if (uc != uc) return false;
        st.u = fmaf(fmaf(-shift, sc, uc), f, st.u);
    }
    st.s = fmaf(sc, f, st.s);
    return true;
}
template <int DT, bool ENT, int NV>
__device__ inline bool add_or_clamp(LpState &st, const uint4 (&raw)[NV], float k) {
    if (add_vectors<DT, ENT, NV>(st, raw, k)) return true;
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
        uint4 r = raw[0];
#pragma unroll
        for (int n = 1; n < NV; ++n) r = n == i ? raw[n] : r;
        float x[Fmt<DT>::kVec];
        Fmt<DT>::unpack(r, x);
        lp_add<ENT, Fmt<DT>::kVec>(st, x, Fmt<DT>::vmax(r), k);
    }
    return false;
}

// How the second pass forms its exponents log2 p: from x - M (SLOW: held at
// kLpMinExp where the entropy's part multiplies them), or on 16-bit rows with
// one FMA, x k + c with c = log2(1 / d) - M k rounded once: while |c| < 64
// that moves p by less than 2^-18, against half steps of 2^-9 and 2^-11.
constexpr float kFoldC = 64.f;
template <int DT, bool E, bool SLOW>
__device__ inline void grad_vec(const LpGrad &g, float c, const float *x, float k, float *out) {
    constexpr int VEC = Fmt<DT>::kVec;
    if (SLOW) {
        lp_grad_vec<E, VEC>(g, x, k, out);
        return;
    }
    const F2 kk = f2(k, k), A = f2(g.A, g.A), B = f2(g.B, g.B), cc = f2(c, c), mm = f2(g.M, g.M);
#pragma unroll
    for (int p = 0; p < VEC / 2; ++p) {
        const F2 xx = f2(x[2 * p], x[2 * p + 1]);
        const F2 e = Fmt<DT>::kBytes == 2 ? f2_fma(xx, kk, cc) : f2_fma(f2_sub(xx, mm), kk, cc);
        f2_split(f2_mul(f2_ex2(e), E ? f2_fma(B, e, A) : A), out[2 * p], out[2 * p + 1]);
    }
}

template <int DT, int MODE, bool ENT>
__global__ void __launch_bounds__(kLpThreads, kLpCtasPerSm) lp_rows_kernel(LpArgs a) {
    using F = Fmt<DT>;
    constexpr int VEC = F::kVec, KB = F::kBytes, NCT = kLpConsumers;
    constexpr int VPC = kStreamChunk / 16, VPT = VPC / NCT;
    static_assert(VPC % NCT == 0, "a full chunk gives every consumer the same vectors");
    constexpr bool POLICY = MODE == LP_POLICY;
    extern __shared__ __align__(128) uint8_t smem[];
    LpSmem &S = *reinterpret_cast<LpSmem *>(smem + kLpSlots * kStreamChunk);
    const uint32_t ring = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int V = static_cast<int>(a.vocab);
    const uint32_t cl = cluster_nctarank(), rank = cluster_ctarank();
    const int64_t q0 = cluster_id_x(), nq = nclusters_x();
    // this CTA's columns [lo, lo + L) of every row
    const int64_t part = (static_cast<int64_t>(V + cl - 1) / cl + VEC - 1) / VEC * VEC;
    const int64_t lo64 = rank * part;
    const int lo = static_cast<int>(lo64 < V ? lo64 : V);
    const int L = static_cast<int>(lo + part < V ? part : V - lo);
    const char *const xbase = reinterpret_cast<const char *>(a.x) + static_cast<int64_t>(lo) * KB;
    char *const gbase = POLICY ? reinterpret_cast<char *>(a.grad) + static_cast<int64_t>(lo) * KB : nullptr;
    const int64_t xstep = a.ld * KB, gstep = a.ld_grad * KB;

    if (tid == 0) {
        for (int s = 0; s < kLpSlots; ++s) {
            mbar_init(smem_u32(&S.full[s]), 1);
            mbar_init(smem_u32(&S.empty[s]), kLpWarps);
        }
        mbar_init(smem_u32(&S.xbar[0]), cl);
        mbar_init(smem_u32(&S.xbar[1]), cl);
        S.abort = 0;
        S.cta_sum = 0.0;
        fence_mbar_init_cluster();
    }
    __syncthreads();
    if (cl > 1) cluster_sync_all();  // the peers' barriers exist before any remote arrive
    volatile int *abort = &S.abort;

    // forward of the preference loss: rows outside of the sequences are skipped
    int64_t row_lo = 0, row_hi = a.n_rows;
    if (!POLICY && a.offsets) {
        row_lo = load_target(a.offsets, a.off32, 0);
        row_hi = load_target(a.offsets, a.off32, a.n_seqs);
        if (blockIdx.x == 0 && tid == 0) {  // its later kernels count and flag here
            a.ctl->status = 0u;
            a.ctl->n_correct = 0u;
        }
    }
    auto row_live = [&](int64_t row, int64_t t) {
        if (POLICY) return policy_row_live(a, row, t);
        return target_valid(t, a.ignore_index, V) && row >= row_lo && row < row_hi;
    };
    // The gradient's vectors lie where the logits' do only when both rows
    // start at the same offset from a 16-byte boundary.
    auto same_align = [&](int64_t row) {
        return (((reinterpret_cast<uintptr_t>(xbase) + row * xstep) ^ (reinterpret_cast<uintptr_t>(gbase) + row * gstep)) &
                15u) == 0;
    };

    if (warp == kLpWarps) {
        // -------------------------------------------------------------- producer
        if (lane == 0) {
            const uint64_t drop = policy_evict_first(), hold = policy_keep(), normal = createpolicy_normal();
            uint32_t it = 0;
            int64_t t_next = q0 < a.n_rows ? load_target(a.target, a.tgt32, q0) : 0;
            for (int64_t row = q0; row < a.n_rows; row += nq) {
                const int64_t t = t_next;
                if (row + nq < a.n_rows) t_next = load_target(a.target, a.tgt32, row + nq);
                if (!row_live(row, t)) continue;
                const char *slice = xbase + row * xstep;
                const RowGeom gm = row_geom<KB>(slice, lo, L);
                const char *src = slice + gm.nhead * KB;
                const bool twice = POLICY && same_align(row);
                const int nkeep = twice ? min(gm.nch, kLpSlots) : 0;
                for (int pass = 0; pass < (twice ? 2 : 1); ++pass) {
                    const int nc = pass == 0 ? gm.nch : gm.nch - nkeep;
                    for (int i = 0; i < nc; ++i, ++it) {
                        const int c = pass == 0 ? i : nc - 1 - i;
                        const uint64_t pol = pass == 1 ? drop : (c < gm.nch - nkeep && POLICY ? hold : normal);
                        const uint32_t s = it % kLpSlots, r = it / kLpSlots;
                        if (r > 0) mbar_wait_bounded<false, kStreamSleepP>(smem_u32(&S.empty[s]), (r - 1) & 1u, abort);
                        const int64_t off = static_cast<int64_t>(c) * kStreamChunk;
                        const uint32_t bytes =
                            static_cast<uint32_t>(gm.bytes - off < kStreamChunk ? gm.bytes - off : kStreamChunk);
                        mbar_expect_tx(smem_u32(&S.full[s]), bytes);
                        bulk_g2s_hint(ring + s * kStreamChunk, src + off, bytes, smem_u32(&S.full[s]), pol);
                    }
                }
            }
            // drain: every issued copy has landed before the CTA may exit
            for (uint32_t i = 0; i < kLpSlots && i < it; ++i) {
                const uint32_t c = it - 1 - i;
                mbar_wait_bounded<false, kStreamSleepP>(smem_u32(&S.full[c % kLpSlots]), (c / kLpSlots) & 1u, abort);
            }
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------- consumers
        const float k = a.k;
        bool have_norm = false;
        float w_sum = 0.f;
        uint32_t it = 0, j = 0;  // ring position; live rows done (parities)
        int64_t t_next = q0 < a.n_rows ? load_target(a.target, a.tgt32, q0) : 0;
        for (int64_t row = q0; row < a.n_rows; row += nq) {
            const int64_t t = t_next;
            if (row + nq < a.n_rows) t_next = load_target(a.target, a.tgt32, row + nq);
            const bool writer = tid == 0 && rank == 0;
            if (!row_live(row, t)) {
                if (POLICY) {
                    lp_zero_span<DT>(gbase + row * gstep, 0, L, tid, NCT);
                    if (writer) {
                        if (a.reduction == CE_RED_NONE) a.loss[row] = 0.f;
                        if (a.row_stats) a.row_stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                } else if (writer) {
                    // ignored: 0; a target outside [0, vocab): NaN (0 inside the preference loss, which flags it)
                    const float none = t == a.ignore_index || a.offsets ? 0.f : NAN;
                    if (a.logp) a.logp[row] = none;
                    if (a.entropy) a.entropy[row] = none;
                    if (a.stats) a.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                continue;
            }
            const char *xrow = xbase + row * xstep;
            const RowGeom gm = row_geom<KB>(xrow, lo, L);
            const int nvec = gm.nvec, nch = gm.nch, nedge = gm.nhead + gm.ntail;
            const int vlo = static_cast<int>(gm.vlo) - lo, tail0 = static_cast<int>(gm.tail0) - lo;
            const int yc = static_cast<int>(t) - lo;  // target column of the slice (it may lie outside)
            const int y = yc >= vlo && yc < tail0 ? yc - vlo : -1;
            const bool twice = POLICY && same_align(row);
            const int nkeep = twice ? min(nch, kLpSlots) : 0;
            const uint32_t rp = j & 1u, it_row = it;
            PolicyIn in{};
            if (POLICY && warp == 0) in = policy_load(a, row);  // its latency hides under the first pass
            // ------------------------------------------------ pass 1: statistics
            LpState st = lp_empty();
            uint32_t held = 0;
            for (int c = 0; c < nch; ++c, ++it) {
                const uint32_t s = it % kLpSlots;
                mbar_wait_bounded<false, kStreamSleepConsumer>(smem_u32(&S.full[s]), (it / kLpSlots) & 1u, abort);
                const uint32_t base_s = ring + s * kStreamChunk;
                const int v0 = c * VPC, nv = min(VPC, nvec - v0);
                const int vy = y >= 0 ? y / VEC - v0 : -1;
                if (vy >= 0 && vy < nv && vy % NCT == tid) {
                    // the target's column leaves the chunk: this thread alone reads its vector
                    S.xy[rp] = take_out<DT>(base_s + 16u * vy + static_cast<uint32_t>(y % VEC) * KB);
                    fence_async_shared();  // before a copy may overwrite the slot
                }
                bool plain = true;
                if (nv == VPC) {
                    uint4 raw[VPT];
#pragma unroll
                    for (int i = 0; i < VPT; ++i) raw[i] = ld_shared_v4(base_s + 16u * (tid + i * NCT));
                    plain = add_or_clamp<DT, ENT, VPT>(st, raw, k);
                } else {
                    for (int v = tid; v < nv; v += NCT) {
                        const uint4 raw[1] = {ld_shared_v4(base_s + 16u * v)};
                        plain = add_or_clamp<DT, ENT, 1>(st, raw, k) && plain;
                    }
                }
                // chunks whose exponents the second pass has to hold as well (31: any later one)
                if (POLICY && ENT && !plain) held |= 1u << min(c, 31);
                __syncwarp();
                if (lane == 0 && c < nch - nkeep) mbar_arrive(smem_u32(&S.empty[s]));
            }
            // columns before the first and after the last 16-byte boundary
            const int edge_c = tid < gm.nhead ? tid : tail0 + (tid - gm.nhead);
            if (tid < nedge) {
                const float x = F::load1(xrow, edge_c);
                if (edge_c == yc) S.xy[rp] = x;
                else lp_add1<ENT>(st, x, k);
            }
            // ------------------------------------------------ merge and row scalars
            // warp 0 merges the CTA's partials (and the cluster's), forms the row's
            // scalars and hands the gradient's to the others
            st = lp_warp_merge<ENT>(st, k);
            if (lane == 0) S.red[rp][warp] = st;
            lp_consumer_sync();
            if (warp == 0) {
                st = lp_warp_merge<ENT, kLpWarps>(S.red[rp][lane & (kLpWarps - 1)], k);
                float xy = yc >= 0 && yc < L ? S.xy[rp] : 0.f;
                if (cl > 1) {
                    const uint32_t my_bar = smem_u32(&S.xbar[rp]);
                    if (lane < static_cast<int>(cl)) {
                        st_cluster_v4(mapa_shared(smem_u32(&S.slot[rp][rank]), lane), st.m, st.s, st.u, xy);
                        mbar_arrive_remote(mapa_shared(my_bar, lane));
                    }
                    mbar_wait_bounded<true, kStreamSleepConsumer>(my_bar, (j >> 1) & 1u, abort);
                    st = lp_empty();
                    for (uint32_t d = 0; d < cl; ++d) {
                        const float4 q = S.slot[rp][d];
                        st = lp_merge<ENT>(st, LpState{q.x, q.y, q.z}, k);
                    }
                    xy = S.slot[rp][t / part].w;
                }
                float4 stats = lp_row_stats(st, xy, k);
                const LpRow r = lp_row(stats, k, a.inv_t);
                if (!POLICY) {
                    if (writer) {
                        const bool gone = *abort != 0;  // a wait gave up: no workspace to flag it in
                        if (a.logp) a.logp[row] = gone ? NAN : r.logp;
                        if (ENT && a.entropy) a.entropy[row] = gone ? NAN : r.entropy;
                        if (!ENT || gone) stats.w = NAN;
                        if (gone) stats.x = NAN;
                        if (a.stats) a.stats[row] = stats;
                    }
                } else {
                    const PolicyOut o = policy_row(a, in, r, r.entropy);
                    if (!have_norm) {
                        pdl_wait();
                        w_sum = a.ctl->w_y;
                        have_norm = true;
                    }
                    if (writer) {
                        if (a.reduction == CE_RED_NONE) a.loss[row] = o.loss;
                        else S.cta_sum += static_cast<double>(o.loss);
                        if (a.row_stats) a.row_stats[row] = make_float4(r.logp, ENT ? r.entropy : 0.f, o.ratio, o.kl);
                    }
                    const float scale = policy_scale(a, row, w_sum);
                    if (lane == 0) S.grad[rp] = lp_grad(stats, r, a.inv_t, o.g * scale, o.h * scale);
                }
            }
            ++j;
            if (!POLICY) continue;
            lp_consumer_sync();
            const LpGrad g = S.grad[rp];
            // ------------------------------------------------ pass 2: gradient
            char *grow = gbase + row * gstep;
            if (!twice) {
                lp_grad_span<DT, ENT>(xrow, grow, 0, L, yc, g, k, tid, NCT);
                continue;
            }
            uint4 *vp = reinterpret_cast<uint4 *>(grow + static_cast<int64_t>(vlo) * KB);
            const float fold = fmaf(-g.M, k, g.neg_log2d);
            const float cexp = KB == 2 ? fold : g.neg_log2d;
            // the whole row takes the slow form where the folded constant is too large,
            // and on fp32 rows where M might carry x - M out of range
            if (!(fabsf(KB == 2 ? fold : g.M) < (KB == 2 ? kFoldC : 1e30f))) held = ~0u;
            auto pass2 = [&](auto ent_tag) {
                constexpr bool E = decltype(ent_tag)::value;
                for (int i = 0; i < nch; ++i) {
                    // the kept chunks, from the slots the first pass filled, then the earlier ones
                    const bool in_ring = i < nkeep;
                    const int c = in_ring ? nch - nkeep + i : nch - 1 - i;
                    const uint32_t s = (in_ring ? it_row + static_cast<uint32_t>(c) : it) % kLpSlots;
                    if (!in_ring) {
                        mbar_wait_bounded<false, kStreamSleepConsumer>(smem_u32(&S.full[s]), (it / kLpSlots) & 1u, abort);
                        ++it;
                    }
                    const uint32_t base_s = ring + s * kStreamChunk;
                    const int v0 = c * VPC, nv = min(VPC, nvec - v0);
                    if (!((held >> min(c, 31)) & 1u)) {
                        for (int v = tid; v < nv; v += NCT) {
                            float x[VEC], og[VEC];
                            F::unpack(ld_shared_v4(base_s + 16u * v), x);
                            grad_vec<DT, E, false>(g, cexp, x, k, og);
                            st_stream(vp + v0 + v, F::pack(og));
                        }
                    } else {
                        for (int v = tid; v < nv; v += NCT) {
                            float x[VEC], og[VEC];
                            F::unpack(ld_shared_v4(base_s + 16u * v), x);
                            grad_vec<DT, E, true>(g, cexp, x, k, og);
                            st_stream(vp + v0 + v, F::pack(og));
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&S.empty[s]));
                }
            };
            if (ENT && g.B != 0.f) pass2(std::integral_constant<bool, ENT>{});
            else pass2(std::integral_constant<bool, false>{});
            // the target column of the interior, by the thread that stored its vector, after that store
            if (y >= 0 && (y / VEC) % NCT == tid) F::store1(grow, vlo + y, g.dy);
            if (tid < nedge)
                F::store1(grow, edge_c, edge_c == yc ? g.dy : lp_grad_elem<ENT>(g, F::load1(xrow, edge_c), k));
        }
        // ---------------------------------------------------- batch loss (last cluster)
        if (POLICY && a.reduction != CE_RED_NONE && rank == 0) {
            if (!have_norm) pdl_wait();
            if (tid == 0) {
                a.part[q0] = S.cta_sum;
                __threadfence();
                S.last = atomicAdd(&a.ctl->done, 1u) == static_cast<unsigned>(nq) - 1u ? 1u : 0u;
            }
            lp_consumer_sync();
            if (S.last) {
                __threadfence();
                double sum = 0.0;  // in cluster order, then a fixed tree
                for (int64_t i = tid; i < nq; i += NCT) sum += __ldcg(a.part + i);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (lane == 0) S.sum[warp] = sum;
                lp_consumer_sync();
                if (tid == 0) {
                    double tot = 0.0;
                    for (int w = 0; w < kLpWarps; ++w) tot += S.sum[w];
                    if (a.reduction == CE_RED_MEAN) {
                        const float w_all = a.ctl->w_y;
                        tot = w_all != 0.f ? tot / static_cast<double>(w_all) : 0.0;
                    }
                    a.loss[0] = static_cast<float>(tot);
                }
            }
        }
    }
    __syncthreads();
    if (tid == 0 && S.abort && a.ctl) {
        if (POLICY) pdl_wait();
        atomicOr(&a.ctl->status, CE_FLAG_WAIT_TIMEOUT);
    }
    if (cl > 1) cluster_sync_all();  // no CTA leaves while a peer may still write into it
}

template <int DT>
static const void *rows_fn(int mode, bool ent) {
    if (mode == LP_FWD)
        return ent ? reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_FWD, true>)
                   : reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_FWD, false>);
    return ent ? reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_POLICY, true>)
               : reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_POLICY, false>);
}

// The launch attributes of a kernel and cluster size on the current context,
// set and asked for once: how many clusters can be resident, and the SM count.
static cudaError_t rows_ready(const void *fn, int cl, int *clusters, int *sms) {
    struct Entry {
        const void *fn;
        unsigned long long ctx;
        int dev, cl, clusters, sms;
    };
    static Entry cache[256];
    static int used = 0;
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lk(mu);
    if (ctx != 0)
        for (int i = 0; i < used; ++i)
            if (cache[i].fn == fn && cache[i].ctx == ctx && cache[i].dev == dev && cache[i].cl == cl) {
                *clusters = cache[i].clusters;
                *sms = cache[i].sms;
                return cudaSuccess;
            }
    if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpSmemBytes)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(*sms * kLpCtasPerSm / cl * cl));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = kLpSmemBytes;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cl;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(clusters, fn, &cfg)) != cudaSuccess) return e;
    if (*clusters < 1) return cudaErrorInvalidConfiguration;
    const unsigned long long ctx2 = current_context_id();
    if (ctx2 != 0 && used < 256) cache[used++] = Entry{fn, ctx2, dev, cl, *clusters, *sms};
    return cudaSuccess;
}

cudaError_t launch_lp_rows(const LpArgs &a0, int dtype, int mode, bool entropy, bool after_prep, cudaStream_t s) {
    LpArgs a = a0;
    const void *fn = dtype == CE_DT_F32 ? rows_fn<CE_DT_F32>(mode, entropy)
                   : dtype == CE_DT_BF16 ? rows_fn<CE_DT_BF16>(mode, entropy) : rows_fn<CE_DT_F16>(mode, entropy);
    const int64_t row_bytes = a.vocab * (dtype == CE_DT_F32 ? 4 : 2);
    int clusters = 0, sms = 0;
    cudaError_t e = rows_ready(fn, 1, &clusters, &sms);
    if (e != cudaSuccess) return e;
    const int64_t slots = static_cast<int64_t>(sms) * kLpCtasPerSm;
    // With two passes the parts that wait in L2 for their second one (three
    // CTAs per SM) stay well inside it: 176 KB a CTA.
    int cl = 1;
    if (mode == LP_POLICY)
        while (cl < kLpMaxCluster && row_bytes > cl * (int64_t(176) << 10)) cl *= 2;
    // Few rows: split them over more CTAs, down to one chunk each.
    while (cl < kLpMaxCluster && a.n_rows * cl * 2 <= slots && row_bytes >= cl * 2 * kStreamChunk) cl *= 2;
    if (cl > 1 && (e = rows_ready(fn, cl, &clusters, &sms)) != cudaSuccess) return e;
    if (clusters > a.n_rows) clusters = static_cast<int>(a.n_rows);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * cl));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = kLpSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cl;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = after_prep ? 2 : 1;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace ce
