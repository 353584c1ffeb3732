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
// row's statistics are merged; of rows that fill no more than half of it, the
// next one's first pass comes in between. Every wait is bounded.
#include <mutex>

#include "ce_host.h"
#include "ce_stream.cuh"
#include "lp_policy.cuh"

namespace ce {

constexpr int kLpWarps = 8;                    // consumers
constexpr int kLpConsumers = kLpWarps * 32;
constexpr int kLpThreads = kLpConsumers + 64;  // and the producer and the scalar warp
constexpr int kLpSlots = 6;
constexpr int kLpCtasPerSm = 2;
constexpr int kLpMaxCluster = 8;
constexpr int kLpLagChunks = 3;  // two such rows fill the ring
// Rows are shared out per window of at most kLpWindow rows and kLpList rows a cluster
constexpr int kLpWindow = 8192;
constexpr int kLpList = 256;
constexpr int kLpCtlBytes = 6144;
constexpr int kLpSmemBytes = kLpSlots * kStreamChunk + 2 * kLpConsumers * 16 + kLpCtlBytes;

struct LpSmem {
    uint64_t full[kLpSlots], empty[kLpSlots];
    uint64_t xbar[2];
    uint64_t done[2], taken[2];     // per row parity: the consumers' statistics are there; they have been used
    float4 slot[2][kLpMaxCluster];  // each CTA's {m, s, u, target logit}
    LpGrad grad[2];                 // the row's gradient scalars
    float xy[2];
    int abort, drain_abort;           // a wait gave up; the wait for copies in flight did
    int n_live, n_dead;               // this cluster's rows of the window
    int live[kLpList + 1], dead[kLpList + 1];
    uint32_t mask[kLpWindow / 32];    // which rows of the window take part
    int before[kLpWindow / 32];       // how many of them lie before each 32
};
static_assert(sizeof(LpSmem) <= kLpCtlBytes, "control block too large");

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

// How add_vectors forms its exponents.
// DIFF false: one packed FMA a pair, a' = x k - mu with mu = m k rounded. The FMA
//   rounds a' alone. What mu's rounding shifted, the same for every term, is
//   taken out of the vectors' sums by 2^-shift to second order: shift is at most
//   half a unit in the last place of mu, 2^-7 while |mu| < kLpFmaMax, so the rest
//   is below (2^-7 ln 2)^3 / 6 = 2.7e-8 of a term. It grows with mu^3 (from 2^25
//   on a shift is no longer small against 1), so a larger |mu| takes the
//   difference. With the entropy, a logit that is -inf makes 0 * inf = NaN in u,
//   and the vectors are taken again with the difference.
// DIFF true: (x - m) k, the difference first, at any finite m: a packed operation
//   more a pair, and with the entropy exponents held at kLpMinExp, which `low`
//   counts. (8192 x 128256 bf16, all chunks in this form instead of the first:
//   forward 300 us against 302, with the entropy 361 against 310.)
constexpr float kLpFmaMax = 131072.f;

// Add NV vectors of one thread to its statistics. False where the form does not
// take them, with st moved to the new maximum but nothing added. ALL: every
// vector counts; else the first n do, and the others hold -inf.
template <int DT, bool ENT, int NV, bool DIFF, bool ALL>
__device__ inline bool add_vectors(LpState &st, const uint4 (&raw)[NV], int n, float k, int &low) {
    using F = Fmt<DT>;
    constexpr int VEC = F::kVec;
    float cm = F::vmax(raw[0]);
#pragma unroll
    for (int i = 1; i < NV; ++i) cm = fmaxf(cm, F::vmax(raw[i]));
    if (cm > st.m) lp_rebase<ENT>(st, cm, k);
    const float mu = st.m * k;
    if (DIFF ? !(fabsf(st.m) < INFINITY) : !(fabsf(mu) < kLpFmaMax)) return false;
    const F2 kk = f2(k, k), nm = DIFF ? f2(st.m, st.m) : f2(-mu, -mu);
    F2 s2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)}, u2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!ALL && i >= n) continue;
        float x[VEC];
        F::unpack(raw[i], x);
#pragma unroll
        for (int p = 0; p < VEC / 2; ++p) {
            const F2 xx = f2(x[2 * p], x[2 * p + 1]);
            F2 e = DIFF ? f2_mul(f2_sub(xx, nm), kk) : f2_fma(xx, kk, nm);
            if (DIFF && ENT) {
                float a0, a1;
                f2_split(e, a0, a1);
                a0 = lp_clamp(a0);
                a1 = lp_clamp(a1);
                low += (a0 == kLpMinExp ? 1 : 0) + (a1 == kLpMinExp ? 1 : 0);
                e = f2(a0, a1);
            }
            const F2 ex = f2_ex2(e);
            s2[p & 1] = f2_add(s2[p & 1], ex);
            if (ENT) u2[p & 1] = f2_fma(ex, e, u2[p & 1]);
        }
    }
    float s0, s1, sc, uc = 0.f;
    f2_split(f2_add(s2[0], s2[1]), s0, s1);
    sc = s0 + s1;
    if (ENT) {
        f2_split(f2_add(u2[0], u2[1]), s0, s1);
        uc = s0 + s1;
    }
    if (DIFF) {
        st.s += sc;
        if (ENT) st.u += uc;
        return true;
    }
    if (ENT && uc != uc) return false;
    const float shift = fmaf(st.m, k, -mu), d = shift * kLn2, f = fmaf(d, fmaf(d, 0.5f, -1.f), 1.f);
    if (ENT) st.u = fmaf(fmaf(-shift, sc, uc), f, st.u);
    st.s = fmaf(sc, f, st.s);
    return true;
}

// The same for any vectors. y_warp: one of the warp's lanes holds the row's
// target column among them, set to -inf (own: this one), so that the warp takes
// the held exponents at once instead of one lane after the others. Returns
// whether the second pass needs no held exponents for these vectors (the
// target's column it writes apart; far below another maximum than this thread's
// so far, an exponent that was not held here can leave fp32's range there).
template <int DT, bool ENT, int NV, bool ALL>
__device__ inline bool add_any(LpState &st, const uint4 (&raw)[NV], int n, float k, bool y_warp, bool own) {
    int low = 0;
    if (!(ENT && y_warp) && add_vectors<DT, ENT, NV, false, ALL>(st, raw, n, k, low)) return true;
    if (add_vectors<DT, ENT, NV, true, ALL>(st, raw, n, k, low)) return low <= (own ? 1 : 0) && fabsf(st.m * k) < kLpFmaMax;
    // no finite maximum: every value -inf or NaN so far, or +inf among them
#pragma unroll 1
    for (int i = 0; i < (ALL ? NV : n); ++i) {
        uint4 r = raw[0];
#pragma unroll
        for (int v = 1; v < NV; ++v) r = v == i ? raw[v] : r;
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

// Where one row's slice of L columns sits against 16-byte boundaries, in 32-bit
// arithmetic (it is formed once a row by every thread): columns before the
// first, vectors from there, columns after the last.
struct LpGeom {
    int head, nvec, tail0, nch;
};
template <int KB>
__device__ inline LpGeom lp_geom(const char *slice, int L) {
    LpGeom g;
    g.head = min(static_cast<int>((16u - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(slice)) & 15u)) & 15u) / KB, L);
    g.nvec = (L - g.head) / (16 / KB);
    g.tail0 = g.head + g.nvec * (16 / KB);
    g.nch = (g.nvec + kStreamChunk / 16 - 1) / (kStreamChunk / 16);
    return g;
}

// A position in the ring: slots are used one after the other, phase changes
// with every round.
struct RingPos {
    uint32_t slot, phase;
    __device__ inline void next() {
        if (++slot == kLpSlots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

template <class T>
__device__ inline void swap_values(T &a, T &b) {
    const T c = a;
    a = b;
    b = c;
}

// LAG: rows of at most kLpLagChunks chunks. Their second pass comes after the
// next row's first, both rows in the ring, so that a row's statistics are merged
// meanwhile (8192 bf16 rows, without / with entropy: 10000 columns 115 / 128 us
// to 97 / 113, 16384 121 / 135 to 105 / 120, 24000 154 / 173 to 146 / 171).
// Compiled apart, since what it carries from row to row costs longer rows 3%.
template <int DT, int MODE, bool ENT, bool LAG>
__global__ void __launch_bounds__(kLpThreads, kLpCtasPerSm) lp_rows_kernel(LpArgs a) {
    using F = Fmt<DT>;
    constexpr int VEC = F::kVec, KB = F::kBytes, NCT = kLpConsumers;
    constexpr int VPC = kStreamChunk / 16, VPT = VPC / NCT;
    static_assert(VPC % NCT == 0, "a full chunk gives every consumer the same vectors");
    constexpr bool POLICY = MODE == LP_POLICY;
    extern __shared__ __align__(128) uint8_t smem[];
    float4 *const parts = reinterpret_cast<float4 *>(smem + kLpSlots * kStreamChunk);  // [2][NCT] {m, s, u, -}
    LpSmem &S = *reinterpret_cast<LpSmem *>(parts + 2 * NCT);
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
        for (int p = 0; p < 2; ++p) {
            mbar_init(smem_u32(&S.xbar[p]), cl);
            mbar_init(smem_u32(&S.done[p]), kLpWarps);
            mbar_init(smem_u32(&S.taken[p]), 1);
        }
        S.abort = S.drain_abort = 0;
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
    // Which rows this cluster takes. Up to one row a cluster: its own number.
    // Otherwise the rows that take part and those that do not are dealt out
    // separately, window by window, every cluster getting the same number of each
    // (dealt together, a cluster's share of the former varies: 8192 x 128256
    // bf16 with 30% left out 658 us against 636). A window's lists are
    // built by the whole CTA from one read of the targets.
    const bool single = a.n_rows <= nq;
    const int64_t window = single ? a.n_rows : (kLpList * nq < kLpWindow ? kLpList * nq : kLpWindow);
    RingPos pos{0u, 0u};     // producer and consumers
    uint32_t issued = 0;     // producer: copies so far
    uint32_t j = 0, j2 = 0;  // live rows done (their parities), and with LAG second passes
    bool have_norm = false;  // scalar warp: the batch's weight sum, this cluster's row losses (lane 0 of its first CTA)
    float w_sum = 0.f;
    double cta_sum = 0.0;
    const auto dead_outputs = [&](int64_t row, int64_t t) {
        if (POLICY) {
            if (a.reduction == CE_RED_NONE) a.loss[row] = 0.f;
            if (a.row_stats) a.row_stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            // ignored: 0; a target outside [0, vocab): NaN (0 inside the preference loss, which flags it)
            const float none = t == a.ignore_index || a.offsets ? 0.f : NAN;
            if (a.logp) a.logp[row] = none;
            if (a.entropy) a.entropy[row] = none;
            if (a.stats) a.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    const auto zero_row = [&](int64_t row) {
        if (POLICY) lp_zero_span<DT>(gbase + row * gstep, 0, L, tid, NCT);
    };
    for (int64_t w0 = 0; w0 < a.n_rows; w0 += window) {
    int n_live, n_dead;
    if (single) {
        const int64_t t = load_target(a.target, a.tgt32, q0);  // at most one cluster a row is launched
        n_live = row_live(q0, t) ? 1 : 0;
        n_dead = POLICY ? 1 - n_live : 0;
        if (tid == 0) {
            S.live[0] = S.dead[0] = static_cast<int>(q0);
            if (n_live == 0 && rank == 0) dead_outputs(q0, t);
        }
        __syncthreads();
    } else {
        const int cnt = static_cast<int>(a.n_rows - w0 < window ? a.n_rows - w0 : window);
        const int words = (cnt + 31) / 32;
        // the targets of several words at once: their latency is the window's start-up
        constexpr int NWARP = kLpThreads / 32, U = 13;
        for (int base = warp; base < words; base += U * NWARP) {
            int64_t t[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int at = (base + i * NWARP) * 32 + lane;
                t[i] = at < cnt ? load_target(a.target, a.tgt32, w0 + at) : -1;
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int wd = base + i * NWARP;
                if (wd < words) {
                    const uint32_t m = __ballot_sync(0xffffffffu, wd * 32 + lane < cnt && row_live(w0 + wd * 32 + lane, t[i]));
                    if (lane == 0) S.mask[wd] = m;
                }
            }
        }
        __syncthreads();
        if (warp == 0) {
            constexpr int PER = kLpWindow / 32 / 32;  // words of a lane
            int c[PER], sum = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int wd = lane * PER + i;
                c[i] = sum;
                sum += wd < words ? __popc(S.mask[wd]) : 0;
            }
            int incl = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) S.before[lane * PER + i] = incl - sum + c[i];
            if (lane == 31) {
                // this cluster's rows have the ranks q0, q0 + nq, ... among each kind
                const int q = static_cast<int>(q0), n = static_cast<int>(nq), live = incl, dead = cnt - incl;
                S.n_live = q < live ? (live - q - 1) / n + 1 : 0;
                S.n_dead = q < dead ? (dead - q - 1) / n + 1 : 0;
            }
        }
        __syncthreads();
        for (int wd = warp; wd < words; wd += kLpThreads / 32) {
            const int i = wd * 32 + lane;
            const uint32_t m = S.mask[wd];
            const int lr = S.before[wd] + __popc(m & ((1u << lane) - 1u));
            const bool live = (m >> lane) & 1u;
            const uint32_t r = live ? lr : i - lr;
            const uint32_t at = r / static_cast<uint32_t>(nq);
            if (i < cnt && r - at * static_cast<uint32_t>(nq) == static_cast<uint32_t>(q0)) {
                (live ? S.live : S.dead)[at] = static_cast<int>(w0) + i;
                if (!live && rank == 0) dead_outputs(w0 + i, load_target(a.target, a.tgt32, w0 + i));
            }
        }
        __syncthreads();
        n_live = S.n_live;
        n_dead = POLICY ? S.n_dead : 0;
    }
    const auto live_row = [&](int i) { return static_cast<int64_t>(S.live[i]); };
    const auto dead_row = [&](int i) { return static_cast<int64_t>(S.dead[i]); };

    if (warp == kLpWarps) {
        // -------------------------------------------------------------- producer
        if (lane == 0) {
            const uint64_t drop = policy_evict_first(), hold = policy_keep(), normal = createpolicy_normal();
            for (int li = 0; li < n_live; ++li) {
                const int64_t row = live_row(li);
                const char *slice = xbase + row * xstep;
                const LpGeom gm = lp_geom<KB>(slice, L);
                const char *src = slice + gm.head * KB;
                const int nkeep = POLICY ? min(gm.nch, kLpSlots) : 0;
                for (int pass = 0; pass < (POLICY ? 2 : 1); ++pass) {
                    const int nc = pass == 0 ? gm.nch : gm.nch - nkeep;
                    for (int i = 0; i < nc; ++i) {
                        const int c = pass == 0 ? i : nc - 1 - i;
                        const uint64_t pol = pass == 1 ? drop : (c < gm.nch - nkeep && POLICY ? hold : normal);
                        const uint32_t full = smem_u32(&S.full[pos.slot]);
                        if (issued >= kLpSlots)
                            mbar_wait_bounded<false, kStreamSleepP>(smem_u32(&S.empty[pos.slot]), pos.phase ^ 1u, abort);
                        const uint32_t bytes = 16u * static_cast<uint32_t>(min(VPC, gm.nvec - c * VPC));
                        mbar_expect_tx(full, bytes);
                        bulk_g2s_hint(ring + pos.slot * kStreamChunk, src + static_cast<int64_t>(c) * kStreamChunk, bytes, full,
                                      pol);
                        pos.next();
                        ++issued;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == kLpWarps + 1) {
        // -------------------------------------------------------------- scalar warp
        // Merges the consumers' statistics of each row (and the cluster's), forms the
        // row's scalars, writes its results and hands the gradient's scalars back,
        // so that in the forward the consumers go on with the next row meanwhile.
        const float k = a.k;
        int64_t t_next = 0;  // read a row ahead
        PolicyIn in_next{};
        const auto fetch = [&](int li) {
            if (li >= n_live) return;
            t_next = load_target(a.target, a.tgt32, live_row(li));
            if (POLICY) in_next = policy_load(a, live_row(li));
        };
        fetch(0);
        for (int li = 0; li < n_live; ++li) {
            const int64_t row = live_row(li), t = t_next;
            const PolicyIn in = in_next;
            fetch(li + 1);
            const uint32_t rp = j & 1u, ph = (j >> 1) & 1u;
            ++j;
            const bool writer = lane == 0 && rank == 0;
            mbar_wait_bounded<false, kStreamSleepConsumer>(smem_u32(&S.done[rp]), ph, abort);
            const float4 *const pp = parts + rp * NCT;
            float M = -INFINITY;
#pragma unroll
            for (int i = 0; i < kLpWarps; ++i) M = fmaxf(M, pp[lane + 32 * i].x);
            LpState st{M, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kLpWarps; ++i) {
                const float4 q = pp[lane + 32 * i];
                LpState o{q.x, q.y, q.z};
                if (M != -INFINITY) lp_rebase<ENT>(o, M, k);
                st.s += o.s;
                if (ENT) st.u += o.u;
            }
            st = lp_warp_merge<ENT>(st, k);
            float xy = S.xy[rp];
            if (cl > 1) {
                const uint32_t my_bar = smem_u32(&S.xbar[rp]);
                if (lane < static_cast<int>(cl)) {
                    st_cluster_v4(mapa_shared(smem_u32(&S.slot[rp][rank]), lane), st.m, st.s, st.u, xy);
                    mbar_arrive_remote(mapa_shared(my_bar, lane));
                }
                mbar_wait_bounded<true, kStreamSleepConsumer>(my_bar, ph, abort);
                // lanes from cl on repeat its last CTA's entry as an empty state
                const float4 q = S.slot[rp][lane < static_cast<int>(cl) ? lane : 0];
                st = lane < static_cast<int>(cl) ? LpState{q.x, q.y, q.z} : lp_empty();
                st = lp_warp_merge<ENT>(st, k);
                xy = S.slot[rp][t / part].w;
            }
            float4 stats = lp_row_stats(st, xy, k);
            const LpRow r = lp_row(stats, k, a.inv_t);
            if (!POLICY) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&S.taken[rp]));
                if (writer) {
                    const bool gone = *abort != 0;  // a wait gave up: no workspace to flag it in
                    if (a.logp) a.logp[row] = gone ? NAN : r.logp;
                    if (ENT && a.entropy) a.entropy[row] = gone ? NAN : r.entropy;
                    if (!ENT || gone) stats.w = NAN;
                    if (gone) stats.x = NAN;
                    if (a.stats) a.stats[row] = stats;
                }
                continue;
            }
            const PolicyOut o = policy_row(a, in, r, r.entropy);
            if (!have_norm) {
                pdl_wait();
                w_sum = policy_weight_sum(a);
                have_norm = true;
            }
            const float scale = policy_scale(a, row, w_sum);
            if (lane == 0) {
                S.grad[rp] = lp_grad(stats, r, a.inv_t, o.g * scale, o.h * scale);
                mbar_arrive(smem_u32(&S.taken[rp]));
            }
            if (writer) {
                if (a.reduction == CE_RED_NONE) a.loss[row] = o.loss;
                else cta_sum += static_cast<double>(o.loss);
                if (a.row_stats) a.row_stats[row] = make_float4(r.logp, ENT ? r.entropy : 0.f, o.ratio, o.kl);
            }
        }
    } else {
        // -------------------------------------------------------------- consumers
        const float k = a.k;
        // the row's target column in this slice (it may lie outside), read a row ahead
        const auto target_column = [&](int i) { return static_cast<int>(load_target(a.target, a.tgt32, live_row(i))) - lo; };
        int yc_next = n_live > 0 ? target_column(0) : 0;
        constexpr int lag = LAG ? 1 : 0;
        uint32_t held = 0, keep_slot = 0;           // the second pass's: chunks that need held exponents, its first kept slot
        uint32_t held_before = 0, keep_before = 0;  // and those of the row before
        int yc = 0, yc_before = 0;
        for (int li = 0; li < n_live + lag; ++li) {
            if (!LAG || li < n_live) {
            yc = yc_next;
            if (li + 1 < n_live) yc_next = target_column(li + 1);
            const char *xrow = xbase + live_row(li) * xstep;
            const LpGeom gm = lp_geom<KB>(xrow, L);
            const int nvec = gm.nvec, nch = gm.nch, vlo = gm.head, tail0 = gm.tail0, nedge = vlo + L - tail0;
            const int y = yc >= vlo && yc < tail0 ? yc - vlo : -1;
            // the chunk with the target's column, for the warp that reads its vector
            const int y_thread = y >= 0 ? (y / VEC) % NCT : -32;
            const int y_chunk = y_thread / 32 == warp ? y / VEC / VPC : -1;
            const int nkeep = POLICY ? min(nch, kLpSlots) : 0;
            const uint32_t rp = j & 1u;
            // (the policy loss's wait for its gradient scalars has covered this)
            if (!POLICY && j > 1)
                mbar_wait_bounded<false, kStreamSleepConsumer>(smem_u32(&S.taken[rp]), ((j >> 1) - 1u) & 1u, abort);
            // ------------------------------------------------ pass 1: statistics
            LpState st = lp_empty();
            held = 0;
            for (int c = 0; c < nch; ++c) {
                if (c == nch - nkeep) keep_slot = pos.slot;
                mbar_wait_bounded<false, kStreamSleepConsumer>(smem_u32(&S.full[pos.slot]), pos.phase, abort);
                const uint32_t base_s = ring + pos.slot * kStreamChunk, mine = base_s + 16u * tid;
                const int nv = min(VPC, nvec - c * VPC);
                const bool y_warp = c == y_chunk, own = y_warp && y_thread == tid;
                if (own) {
                    // the target's column leaves the chunk: this thread alone reads its vector
                    S.xy[rp] = take_out<DT>(base_s + static_cast<uint32_t>(y - c * VPC * VEC) * KB);
                    fence_async_shared();  // before a copy may overwrite the slot
                }
                bool plain = true;
                if (nv == VPC) {
                    uint4 raw[VPT];
#pragma unroll
                    for (int i = 0; i < VPT; ++i) raw[i] = ld_shared_v4(mine + 16u * i * NCT);
                    plain = add_any<DT, ENT, VPT, true>(st, raw, VPT, k, y_warp, own);
                } else {
                    // the row's last chunk, as many vectors as reach this thread, all at once (8192 x
                    // 16000 bf16, whose last chunk is 95% full, policy with entropy: 140 us against
                    // 166 with its vectors in pairs, one pair after the other)
                    const int n = tid < nv ? (nv - 1 - tid) / NCT + 1 : 0;
                    if (n > 0) {
                        uint4 raw[VPT];
#pragma unroll
                        for (int i = 0; i < VPT; ++i) {
                            constexpr uint32_t none = F::kNegInfWord;
                            raw[i] = i < n ? ld_shared_v4(mine + 16u * i * NCT) : make_uint4(none, none, none, none);
                        }
                        plain = add_any<DT, ENT, VPT, false>(st, raw, n, k, y_warp, own);
                    }
                }
                if (POLICY && ENT && !plain) held |= 1u << min(c, 31);  // 31: any later one
                __syncwarp();
                if (lane == 0 && c < nch - nkeep) mbar_arrive(smem_u32(&S.empty[pos.slot]));
                pos.next();
            }
            // columns before the first and after the last 16-byte boundary
            const int edge_c = tid < vlo ? tid : tail0 + (tid - vlo);
            if (tid < nedge) {
                const float x = F::load1(xrow, edge_c);
                if (edge_c == yc) S.xy[rp] = x;
                else lp_add1<ENT>(st, x, k);
            }
            // ------------------------------------------------ to the scalar warp
            parts[rp * NCT + tid] = make_float4(st.m, st.s, st.u, 0.f);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.done[rp]));
            ++j;
            }
            if (!POLICY) continue;
            if (LAG) {  // on to the row before
                swap_values(yc, yc_before);
                swap_values(held, held_before);
                swap_values(keep_slot, keep_before);
                if (li == 0) continue;
            }
            const int64_t row = live_row(li - lag);
            const char *xrow = xbase + row * xstep;
            const LpGeom gm = lp_geom<KB>(xrow, L);
            const int nvec = gm.nvec, nch = gm.nch, vlo = gm.head, tail0 = gm.tail0;
            const int y = yc >= vlo && yc < tail0 ? yc - vlo : -1;
            const int nkeep = min(nch, kLpSlots);
            const uint32_t at = LAG ? j2++ : j - 1u, rp = at & 1u;
            mbar_wait_bounded<false, kStreamSleepConsumer>(smem_u32(&S.taken[rp]), (at >> 1) & 1u, abort);
            const LpGrad g = S.grad[rp];
            // ------------------------------------------------ pass 2: gradient
            char *grow = gbase + row * gstep;
            char *const gv = grow + static_cast<int64_t>(vlo) * KB;
            uint4 *vp = reinterpret_cast<uint4 *>(gv);
            // gradient rows at another offset from a 16-byte boundary than the logits'
            const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(gv)) & 15u;
            const float fold = fmaf(-g.M, k, g.neg_log2d);
            const float cexp = KB == 2 ? fold : g.neg_log2d;
            // the whole row takes the slow form where the folded constant is too large, on
            // fp32 rows where M might carry the exponent out of range, and where B times
            // an exponent of down to -3.4e38 (a far finite mask) would be -inf, 0 * inf
            if (!(fabsf(KB == 2 ? fold : g.M * k) < (KB == 2 ? kFoldC : 1e20f))) held = ~0u;
            if (ENT && !(fabsf(g.B) < 1.f)) held = ~0u;
            auto pass2 = [&](auto ent_tag) {
                constexpr bool E = decltype(ent_tag)::value;
                for (int i = 0; i < nch; ++i) {
                    // the kept chunks, from the slots the first pass filled, then the earlier ones
                    const bool in_ring = i < nkeep;
                    const int c = in_ring ? nch - nkeep + i : nch - 1 - i;
                    const uint32_t s = in_ring ? keep_slot : pos.slot;
                    if (in_ring) {
                        if (++keep_slot == kLpSlots) keep_slot = 0;
                    } else {
                        mbar_wait_bounded<false, kStreamSleepConsumer>(smem_u32(&S.full[s]), pos.phase, abort);
                        pos.next();
                    }
                    const uint32_t base_s = ring + s * kStreamChunk;
                    const int v0 = c * VPC, nv = min(VPC, nvec - v0);
                    if (mis != 0) {
                        // vector o of the gradient is the last mis bytes of the logits' vector o and
                        // the first 16 - mis of o + 1 (past the chunk's end read from L2)
#pragma unroll 2
                        for (int v = tid; v < nv && v0 + v + 1 < nvec; v += NCT) {
                            const uint4 r0 = ld_shared_v4(base_s + 16u * v);
                            const uint4 r1 = v + 1 < nv ? ld_shared_v4(base_s + 16u * (v + 1))
                                                        : ld_stream(xrow + vlo * KB + 16 * static_cast<int64_t>(v0 + v + 1));
                            float x[VEC], og[VEC];
                            F::unpack(shift16<KB>(r0, r1, 16u - mis), x);
                            grad_vec<DT, E, true>(g, cexp, x, k, og);
                            st_stream(gv + 16 * static_cast<int64_t>(v0 + v) + (16u - mis), F::pack(og));
                        }
                    } else if (!((held >> min(c, 31)) & 1u)) {
                        uint4 *const out = vp + v0 + tid;
                        if (nv == VPC) {
#pragma unroll
                            for (int i = 0; i < VPT; ++i) {
                                float x[VEC], og[VEC];
                                F::unpack(ld_shared_v4(base_s + 16u * tid + 16u * i * NCT), x);
                                grad_vec<DT, E, false>(g, cexp, x, k, og);
                                st_stream(out + i * NCT, F::pack(og));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < VPT; ++i) {
                                if (tid + i * NCT >= nv) continue;
                                float x[VEC], og[VEC];
                                F::unpack(ld_shared_v4(base_s + 16u * tid + 16u * i * NCT), x);
                                grad_vec<DT, E, false>(g, cexp, x, k, og);
                                st_stream(out + i * NCT, F::pack(og));
                            }
                        }
                    } else {
#pragma unroll 1
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
            // The target column of the vectors, by the thread that stored its vector,
            // after that store; the columns outside of them. Shifted vectors leave the
            // first 16 - mis bytes of the interior and its last mis out as well.
            const int lead = mis != 0 && nvec > 0 ? static_cast<int>(16u - mis) / KB : 0;
            const int trail = mis != 0 && nvec > 0 ? static_cast<int>(mis) / KB : 0;
            const int yo = y - lead;
            if (y >= 0 && yo >= 0 && y < nvec * VEC - trail && (yo / VEC) % NCT == tid) F::store1(grow, vlo + y, g.dy);
            const int nh = vlo + lead, ne = nh + trail + L - tail0;
            if (tid < ne) {
                const int c = tid < nh ? tid : tail0 - trail + (tid - nh);
                F::store1(grow, c, c == yc ? g.dy : lp_grad_elem<ENT>(g, F::load1(xrow, c), k));
            }
            // one of the rows that take no part, between two that do
            if (li - lag < n_dead) zero_row(dead_row(li - lag));
        }
        if (POLICY)
            for (int di = n_live; di < n_dead; ++di) zero_row(dead_row(di));
    }
    if (!single && w0 + window < a.n_rows) __syncthreads();  // the lists are rebuilt
    }
    if (warp == kLpWarps && lane == 0) {
        // drain: every issued copy has landed before the CTA may exit (waited for
        // with a limit of its own where another wait gave up)
        for (uint32_t i = 0; i < kLpSlots && i < issued; ++i) {
            // the last copy of each used slot, latest first
            if (pos.slot == 0) {
                pos.slot = kLpSlots;
                pos.phase ^= 1u;
            }
            --pos.slot;
            mbar_wait_bounded<false, kStreamSleepP>(smem_u32(&S.full[pos.slot]), pos.phase, &S.drain_abort);
        }
    }
    // ---------------------------------------------------- batch loss (last cluster)
    if (POLICY && warp == kLpWarps + 1 && a.reduction != CE_RED_NONE && rank == 0) {
        if (!have_norm) pdl_wait();
        unsigned last = 0;
        if (lane == 0) {
            a.part[q0] = cta_sum;
            __threadfence();
            last = atomicAdd(&a.ctl->done, 1u) == static_cast<unsigned>(nq) - 1u ? 1u : 0u;
        }
        if (__shfl_sync(0xffffffffu, last, 0)) {
            __threadfence();
            double sum = 0.0;  // in cluster order, then a fixed tree
            for (int64_t i = lane; i < nq; i += 32) sum += __ldcg(a.part + i);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (a.reduction == CE_RED_MEAN) {
                const float w_all = policy_weight_sum(a);
                sum = w_all != 0.f ? sum / static_cast<double>(w_all) : 0.0;
            }
            if (lane == 0) a.loss[0] = static_cast<float>(sum);
        }
    }
    if (POLICY && blockIdx.x == 0 && tid == 0) {
        pdl_wait();
        policy_flags(a);
    }
    __syncthreads();
    if (tid == 0 && S.abort && a.ctl) {
        if (POLICY) pdl_wait();
        atomicOr(&a.ctl->status, CE_FLAG_WAIT_TIMEOUT);
    }
    if (cl > 1) cluster_sync_all();  // no CTA leaves while a peer may still write into it
}

template <int DT>
static const void *rows_fn(int mode, bool ent, bool lag) {
    if (mode == LP_FWD)
        return ent ? reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_FWD, true, false>)
                   : reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_FWD, false, false>);
    if (lag)
        return ent ? reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_POLICY, true, true>)
                   : reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_POLICY, false, true>);
    return ent ? reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_POLICY, true, false>)
               : reinterpret_cast<const void *>(&lp_rows_kernel<DT, LP_POLICY, false, false>);
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
    const int64_t row_bytes = a.vocab * (dtype == CE_DT_F32 ? 4 : 2);
    const bool lag = mode == LP_POLICY && row_bytes <= kLpLagChunks * kStreamChunk;
    const void *fn = dtype == CE_DT_F32 ? rows_fn<CE_DT_F32>(mode, entropy, lag)
                   : dtype == CE_DT_BF16 ? rows_fn<CE_DT_BF16>(mode, entropy, lag) : rows_fn<CE_DT_F16>(mode, entropy, lag);
    int clusters = 0, sms = 0;
    cudaError_t e = rows_ready(fn, 1, &clusters, &sms);
    if (e != cudaSuccess) return e;
    // Rows of up to 16 KB: a group of warps a row (GB300, 8192 rows with the
    // entropy, forward / policy: 2 KB rows 17 / 39 us against 39 / 91 here, 8 KB
    // 27 / 58 against 46 / 108, 16 KB 48 / 95 against 57 / 137; at 32 KB, with
    // groups of eight warps, 80 / 192 against 66 / 120).
    if (lp_short_takes(a.vocab, dtype)) return launch_lp_short(a, dtype, mode, entropy, after_prep, sms, s);
    const int64_t slots = static_cast<int64_t>(sms) * kLpCtasPerSm;
    int cl = 1;
    // Two passes over many rows: the rows in flight, whose first chunks wait in
    // L2 for the second pass, kept to 60 MB (GB300, L2 flushed, with the
    // entropy, 30% of the first's rows left out: 8192 x 128256 bf16 one CTA a
    // row 709 us, pairs 686, quads 781; 4096 x 256000 891, 769, 773; 2048 x
    // 128256 fp32 438, 389, 354; below the limit 8192 x 64000 364, 467, 647 and
    // 8192 x 32000 220, 324, 481).
    if (mode == LP_POLICY && a.n_rows > slots)
        while (cl < kLpMaxCluster && slots / cl * row_bytes > (int64_t(60) << 20)) cl *= 2;
    // Few rows: split over more CTAs while all rows still run at once, down to
    // one chunk each (8 x 128256 bf16, with the gradient: one CTA a row 25.6 us,
    // 2 19.5, 4 15.4, 8 15.0; 64 x 32000 fp16 the same for 1 to 4, 8 slower).
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
