// verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers. Per sequence b and position i with
// p = softmax(z / T), q = softmax(y / T) (or 1 at the draft t without a draft model):
//
//   draft i stays while u_i q_i(t) < p_i(t); n = the drafts that stay before the first that does not
//   token n: the lowest v with  sum_{c <= v} w_c > r sum_c w_c,
//            w = max(p_n - q_n, 0) where position n has a draft, p_n otherwise (and where that sum is 0)
//   T = 0: draft i stays where it is the lowest index of the row's maximum, which is also token n
//
// Two kernels. The first forms, for parts of every row, M = max x, its lowest index,
// and the sum of the other terms 2^((x - M) k), k = log2(e) / T. The second (a
// cluster of CTAs per sequence) merges them in a fixed order, decides, and reads
// row n once more to draw the token: every warp sums w over a contiguous range,
// the ranges' sums (fp64) meet in the cluster, and the CTA whose range holds
// r sum w walks it. Exponents are formed by the difference x - M first, so that
// equal logits have equal probabilities whatever part they lie in.
// Bound by HBM: rows of both models once, and one row of each again from L2.
#include "ce_device.cuh"
#include "ce_kernels.h"
#include "fp8.h"

namespace ce {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxDrafts = 255;
constexpr int kNone = 0x7fffffff;

struct VfPart {
    float m, s;
    int at;      // lowest index of the maximum
    float pad;
};

struct VfArgs {
    const void *x, *y;               // target logits [B][K + 1][V], draft logits [B][K][V] or NULL
    int64_t xs, xr, ys, yr;          // strides of a sequence and of a row, elements
    int B, K, V;
    const void *draft;
    int tok32;
    const float *u, *r;              // [B][K], [B]
    const float *temps;              // [B] or NULL
    float temp;
    int parts, part_len;
    VfPart *px, *py;                 // [B][K + 1][parts], [B][K][parts]
    int *accepted;
    void *tokens;                    // [B][K + 1]
    float *logp;
};

__device__ inline int64_t vf_draft(const VfArgs &a, int b, int i) {
    return load_target(a.draft, a.tok32, static_cast<int64_t>(b) * a.K + i);
}
__device__ inline bool vf_valid(const VfArgs &a, int64_t t) { return t >= 0 && t < a.V; }
__device__ inline float vf_temp(const VfArgs &a, int b) { return a.temps ? __ldg(a.temps + b) : a.temp; }
__device__ inline bool vf_temp_ok(float t) { return t == 0.f || (t >= 1e-4f && t <= 1e4f); }
// log2(e) / T; greedy sequences report log-probabilities at T = 1
__device__ inline float vf_k(float t) { return t == 0.f ? kLog2e : kLog2e / t; }

// Statistics of a set of logits: the maximum m, its lowest index, and the sum s of
// the other terms 2^((x - m) k). The maximum's own term is exactly 1 and kept
// out of the sum, so that the log-probability -log1p(s) of a likely token forms
// without cancellation. Empty (or -inf alone): m = -inf, s = 0; NaN stays in s.
struct VfState {
    float m, s;
    int at;
};
// what a set with maximum m and sum s adds to the others of a set whose maximum M >= m is another element
__device__ inline float vf_shift(float m, float s, float M, float k) {
    return m == -INFINITY ? s : (1.f + s) * ex2_hw((m - M) * k);
}
__device__ inline VfState vf_merge(const VfState &a, const VfState &b, float k) {
    const bool first = a.m > b.m || (a.m == b.m && a.at <= b.at);
    const VfState &hi = first ? a : b, &lo = first ? b : a;
    return VfState{hi.m, hi.s + vf_shift(lo.m, lo.s, hi.m, k), hi.at};
}

// Statistics of elements [lo, hi) of one row by the whole CTA; the result in thread 0.
template <int DT>
__device__ inline VfState vf_row_part(const void *row, int lo, int hi, float k, VfState *red) {
    constexpr int N = Fmt<DT>::kVec;
    const char *p = reinterpret_cast<const char *>(row) + static_cast<int64_t>(lo) * Fmt<DT>::kBytes;
    int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / Fmt<DT>::kBytes;
    if (head > hi - lo) head = hi - lo;
    const int vecs = (hi - lo - head) / N, tail = lo + head + vecs * N;
    const uint4 *v4 = reinterpret_cast<const uint4 *>(p + head * Fmt<DT>::kBytes);
    VfState st{-INFINITY, 0.f, kNone};
    const auto one = [&](int i) {
        const float x = Fmt<DT>::load1(row, i);
        if (x > st.m) st = VfState{x, x == INFINITY ? NAN : vf_shift(st.m, st.s, x, k), i};
        else st.s += st.m == -INFINITY ? (x != x ? x : 0.f) : ex2_hw((x - st.m) * k);
    };
    const int t = threadIdx.x;
    if (t < head) one(lo + t);
    constexpr int U = 4;
    for (int i = t; i < vecs; i += U * kThreads) {
        uint4 raw[U];
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (i + q * kThreads < vecs) raw[q] = ld_stream_ro(v4 + i + q * kThreads);
#pragma unroll
        for (int q = 0; q < U; ++q) {
            if (i + q * kThreads < vecs) {
                float x[N];
                Fmt<DT>::unpack(raw[q], x);
                const float vmax = Fmt<DT>::vmax(raw[q]);
                if (vmax > st.m) {
                    // the vector's first maximum leaves the sum, what was there joins it
                    float sum = vmax == INFINITY ? NAN : vf_shift(st.m, st.s, vmax, k);
                    int at = -1;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        if (at < 0 && x[j] == vmax) at = j;
                        else sum += ex2_hw((x[j] - vmax) * k);
                    }
                    st = VfState{vmax, sum, lo + head + (i + q * kThreads) * N + at};
                } else {
                    const float m = st.m == -INFINITY ? 0.f : st.m;
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < N; ++j) s += ex2_hw((x[j] - m) * k);
                    st.s += s;
                }
            }
        }
    }
    if (t < hi - tail) one(tail + t);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        VfState o;
        o.m = __shfl_xor_sync(0xffffffffu, st.m, off);
        o.s = __shfl_xor_sync(0xffffffffu, st.s, off);
        o.at = __shfl_xor_sync(0xffffffffu, st.at, off);
        st = vf_merge(st, o, k);
    }
    if ((t & 31) == 0) red[t >> 5] = st;
    __syncthreads();
    if (t == 0)
        for (int w = 1; w < kWarps; ++w) st = vf_merge(st, red[w], k);
    __syncthreads();
    return st;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) vf_stats_kernel(VfArgs a) {
    __shared__ VfState red[kWarps];
    pdl_launch_dependents();
    // position by position, so that a batch's first rows come first
    const int part = blockIdx.x % a.parts, rest = blockIdx.x / a.parts, b = rest % a.B, i = rest / a.B;
    const float temp = vf_temp(a, b), k = vf_k(temp);
    if (!vf_temp_ok(temp)) return;
    // a missing draft ends the sequence: rows behind it are not read
    bool ended = false;
    for (int j = threadIdx.x; j < i; j += kThreads) ended |= !vf_valid(a, vf_draft(a, b, j));
    if (__syncthreads_or(ended)) return;
    const int lo = part * a.part_len, hi = min(a.V, lo + a.part_len);
    const char *x = reinterpret_cast<const char *>(a.x) + (b * a.xs + i * a.xr) * Fmt<DT>::kBytes;
    const VfState sx = vf_row_part<DT>(x, lo, hi, k, red);
    if (threadIdx.x == 0)
        a.px[(static_cast<int64_t>(b) * (a.K + 1) + i) * a.parts + part] = VfPart{sx.m, sx.s, sx.at, 0.f};
    if (a.y && i < a.K && temp != 0.f && vf_valid(a, vf_draft(a, b, i))) {
        const char *y = reinterpret_cast<const char *>(a.y) + (b * a.ys + i * a.yr) * Fmt<DT>::kBytes;
        const VfState sy = vf_row_part<DT>(y, lo, hi, k, red);
        if (threadIdx.x == 0)
            a.py[(static_cast<int64_t>(b) * a.K + i) * a.parts + part] = VfPart{sy.m, sy.s, sy.at, 0.f};
    }
}

// a row's statistics from its parts, by one warp, the same in every lane
__device__ inline VfState vf_row(const VfPart *p, int parts, float k) {
    const int lane = threadIdx.x & 31;
    VfState st{-INFINITY, 0.f, kNone};
    for (int j = lane; j < parts; j += 32) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + j));
        st = vf_merge(st, VfState{v.x, v.y, __float_as_int(v.z)}, k);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        VfState o;
        o.m = __shfl_xor_sync(0xffffffffu, st.m, off);
        o.s = __shfl_xor_sync(0xffffffffu, st.s, off);
        o.at = __shfl_xor_sync(0xffffffffu, st.at, off);
        st = vf_merge(st, o, k);
    }
    return st;
}
__device__ inline bool vf_defined(const VfState &s) { return s.s < INFINITY && fabsf(s.m) < INFINITY; }
__device__ inline float vf_total(const VfState &s) { return 1.f + s.s; }

// Sums over a vocabulary as pairs of fp32 (value hi + lo, |lo| at most half a
// unit of hi; each addition exact to about 2^-46): fp64 additions run at 1/64 of
// the fp32 rate and less here.
struct alignas(8) FF {
    float hi, lo;
};
__device__ inline FF ff_add(FF a, FF b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float hi = s + e;
    return FF{hi, e - (hi - s)};
}
__device__ inline FF ff_scale(FF a, float r) {
    const float p = r * a.hi, e = fmaf(r, a.lo, fmaf(r, a.hi, -p)), hi = p + e;
    return FF{hi, e - (hi - p)};
}
__device__ inline bool ff_above(FF a, FF b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ inline FF ff_shfl_xor(FF a, int off) {
    return FF{__shfl_xor_sync(0xffffffffu, a.hi, off), __shfl_xor_sync(0xffffffffu, a.lo, off)};
}
__device__ inline FF ff_shfl_up(FF a, int off) {
    return FF{__shfl_up_sync(0xffffffffu, a.hi, off), __shfl_up_sync(0xffffffffu, a.lo, off)};
}
__device__ inline FF ff_shfl(FF a, int lane) {
    return FF{__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
// sums over the lanes up to and with this one
__device__ inline FF ff_scan(FF a) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const FF o = ff_shfl_up(a, off);
        if ((threadIdx.x & 31) >= off) a = ff_add(o, a);
    }
    return a;
}
__device__ inline void st_cluster_ff(uint32_t addr, FF v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.hi), "f"(v.lo) : "memory");
}

// What row n's token is drawn from.
template <int DT>
struct VfWeights {
    const void *x, *y;    // y: NULL without a draft model at this position
    float mx, ix, my, iy; // maxima and 1 / sums
    float k;
    int drop;             // the draft without a draft model, or -1
    // eight weights from element c on (zeros from `end` on)
    __device__ inline void get(int c, int end, float (&w)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = 0.f;
            if (c + j < end) {
                v = ex2_hw((Fmt<DT>::load1(x, c + j) - mx) * k) * ix;
                if (y) v = fmaxf(v - ex2_hw((Fmt<DT>::load1(y, c + j) - my) * k) * iy, 0.f);
                if (c + j == drop) v = 0.f;
            }
            w[j] = v;
        }
    }
};

template <int DT>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) vf_pick_kernel(VfArgs a) {
    __shared__ VfState sx[kMaxDrafts + 1], sy[kMaxDrafts];
    __shared__ FF ranges[2][kCluster * kWarps];
    __shared__ FF scan[kWarps], from, goal;
    __shared__ float mass;
    __shared__ int count, bad, pick, last, own;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank()), b = blockIdx.x / kCluster;
    const float temp = vf_temp(a, b), k = vf_k(temp);
    const bool greedy = temp == 0.f;
    if (tid == 0) {
        count = a.K;
        bad = vf_temp_ok(temp) ? 0 : 1;
        last = -1;
        pick = kNone;
    }
    __syncthreads();
    cluster_sync_all();  // every CTA of the cluster runs before one writes into another
    pdl_wait();
    const bool usable = !bad;
    // every row's statistics and whether its draft stays
    for (int i = warp; i <= a.K && usable; i += kWarps) {
        bool ended = false;
        for (int j = lane; j < i; j += 32) ended |= !vf_valid(a, vf_draft(a, b, j));
        if (__any_sync(0xffffffffu, ended)) break;
        const VfState p = vf_row(a.px + (static_cast<int64_t>(b) * (a.K + 1) + i) * a.parts, a.parts, k);
        const int64_t t = i < a.K ? vf_draft(a, b, i) : -1;
        const bool has = vf_valid(a, t);
        VfState q{0.f, 0.f, 0};
        const bool model = a.y && has && !greedy;
        if (model) q = vf_row(a.py + (static_cast<int64_t>(b) * a.K + i) * a.parts, a.parts, k);
        if (lane == 0) {
            sx[i] = p;
            if (i < a.K) sy[i] = q;
            bool stays = has && vf_defined(p) && vf_defined(q);
            if (stays && greedy) stays = p.at == static_cast<int>(t);
            if (stays && !greedy) {
                const float pt = ex2_hw((Fmt<DT>::load1(a.x, b * a.xs + i * a.xr + t) - p.m) * k);
                const float qt = model ? ex2_hw((Fmt<DT>::load1(a.y, b * a.ys + i * a.yr + t) - q.m) * k) : 1.f;
                stays = __ldg(a.u + static_cast<int64_t>(b) * a.K + i) * qt * vf_total(p) < pt * vf_total(q);
            }
            if (!stays && i < a.K) atomicMin(&count, i);
        }
    }
    __syncthreads();
    const int n = usable ? count : 0;
    const int64_t tn = n < a.K ? vf_draft(a, b, n) : -1;
    const bool turned = usable && vf_valid(a, tn), model = turned && a.y && !greedy;
    const VfState p = usable ? sx[n] : VfState{0.f, 0.f, 0};
    const VfState q = model ? sy[n] : VfState{0.f, 0.f, 0};
    const bool defined = usable && vf_defined(p) && vf_defined(q);
    const int64_t row = static_cast<int64_t>(b) * (a.K + 1);
    const float ln2_k = k * 0.6931471805599453f;  // 1 / T
    // accepted tokens, and what lies behind the last one
    if (rank == 0) {
        if (tid == 0) a.accepted[b] = n;
        for (int i = tid; i <= a.K; i += kThreads) {
            if (i == n) continue;
            int64_t t = -1;
            float lp = 0.f;
            if (i < n) {
                t = vf_draft(a, b, i);
                lp = (Fmt<DT>::load1(a.x, b * a.xs + i * a.xr + t) - sx[i].m) * ln2_k - log1pf(sx[i].s);
            }
            if (a.tok32) reinterpret_cast<int32_t *>(a.tokens)[row + i] = static_cast<int32_t>(t);
            else reinterpret_cast<int64_t *>(a.tokens)[row + i] = t;
            a.logp[row + i] = lp;
        }
    }
    const int64_t xrow = b * a.xs + n * a.xr;
    const auto emit = [&](int t) {
        const float lp = t < 0 ? NAN : (Fmt<DT>::load1(a.x, xrow + t) - p.m) * ln2_k - log1pf(p.s);
        if (a.tok32) reinterpret_cast<int32_t *>(a.tokens)[row + n] = t;
        else reinterpret_cast<int64_t *>(a.tokens)[row + n] = t;
        a.logp[row + n] = lp;
    };
    if (!defined || greedy) {  // the same in every CTA of the cluster
        if (rank == 0 && tid == 0) emit(defined ? p.at : -1);
        return;
    }
    VfWeights<DT> w;
    w.x = reinterpret_cast<const char *>(a.x) + xrow * Fmt<DT>::kBytes;
    w.y = model ? reinterpret_cast<const char *>(a.y) + (b * a.ys + n * a.yr) * Fmt<DT>::kBytes : nullptr;
    w.mx = p.m; w.ix = 1.f / vf_total(p); w.my = q.m; w.iy = 1.f / vf_total(q); w.k = k;
    w.drop = turned && !a.y ? static_cast<int>(tn) : -1;
    // contiguous ranges of the row, one a warp of the cluster, in steps of 256 elements
    const int steps = (a.V + 255) / 256, all = kCluster * kWarps;
    for (int pass = 0;; ++pass) {
        const int g = rank * kWarps + warp;
        const int s0 = static_cast<int>(static_cast<int64_t>(steps) * g / all);
        const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (g + 1) / all);
        FF sum{0.f, 0.f};
        for (int st = s0; st < s1; ++st) {
            float v[8], t = 0.f;
            w.get(st * 256 + lane * 8, a.V, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) t += v[j];
            sum = ff_add(sum, FF{t, 0.f});
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum = ff_add(sum, ff_shfl_xor(sum, off));
        if (lane < kCluster) st_cluster_ff(mapa_shared(smem_u32(&ranges[pass][g]), lane), sum);
        cluster_sync_all();
        // Every CTA finds the same range: the first whose end lies above the aim;
        // rounding may leave none, then the last that holds anything.
        if (warp == 0) {
            static_assert(kCluster * kWarps == 64, "two ranges a lane");
            const FF v0 = ranges[pass][2 * lane], v1 = ranges[pass][2 * lane + 1];
            const FF incl = ff_scan(ff_add(v0, v1));
            FF before = ff_shfl_up(incl, 1);
            if (lane == 0) before = FF{0.f, 0.f};
            const FF sum_all = ff_shfl(incl, 31), aim = ff_scale(sum_all, __ldg(a.r + b));
            const FF mid = ff_add(before, v0);
            const int hit = ff_above(mid, aim) ? 2 * lane : (ff_above(incl, aim) ? 2 * lane + 1 : -1);
            const int full = v1.hi > 0.f ? 2 * lane + 1 : (v0.hi > 0.f ? 2 * lane : -1);
            const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), fulls = __ballot_sync(0xffffffffu, full >= 0);
            const int src = hits ? __ffs(hits) - 1 : (fulls ? 31 - __clz(fulls) : 0);
            const int found = hits ? hit : full;
            if (lane == src) {
                own = found;
                from = (found & 1) ? mid : before;
                goal = aim;
                mass = sum_all.hi;
            }
        }
        __syncthreads();
        // p <= q everywhere (p = q): drawn from p
        if (mass > 0.f || pass == 1) break;
        w.y = nullptr;
        w.drop = -1;
    }
    const int range = own;
    if (range < 0) {  // nothing to draw from
        if (rank == 0 && tid == 0) emit(-1);
        return;
    }
    if (range / kWarps != rank) return;
    // the CTA walks its warp's range, 2048 elements at a time
    const FF aim = goal;
    FF below = from;
    const int e0 = static_cast<int>(static_cast<int64_t>(steps) * range / all) * 256;
    const int64_t end = static_cast<int64_t>(steps) * (range + 1) / all * 256;
    const int e1 = end < a.V ? static_cast<int>(end) : a.V;
    for (int c0 = e0; c0 < e1; c0 += kThreads * 8) {
        float v[8], t = 0.f;
        const int c = c0 + tid * 8;
        w.get(c, e1, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) t += v[j];
        const FF incl = ff_scan(FF{t, 0.f});
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        FF start = below;
        for (int j = 0; j < warp; ++j) start = ff_add(start, scan[j]);
        FF before = ff_shfl_up(incl, 1);
        before = lane == 0 ? start : ff_add(start, before);
        int found = -1, lastpos = -1;
        float run = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            run += v[j];
            if (v[j] > 0.f) {
                lastpos = c + j;
                if (found < 0 && ff_above(ff_add(before, FF{run, 0.f}), aim)) found = c + j;
            }
        }
        if (found >= 0) atomicMin(&pick, found);
        if (lastpos >= 0) atomicMax(&last, lastpos);
        for (int j = 0; j < kWarps; ++j) below = ff_add(below, scan[j]);
        __syncthreads();
        if (pick != kNone) break;  // written before the barrier above, read after it
    }
    if (tid == 0) emit(pick != kNone ? pick : last);
}

}  // namespace

static int vf_part_len(int64_t rows, int64_t vocab, int dtype) {
    // parts of at most 64 KB, more of them while the rows do not fill the GPU, none under 2048 elements
    const int64_t most = 65536 / fp8_elem(dtype);
    int64_t parts = (vocab + most - 1) / most;
    const int64_t want = rows > 0 ? (1216 + rows - 1) / rows : 1, fit = (vocab + 2047) / 2048;
    if (parts < want) parts = want;
    if (parts > fit) parts = fit;
    const int64_t len = (vocab + parts - 1) / parts;
    return static_cast<int>((len + 7) / 8 * 8);
}

static int64_t vf_parts(int64_t rows, int64_t vocab, int dtype) {
    const int64_t len = vf_part_len(rows, vocab, dtype);
    return (vocab + len - 1) / len;
}

}  // namespace ce

using namespace ce;

namespace {

ce_status vf_check(const ce_verify_params *p) {
    if (!p || p->n_seqs < 0 || p->n_drafts < 0 || p->vocab < 1 || p->reserved != 0) return CE_ERR_INVALID_ARG;
    if (!fp8_dtype_ok(p->dtype)) return CE_ERR_INVALID_ARG;
    if (p->token_is_int32 != 0 && p->token_is_int32 != 1) return CE_ERR_INVALID_ARG;
    if (!(p->temperature == 0.f || (p->temperature >= 1e-4f && p->temperature <= 1e4f))) return CE_ERR_INVALID_ARG;
    if (p->ld < p->vocab || p->ld_draft < p->vocab || p->seq_stride < 0 || p->draft_seq_stride < 0) return CE_ERR_INVALID_ARG;
    constexpr int64_t kMost = (int64_t(1) << 31) - 4096;
    if (p->n_drafts > kMaxDrafts || p->vocab > kMost || p->n_seqs > kMost / kCluster ||
        p->n_seqs * (p->n_drafts + 1) > kMost / vf_parts(p->n_seqs * (p->n_drafts + 1), p->vocab, p->dtype))
        return CE_ERR_UNSUPPORTED;
    return CE_OK;
}

size_t vf_bytes(const ce_verify_params *p) {
    const int64_t rows = p->n_seqs * (p->n_drafts + 1);
    return static_cast<size_t>(vf_parts(rows, p->vocab, p->dtype) * (rows + p->n_seqs * p->n_drafts)) * sizeof(VfPart) + 256;
}

}  // namespace

extern "C" {

ce_status ce_verify_workspace_size(const ce_verify_params *p, size_t *bytes) {
    const ce_status st = vf_check(p);
    if (st != CE_OK) return st;
    if (!bytes) return CE_ERR_INVALID_ARG;
    *bytes = vf_bytes(p);
    return CE_OK;
}

ce_status ce_verify_drafts(const ce_verify_params *p, const void *logits, const void *draft_logits,
                           const void *draft_token, const float *accept_uniform, const float *sample_uniform,
                           const float *temperatures, int32_t *accepted, void *tokens, float *logp, void *ws,
                           size_t ws_size, void *stream) {
    ce_status st = vf_check(p);
    if (st != CE_OK) return st;
    if (p->n_seqs == 0) return CE_OK;
    if (!ws || !fp8_on(ws, 256) || ws_size < vf_bytes(p)) return CE_ERR_WORKSPACE;
    const int esz = fp8_elem(p->dtype), tsz = p->token_is_int32 ? 4 : 8;
    if (!logits || !sample_uniform || !accepted || !tokens || !logp) return CE_ERR_INVALID_ARG;
    if (p->n_drafts > 0 && (!draft_token || !accept_uniform)) return CE_ERR_INVALID_ARG;
    if (!fp8_on(logits, esz) || !fp8_on(draft_logits, esz) || !fp8_on(draft_token, tsz) || !fp8_on(tokens, tsz) ||
        !fp8_on(accept_uniform, 4) || !fp8_on(sample_uniform, 4) || !fp8_on(temperatures, 4) || !fp8_on(accepted, 4) || !fp8_on(logp, 4))
        return CE_ERR_INVALID_ARG;
    // every output apart from every other buffer
    const int64_t B = p->n_seqs, K = p->n_drafts;
    const struct { const void *at; int64_t bytes; } bufs[] = {
        {accepted, B * 4}, {tokens, B * (K + 1) * tsz}, {logp, B * (K + 1) * 4}, {ws, static_cast<int64_t>(vf_bytes(p))},
        {draft_token, B * K * tsz}, {accept_uniform, B * K * 4}, {sample_uniform, B * 4}, {temperatures, B * 4},
        {logits, ((B - 1) * p->seq_stride + K * p->ld + p->vocab) * esz},
        {draft_logits, ((B - 1) * p->draft_seq_stride + (K - 1) * p->ld_draft + p->vocab) * esz}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 10; ++j)
            if (bufs[j].at && bufs[j].bytes > 0 && !fp8_apart(bufs[i].at, bufs[i].bytes, bufs[j].at, bufs[j].bytes))
                return CE_ERR_INVALID_ARG;
    VfArgs a{};
    a.x = logits;
    a.y = p->n_drafts > 0 ? draft_logits : nullptr;
    a.xs = p->seq_stride; a.xr = p->ld; a.ys = p->draft_seq_stride; a.yr = p->ld_draft;
    a.B = static_cast<int>(p->n_seqs);
    a.K = static_cast<int>(p->n_drafts);
    a.V = static_cast<int>(p->vocab);
    a.draft = draft_token;
    a.tok32 = p->token_is_int32;
    a.u = accept_uniform;
    a.r = sample_uniform;
    a.temps = temperatures;
    a.temp = p->temperature;
    const int64_t rows = p->n_seqs * (p->n_drafts + 1);
    a.part_len = vf_part_len(rows, p->vocab, p->dtype);
    a.parts = static_cast<int>(vf_parts(rows, p->vocab, p->dtype));
    a.px = reinterpret_cast<VfPart *>(ws);
    a.py = a.px + rows * a.parts;
    a.accepted = accepted;
    a.tokens = tokens;
    a.logp = logp;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    using Fn = void (*)(VfArgs);
    static const Fn stats[3] = {vf_stats_kernel<CE_DT_F32>, vf_stats_kernel<CE_DT_BF16>, vf_stats_kernel<CE_DT_F16>};
    static const Fn picks[3] = {vf_pick_kernel<CE_DT_F32>, vf_pick_kernel<CE_DT_BF16>, vf_pick_kernel<CE_DT_F16>};
    void *args[] = {&a};
    cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void *>(stats[p->dtype]),
                                     dim3(static_cast<unsigned>(rows * a.parts)), dim3(kThreads), args, 0, s);
    if (e != cudaSuccess) return cuda_fail(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(picks[p->dtype]), args);
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

}  // extern "C"
