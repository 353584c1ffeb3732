// verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers. Per sequence b and position i with
// p = softmax(z / T), q = softmax(y / T) (or 1 at the draft t without a draft model):
//
//   draft i stays while u_i q_i(t) < p_i(t); n = the drafts that stay before the first that does not
//   token n: the lowest v with  sum_{c <= v} w_c > r sum_c w_c,
//            w = max(p_n - q_n, 0) where position n has a draft, p_n otherwise (and where that sum is 0)
//   T = 0: draft i stays where it is the lowest index of the row's maximum, which is also token n
//
// A row's statistics are M = max x, its lowest index, and the sum of the other terms
// 2^((x - M) k), k = log2(e) / T. Exponents are formed by the difference x - M first,
// so that equal logits have equal probabilities wherever in the row they lie.
//
// Long rows of many sequences: one kernel, a cluster of CTAs per sequence. Position by
// position the cluster reads the row of both models (a contiguous slice a CTA), its
// warps exchange statistics through distributed shared memory, every warp merges them
// in the same order and decides; of the rows behind the first draft that is turned
// down only the first copies of the next one are made, ahead of the decision. Few or
// short rows would leave the memory idle that way: there a first kernel forms the
// statistics of parts of all rows at once, and a second (a cluster a sequence) merges
// them and decides (vf_at_once). Either draws the token by reading row n once more,
// mostly from L2: every warp sums w over a contiguous range, the ranges' sums meet in
// the cluster, and the CTA whose range holds r sum w walks it.
//
// Bound by the chain of dependent steps: a launch, a row's reading, an exchange and
// the draw where sequences are few (1 of 3 drafts and 128256 bf16 logits with a draft
// model: 17 us), the longest sequence's positions where they are many (128 of 4
// drafts: 74 us, of which the rows that decide would take 24 at the copy rate).
// Tried for many sequences and slower (the latter): parts of all rows dealt out
// position by position, the CTA or warp that completes a row by a counter deciding
// whether the next ones are read: 108 and 224 us; its fences and atomics took longer
// than the reading. The ring's loop rolled up (a fifth of the stalls are waits for
// instructions): no change.
#include <atomic>

#include "ce_device.cuh"
#include "ce_kernels.h"
#include "fp8.h"

namespace ce {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;  // CTAs of a cluster at most
constexpr int kMaxDrafts = 255;
constexpr int kNone = 0x7fffffff;

struct alignas(16) VfPart {
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
    int parts;                       // of a row
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

// U vectors of 16 bytes a thread of a row: vector v0 and every `stride`-th after it,
// counted from the 16-byte boundary at or before the row's first element.
template <int DT, int U> struct VfTile {
    static constexpr int N = Fmt<DT>::kVec;
    uint4 raw[U];
    int first, step;  // index of the first vector's first element (negative before the row), elements between vectors

    // (the first `limit` of the U vectors)
    __device__ inline void load(const void *row, int V, int v0, int stride, int limit = U) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row);
        const int before = static_cast<int>(at & 15u) / Fmt<DT>::kBytes;
        const uint4 *base = reinterpret_cast<const uint4 *>(at & ~static_cast<uintptr_t>(15));
        first = v0 * N - before;
        step = stride * N;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = first + u * step;
            if (u < limit && c >= 0 && c + N <= V) {
                raw[u] = ld_stream_ro(base + v0 + u * stride);
            } else {
                float x[N];
#pragma unroll
                for (int j = 0; j < N; ++j) x[j] = u < limit && c + j >= 0 && c + j < V ? Fmt<DT>::load1(row, c + j) : -INFINITY;
                raw[u] = Fmt<DT>::pack(x);
            }
        }
    }
    // this lane's statistics
    __device__ inline VfState stats(float k) {
        float top[U], m = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            top[u] = Fmt<DT>::vmax(raw[u]);
            m = fmaxf(m, top[u]);
        }
        VfState st{m, 0.f, kNone};
        if (m == -INFINITY || m == INFINITY) {  // nothing but -inf and NaN, or +inf
            float nan = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[N];
                Fmt<DT>::unpack(raw[u], x);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (x[j] != x[j]) nan = x[j];
            }
            st.s = m == INFINITY ? NAN : nan;
            return st;
        }
        // the lowest element that holds the maximum leaves the sum
        uint4 hit = raw[U - 1];
        int at = U - 1;
#pragma unroll
        for (int u = U - 2; u >= 0; --u)
            if (top[u] == m) {
                hit = raw[u];
                at = u;
            }
        float h[N];
        Fmt<DT>::unpack(hit, h);
        int j0 = 0;
#pragma unroll
        for (int j = N - 1; j >= 0; --j) j0 = h[j] == m ? j : j0;
        st.at = first + at * step + j0;
        const F2 mm = f2(m, m), kk = f2(k, k);
        F2 sum = f2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[N];
            Fmt<DT>::unpack(raw[u], x);
            const int skip = at == u ? j0 : -1;
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const F2 v = f2(skip == j ? -INFINITY : x[j], skip == j + 1 ? -INFINITY : x[j + 1]);
                sum = f2_add(sum, f2_ex2(f2_mul(f2_sub(v, mm), kk)));
            }
        }
        float lo, hi;
        f2_split(sum, lo, hi);
        st.s = lo + hi;
        return st;
    }
};

// over the warp, the same in every lane: the maximum first, then one move of each lane's sum to it
__device__ inline VfState vf_reduce(const VfState &st, float k) {
    float M = st.m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    // the lowest index of the maximum: its lane's own term stays out of the sum
    int at = st.m == M ? st.at : kNone;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) at = min(at, __shfl_xor_sync(0xffffffffu, at, off));
    float s = st.m == M && st.at == at ? st.s : vf_shift(st.m, st.s, M, k);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return VfState{M, s, at};
}

// a row's statistics from its parts, by one warp, the same in every lane
__device__ inline VfState vf_row(const VfPart *p, int parts, float k) {
    const int lane = threadIdx.x & 31;
    VfState st{-INFINITY, 0.f, kNone};
    for (int j = lane; j < parts; j += 32) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + j));
        st = vf_merge(st, VfState{v.x, v.y, __float_as_int(v.z)}, k);
    }
    return vf_reduce(st, k);
}
__device__ inline void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// A term's exponent relative to the reference R is x k - r with r = R k rounded once:
// what that rounding shifts is the same for every term of the row, so it leaves the
// probabilities alone. From 2^24 on it may shift by whole powers of two, further up by
// more than fp32 holds, and R k itself may be infinite: there it is (x - R) k. That is an
// instruction more for every two elements, and no row of a model needs it: the loops over
// a row have a plain second form for it.
__device__ inline bool vf_far(float R, float k) { return !(fabsf(R * k) < 0x1p24f); }
__device__ inline float vf_arg(float x, float R, float k) { return vf_far(R, k) ? (x - R) * k : fmaf(x, k, -(R * k)); }
// 2^ those of N values, r = R k, or R itself where that is far
template <int N>
__device__ inline void vf_exps(const float *x, float k, float r, bool far, float *e) {
    const F2 kk = f2(k, k), rr = f2(-r, -r);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const F2 v = f2(x[j], x[j + 1]);
        f2_split(f2_ex2(far ? f2_mul(f2_add(v, rr), kk) : f2_fma(v, kk, rr)), e[j], e[j + 1]);
    }
}

// A row's distribution: p_c = 2^vf_arg(x_c, R, k) / S. M the maximum; at its lowest index
// and s1 = sum of the terms 2^((x - M) k) without that one, where they are known.
struct VfRow {
    float R, S, M, s1;
    int at;
};
// (the terms of a VfState are relative to exactly M: S takes the shift that R k's rounding makes)
__device__ inline VfRow vf_of(const VfState &s, float k) {
    return VfRow{s.m, (1.f + s.s) * ex2_hw(vf_arg(s.m, s.m, k)), s.m, s.s, s.at};
}
__device__ inline VfRow vf_none() { return VfRow{0.f, 1.f, 0.f, 0.f, 0}; }
__device__ inline bool vf_defined(const VfRow &r) {
    return r.S > 0.f && r.S < INFINITY && fabsf(r.M) < INFINITY && fabsf(r.R) < INFINITY;
}

// log p of a logit x from the row's sum (the same exponent as the sum's terms: R k's rounding cancels)
__device__ inline float vf_logp_of(float x, const VfRow &p, float k) {
    return vf_arg(x, p.R, k) * 0.6931471805599453f - logf(p.S);
}

// Whether a draft stays, u q_t < p_t: its logits xt, yt in the rows p, q (model: there
// is a draft model's). In logarithms, so that no probability is too small.
__device__ inline bool vf_stays(int64_t t, float u, float xt, float yt, const VfRow &p, const VfRow &q, bool model,
                                bool greedy, float k) {
    if (!vf_defined(p) || !vf_defined(q)) return false;
    if (greedy) return p.at == static_cast<int>(t);
    const float lp = vf_arg(xt, p.R, k) - log2f(p.S), lq = model ? vf_arg(yt, q.R, k) - log2f(q.S) : 0.f;
    return log2f(u) + lq < lp;
}

// Few sequences: one warp a part of a row, parts dealt out round robin.
template <int DT, int U>
__global__ void __launch_bounds__(kThreads, 3) vf_stats_kernel(VfArgs a) {
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warps = gridDim.x * kWarps, items = a.B * (a.K + 1) * a.parts;
    for (int item = blockIdx.x * kWarps + (threadIdx.x >> 5); item < items;) {
        const int part = item % a.parts, rest = item / a.parts, b = rest % a.B, i = rest / a.B;
        item = item < items - warps ? item + warps : items;
        const float temp = vf_temp(a, b), k = vf_k(temp);
        // a missing draft ends the sequence: rows behind it are not read
        bool ended = !vf_temp_ok(temp);
        for (int j = lane; j < i; j += 32) ended |= !vf_valid(a, vf_draft(a, b, j));
        if (__any_sync(0xffffffffu, ended)) continue;
        const bool model = a.y && temp != 0.f && i < a.K && vf_valid(a, vf_draft(a, b, i));
        VfTile<DT, U> tx, ty;
        tx.load(reinterpret_cast<const char *>(a.x) + (b * a.xs + i * a.xr) * Fmt<DT>::kBytes, a.V, part * U * 32 + lane, 32);
        if (model) ty.load(reinterpret_cast<const char *>(a.y) + (b * a.ys + i * a.yr) * Fmt<DT>::kBytes, a.V, part * U * 32 + lane, 32);
        const VfState sx = vf_reduce(tx.stats(k), k);
        if (lane == 0) a.px[(static_cast<int64_t>(b) * (a.K + 1) + i) * a.parts + part] = VfPart{sx.m, sx.s, sx.at, 0.f};
        if (!model) continue;
        const VfState sy = vf_reduce(ty.stats(k), k);
        if (lane == 0) a.py[(static_cast<int64_t>(b) * a.K + i) * a.parts + part] = VfPart{sy.m, sy.s, sy.at, 0.f};
    }
}

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
// A row as vectors of 16 bytes, counted from the boundary at or before its first
// element; elements outside of the row read as -inf.
template <int DT> struct VfRowIn {
    static constexpr int N = Fmt<DT>::kVec;
    const char *row;
    int before, V;  // elements of vector 0 before the row, elements of the row
    __device__ inline VfRowIn(const void *p, int vocab)
        : row(reinterpret_cast<const char *>(p)), before(static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / Fmt<DT>::kBytes), V(vocab) {}
    __device__ inline int first(int v) const { return v * N - before; }
    __device__ inline bool whole(int v) const { return first(v) >= 0 && first(v) + N <= V; }
    __device__ inline const void *at(int v) const { return row + static_cast<int64_t>(first(v)) * Fmt<DT>::kBytes; }
    __device__ inline uint4 edge(int v) const {  // element by element
        float t[N];
#pragma unroll
        for (int j = 0; j < N; ++j) t[j] = first(v) + j >= 0 && first(v) + j < V ? Fmt<DT>::load1(row, first(v) + j) : -INFINITY;
        return Fmt<DT>::pack(t);
    }
    __device__ inline uint4 get(int v) const { return whole(v) ? __ldg(reinterpret_cast<const uint4 *>(at(v))) : edge(v); }
};

// A thread's vectors v0, v0 + stride, ... < v1 of two rows (two: is there a second) on
// their way through its own slots of shared memory, kDepth of them in flight: 64 KB
// a CTA, so that one CTA alone on an SM reads at the rate that it could read at.
// Vectors that reach over an end of either row are taken element by element,
// before and after; `apart`: the second row's elements lie elsewhere in their
// vectors than the first's, and are wanted at the first's places.
constexpr int kDepth = 8;
constexpr int kRing = kDepth * 2 * kThreads * 16;  // bytes of dynamic shared memory
template <int DT> struct VfStream {
    static constexpr int N = Fmt<DT>::kVec;
    VfRowIn<DT> x, y;
    bool two, apart;
    int v, v1, stride, left, ahead;  // the next vector; whole vectors to use, and to ask for
    const char *px, *py;
    uint32_t mine;

    __device__ inline void ask(int slot) {
        if (ahead > 0) {
            cp_async16(mine + slot * 2 * kThreads * 16, px);
            if (two) cp_async16(mine + (slot * 2 + 1) * kThreads * 16, py);
            px += static_cast<int64_t>(stride) * 16;
            py += static_cast<int64_t>(stride) * 16;
            --ahead;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // the first copies; `use` of run() follows, or drop()
    __device__ inline VfStream(const VfRowIn<DT> &x_, const VfRowIn<DT> &y_, bool two_, bool apart_, int v0, int v1_, int stride_,
                               uint4 *ring)
        : x(x_), y(y_), two(two_), apart(apart_), v(v0), v1(v1_), stride(stride_), mine(smem_u32(ring + threadIdx.x)) {
        // where whole vectors of both rows begin (at vector 0 or 1) and end
        const int v_in = v == 0 && (!x.whole(0) || (two && !y.whole(0))) ? v + stride : v;
        int end = (x.V + x.before) / N;
        if (two) end = min(end, (y.V + y.before) / N);
        end = min(end, v1);
        left = !(two && apart) && v_in < end ? (end - v_in + stride - 1) / stride : 0;
        ahead = left;
        px = reinterpret_cast<const char *>(x.at(v_in));
        py = reinterpret_cast<const char *>(y.at(v_in));
#pragma unroll
        for (int j = 0; j < kDepth - 2; ++j) ask(j);
    }
    __device__ inline void drop() { asm volatile("cp.async.wait_all;" ::: "memory"); }
    // every vector without the ring, whose copies have been dropped
    template <typename F> __device__ inline void all(F use) {
        while (__any_sync(0xffffffffu, v < v1))
            if (v < v1) slow(use);
    }
    template <typename F> __device__ inline void slow(F use) {
        uint4 ry = make_uint4(0u, 0u, 0u, 0u);
        if (two && apart) {
            float t[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int c = x.first(v) + j;
                t[j] = c >= 0 && c < y.V ? Fmt<DT>::load1(y.row, c) : -INFINITY;
            }
            ry = Fmt<DT>::pack(t);
        } else if (two) {
            ry = y.get(v);
        }
        use(v, x.get(v), ry);
        v += stride;
    }
    template <typename F> __device__ inline void run(F use) {
        if (!(two && apart) && v == 0 && v < v1 && (!x.whole(0) || (two && !y.whole(0)))) slow(use);
        // two vectors at a time, so that their arithmetic overlaps
        while (left > 0) {
#pragma unroll
            for (int j = 0; j < kDepth; j += 2) {
                if (left <= 0) break;
                ask((j + kDepth - 2) % kDepth);
                ask((j + kDepth - 1) % kDepth);
                asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
                const uint4 none = make_uint4(0u, 0u, 0u, 0u);
                const uint4 rx0 = ld_shared_v4(mine + j * 2 * kThreads * 16), rx1 = ld_shared_v4(mine + (j + 1) * 2 * kThreads * 16);
                uint4 ry0 = none, ry1 = none;
                if (two) {
                    ry0 = ld_shared_v4(mine + (j * 2 + 1) * kThreads * 16);
                    ry1 = ld_shared_v4(mine + (j * 2 + 3) * kThreads * 16);
                }
                if (left == 1) {
                    use(v, rx0, ry0);
                    v += stride;
                    left = 0;
                    break;
                }
                use(v, rx0, ry0, v + stride, rx1, ry1);
                v += 2 * stride;
                left -= 2;
            }
        }
        drop();
        // The warp's lanes leave together. They come here by loops of different lengths, and the compiler may give lanes that
        // leave in different places a copy each of what follows, shuffles included, which then miss one another.
        while (__any_sync(0xffffffffu, v < v1))
            if (v < v1) slow(use);
    }
};

// What row n's token is drawn from: w_c = max(p_c - q_c, 0), or p_c.
// Where little is left over, the roundings of p, q and S would be drawn from: below
// kLittle of all probability the terms of both rows are summed once more, by the
// difference and in the same order, as pairs, and p - q is formed of those with a
// remainder (VF_FINE): equal rows leave exactly nothing then, and are drawn from p.
constexpr float kLittle = 0x1p-8f;
enum { VF_FAR_X = 1, VF_FAR_Y = 2, VF_FINE = 4 };
template <int DT> struct VfWeights {
    static constexpr int N = Fmt<DT>::kVec;
    VfRowIn<DT> x, y;
    bool two, apart;  // a draft model at this position; its row starts elsewhere in its 16 bytes than x's
    float rx, ix, ry, iy, k;  // R k, or R where that is far; 1 / S
    int drop;                 // the draft without a draft model, or kNone
    int form;                 // VF_FAR_X | VF_FAR_Y | VF_FINE

    // y's elements in the places of x's vector v
    __device__ inline uint4 second(int v) const {
        if (!two) return make_uint4(0u, 0u, 0u, 0u);
        if (!apart) return y.get(v);
        float t[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = x.first(v) + j;
            t[j] = c >= 0 && c < y.V ? Fmt<DT>::load1(y.row, c) : -INFINITY;
        }
        return Fmt<DT>::pack(t);
    }
    // the weights of vector v from its logits; e, d: p's and q's terms (not scaled). NEAR: form is 0; low: VF_FINE's 1 / S less ix, iy
    template <bool NEAR>
    __device__ inline void get(int v, const uint4 &ux, const uint4 &uy, const float2 &low, float (&e)[N], float (&d)[N], float (&w)[N]) const {
        float t[N];
        Fmt<DT>::unpack(ux, t);
        vf_exps<N>(t, k, rx, !NEAR && (form & VF_FAR_X), e);
        const F2 sx = f2(ix, ix);
        if (two) {
            Fmt<DT>::unpack(uy, t);
            vf_exps<N>(t, k, ry, !NEAR && (form & VF_FAR_Y), d);
            const F2 sy = f2(-iy, -iy);
            if (!NEAR && (form & VF_FINE)) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    // (no product here may be fused into a difference: both sides are rounded alike)
                    const float u = __fmul_rn(d[j], iy), r = fmaf(d[j], iy, -u);
                    w[j] = fmaxf((fmaf(e[j], ix, -u) - r) + (__fmul_rn(e[j], low.x) - __fmul_rn(d[j], low.y)), 0.f);
                }
                return;
            }
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                f2_split(f2_fma(sy, f2(d[j], d[j + 1]), f2_mul(f2(e[j], e[j + 1]), sx)), w[j], w[j + 1]);
                w[j] = fmaxf(w[j], 0.f);
                w[j + 1] = fmaxf(w[j + 1], 0.f);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; j += 2) f2_split(f2_mul(f2(e[j], e[j + 1]), sx), w[j], w[j + 1]);
        }
        const unsigned rel = static_cast<unsigned>(drop) - static_cast<unsigned>(x.first(v));
        if (rel < static_cast<unsigned>(N)) {
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = static_cast<unsigned>(j) == rel ? 0.f : w[j];
        }
    }
};

__device__ inline void vf_put(const VfArgs &a, int64_t at, int64_t token, float lp) {
    if (a.tok32) reinterpret_cast<int32_t *>(a.tokens)[at] = static_cast<int32_t>(token);
    else reinterpret_cast<int64_t *>(a.tokens)[at] = token;
    a.logp[at] = lp;
}
// log p of a token with logit x from the sum beside the maximum's term; ln2_k = 1 / T
__device__ inline float vf_logp(float x, float M, float s1, float ln2_k) { return (x - M) * ln2_k - log1pf(s1); }

// Every warp of the cluster gives 16 bytes to all, and all go on once they have
// them: asynchronous stores that count on each CTA's mbarrier, two sets of slots by
// turns. (A cluster barrier's release waits for the copies in flight too.) A warp
// gives for the next turn only after it has read this one's, so no slot is written
// while it is read.
struct VfMeetMem {
    float4 slot[2][kCluster * kWarps];
    uint64_t bar[2];
    int abort;
};
struct VfMeet {
    VfMeetMem &m;
    int rank, size, turn;
    __device__ inline VfMeet(VfMeetMem &mem) : m(mem), rank(cluster_ctarank()), size(cluster_nctarank()), turn(0) {
        if (threadIdx.x == 0) {
            m.abort = 0;
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&m.bar[i]), 1);
            }
            fence_mbar_init_cluster();
            for (int i = 0; i < 2; ++i) mbar_expect_tx(smem_u32(&m.bar[i]), size * kWarps * 16);
        }
        __syncthreads();
        cluster_sync_all();  // every CTA of the cluster runs, and its barriers exist, before one writes into another
    }
    __device__ inline const float4 *all(float a, float b, float c, float d) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, set = turn & 1;
        const uint32_t bar = smem_u32(&m.bar[set]);
        __syncwarp();  // every lane has read the last turn's
        if (lane < size) {
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                             mapa_shared(smem_u32(&m.slot[set][rank * kWarps + warp]), lane)),
                         "f"(a), "f"(b), "f"(c), "f"(d), "r"(mapa_shared(bar, lane))
                         : "memory");
        }
        mbar_wait_bounded<true>(bar, (turn >> 1) & 1, &m.abort);
        if (threadIdx.x == 0) mbar_expect_tx(bar, size * kWarps * 16);  // the turn after the next
        ++turn;
        return m.slot[set];
    }
    // no CTA leaves while another may still write into it (one whose wait gave up may be early)
    __device__ inline void leave() {
        __syncthreads();
        cluster_sync_all();
    }
    __device__ inline bool failed() const { return *const_cast<volatile int *>(&m.abort) != 0; }
};

struct VfDrawMem {
    FF scan[kWarps], from, goal;
    float2 refs, low;  // R of both rows, VF_FINE's 1 / S less their fp32
    float mass, s1;
    int own, pick, last;
};

// Token n of sequence b, by its whole cluster, and what lies behind it. p, q: the
// rows (q: vf_none() without a draft model at n), the same in every thread of the
// cluster; turned: position n has a draft; S1: p.s1 is known (else it is formed
// here, for the log-probability of a token that holds the maximum). The CTAs have
// met in a cluster barrier since they started.
template <int DT, bool S1>
__device__ inline void vf_draw(const VfArgs &a, int b, int n, const VfRow &p, const VfRow &q, bool turned, bool model,
                               bool usable, bool greedy, float k, VfDrawMem &m, VfMeet &meet, uint4 *ring) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank()), size = static_cast<int>(cluster_nctarank());
    const int64_t row = static_cast<int64_t>(b) * (a.K + 1), xrow = b * a.xs + n * a.xr;
    const float ln2_k = k * 0.6931471805599453f;
    if (rank == 0) {
        if (tid == 0) a.accepted[b] = n;
        for (int i = n + 1 + tid; i <= a.K; i += kThreads) vf_put(a, row + i, -1, 0.f);
    }
    const auto emit = [&](int t) {
        float lp = NAN;
        if (t >= 0) {
            const float x = Fmt<DT>::load1(a.x, xrow + t);
            if (S1 || greedy) lp = vf_logp(x, p.M, p.s1, ln2_k);
            else lp = x == p.M ? -log1pf(m.s1) : vf_logp_of(x, p, k);
        }
        vf_put(a, row + n, t, lp);
    };
    const bool defined = usable && vf_defined(p) && vf_defined(q);
    if (!defined || greedy) {  // the same in every CTA of the cluster
        if (rank == 0 && tid == 0) emit(defined ? p.at : -1);
        return;
    }
    constexpr int N = Fmt<DT>::kVec;
    const char *px = reinterpret_cast<const char *>(a.x) + xrow * Fmt<DT>::kBytes;
    const char *py = model ? reinterpret_cast<const char *>(a.y) + (b * a.ys + n * a.yr) * Fmt<DT>::kBytes : px;
    const bool far_x = vf_far(p.R, k), far_y = vf_far(q.R, k);
    VfWeights<DT> w{VfRowIn<DT>(px, a.V), VfRowIn<DT>(py, a.V), model, false, far_x ? p.R : p.R * k, 1.f / p.S,
                    far_y ? q.R : q.R * k, 1.f / q.S, k, turned && !model ? static_cast<int>(vf_draft(a, b, n)) : kNone,
                    (far_x ? VF_FAR_X : 0) | (far_y ? VF_FAR_Y : 0)};
    if (tid == 0) m.refs = make_float2(p.R, q.R);  // (read behind a barrier)
    w.apart = w.x.before != w.y.before;
    // contiguous ranges of the row, one a warp of the cluster, in steps of 32 vectors
    const int steps = (a.V + N - 1 + 32 * N - 1) / (32 * N), all = size * kWarps;
    const auto step_of = [&](int range) { return static_cast<int>(static_cast<int64_t>(steps) * range / all); };
    bool terms = false;  // this pass sums the terms for VF_FINE
    for (int pass = 0;; ++pass) {
        const int g = rank * kWarps + warp, s0 = step_of(g), s1 = step_of(g + 1);
        FF sum{0.f, 0.f};
        float rest = 0.f, tops = 0.f;
        const auto one = [&](int v, const uint4 &ux, const uint4 &uy, float &r) {
            float e[N], d[N], g[N];
            w.template get<true>(v, ux, uy, make_float2(0.f, 0.f), e, d, g);
            F2 t = f2(g[0], g[1]);
#pragma unroll
            for (int j = 2; j < N; j += 2) t = f2_add(t, f2(g[j], g[j + 1]));
            if (!S1) {
                // p's terms off the maximum, and how many elements hold it
                if (Fmt<DT>::vmax(ux) == p.M) {
                    float x[N];
                    Fmt<DT>::unpack(ux, x);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        tops += x[j] == p.M ? 1.f : 0.f;
                        e[j] = x[j] == p.M ? 0.f : e[j];
                    }
                }
                F2 o = f2(e[0], e[1]);
#pragma unroll
                for (int j = 2; j < N; j += 2) o = f2_add(o, f2(e[j], e[j + 1]));
                float lo, hi;
                f2_split(o, lo, hi);
                r += lo + hi;
            }
            float lo, hi;
            f2_split(t, lo, hi);
            return lo + hi;
        };
        if (w.form == 0) {
            VfStream<DT> in(w.x, w.y, w.two, w.apart, s0 * 32 + lane, s1 * 32, 32, ring);
            float rest2 = 0.f;
            struct Use {
                const decltype(one) &f;
                FF &sum;
                float &rest, &rest2;
                __device__ inline void operator()(int v, const uint4 &ux, const uint4 &uy) const { sum = ff_add(sum, FF{f(v, ux, uy, rest), 0.f}); }
                __device__ inline void operator()(int v, const uint4 &ux, const uint4 &uy, int v2, const uint4 &ux2, const uint4 &uy2) const {
                    const float t = f(v, ux, uy, rest), t2 = f(v2, ux2, uy2, rest2);
                    sum = ff_add(ff_add(sum, FF{t, 0.f}), FF{t2, 0.f});
                }
            };
            in.run(Use{one, sum, rest, rest2});
            rest += rest2;
        } else {
            FF more{0.f, 0.f};  // terms: sum and more are those of p's terms and of q's
            const float2 low = m.low;
#pragma unroll 1
            for (int step = s0; step < s1; ++step) {
                const int v = step * 32 + lane;
                const uint4 ux = w.x.get(v);
                float x[N], e[N], d[N] = {}, g[N], se = 0.f, sd = 0.f;
                w.template get<false>(v, ux, w.second(v), low, e, d, g);
                Fmt<DT>::unpack(ux, x);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    se += terms ? e[j] : g[j];
                    sd += d[j];
                    tops += x[j] == p.M ? 1.f : 0.f;
                    rest += x[j] == p.M ? 0.f : e[j];
                }
                sum = ff_add(sum, FF{se, 0.f});
                more = ff_add(more, FF{sd, 0.f});
                __syncwarp();
            }
            if (terms) {
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    sum = ff_add(sum, ff_shfl_xor(sum, off));
                    more = ff_add(more, ff_shfl_xor(more, off));
                }
                const float4 *given = meet.all(sum.hi, sum.lo, more.hi, more.lo);
                sum = more = FF{0.f, 0.f};
                for (int j = 0; j < all; ++j) {
                    sum = ff_add(sum, FF{given[j].x, given[j].y});
                    more = ff_add(more, FF{given[j].z, given[j].w});
                }
                w.ix = 1.f / sum.hi;
                w.iy = 1.f / more.hi;
                w.form |= VF_FINE;
                terms = false;
                // the same value from every thread
                m.low = make_float2(fmaf(-w.ix, sum.lo, fmaf(-w.ix, sum.hi, 1.f)) * w.ix,
                                    fmaf(-w.iy, more.lo, fmaf(-w.iy, more.hi, 1.f)) * w.iy);
                __syncthreads();
                continue;
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            sum = ff_add(sum, ff_shfl_xor(sum, off));
            if (!S1) {
                rest += __shfl_xor_sync(0xffffffffu, rest, off);
                tops += __shfl_xor_sync(0xffffffffu, tops, off);
            }
        }
        const float4 *ranges = meet.all(sum.hi, sum.lo, rest, tops);
        // Every CTA finds the same range: the first whose end lies above the aim;
        // rounding may leave none, then the last that holds anything.
        if (warp == 0) {
            static_assert(kCluster * kWarps == 64, "two ranges a lane");
            const FF zero{0.f, 0.f};
            const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 r0 = 2 * lane < all ? ranges[2 * lane] : none, r1 = 2 * lane < all ? ranges[2 * lane + 1] : none;
            const FF v0{r0.x, r0.y}, v1{r1.x, r1.y};
            if (!S1 && pass == 0) {
                float rest_all = r0.z + r1.z, tops_all = r0.w + r1.w;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    rest_all += __shfl_xor_sync(0xffffffffu, rest_all, off);
                    tops_all += __shfl_xor_sync(0xffffffffu, tops_all, off);
                }
                // from terms relative to R to those relative to M
                if (lane == 0) m.s1 = (tops_all - 1.f) + rest_all / ex2_hw(vf_arg(p.M, p.R, k));
            }
            const FF incl = ff_scan(ff_add(v0, v1));
            FF before = ff_shfl_up(incl, 1);
            if (lane == 0) before = zero;
            const FF sum_all = ff_shfl(incl, 31), aim = ff_scale(sum_all, __ldg(a.r + b));
            const FF mid = ff_add(before, v0);
            const int hit = ff_above(mid, aim) ? 2 * lane : (ff_above(incl, aim) ? 2 * lane + 1 : -1);
            const int full = v1.hi > 0.f ? 2 * lane + 1 : (v0.hi > 0.f ? 2 * lane : -1);
            const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), fulls = __ballot_sync(0xffffffffu, full >= 0);
            const int src = hits ? __ffs(hits) - 1 : (fulls ? 31 - __clz(fulls) : 0);
            const int found = hits ? hit : full;
            if (lane == src) {
                m.own = meet.failed() ? -1 : found;  // a wait that gave up leaves no token
                m.from = (found & 1) ? mid : before;
                m.goal = aim;
                m.mass = meet.failed() ? 1.f : sum_all.hi;
                m.pick = kNone;
                m.last = -1;
            }
        }
        __syncthreads();
        if (w.two && !(w.form & VF_FINE) && m.mass <= kLittle) {
            terms = true;
            w.form = VF_FAR_X | VF_FAR_Y;
            w.rx = m.refs.x;
            w.ry = m.refs.y;
            continue;
        }
        if (m.mass > 0.f || (!w.two && w.drop == kNone)) break;
        // p <= q everywhere (p = q): drawn from p
        w.two = false;
        w.drop = kNone;
    }
    const int range = m.own;
    if (range < 0) {  // nothing to draw from
        if (rank == 0 && tid == 0) emit(-1);
        return;
    }
    if (range / kWarps != rank) return;
    // the CTA walks its warp's range, a vector a thread at a time
    const FF aim = m.goal;
    FF below = m.from;
    const int v1 = step_of(range + 1) * 32;
    for (int v0 = step_of(range) * 32; v0 < v1; v0 += kThreads) {
        float v[N], t = 0.f;
        const int c = w.x.first(v0 + tid);
        if (v0 + tid < v1) {
            float e[N], d[N];
            w.template get<false>(v0 + tid, w.x.get(v0 + tid), w.second(v0 + tid), m.low, e, d, v);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) t += v[j];
        const FF incl = ff_scan(FF{t, 0.f});
        if (lane == 31) m.scan[warp] = incl;
        __syncthreads();
        FF start = below;
        for (int j = 0; j < warp; ++j) start = ff_add(start, m.scan[j]);
        FF before = ff_shfl_up(incl, 1);
        before = lane == 0 ? start : ff_add(start, before);
        int found = -1, lastpos = -1;
        float run = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            run += v[j];
            if (v[j] > 0.f) {
                lastpos = c + j;
                if (found < 0 && ff_above(ff_add(before, FF{run, 0.f}), aim)) found = c + j;
            }
        }
        if (found >= 0) atomicMin(&m.pick, found);
        if (lastpos >= 0) atomicMax(&m.last, lastpos);
        for (int j = 0; j < kWarps; ++j) below = ff_add(below, m.scan[j]);
        __syncthreads();
        if (m.pick != kNone) break;  // written before the barrier above, read after it
    }
    // rounding may leave no such element: then the last that holds anything
    if (tid == 0) emit(m.pick != kNone ? m.pick : m.last);
}

// Few sequences, after vf_stats_kernel.
template <int DT>
__global__ void __launch_bounds__(kThreads, 2) vf_pick_kernel(VfArgs a) {
    extern __shared__ uint4 ring[];
    __shared__ VfState sx[kMaxDrafts + 1], sy[kMaxDrafts];
    __shared__ VfDrawMem mem;
    __shared__ VfMeetMem meeting;
    __shared__ int count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank()), b = blockIdx.x / cluster_nctarank();
    const float temp = vf_temp(a, b), k = vf_k(temp);
    const bool greedy = temp == 0.f, usable = vf_temp_ok(temp);
    if (tid == 0) count = a.K;
    VfMeet meet(meeting);
    pdl_wait();
    // every row's statistics and whether its draft stays
    for (int i = warp; i <= a.K && usable; i += kWarps) {
        bool ended = false;
        for (int j = lane; j < i; j += 32) ended |= !vf_valid(a, vf_draft(a, b, j));
        if (__any_sync(0xffffffffu, ended)) break;
        const int64_t t = i < a.K ? vf_draft(a, b, i) : -1;
        const bool has = vf_valid(a, t), model = a.y && has && !greedy;
        const float u = has ? __ldg(a.u + static_cast<int64_t>(b) * a.K + i) : 0.f;
        const float xt = has ? Fmt<DT>::load1(a.x, b * a.xs + i * a.xr + t) : 0.f;
        const float yt = model ? Fmt<DT>::load1(a.y, b * a.ys + i * a.yr + t) : 0.f;
        const VfState p = vf_row(a.px + (static_cast<int64_t>(b) * (a.K + 1) + i) * a.parts, a.parts, k);
        VfState q{0.f, 0.f, 0};
        if (model) q = vf_row(a.py + (static_cast<int64_t>(b) * a.K + i) * a.parts, a.parts, k);
        if (lane == 0) {
            sx[i] = p;
            if (i < a.K) {
                sy[i] = q;
                if (!has || !vf_stays(t, u, xt, yt, vf_of(p, k), model ? vf_of(q, k) : vf_none(), model, greedy, k)) atomicMin(&count, i);
            }
        }
    }
    __syncthreads();
    const int n = usable ? count : 0;
    if (rank == 0) {
        for (int i = tid; i < n; i += kThreads) {
            const int64_t t = vf_draft(a, b, i);
            vf_put(a, static_cast<int64_t>(b) * (a.K + 1) + i, t,
                   vf_logp(Fmt<DT>::load1(a.x, b * a.xs + i * a.xr + t), sx[i].m, sx[i].s, k * 0.6931471805599453f));
        }
    }
    const bool turned = usable && n < a.K && vf_valid(a, vf_draft(a, b, n)), model = turned && a.y && !greedy;
    vf_draw<DT, true>(a, b, n, usable ? vf_of(sx[n], k) : vf_none(), model ? vf_of(sy[n], k) : vf_none(), turned, model, usable,
                      greedy, k, mem, meet, ring);
    meet.leave();
}

// Adds 2^(x k - r) of a vector whose first element is c, without element `skip`, and
// follows the maximum (with it): a conversion, half a multiplication, an
// exponential, half an addition and half a maximum an element.
template <int DT> struct VfAdd {
    static constexpr int N = Fmt<DT>::kVec;
    F2 sum = f2(0.f, 0.f);
    uint32_t top16 = Fmt<DT>::kNegInfWord;  // packed maxima of 16-bit types
    float top = -INFINITY;
    // (rk: R k, or R itself where that is far)
    __device__ inline void add(const uint4 &r, int c, float k, float rk, int skip, bool far = false) {
        float x[N];
        Fmt<DT>::unpack(r, x);
        if constexpr (DT == CE_DT_F32) top = fmaxf(top, Fmt<DT>::vmax(r));
        else top16 = Fmt<DT>::hmax2(top16, Fmt<DT>::hmax2(Fmt<DT>::hmax2(r.x, r.y), Fmt<DT>::hmax2(r.z, r.w)));
        const unsigned rel = static_cast<unsigned>(skip) - static_cast<unsigned>(c);
        if (rel < static_cast<unsigned>(N)) {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = static_cast<unsigned>(j) == rel ? -INFINITY : x[j];
        }
        const F2 kk = f2(k, k), rr = f2(-rk, -rk);
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const F2 v = f2(x[j], x[j + 1]);
            sum = f2_add(sum, f2_ex2(far ? f2_mul(f2_add(v, rr), kk) : f2_fma(v, kk, rr)));
        }
    }
    __device__ inline void join(const VfAdd &o) {
        sum = f2_add(sum, o.sum);
        top = fmaxf(top, o.top);
        if constexpr (DT != CE_DT_F32) top16 = Fmt<DT>::hmax2(top16, o.top16);
    }
    __device__ inline void finish(float &m, float &s) const {
        float lo, hi;
        f2_split(sum, lo, hi);
        s = lo + hi;
        m = top;
        if constexpr (DT != CE_DT_F32) {
            Fmt<DT>::unpack2(top16, lo, hi);
            m = fmaxf(lo, hi);
        }
    }
};

// Many sequences: everything of one by its cluster, position by position. Sums are
// taken from a reference R that every thread knows at the start, the draft's own
// logit x_t (then log p_t = -log1p(s), s without the draft's term), or the largest
// of 32 spread elements: no running maximum, no rebasing, and the warps' sums
// just add up. Where the maximum turns out 2^60 or more away, the row is taken
// again from its maximum. (With each thread's running maximum and its element kept
// out of the sum the instructions took twice as long as the reading: 108 us for
// 128 sequences of 4 drafts and 128256 columns of bf16.)
template <int DT>
__global__ void __launch_bounds__(kThreads, 3) vf_seq_kernel(VfArgs a) {
    extern __shared__ uint4 ring[];
    constexpr int N = Fmt<DT>::kVec;
    constexpr float kFar = 60.f;
    __shared__ VfMeetMem meeting;
    __shared__ int drafts[kMaxDrafts + 1];         // -1: none
    __shared__ float us[kMaxDrafts + 1], xts[kMaxDrafts + 1], yts[kMaxDrafts + 1];
    __shared__ VfDrawMem mem;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank()), size = static_cast<int>(cluster_nctarank()), b = blockIdx.x / size;
    const float temp = vf_temp(a, b), k = vf_k(temp), ln2_k = k * 0.6931471805599453f;
    const bool greedy = temp == 0.f, usable = vf_temp_ok(temp);
    // Every position's scalars; a position behind a missing draft has none, for its rows are not read. (A warp looks at the
    // drafts before its own itself: a barrier instead took 1 us.)
    static_assert(kMaxDrafts < kThreads, "a position a thread");
    int64_t t = -1;
    unsigned missing = 0;
    for (int c = 0; c <= tid >> 5; ++c) {
        t = c * 32 + lane < a.K && !missing ? vf_draft(a, b, c * 32 + lane) : -1;
        missing = __ballot_sync(0xffffffffu, !vf_valid(a, t));
    }
    if (tid <= a.K) {
        const int i = tid;
        const bool has = !(missing & ((2u << lane) - 1u));
        drafts[i] = has ? static_cast<int>(t) : -1;
        us[i] = has ? __ldg(a.u + static_cast<int64_t>(b) * a.K + i) : 0.f;
        xts[i] = has ? Fmt<DT>::load1(a.x, b * a.xs + i * a.xr + t) : 0.f;
        yts[i] = has && a.y && !greedy ? Fmt<DT>::load1(a.y, b * a.ys + i * a.yr + t) : 0.f;
    }
    VfMeet meet(meeting);
    // this CTA's slice of a row, in steps of a vector a thread
    const int steps = (a.V + N - 1 + kThreads * N - 1) / (kThreads * N);
    const int t0 = static_cast<int>(static_cast<int64_t>(steps) * rank / size), t1 = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / size);
    // position i's rows on their way (the rows' vectors need not lie alike: each row's slice is its own)
    const auto stream = [&](int i) {
        const bool two = a.y && drafts[i] >= 0 && !greedy;
        const VfRowIn<DT> in(reinterpret_cast<const char *>(a.x) + (b * a.xs + i * a.xr) * Fmt<DT>::kBytes, a.V);
        const VfRowIn<DT> yin(two ? reinterpret_cast<const char *>(a.y) + (b * a.ys + i * a.yr) * Fmt<DT>::kBytes : in.row, a.V);
        return VfStream<DT>(in, yin, two, false, t0 * kThreads + tid, usable ? t1 * kThreads : 0, kThreads, ring);
    };
    // the largest of 32 elements spread over a row (0 if none is finite)
    const auto sample = [&](const void *row) {
        float v = Fmt<DT>::load1(row, static_cast<int>(static_cast<int64_t>(a.V) * lane / 32));
        v = fabsf(v) < INFINITY ? v : -INFINITY;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
        return v == -INFINITY ? 0.f : v;
    };
    VfRow p = vf_none(), q = vf_none();
    bool has = false, model = false;
    int n = 0;
    VfStream<DT> in = stream(0);
    for (; usable; ++n) {
        const int t = drafts[n];
        has = t >= 0;
        model = a.y && has && !greedy;
        const char *x = reinterpret_cast<const char *>(a.x) + (b * a.xs + n * a.xr) * Fmt<DT>::kBytes;
        const char *y = reinterpret_cast<const char *>(a.y) + (b * a.ys + n * a.yr) * Fmt<DT>::kBytes;
        const float u = us[n], xt = xts[n], yt = yts[n];
        const int skip = has ? t : kNone;
        q = vf_none();
        if (greedy) {
            // the maximum's lowest index, through the same ring (200 sequences of 6 drafts, 50257 fp32 logits: 64 us; 74 with
            // a tile's loads in registers, none of the next row's under way)
            VfState st{-INFINITY, 0.f, kNone};
            struct Use {
                VfState &st;
                const VfStream<DT> &in;
                float k;
                __device__ inline void operator()(int v, const uint4 &ux, const uint4 &) const {
                    VfTile<DT, 1> tx;
                    tx.raw[0] = ux;
                    tx.first = in.x.first(v);
                    tx.step = 0;
                    st = vf_merge(st, tx.stats(k), k);
                }
                __device__ inline void operator()(int v, const uint4 &ux, const uint4 &, int v2, const uint4 &ux2, const uint4 &) const {
                    VfTile<DT, 2> tx;
                    tx.raw[0] = ux;
                    tx.raw[1] = ux2;
                    tx.first = in.x.first(v);
                    tx.step = in.x.first(v2) - tx.first;
                    st = vf_merge(st, tx.stats(k), k);
                }
            };
            in.run(Use{st, in, k});
            if (has) in = stream(n + 1);
            st = vf_reduce(st, k);
            const float4 *all = meet.all(st.m, st.s, __int_as_float(st.at), 0.f);
            st = VfState{-INFINITY, 0.f, kNone};
            for (int j = lane; j < size * kWarps; j += 32) st = vf_merge(st, VfState{all[j].x, all[j].y, __float_as_int(all[j].z)}, k);
            p = vf_of(vf_reduce(st, k), k);
        } else {
            float R = has && !vf_far(xt, k) ? xt : sample(x), Q = 0.f;  // (no NaN or infinity, and rather no far one)
            if (model) Q = !vf_far(yt, k) ? yt : sample(y);
            for (int again = 0;; ++again) {
                VfAdd<DT> ax, ay;
                const float rk = R * k, qk = Q * k;
                VfAdd<DT> bx, by;  // of every second vector
                struct Use {
                    VfAdd<DT> &ax, &ay, &bx, &by;
                    const VfStream<DT> &in;
                    float k, rk, qk;
                    int skip;
                    bool model;
                    __device__ inline void operator()(int v, const uint4 &ux, const uint4 &uy) const {
                        ax.add(ux, in.x.first(v), k, rk, skip);
                        if (model) ay.add(uy, in.y.first(v), k, qk, kNone);
                    }
                    __device__ inline void operator()(int v, const uint4 &ux, const uint4 &uy, int v2, const uint4 &ux2, const uint4 &uy2) const {
                        ax.add(ux, in.x.first(v), k, rk, skip);
                        bx.add(ux2, in.x.first(v2), k, rk, skip);
                        if (model) {
                            ay.add(uy, in.y.first(v), k, qk, kNone);
                            by.add(uy2, in.y.first(v2), k, qk, kNone);
                        }
                    }
                };
                const bool far_x = vf_far(R, k), far_y = model && vf_far(Q, k);
                if (!far_x && !far_y) {
                    in.run(Use{ax, ay, bx, by, in, k, rk, qk, skip, model});
                } else {
                    in.drop();
                    in.all([&](int v, const uint4 &ux, const uint4 &uy) {
                        ax.add(ux, in.x.first(v), k, far_x ? R : rk, skip, far_x);
                        if (model) ay.add(uy, in.y.first(v), k, far_y ? Q : qk, kNone, far_y);
                    });
                }
                ax.join(bx);
                ay.join(by);
                // the next position's rows, in case this draft stays
                if (has) in = stream(n + 1);
                float mx, vx, my, vy;
                ax.finish(mx, vx);
                ay.finish(my, vy);
                const auto over = [&](float &m0, float &v0, float &m1, float &v1) {
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) {
                        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, off));
                        v0 += __shfl_xor_sync(0xffffffffu, v0, off);
                        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, off));
                        v1 += __shfl_xor_sync(0xffffffffu, v1, off);
                    }
                };
                over(mx, vx, my, vy);
                const float4 *all = meet.all(mx, vx, my, vy);
                const int slots = size * kWarps;
                const float4 none = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                const float4 f0 = lane < slots ? all[lane] : none, f1 = lane + 32 < slots ? all[lane + 32] : none;
                mx = fmaxf(f0.x, f1.x);
                vx = f0.y + f1.y;
                my = fmaxf(f0.z, f1.z);
                vy = f0.w + f1.w;
                over(mx, vx, my, vy);
                // the draft's own term beside the others' sum; a NaN in the draft's place shows in xt
                const float et = has ? ex2_hw(vf_arg(xt, R, k)) : 0.f;
                p = VfRow{R, et + vx, mx, R == xt ? vx / et : vx, kNone};
                if (model) q = VfRow{Q, vy, my, 0.f, kNone};
                // (the maximum of a row with NaN is that of the others: its sum is NaN)
                const bool far = fabsf(mx) < INFINITY && !(fabsf((mx - R) * k) <= kFar) && R != mx;
                const bool qfar = model && fabsf(my) < INFINITY && !(fabsf((my - Q) * k) <= kFar) && Q != my;
                if (again || !(far || qfar)) break;
                if (far) R = mx;
                if (qfar) Q = my;
                in.drop();
                in = stream(n);
            }
        }
        if (!has || !vf_stays(t, u, xt, yt, p, q, model, greedy, k)) break;
        if (rank == 0 && tid == 0) {
            float lp;
            if (greedy) lp = vf_logp(xt, p.M, p.s1, ln2_k);
            else lp = p.R == xt ? -log1pf(p.s1) : vf_logp_of(xt, p, k);
            vf_put(a, static_cast<int64_t>(b) * (a.K + 1) + n, t, lp);
        }
    }
    in.drop();
    if (meet.failed()) p.S = NAN;  // (no result: token -1)
    vf_draw<DT, false>(a, b, n, p, q, has, model, usable, greedy, k, mem, meet, ring);
    meet.leave();
}

}  // namespace

// How the rows are cut: U vectors a lane (4, or fewer while that leaves warps
// without a part), and how many parts a row has wherever it starts.
constexpr int kStatsWarps = 152 * 3 * kWarps;  // three CTAs an SM
struct VfCut {
    int U;
    int64_t parts;
};
static VfCut vf_cut(int64_t rows, int64_t vocab, int dtype) {
    const int N = 16 / fp8_elem(dtype);
    VfCut c{};
    for (int U = 4; U >= 1; U >>= 1) {
        c.U = U;
        const int per = U * 32 * N;
        c.parts = (vocab + N - 1 + per - 1) / per;
        if (rows * c.parts >= kStatsWarps) break;
    }
    return c;
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
    constexpr int64_t kMost = (int64_t(1) << 31) - 65536;  // element indices are 32-bit
    if (p->n_drafts > kMaxDrafts || p->vocab > kMost || p->n_seqs > kMost / kCluster ||
        p->n_seqs * (p->n_drafts + 1) > kMost / vf_cut(p->n_seqs * (p->n_drafts + 1), p->vocab, p->dtype).parts)
        return CE_ERR_UNSUPPORTED;
    return CE_OK;
}

size_t vf_bytes(const ce_verify_params *p) {
    const int64_t rows = p->n_seqs * (p->n_drafts + 1);
    return static_cast<size_t>(vf_cut(rows, p->vocab, p->dtype).parts * (rows + p->n_seqs * p->n_drafts)) * sizeof(VfPart) + 256;
}

// the shared-memory limit is a per-device attribute of each kernel: set once per device
cudaError_t vf_allow_ring(const void *fn, int which, int dev) {
    static std::atomic<uint64_t> done[6];
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit && (done[which].load() & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
    if (e == cudaSuccess) done[which].fetch_or(bit);
    return e;
}

// Clusters of c CTAs that are resident at once (asked once a device): a cluster lies within one of the GPU's
// partitions, so that fewer fit than the SMs' room says.
int vf_resident(const void *fn, int which, int dev, int c) {
    constexpr int kDevs = 64;
    static std::atomic<int> known[6][kDevs][kCluster + 1];
    int n = 0;
    if (dev < kDevs && (n = known[which][dev][c].load()) > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(c);
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(c) * 64);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRing;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) n = 1;
    (void)cudaGetLastError();
    if (dev < kDevs) known[which][dev][c].store(n);
    return n;
}

// CTAs a sequence: as many as let all sequences run at once, two at least (64 sequences of 2 drafts, 128256 columns of
// bf16: 26 us with clusters of 6, 36 with clusters of 7, some of which wait for a second wave). The clusters that start
// while the statistics are still being formed want more room: half of it again (32 sequences of 6 drafts, 32000 bf16
// logits: 19 us with clusters of 5, 26 with clusters of 8, of which the device would hold 36).
int vf_cluster(const void *fn, int which, int dev, int64_t seqs) {
    int c = kCluster;
    while (c > 2 && vf_resident(fn, which, dev, c) < (which < 3 ? seqs : seqs * 3 / 2)) --c;
    return c;
}

// Whether the rows of all positions are read at once: where one position's rows, of all sequences and both models, are
// few enough that reading them takes less than the steps that a cluster a sequence takes from a position to the next. All
// at once / a cluster a sequence (us, 6 drafts): 48 sequences of 32000 bf16 logits (3 MB a position) 18 / 25, of 50257
// fp32 (10 MB) 32 / 32, of 128256 bf16 with a draft model (23 MB) 63 / 49; over 168 sizes of 1 to 200 sequences, 0 to 6
// drafts the rule's choice is 1% slower than the better one.
constexpr int64_t kAtOnce = int64_t(8) << 20;
bool vf_at_once(const VfArgs &a, int esz) {
    const int64_t rows = static_cast<int64_t>(a.B) * (a.K + 1 + (a.y ? a.K : 0));
    return rows * a.V * esz <= kAtOnce * (a.K + 1);
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
    const VfCut cut = vf_cut(rows, p->vocab, p->dtype);
    a.parts = static_cast<int>(cut.parts);
    a.px = reinterpret_cast<VfPart *>(ws);
    a.py = a.px + rows * a.parts;
    a.accepted = accepted;
    a.tokens = tokens;
    a.logp = logp;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    using Fn = void (*)(VfArgs);
#define CE_STATS(DT) {vf_stats_kernel<DT, 1>, vf_stats_kernel<DT, 2>, vf_stats_kernel<DT, 4>}
    static const Fn stats[3][3] = {CE_STATS(CE_DT_F32), CE_STATS(CE_DT_BF16), CE_STATS(CE_DT_F16)};
#undef CE_STATS
    static const Fn picks[3] = {vf_pick_kernel<CE_DT_F32>, vf_pick_kernel<CE_DT_BF16>, vf_pick_kernel<CE_DT_F16>};
    static const Fn seqs[3] = {vf_seq_kernel<CE_DT_F32>, vf_seq_kernel<CE_DT_BF16>, vf_seq_kernel<CE_DT_F16>};
    void *args[] = {&a};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRing;
    cfg.stream = s;
    cfg.attrs = at;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const bool seq = !vf_at_once(a, esz);
    const void *fn = reinterpret_cast<const void *>(seq ? seqs[p->dtype] : picks[p->dtype]);
    const int which = seq ? p->dtype : 3 + p->dtype;
    e = vf_allow_ring(fn, which, dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const int c = vf_cluster(fn, which, dev, p->n_seqs);
    at[0].val.clusterDim.x = static_cast<unsigned>(c);
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * c);
    cfg.numAttrs = seq ? 1 : 2;
    if (!seq) {
        const int64_t warps = rows * a.parts;
        e = cudaLaunchKernel(reinterpret_cast<const void *>(stats[p->dtype][cut.U >> 1]),
                             dim3(static_cast<unsigned>(warps < kStatsWarps ? (warps + kWarps - 1) / kWarps : kStatsWarps / kWarps)),
                             dim3(kThreads), args, 0, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    e = cudaLaunchKernelExC(&cfg, fn, args);
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

}  // extern "C"
