// lp_grad.cu -- the gradient of token log-probabilities from saved row
// statistics, the normalisers of the policy loss, and the sequence-level
// kernels of the preference loss.
#include "ce_host.h"
#include "lp_device.cuh"
#include "lp_kernels.h"

namespace ce {

// ------------------------------------------------------------------ policy normalisers
constexpr int kLpPrepThreads = 1024;

// Up to kPrepParts blocks, each over its share of the rows: the sum of the
// weights of those that take part (fp64, fixed order) and the target check, to
// the control block; the row kernel adds the blocks up. It may start at once
// and waits for this kernel where it reads the sums. Eight rows in flight a
// thread: with one, 60000 rows took longer here than their 1000-column rows.
__global__ void __launch_bounds__(kLpPrepThreads) lp_prep_kernel(LpArgs a) {
    pdl_launch_dependents();
    __shared__ double sh_w[kLpPrepThreads / 32];
    constexpr int U = 8;
    const int tid = threadIdx.x;
    double w = 0.0;
    bool bad = false;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kLpPrepThreads + tid; base < a.n_rows;
         base += static_cast<int64_t>(U) * gridDim.x * kLpPrepThreads) {
        int64_t t[U];
        float wt[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t r = base + static_cast<int64_t>(i) * gridDim.x * kLpPrepThreads;
            t[i] = r < a.n_rows ? load_target(a.target, a.tgt32, r) : a.ignore_index;
            wt[i] = a.row_weight && r < a.n_rows ? __ldg(a.row_weight + r) : 1.f;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (target_valid(t[i], a.ignore_index, a.vocab)) w += static_cast<double>(wt[i]);
            else if (t[i] != a.ignore_index) bad = true;
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
    if ((tid & 31) == 0) sh_w[tid >> 5] = w;
    const int any_bad = __syncthreads_or(bad);
    static_assert(kLpPrepThreads == 1024, "one warp adds the warps up");
    double sum = tid < 32 ? sh_w[tid] : 0.0;
    if (tid < 32) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
    if (tid == 0) {
        a.ctl->prep_part[blockIdx.x][0] = sum;
        a.ctl->prep_bad[blockIdx.x] = any_bad ? 1u : 0u;
        if (blockIdx.x == 0) {
            a.ctl->done = 0u;
            // without rows no row kernel follows to set the bits
            a.ctl->status = a.n_rows == 0 && a.reduction == CE_RED_MEAN ? CE_FLAG_NO_VALID_ROWS : 0u;
        }
    }
}

// ------------------------------------------------------------------ gradient from statistics
constexpr int kLpGradThreads = 256;
constexpr int kPairThreads = 256;
// A row goes to one item in equal parts of at most 128 KB; with few rows in as
// many parts as give every resident block one, of at least 8 KB (GB300, both
// gradients: 8192 x 128256 bf16 645 us, with parts of 64 KB 655 and of 32 KB
// 815; 8 x 128256 8 us against 17 with 128 KB parts).
constexpr int64_t kLpGradMaxBytes = 131072, kLpGradMinBytes = 8192;
constexpr int kLpGradCtasPerSm = 5;

// fixed-order block sum of two doubles, to every thread
__device__ inline void block_sum2(double &x, double &y, double (&sh)[kPairThreads / 32][2]) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, off);
        y += __shfl_xor_sync(0xffffffffu, y, off);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        sh[threadIdx.x >> 5][0] = x;
        sh[threadIdx.x >> 5][1] = y;
    }
    __syncthreads();
    x = y = 0.0;
    for (int i = 0; i < kPairThreads / 32; ++i) {
        x += sh[i][0];
        y += sh[i][1];
    }
}

// The batch's part of a preference coefficient: grad_output (for reduction
// none it is in the coefficients already) over the number of live pairs.
__device__ inline float lp_pair_scale(const LpArgs &a) {
    if (a.reduction == CE_RED_NONE) return 1.f;
    const float up = a.grad_output ? __ldg(a.grad_output) : 1.f;
    if (a.reduction != CE_RED_MEAN) return up;
    const unsigned live = __ldcg(&a.ctl->n_correct);
    return live ? up / static_cast<float>(live) : 0.f;
}

// The batch loss from the pair losses, by one block (fixed order, fp64).
__device__ inline void lp_pair_loss(const LpArgs &a) {
    __shared__ double sh[kPairThreads / 32][2];
    const unsigned live = __ldcg(&a.ctl->n_correct);
    if (a.reduction != CE_RED_NONE) {
        double s = 0.0, none = 0.0;
        for (int64_t p = threadIdx.x; p < a.n_seqs / 2; p += kPairThreads) s += __ldcg(a.part + p);
        block_sum2(s, none, sh);
        if (a.reduction == CE_RED_MEAN && live) s /= static_cast<double>(live);
        if (threadIdx.x == 0) a.loss[0] = static_cast<float>(s);
    }
    if (threadIdx.x == 0 && live == 0u && !(__ldcg(&a.ctl->status) & CE_FLAG_BAD_OFFSETS))
        atomicOr(&a.ctl->status, CE_FLAG_NO_VALID_ROWS);
}
static_assert(kPairThreads == kLpGradThreads, "the gradient kernel's first block forms the batch loss");

// The logits once more, the gradient written: a map over (row, part) items, last rows first, so that what the forward read last is still in L2.
// Bound by HBM; 4 vectors in flight per thread.
template <int DT, bool ENT>
__global__ void __launch_bounds__(kLpGradThreads, kLpGradCtasPerSm) lp_grad_kernel(LpArgs a, int64_t parts, int64_t span) {
    using F = Fmt<DT>;
    constexpr int KB = F::kBytes;
    const int tid = threadIdx.x;
    float batch = 1.f;  // preference: what every row's coefficient is still to be multiplied by
    if (a.row_coef) {
        pdl_wait();
        batch = lp_pair_scale(a);
        if (blockIdx.x == 0) lp_pair_loss(a);
    }
    for (int64_t i = blockIdx.x; i < a.n_rows * parts; i += gridDim.x) {
        const int64_t row = a.n_rows - 1 - i / parts, c0 = (i % parts) * span;
        const int64_t c1 = c0 + span < a.vocab ? c0 + span : a.vocab;
        char *grow = reinterpret_cast<char *>(a.grad) + row * a.ld_grad * KB;
        const int64_t t = load_target(a.target, a.tgt32, row);
        const bool valid = target_valid(t, a.ignore_index, a.vocab);
        const float g = valid && a.g_logp ? __ldg(a.g_logp + row) * batch : 0.f;
        const float h = valid && ENT && a.g_entropy ? __ldg(a.g_entropy + row) : 0.f;
        if (!valid || (a.row_coef && g == 0.f)) {
            lp_zero_span<DT>(grow, c0, c1, tid, kLpGradThreads);
            continue;
        }
        const float4 st = __ldg(a.stats + row);
        const LpRow r = lp_row(st, a.k, a.inv_t);
        const LpGrad lg = lp_grad(st, r, a.inv_t, g, h);
        lp_grad_span<DT, ENT>(reinterpret_cast<const char *>(a.x) + row * a.ld * KB, grow, c0, c1, static_cast<int>(t), lg,
                              a.k, tid, kLpGradThreads);
    }
}

// ------------------------------------------------------------------ preference pairs
// One block per pair (p: sequences p and P + p of the 2 P): their log
// probability sums in fp64, the pair's loss and the coefficient dL/dlogp of
// each of their rows, written over the row's log-probability (rows whose
// target takes no part already hold 0). The divisor of the mean (pairs with a
// valid target on both sides, counted here) and grad_output are left to the
// gradient kernel (lp_pair_scale).
// Offsets that fall, or leave [0, n_rows], make the whole batch void: loss
// NaN, gradient 0, a status bit. Every block checks all of them itself.
__global__ void __launch_bounds__(kPairThreads) lp_pair_kernel(PairArgs a) {
    constexpr int HALF = kPairThreads / 2, W = HALF / 32;
    __shared__ double sh[2][W][2];  // per side and warp: log-probabilities, valid targets
    const int tid = threadIdx.x;
    const int side_t = tid / HALF, ht = tid - side_t * HALF;  // half of the block a sequence
    bool bad = false;
    for (int64_t j = tid; j < 2 * a.n_pairs; j += kPairThreads) {
        const int64_t b = load_target(a.offsets, a.off32, j), e = load_target(a.offsets, a.off32, j + 1);
        if (b < 0 || e < b || e > a.n_rows) bad = true;
    }
    const bool void_batch = __syncthreads_or(bad);
    pdl_wait();  // the log-probabilities
    if (void_batch) {
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPairThreads + tid; i < a.n_rows;
             i += static_cast<int64_t>(gridDim.x) * kPairThreads)
            a.row[i] = 0.f;
        for (int64_t p = static_cast<int64_t>(blockIdx.x) * kPairThreads + tid; p < a.n_pairs;
             p += static_cast<int64_t>(gridDim.x) * kPairThreads) {
            a.pair_loss[p] = NAN;
            if (a.reduction == CE_RED_NONE) a.loss[p] = NAN;
            if (a.seq_logp) a.seq_logp[p] = a.seq_logp[a.n_pairs + p] = NAN;
        }
        if (blockIdx.x == 0 && tid == 0) atomicOr(&a.ctl->status, CE_FLAG_BAD_OFFSETS);
        return;
    }
    for (int64_t p = blockIdx.x; p < a.n_pairs; p += gridDim.x) {
        const int64_t seq = p + side_t * a.n_pairs;
        const int64_t b = load_target(a.offsets, a.off32, seq), e = load_target(a.offsets, a.off32, seq + 1);
        bool oob = false;
        double s = 0.0, n = 0.0;
        for (int64_t i = b + ht; i < e; i += HALF) {
            const int64_t t = load_target(a.target, a.tgt32, i);
            const float lp = a.row[i];  // 0 where the target takes no part
            if (target_valid(t, a.ignore_index, a.vocab)) {
                s += static_cast<double>(lp);
                n += 1.0;
            } else if (t != a.ignore_index) {
                oob = true;
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, off);
            n += __shfl_xor_sync(0xffffffffu, n, off);
        }
        if ((tid & 31) == 0) {
            sh[side_t][ht / 32][0] = s;
            sh[side_t][ht / 32][1] = n;
        }
        if (__syncthreads_or(oob) && tid == 0) atomicOr(&a.ctl->status, CE_FLAG_TARGET_OUT_OF_RANGE);
        double sum[2] = {}, cnt[2] = {};
        for (int side = 0; side < 2; ++side)
            for (int w = 0; w < W; ++w) {
                sum[side] += sh[side][w][0];
                cnt[side] += sh[side][w][1];
            }
        const bool live = cnt[0] > 0.0 && cnt[1] > 0.0;
        double v[2];
        for (int side = 0; side < 2; ++side) v[side] = a.normalize && cnt[side] > 0.0 ? sum[side] / cnt[side] : sum[side];
        // h in fp64 (a difference of long sums), what follows from it in fp32 (every
        // thread forms it, and fp64 exponentials are slow here)
        float loss = 0.f, slope = 0.f;
        if (live) {
            double h = v[0] - v[1];
            if (a.ref) h -= static_cast<double>(__ldg(a.ref + p)) - static_cast<double>(__ldg(a.ref + a.n_pairs + p));
            const float be = a.beta, z = static_cast<float>(static_cast<double>(be) * h), eps = a.smoothing;
            if (a.kind == CE_PREF_SIGMOID) {
                // softplus(+-z) and the logistic function through e^-|z|, which cannot overflow
                const float q = expf(-fabsf(z)), l = log1pf(q), inv = 1.f / (1.f + q);
                const float sp_pos = (z > 0.f ? z : 0.f) + l, sp_neg = (z > 0.f ? 0.f : -z) + l;
                const float s_pos = z > 0.f ? inv : q * inv, s_neg = z > 0.f ? q * inv : inv;
                loss = (1.f - eps) * sp_neg;
                if (eps != 0.f) loss += eps * sp_pos;  // sp_pos is inf where the rejected side has probability 0
                slope = be * (eps * s_pos - (1.f - eps) * s_neg);
            } else if (a.kind == CE_PREF_HINGE) {
                loss = z < 1.f ? 1.f - z : (z >= 1.f ? 0.f : z);  // NaN stays
                slope = z < 1.f ? -be : (z >= 1.f ? 0.f : z);
            } else {
                const float m = static_cast<float>(h - 0.5 / static_cast<double>(be));
                loss = m * m;
                slope = 2.f * m;
            }
        }
        if (tid == 0) {
            a.pair_loss[p] = loss;
            if (a.reduction == CE_RED_NONE) a.loss[p] = loss;
            if (a.seq_logp) {
                a.seq_logp[p] = static_cast<float>(v[0]);
                a.seq_logp[a.n_pairs + p] = static_cast<float>(v[1]);
            }
            if (live) atomicAdd(&a.ctl->n_correct, 1u);  // integers: the order does not matter
        }
        if (a.reduction == CE_RED_NONE && a.grad_output) slope *= __ldg(a.grad_output + p);
        float c = side_t == 0 ? slope : -slope;
        if (a.normalize && live) c /= static_cast<float>(cnt[side_t]);
        for (int64_t i = b + ht; i < e; i += HALF) {
            const int64_t t = load_target(a.target, a.tgt32, i);
            a.row[i] = target_valid(t, a.ignore_index, a.vocab) ? c : 0.f;
        }
        __syncthreads();  // the sums are used up
    }
}

// ------------------------------------------------------------------ launches
static cudaLaunchConfig_t dep_config(int64_t grid, int threads, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid < 1 ? 1 : grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    return cfg;
}
// may start before the kernel in front of it has ended (it waits inside)
static cudaLaunchAttribute dep_attribute() {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    return at;
}

cudaError_t launch_lp_prep(LpArgs &a, cudaStream_t s) {
    const int64_t want = (a.n_rows + kLpPrepThreads - 1) / kLpPrepThreads;
    a.n_prep = static_cast<int>(want < 1 ? 1 : (want < kPrepParts ? want : kPrepParts));
    cudaLaunchConfig_t cfg = dep_config(a.n_prep, kLpPrepThreads, s);
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&lp_prep_kernel), args);
}

template <int DT>
static const void *grad_fn(bool ent) {
    return ent ? reinterpret_cast<const void *>(&lp_grad_kernel<DT, true>)
               : reinterpret_cast<const void *>(&lp_grad_kernel<DT, false>);
}

cudaError_t launch_lp_grad(const LpArgs &a0, int dtype, bool entropy, bool dependent, cudaStream_t s) {
    LpArgs a = a0;
    const void *fn = dtype == CE_DT_F32 ? grad_fn<CE_DT_F32>(entropy)
                   : dtype == CE_DT_BF16 ? grad_fn<CE_DT_BF16>(entropy) : grad_fn<CE_DT_F16>(entropy);
    const int64_t esz = dtype == CE_DT_F32 ? 4 : 2, row = a.vocab * esz;
    int64_t want = a.n_rows > 0 ? (device_sms() * kLpGradCtasPerSm + a.n_rows - 1) / a.n_rows : 1;
    if (want > row / kLpGradMinBytes) want = row / kLpGradMinBytes;
    const int64_t least = (row + kLpGradMaxBytes - 1) / kLpGradMaxBytes;
    int64_t parts = want > least ? want : least;
    int64_t span = ((row + parts - 1) / parts + 127) / 128 * 128 / esz;  // columns of a part
    const int64_t items = a.n_rows * parts, cap = int64_t(1) << 20;
    cudaLaunchConfig_t cfg = dep_config(items < cap ? items : cap, kLpGradThreads, s);
    cudaLaunchAttribute at = dep_attribute();
    cfg.attrs = &at;
    cfg.numAttrs = dependent ? 1 : 0;
    void *args[] = {&a, &parts, &span};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

cudaError_t launch_lp_pairs(const PairArgs &a0, cudaStream_t s) {
    PairArgs a = a0;
    cudaLaunchConfig_t cfg = dep_config(a.n_pairs < 512 ? a.n_pairs : 512, kPairThreads, s);
    cudaLaunchAttribute at = dep_attribute();
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&lp_pair_kernel), args);
}

}  // namespace ce
