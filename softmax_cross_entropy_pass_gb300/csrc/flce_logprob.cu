// flce_logprob.cu -- token log-probabilities of a linear head and their
// gradient: the logits (hidden W^T + b) / T are formed tile by tile in tensor
// memory and never stored. The forward's product keeps the softmax statistics
// of every 128 columns (16 bytes a row), which one kernel merges
// per row. The backward forms the logits once more and its product's epilogue
// writes their gradient dZ (bf16), from which the two gradient products run.
#include <cmath>

#include "ce_kernels.h"
#include "flce.h"
#include "lp_device.cuh"

namespace ce {

// One warp per row: the row's tile states merged, its log-probability, entropy
// and statistics. `pos` (or NULL: the row itself): the row's place among the
// compacted rows, -1 for rows left out.
struct LpFinishArgs {
    const float4 *part;
    const float *xy;         // the rows' target logits, or NULL: in their part's w
    int tiles;
    int64_t n_rows, vocab;
    const void *target;
    int tgt32;
    int64_t ignore_index;
    const int *pos;
    float k, inv_t;
    float *logp, *entropy;
    float4 *stats;
};
template <bool ENT>
__global__ void __launch_bounds__(256) flce_logprob_finish_kernel(LpFinishArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < a.n_rows;
         row += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t t = load_target(a.target, a.tgt32, row);
        if (!target_valid(t, a.ignore_index, a.vocab)) {
            if (lane == 0) {
                const float none = t == a.ignore_index ? 0.f : NAN;
                if (a.logp) a.logp[row] = none;
                if (a.entropy) a.entropy[row] = none;
                if (a.stats) a.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            continue;
        }
        const float4 *pp = a.part + (a.pos ? static_cast<int64_t>(__ldg(a.pos + row)) : row) * a.tiles;
        // the maximum first, so that the parts' sums are moved to it independently
        float M = -INFINITY;
#pragma unroll 4
        for (int j = lane; j < a.tiles; j += 32) M = fmaxf(M, __ldg(&pp[j].x));
        LpState st{M, 0.f, 0.f};
#pragma unroll 4
        for (int j = lane; j < a.tiles; j += 32) {
            const float4 q = __ldg(pp + j);
            LpState o{q.x, q.y, q.z};
            if (M != -INFINITY) lp_rebase<ENT>(o, M, a.k);
            st.s += o.s;
            if (ENT) st.u += o.u;
        }
        st = lp_warp_merge<ENT>(st, a.k);
        if (lane != 0) continue;
        const float xy = a.xy ? __ldg(a.xy + row) : __ldg(&pp[t / kLpTileN].w);
        float4 stats = lp_row_stats(st, xy, a.k);
        const LpRow r = lp_row(stats, a.k, a.inv_t);
        if (!ENT) stats.w = NAN;
        if (a.logp) a.logp[row] = r.logp;
        if (ENT && a.entropy) a.entropy[row] = r.entropy;
        if (a.stats) a.stats[row] = stats;
    }
}

// The gradient scalars of the compacted rows.
__global__ void __launch_bounds__(256) flce_logprob_rows_kernel(const float4 *stats, const float *g_logp,
                                                                const float *g_entropy, const int *idx,
                                                                const int64_t *tgt, const int *count, float k,
                                                                float inv_t, LpMapRow *rows) {
    const int n = __ldg(count);
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
        const int row = __ldg(idx + i);
        const float4 st = __ldg(stats + row);
        const LpRow r = lp_row(st, k, inv_t);
        const LpGrad g = lp_grad(st, r, inv_t, g_logp ? __ldg(g_logp + row) : 0.f, g_entropy ? __ldg(g_entropy + row) : 0.f);
        rows[i] = LpMapRow{g.M, g.neg_log2d, g.A, g.B, g.dy, static_cast<int>(tgt[i]), 0.f, 0.f};
    }
}

// grad_bias (+)= the column sums of dZ: a block takes 256 columns, 8 to a lane,
// its 16 warps every 16th row each, and adds the warps up in order. Bound by
// reading dZ once.
constexpr int kColsumWarps = 16;
__global__ void __launch_bounds__(kColsumWarps * 32) flce_logprob_colsum_kernel(const uint4 *dz, int64_t ld8, int rows,
                                                                                int64_t V, float *gb, int accumulate,
                                                                                const int *count, int off) {
    __shared__ float sh[kColsumWarps][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t v = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // this lane's vector of a row
    int n = __ldg(count) - off;
    n = n < rows ? n : rows;
    float s[8] = {};
    if (v * 8 < V) {
        const uint4 *p = dz + v;
#pragma unroll 4
        for (int r = warp; r < n; r += kColsumWarps) {
            float x[8];
            Fmt<CE_DT_BF16>::unpack(__ldg(p + r * ld8), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += x[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[warp][lane * 8 + e] = s[e];
    __syncthreads();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (threadIdx.x < 256 && c < V) {
        float t = 0.f;
        for (int w = 0; w < kColsumWarps; ++w) t += sh[w][threadIdx.x];
        gb[c] = accumulate ? gb[c] + t : t;
    }
}

}  // namespace ce

using namespace ce;

namespace {

// up to one row tile of the product there is nothing to skip: no compaction in the forward
constexpr int64_t kCompactAbove = 128;

bool on(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up(size_t a, size_t b) { return (a + b - 1) / b * b; }

// Split count of grad_hidden = dZ W: with few output tiles (128 x 256) as many
// parts of K = V as give every SM of a full GB300 a tile (GB300, 16 x 4096 x
// 128256, 16 tiles: the whole backward 662 us with 4 parts, 618 with 9),
// otherwise the fused-linear path's rule. A function of the sizes alone.
int lp_dh_splits(int64_t chunk, int64_t H, int64_t V) {
    const int64_t tiles = ((chunk + 127) / 128) * ((H + 255) / 256);
    const int least = flce_dh_splits(chunk, H, V);
    const int want = static_cast<int>(152 / tiles);
    return want > least ? gemm_fit_ksplit(static_cast<int>(V), want) : least;
}

struct LpLayout {
    size_t idx, pos, cnt, tgt, hc;       // compaction
    size_t part, xy;                     // forward
    size_t rows, dz, dh;                 // backward
    size_t total;
    int64_t ldd;
    int tiles, splits;
};
// ctl (256 bytes: status, then unused) | compaction | forward or backward buffers
LpLayout lp_layout(int64_t n, int64_t V, int64_t H, int64_t chunk, bool backward) {
    LpLayout L{};
    size_t o = 256;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = up(o + bytes, 1024);
        return at;
    };
    if (backward || n > kCompactAbove) {
        L.idx = take(n * 4);
        L.pos = take(n * 4);
        L.cnt = take(4);
        L.tgt = take(n * 8);
        L.hc = take(static_cast<size_t>(n) * H * 2);
    }
    L.tiles = static_cast<int>((V + kGemmTileN - 1) / kGemmTileN) * (kGemmTileN / kLpTileN);
    if (!backward) {
        if (n <= kFewMaxRows) {
            L.tiles = flce_few_parts(V);
            L.xy = take(n * 4);
        }
        L.part = take(static_cast<size_t>(n) * L.tiles * 16);
    } else {
        L.ldd = (V + 15) / 16 * 16;  // rows on 32-byte boundaries
        L.splits = lp_dh_splits(chunk, H, V);
        L.rows = take(n * sizeof(LpMapRow));
        L.dz = take(static_cast<size_t>(chunk) * L.ldd * 2);
        L.dh = take(L.splits > 1 ? static_cast<size_t>(L.splits) * chunk * H * 4 : 0);
    }
    L.total = o;
    return L;
}

ce_status check(const ce_params *p, int64_t H, float temperature) {
    if (!p || p->n_rows < 0 || p->vocab < 1 || H < 1) return CE_ERR_INVALID_ARG;
    if (p->target_is_int32 != 0 && p->target_is_int32 != 1) return CE_ERR_INVALID_ARG;
    if (p->variant != 0 || p->reserved != 0) return CE_ERR_INVALID_ARG;
    if (!(temperature >= 1e-4f && temperature <= 1e4f)) return CE_ERR_INVALID_ARG;
    if (p->class_weight || p->label_smoothing != 0.f || p->softcap != 0.f || p->z_loss != 0.f || p->accuracy)
        return CE_ERR_UNSUPPORTED;
    if (p->dtype != CE_DT_BF16 || (H % 8)) return CE_ERR_UNSUPPORTED;
    if (p->n_rows > INT32_MAX || p->vocab > INT32_MAX || H > INT32_MAX) return CE_ERR_UNSUPPORTED;
    return CE_OK;
}

int64_t clamp_chunk(int64_t chunk, int64_t n) { return chunk < n ? chunk : (n > 0 ? n : 1); }

float base2(float temperature) { return static_cast<float>(1.4426950408889634 / static_cast<double>(temperature)); }

}  // namespace

extern "C" {

ce_status flce_token_logprob_workspace_size(const ce_params *p, int64_t hidden_dim, int64_t chunk_rows, size_t *bytes) {
    ce_status st = check(p, hidden_dim, 1.f);
    if (st != CE_OK) return st;
    if (!bytes || chunk_rows < 0) return CE_ERR_INVALID_ARG;
    *bytes = lp_layout(p->n_rows, p->vocab, hidden_dim, clamp_chunk(chunk_rows, p->n_rows), chunk_rows > 0).total;
    return CE_OK;
}

ce_status flce_token_logprob(const ce_params *p, int64_t H, float temperature, const void *hidden, const void *weight,
                             const float *bias, const void *target, float *logp, float *entropy, float *stats, void *ws,
                             size_t ws_size, void *stream) {
    ce_status st = check(p, H, temperature);
    if (st != CE_OK) return st;
    const int64_t n = p->n_rows, V = p->vocab;
    if (n == 0) return CE_OK;
    if (!hidden || !weight || !target || (!logp && !entropy && !stats)) return CE_ERR_INVALID_ARG;
    if (!on(target, p->target_is_int32 ? 4 : 8)) return CE_ERR_INVALID_ARG;
    if (!on(hidden, 16) || !on(weight, 16) || !on(bias, 16) || !on(logp, 4) || !on(entropy, 4) || !on(stats, 16))
        return CE_ERR_INVALID_ARG;
    const LpLayout L = lp_layout(n, V, H, 0, false);
    if (!ws || !on(ws, 256) || ws_size < L.total) return CE_ERR_WORKSPACE;
    char *w = reinterpret_cast<char *>(ws);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    WsCtl *ctl = reinterpret_cast<WsCtl *>(ws);
    const bool few = n <= kFewMaxRows, compact = n > kCompactAbove;
    cudaError_t e = few ? cudaSuccess : cudaMemsetAsync(ws, 0, 256, s);  // the few-rows kernel clears its status word itself
    if (e != cudaSuccess) return cuda_fail(e);
    int *idx = reinterpret_cast<int *>(w + L.idx), *pos = reinterpret_cast<int *>(w + L.pos);
    int *cnt = reinterpret_cast<int *>(w + L.cnt);
    int64_t *tgt = reinterpret_cast<int64_t *>(w + L.tgt);
    if (compact) {
        e = flce_compact(target, p->target_is_int32, n, V, p->ignore_index, hidden, H,
                         CompactBufs{idx, pos, cnt, tgt, w + L.hc}, nullptr, nullptr, nullptr, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    GemmLp lp{};
    lp.part = reinterpret_cast<float4 *>(w + L.part);
    lp.target = compact ? static_cast<const void *>(tgt) : target;
    lp.tgt32 = compact ? 0 : p->target_is_int32;
    lp.ignore_index = p->ignore_index;
    lp.k = base2(temperature);
    lp.entropy = entropy != nullptr;
    if (few) {
        e = flce_few(static_cast<int>(n), static_cast<int>(V), static_cast<int>(H), hidden, weight, bias, target,
                     p->target_is_int32, p->ignore_index, lp.k, lp.entropy, lp.part, reinterpret_cast<float *>(w + L.xy),
                     &ctl->status, s);
    } else {
        const GemmDyn rows{cnt, 0, 0, nullptr};
        e = gemm_bf16(static_cast<int>(n), static_cast<int>(V), static_cast<int>(H), compact ? w + L.hc : hidden, H, 0,
                      weight, H, 0, CE_GEMM_F32_STORE, nullptr, V, bias, &ctl->status, s, compact ? &rows : nullptr, nullptr,
                      1, 0, GEMM_AUTO, &lp);
    }
    if (e != cudaSuccess) return cuda_fail(e);
    LpFinishArgs a{};
    a.part = lp.part;
    a.xy = few ? reinterpret_cast<float *>(w + L.xy) : nullptr;
    a.tiles = L.tiles;
    a.n_rows = n;
    a.vocab = V;
    a.target = target;
    a.tgt32 = p->target_is_int32;
    a.ignore_index = p->ignore_index;
    a.pos = compact ? pos : nullptr;
    a.k = lp.k;
    a.inv_t = 1.f / temperature;
    a.logp = logp;
    a.entropy = entropy;
    a.stats = reinterpret_cast<float4 *>(stats);
    void *args[] = {&a};
    const int64_t blocks = (n + 7) / 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < 2048 ? blocks : 2048));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelExC(&cfg,
                            entropy ? reinterpret_cast<const void *>(&flce_logprob_finish_kernel<true>)
                                    : reinterpret_cast<const void *>(&flce_logprob_finish_kernel<false>),
                            args);
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

ce_status flce_token_logprob_backward(const ce_params *p, int64_t H, float temperature, const void *hidden,
                                      const void *weight, const float *bias, const void *target, const float *stats,
                                      const float *grad_logp, const float *grad_entropy, void *grad_hidden,
                                      void *grad_weight, int32_t grad_weight_dtype, float *grad_bias, int64_t chunk_rows,
                                      void *ws, size_t ws_size, void *stream) {
    ce_status st = check(p, H, temperature);
    if (st != CE_OK) return st;
    if (chunk_rows < 1 || (grad_weight_dtype != CE_DT_F32 && grad_weight_dtype != CE_DT_BF16)) return CE_ERR_INVALID_ARG;
    const int64_t n = p->n_rows, V = p->vocab, C = clamp_chunk(chunk_rows, n);
    const bool wide = grad_weight_dtype == CE_DT_F32;
    if (!wide && C < n) return CE_ERR_UNSUPPORTED;  // several chunks add up in fp32
    if (!grad_weight || !on(grad_weight, 16) || (grad_bias && !on(grad_bias, 4)) || !on(bias, 16)) return CE_ERR_INVALID_ARG;
    if (n > 0 && (!hidden || !weight || !target || !stats || !grad_hidden || (!grad_logp && !grad_entropy)))
        return CE_ERR_INVALID_ARG;
    if (!on(target, p->target_is_int32 ? 4 : 8)) return CE_ERR_INVALID_ARG;
    if (!on(hidden, 16) || !on(weight, 16) || !on(grad_hidden, 16) || !on(stats, 16) || !on(grad_logp, 4) ||
        !on(grad_entropy, 4))
        return CE_ERR_INVALID_ARG;
    const LpLayout L = lp_layout(n, V, H, C, true);
    if (!ws || !on(ws, 256) || ws_size < L.total) return CE_ERR_WORKSPACE;
    char *w = reinterpret_cast<char *>(ws);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    WsCtl *ctl = reinterpret_cast<WsCtl *>(ws);
    cudaError_t e = cudaMemsetAsync(ws, 0, 256, s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (n == 0) {
        e = cudaMemsetAsync(grad_weight, 0, static_cast<size_t>(V) * H * (wide ? 4 : 2), s);
        if (e == cudaSuccess && grad_bias) e = cudaMemsetAsync(grad_bias, 0, static_cast<size_t>(V) * 4, s);
        return e == cudaSuccess ? CE_OK : cuda_fail(e);
    }
    int *idx = reinterpret_cast<int *>(w + L.idx), *pos = reinterpret_cast<int *>(w + L.pos);
    int *cnt = reinterpret_cast<int *>(w + L.cnt);
    int64_t *tgt = reinterpret_cast<int64_t *>(w + L.tgt);
    LpMapRow *rows = reinterpret_cast<LpMapRow *>(w + L.rows);
    e = flce_compact(target, p->target_is_int32, n, V, p->ignore_index, hidden, H, CompactBufs{idx, pos, cnt, tgt, w + L.hc},
                     grad_hidden, nullptr, nullptr, s);
    if (e != cudaSuccess) return cuda_fail(e);
    float k = base2(temperature), inv_t = 1.f / temperature;
    {
        const float4 *stp = reinterpret_cast<const float4 *>(stats);
        const int *ci = idx, *cc = cnt;
        const int64_t *ct = tgt;
        void *args[] = {&stp, &grad_logp, &grad_entropy, &ci, &ct, &cc, &k, &inv_t, &rows};
        const int64_t blocks = (n + 255) / 256;
        e = cudaLaunchKernel(reinterpret_cast<const void *>(&flce_logprob_rows_kernel),
                             dim3(static_cast<unsigned>(blocks < 1024 ? blocks : 1024)), dim3(256), args, 0, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    void *dz = w + L.dz;
    for (int64_t r0 = 0; r0 < n; r0 += C) {
        const int64_t c = n - r0 < C ? n - r0 : C;
        const char *h_c = w + L.hc + r0 * H * 2;
        const GemmDyn rows_m{cnt, static_cast<int>(r0), 0, nullptr}, rows_k{cnt, static_cast<int>(r0), 1, nullptr};
        GemmLp lp{};
        lp.rows = rows + r0;
        lp.k = k;
        lp.entropy = grad_entropy != nullptr;
        e = gemm_bf16(static_cast<int>(c), static_cast<int>(V), static_cast<int>(H), h_c, H, 0, weight, H, 0,
                      CE_GEMM_BF16_STORE, dz, L.ldd, bias, &ctl->status, s, &rows_m, nullptr, 1, 0, GEMM_AUTO, &lp);
        if (e != cudaSuccess) return cuda_fail(e);
        e = flce_grad_hidden(c, H, V, dz, L.ldd, weight, L.splits, reinterpret_cast<float *>(w + L.dh), cnt, r0, idx + r0,
                             grad_hidden, &ctl->status, s);
        if (e != cudaSuccess) return cuda_fail(e);
        const int out_kind = wide ? (r0 == 0 ? CE_GEMM_F32_STORE : CE_GEMM_F32_ACCUM) : CE_GEMM_BF16_STORE;
        e = gemm_bf16(static_cast<int>(V), static_cast<int>(H), static_cast<int>(c), dz, L.ldd, 1, h_c, H, 1, out_kind,
                      grad_weight, H, nullptr, &ctl->status, s, &rows_k);
        if (e != cudaSuccess) return cuda_fail(e);
        if (grad_bias) {
            const uint4 *dz8 = reinterpret_cast<const uint4 *>(dz);
            int64_t ld8 = L.ldd / 8, v = V;
            int nr = static_cast<int>(c), accumulate = r0 == 0 ? 0 : 1, off = static_cast<int>(r0);
            const int *cc = cnt;
            void *args[] = {&dz8, &ld8, &nr, &v, &grad_bias, &accumulate, &cc, &off};
            e = cudaLaunchKernel(reinterpret_cast<const void *>(&flce_logprob_colsum_kernel),
                                 dim3(static_cast<unsigned>((V + 255) / 256)), dim3(kColsumWarps * 32), args, 0, s);
            if (e != cudaSuccess) return cuda_fail(e);
        }
    }
    return CE_OK;
}

}  // extern "C"
