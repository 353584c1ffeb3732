// flce.h -- internal declarations of the tensor-core GEMM used by the
// fused-linear cross-entropy.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ce {

// D[M,N] (op)= A[M,K] B[K,N] with bf16 operands and fp32 accumulation.
// a_mn / b_mn: operand stored MN-major (A as [K, M], B as [K, N]) instead of
// K-major (A as [M, K], B as [N, K]). out_kind: 0 fp32 store (+ bias[N]),
// 1 fp32 accumulate, 2 bf16 store.
// `dyn` (optional) makes M or K a device-side value: the kernel uses
// clamp(*count - off, 0, M or K) (dim 0: M, 1: K), and `row_map` sends output
// row r to row row_map[r]. The sizes passed here are then upper bounds.
struct GemmDyn {
    const int *count;
    int off;
    int dim;
    const int *row_map;
};

// `ksplit` > 1 (fp32 store only, static K) computes every tile as ksplit
// partial products over consecutive K ranges, partial p stored at
// out + p * split_stride.
// `stats` (optional, fp32 store only) also writes, for every output row and
// 256-column tile, the tile's softmax state {max, exp-sum without the
// row's target column, smoothing sum, weight sum} to part[row * tiles + t]
// (tiles = ceil(N / 256)); smooth_mode 0: no smoothing sums, 1: plain sum
// of the logits, 2: class-weighted (weight[N]).
struct GemmStats {
    float4 *part;
    const void *target;
    int tgt32;
    int64_t ignore_index;
    int smooth_mode;
    const float *weight;
    float cap;      // softcap c > 0: the stored logits and the states are those of c tanh(x / c)
    float2 *pam;    // or NULL: per row and tile {raw maximum, its first column} (token accuracy)
};
constexpr int kGemmTileN = 256;

// Log-probability epilogues of the logits product (the product itself is not
// stored): `part` set: per output row and kLpTileN columns the state {max m,
// s = sum 2^a without the row's target column, u = sum 2^a a (with entropy),
// the target logit where they hold it} at part[row * 2 ceil(N / 256) + column /
// kLpTileN], a = (x - m) k, x = product + bias. `rows` set: the gradient of every logit, rounded once to bf16 into
// the output, from the row's scalars; rows from M up to the next multiple of
// 64 (within the launch's static M) become zeros.
constexpr int kLpTileN = 128;
struct LpMapRow {
    float m, neg_log2d, A, B;  // (A + B log2 p) p off the target, p = 2^((x - m) k + neg_log2d)
    float dy;                  // at the target column y
    int y;
    float pad0, pad1;
};
static_assert(sizeof(LpMapRow) == 32, "two 16-byte loads per row");
struct GemmLp {
    float4 *part;
    const void *target;
    int tgt32;
    int64_t ignore_index;
    const LpMapRow *rows;
    float k;
    int entropy;
};

// `mode`: GEMM_AUTO (CTA pairs on 256 x 256 tiles when M and N both span at
// least two such tiles, else one CTA per 128 x 256 tile), GEMM_ONE_CTA,
// GEMM_PAIR.
enum { GEMM_AUTO = 0, GEMM_ONE_CTA = 1, GEMM_PAIR = 2 };

cudaError_t gemm_bf16(int M, int N, int K, const void *A, int64_t lda, int a_mn, const void *B,
                      int64_t ldb, int b_mn, int out_kind, void *out, int64_t ldo, const float *bias,
                      unsigned int *status, cudaStream_t s, const GemmDyn *dyn = nullptr,
                      const GemmStats *stats = nullptr, int ksplit = 1, int64_t split_stride = 0,
                      int mode = GEMM_AUTO, const GemmLp *lp = nullptr);

// Ignored-row compaction of n_rows targets (flce.cu): valid rows' indices to
// idx, their positions (or -1) to pos, their targets to tgt, their count to
// cnt; hidden rows [n_rows, H] gathered to hc in that order (zeros past the
// count). grad_hidden (or NULL): rows left out are zeroed. g_in (or NULL):
// gathered to g_out.
struct CompactBufs {
    int *idx, *pos, *cnt;
    int64_t *tgt;
    void *hc;
};
cudaError_t flce_compact(const void *target, int tgt32, int64_t n_rows, int64_t vocab, int64_t ignore_index,
                         const void *hidden, int64_t H, const CompactBufs &b, void *grad_hidden, const float *g_in,
                         float *g_out, cudaStream_t s);
// split count of the grad_hidden product (chunk x H outputs over K = V)
int flce_dh_splits(int64_t chunk, int64_t H, int64_t V);
// grad_hidden rows from dZ (bf16 [c, V], stride ldd): dh = dZ W, each row
// stored at out[row_map[r]] (or r); `parts` holds the split-K partials
cudaError_t flce_grad_hidden(int64_t c, int64_t H, int64_t V, const void *dz, int64_t ldd, const void *weight, int splits,
                             float *parts, const int *count, int64_t off, const int *row_map, void *out,
                             unsigned int *status, cudaStream_t s);
// 2-D bf16 row-major matrix [rows, cols] with row stride ld (elements), box
// of box_cols x box_rows, 128-byte swizzle, zero fill out of bounds.
cudaError_t make_tmap(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_cols,
                      uint32_t box_rows);

// Log-probability statistics of few rows (flce_few.cu): the states of
// flce_few_parts(V) column sets to part[row * flce_few_parts(V) + set] and the
// target logits to xy[row]. n <= kFewMaxRows; arguments as GemmLp's.
constexpr int kFewMaxRows = 64;
int flce_few_parts(int64_t V);
cudaError_t flce_few(int n, int V, int H, const void *hidden, const void *weight, const float *bias, const void *target,
                     int tgt32, int64_t ignore_index, float k, int entropy, float4 *part, float *xy, unsigned int *status,
                     cudaStream_t s);

// K steps of 64 per split-K part: ksplit parts over kiters steps, each
// non-empty (the split count actually used, <= ksplit).
int gemm_fit_ksplit(int K, int ksplit);

}  // namespace ce
