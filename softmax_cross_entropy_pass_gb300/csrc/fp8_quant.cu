// fp8_quant.cu -- e4m3 values with a scale for every block: the root-mean-square
// norm with the residual's addition and an 8-bit output, and plain quantising
// to blocks of 1 x 128 (activations) or 128 x 128 (weights).
//
//   h = x + r,  s = 1 / sqrt(mean h^2 + eps),  y = h s w
//   scale = max(max |y| / 448, 2^-126) over a block,  q = e4m3(y / scale)
//
// h and everything after it is fp32: h is rounded to the residual's type only
// where it is stored, y only where it becomes q. A NaN makes its block's scale
// and values NaN (in the norm its whole row's).
//
// All three are bound by HBM: every element read once, held in registers
// between the reductions, and written once.
#include <cuda_fp8.h>

#include "ce_device.cuh"
#include "ce_kernels.h"
#include "fp8.h"

namespace ce {

namespace {

__device__ inline float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// scale of a block whose largest magnitude is amax; inv = 1 / scale
__device__ inline float block_scale(float amax, float &inv) {
    const float scale = max_nan(amax / kE4m3Max, kFp8MinScale);
    inv = 1.f / scale;
    return scale;
}

__device__ inline uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Eight consecutive elements of a row from column c on, zeros past the last.
// VEC: the row starts on a 16-byte boundary (c is a multiple of 8).
template <int DT, bool VEC>
__device__ inline void load8(const void *row, int64_t c, int64_t cols, float (&x)[8]) {
    if (VEC && c + 8 <= cols) {
        const char *p = reinterpret_cast<const char *>(row) + c * Fmt<DT>::kBytes;
        const uint4 a = ld_stream(p);
        Fmt<DT>::unpack(a, x);
        if (DT == CE_DT_F32) {
            const uint4 b = ld_stream(p + 16);
            Fmt<DT>::unpack(b, x + 4);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = c + j < cols ? Fmt<DT>::load1(row, c + j) : 0.f;
    }
}
template <int DT, bool VEC>
__device__ inline void store8(void *row, int64_t c, int64_t cols, const float (&x)[8]) {
    if (VEC && c + 8 <= cols) {
        uint4 *p = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(row) + c * Fmt<DT>::kBytes);
        p[0] = Fmt<DT>::pack(x);
        if (DT == CE_DT_F32) p[1] = Fmt<DT>::pack(x + 4);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < cols) Fmt<DT>::store1(row, c + j, x[j]);
    }
}
// the rows of q start on 16-byte boundaries, whatever the input's do
__device__ inline void store_q8(uint8_t *row, int64_t c, int64_t cols, const float (&y)[8], float inv) {
    const uint32_t lo = e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    const uint32_t hi = e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
    if (c + 8 <= cols) {
        *reinterpret_cast<uint2 *>(row + c) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < cols) row[c + j] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
}

// the largest of 8 magnitudes over the 16 lanes that hold a block's 128 columns
__device__ inline float block_amax(const float (&y)[8]) {
    float a = fabsf(y[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) a = max_nan(a, fabsf(y[j]));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
    return a;
}

struct NormArgs {
    const void *x, *residual, *weight;
    void *residual_out;
    uint8_t *q;
    float *scale;
    int64_t n_rows, cols, ld_x, ld_res, ld_out, ld_q, blocks;
    int weight_f32;
    float eps;
};

// One CTA per row; thread t holds the vectors of 8 columns t, t + threads, ...
// (16 neighbouring lanes hold a block).
template <int DT, bool VEC, int VPT>
__global__ void __launch_bounds__(1024) norm_fp8_kernel(NormArgs a) {
    __shared__ float part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    const char *x = reinterpret_cast<const char *>(a.x) + row * a.ld_x * Fmt<DT>::kBytes;
    const char *r = reinterpret_cast<const char *>(a.residual) + row * a.ld_res * Fmt<DT>::kBytes;
    float h[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t c = (static_cast<int64_t>(v) * blockDim.x + tid) * 8;
        load8<DT, VEC>(x, c, a.cols, h[v]);
        if (a.residual) {
            float b[8];
            load8<DT, VEC>(r, c, a.cols, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[v][j] += b[j];
        }
    }
    if (a.residual_out) {
        char *o = reinterpret_cast<char *>(a.residual_out) + row * a.ld_out * Fmt<DT>::kBytes;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            store8<DT, VEC>(o, (static_cast<int64_t>(v) * blockDim.x + tid) * 8, a.cols, h[v]);
    }
    // sum over the row of (h f)^2, the same in every thread
    const auto squares = [&](float f) {
        float t = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) t = fmaf(h[v][j] * f, h[v][j] * f, t);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        if (lane == 0) part[warp] = t;
        __syncthreads();
        t = lane < nwarps ? part[lane] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        return t;
    };
    // squares past fp32's range, or under it beside an eps that small, are taken of h 2^-80 or h 2^80
    float f = 1.f, ss = squares(1.f);
    if (ss == INFINITY) f = 0x1p-80f;
    else if (ss < 1e-28f && a.eps < 1e-28f) f = 0x1p80f;
    if (f != 1.f) {
        __syncthreads();
        ss = squares(f);
    }
    const float rstd = f / sqrtf(ss / static_cast<float>(a.cols) + a.eps * f * f);
    uint8_t *q = a.q + row * a.ld_q;
    float *scales = a.scale + row * a.blocks;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t c = (static_cast<int64_t>(v) * blockDim.x + tid) * 8;
        float w[8];
        if (a.weight_f32) load8<CE_DT_F32, true>(a.weight, c, a.cols, w);
        else load8<DT, true>(a.weight, c, a.cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[v][j] = h[v][j] * rstd * w[j];
        float inv;
        const float scale = block_scale(block_amax(h[v]), inv);
        if (c < a.cols) {
            store_q8(q, c, a.cols, h[v], inv);
            if ((lane & 15) == 0) scales[c / kFp8Block] = scale;
        }
    }
}

struct QuantArgs {
    const void *x;
    uint8_t *q;
    float *scale;
    int64_t rows, cols, ld, ld_q, blocks;
    int64_t parts;  // CTAs of a row
};

// 1 x 128: a half warp per block, kRowVecs vectors a thread
constexpr int kRowVecs = 4, kRowQuantThreads = 128;
template <int DT, bool VEC>
__global__ void __launch_bounds__(kRowQuantThreads) quant_rows_kernel(QuantArgs a) {
    const int64_t row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const char *x = reinterpret_cast<const char *>(a.x) + row * a.ld * Fmt<DT>::kBytes;
    float y[kRowVecs][8];
    const int64_t c0 = (part * kRowVecs * kRowQuantThreads + threadIdx.x) * 8;
#pragma unroll
    for (int v = 0; v < kRowVecs; ++v) load8<DT, VEC>(x, c0 + v * kRowQuantThreads * 8, a.cols, y[v]);
#pragma unroll
    for (int v = 0; v < kRowVecs; ++v) {
        const int64_t c = c0 + v * kRowQuantThreads * 8;
        float inv;
        const float scale = block_scale(block_amax(y[v]), inv);
        if (c < a.cols) {
            store_q8(a.q + row * a.ld_q, c, a.cols, y[v], inv);
            if ((threadIdx.x & 15) == 0) a.scale[row * a.blocks + c / kFp8Block] = scale;
        }
    }
}

// 128 x 128: a CTA per block, half a warp per row, 8 rows a half warp
constexpr int kTileThreads = 256, kTileRows = kFp8Block / (kTileThreads / 16);
template <int DT, bool VEC>
__global__ void __launch_bounds__(kTileThreads) quant_tiles_kernel(QuantArgs a) {
    __shared__ float part[kTileThreads / 32];
    const int64_t up = blockIdx.x / a.blocks, across = blockIdx.x % a.blocks;
    const int64_t c = across * kFp8Block + (threadIdx.x & 15) * 8;
    const int64_t r0 = up * kFp8Block + (threadIdx.x >> 4);
    float y[kTileRows][8], amax = 0.f;
#pragma unroll
    for (int v = 0; v < kTileRows; ++v) {
        const int64_t r = r0 + v * (kTileThreads / 16);
        const char *x = reinterpret_cast<const char *>(a.x) + r * a.ld * Fmt<DT>::kBytes;
        load8<DT, VEC>(x, c, r < a.rows ? a.cols : 0, y[v]);
    }
#pragma unroll
    for (int v = 0; v < kTileRows; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(y[v][j]));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = part[0];
#pragma unroll
    for (int i = 1; i < kTileThreads / 32; ++i) amax = max_nan(amax, part[i]);
    float inv;
    const float scale = block_scale(amax, inv);
    if (threadIdx.x == 0) a.scale[blockIdx.x] = scale;
#pragma unroll
    for (int v = 0; v < kTileRows; ++v) {
        const int64_t r = r0 + v * (kTileThreads / 16);
        if (r < a.rows && c < a.cols) store_q8(a.q + r * a.ld_q, c, a.cols, y[v], inv);
    }
}

// Vectors a thread: one while the row's 8-column vectors fit 1024 threads.
cudaError_t launch_norm(const NormArgs &a, int dtype, bool vec, cudaStream_t s) {
    const int64_t vecs = (a.cols + 7) / 8;
    const int vpt = vecs <= 1024 ? 1 : (vecs <= 2048 ? 2 : 4);
    const int threads = static_cast<int>(((vecs + vpt - 1) / vpt + 31) / 32 * 32);
    using Fn = void (*)(NormArgs);
#define CE_NORM(DT) {{norm_fp8_kernel<DT, false, 1>, norm_fp8_kernel<DT, false, 2>, norm_fp8_kernel<DT, false, 4>}, \
                     {norm_fp8_kernel<DT, true, 1>, norm_fp8_kernel<DT, true, 2>, norm_fp8_kernel<DT, true, 4>}}
    static const Fn fns[3][2][3] = {CE_NORM(CE_DT_F32), CE_NORM(CE_DT_BF16), CE_NORM(CE_DT_F16)};
#undef CE_NORM
    NormArgs b = a;
    void *args[] = {&b};
    return cudaLaunchKernel(reinterpret_cast<const void *>(fns[dtype][vec ? 1 : 0][vpt >> 1]),
                            dim3(static_cast<unsigned>(a.n_rows)), dim3(threads), args, 0, s);
}

bool vec_rows(const void *p, int64_t ld, int esz, int64_t rows) {
    return fp8_on(p, 16) && (rows < 2 || (ld * esz) % 16 == 0);
}

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kNormMaxCols = 32768;

int64_t span(int64_t rows, int64_t ld, int64_t cols, int esz) { return rows > 0 ? ((rows - 1) * ld + cols) * esz : 0; }

}  // namespace

}  // namespace ce

using namespace ce;

extern "C" {

ce_status ce_rms_norm_fp8(const ce_norm_params *p, const void *x, const void *residual, const void *weight,
                          void *residual_out, void *q, float *scale, void *stream) {
    if (!p || p->n_rows < 0 || p->cols < 1 || p->reserved != 0) return CE_ERR_INVALID_ARG;
    if (!fp8_dtype_ok(p->dtype) || (p->weight_dtype != p->dtype && p->weight_dtype != CE_DT_F32)) return CE_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f && p->eps < INFINITY)) return CE_ERR_INVALID_ARG;
    if (p->n_rows > kMaxRows || p->cols > kNormMaxCols) return CE_ERR_UNSUPPORTED;
    if (p->ld_x < p->cols || p->ld_q < p->cols || p->ld_q % 16) return CE_ERR_INVALID_ARG;
    if ((residual && p->ld_residual < p->cols) || (residual_out && p->ld_residual_out < p->cols)) return CE_ERR_INVALID_ARG;
    if (!residual && residual_out) return CE_ERR_INVALID_ARG;
    if (p->n_rows == 0) return CE_OK;
    if (!x || !weight || !q || !scale) return CE_ERR_INVALID_ARG;
    const int esz = fp8_elem(p->dtype);
    if (!fp8_on(x, esz) || !fp8_on(residual, esz) || !fp8_on(residual_out, esz) || !fp8_on(weight, 16) ||
        !fp8_on(q, 16) || !fp8_on(scale, 4))
        return CE_ERR_INVALID_ARG;
    const int64_t n = p->n_rows, blocks = (p->cols + kFp8Block - 1) / kFp8Block;
    const int64_t xb = span(n, p->ld_x, p->cols, esz), rb = span(n, p->ld_residual, p->cols, esz);
    const int64_t ob = span(n, p->ld_residual_out, p->cols, esz), qb = span(n, p->ld_q, p->cols, 1);
    const int64_t sb = n * blocks * 4, wb = p->cols * fp8_elem(p->weight_dtype);
    // each output apart from everything but, for residual_out, the input whose place it takes
    if (!fp8_apart(q, qb, x, xb) || !fp8_apart(q, qb, scale, sb) || !fp8_apart(scale, sb, x, xb) ||
        !fp8_apart(q, qb, weight, wb) || !fp8_apart(scale, sb, weight, wb))
        return CE_ERR_INVALID_ARG;
    if (residual && (!fp8_apart(q, qb, residual, rb) || !fp8_apart(scale, sb, residual, rb))) return CE_ERR_INVALID_ARG;
    if (residual_out) {
        if (!fp8_apart(residual_out, ob, q, qb) || !fp8_apart(residual_out, ob, scale, sb) ||
            !fp8_apart(residual_out, ob, weight, wb))
            return CE_ERR_INVALID_ARG;
        const bool over_x = residual_out == x && (n == 1 || p->ld_residual_out == p->ld_x);
        const bool over_r = residual_out == residual && (n == 1 || p->ld_residual_out == p->ld_residual);
        if ((!over_x && !fp8_apart(residual_out, ob, x, xb)) || (!over_r && !fp8_apart(residual_out, ob, residual, rb)))
            return CE_ERR_INVALID_ARG;
    }
    NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.residual_out = residual_out;
    a.q = reinterpret_cast<uint8_t *>(q);
    a.scale = scale;
    a.n_rows = n; a.cols = p->cols;
    a.ld_x = p->ld_x; a.ld_res = p->ld_residual; a.ld_out = p->ld_residual_out; a.ld_q = p->ld_q;
    a.blocks = blocks;
    a.weight_f32 = p->weight_dtype == CE_DT_F32;
    a.eps = p->eps;
    const bool vec = vec_rows(x, a.ld_x, esz, n) && (!residual || vec_rows(residual, a.ld_res, esz, n)) &&
                     (!residual_out || vec_rows(residual_out, a.ld_out, esz, n));
    const cudaError_t e = launch_norm(a, p->dtype, vec, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

ce_status ce_quantize_fp8(int64_t rows, int64_t cols, const void *x, int64_t ld_x, int32_t dtype, int32_t block_rows,
                          void *q, int64_t ld_q, float *scale, void *stream) {
    if (rows < 0 || cols < 1 || !fp8_dtype_ok(dtype) || (block_rows != 1 && block_rows != kFp8Block))
        return CE_ERR_INVALID_ARG;
    if (ld_x < cols || ld_q < cols || ld_q % 16) return CE_ERR_INVALID_ARG;
    if (rows == 0) return CE_OK;
    const int esz = fp8_elem(dtype);
    if (!x || !q || !scale || !fp8_on(x, esz) || !fp8_on(q, 16) || !fp8_on(scale, 4)) return CE_ERR_INVALID_ARG;
    QuantArgs a{};
    a.x = x;
    a.q = reinterpret_cast<uint8_t *>(q);
    a.scale = scale;
    a.rows = rows; a.cols = cols; a.ld = ld_x; a.ld_q = ld_q;
    a.blocks = (cols + kFp8Block - 1) / kFp8Block;
    const int64_t up = block_rows == 1 ? rows : (rows + kFp8Block - 1) / kFp8Block;
    const int64_t per = kRowVecs * kRowQuantThreads * 8;
    a.parts = block_rows == 1 ? (cols + per - 1) / per : a.blocks;
    if (rows > kMaxRows || cols > kMaxRows || up > kMaxRows / a.parts) return CE_ERR_UNSUPPORTED;
    const int64_t xb = span(rows, ld_x, cols, esz), qb = span(rows, ld_q, cols, 1), sb = up * a.blocks * 4;
    if (!fp8_apart(q, qb, x, xb) || !fp8_apart(scale, sb, x, xb) || !fp8_apart(q, qb, scale, sb)) return CE_ERR_INVALID_ARG;
    using Fn = void (*)(QuantArgs);
    static const Fn fns[2][3][2] = {
        {{quant_rows_kernel<CE_DT_F32, false>, quant_rows_kernel<CE_DT_F32, true>},
         {quant_rows_kernel<CE_DT_BF16, false>, quant_rows_kernel<CE_DT_BF16, true>},
         {quant_rows_kernel<CE_DT_F16, false>, quant_rows_kernel<CE_DT_F16, true>}},
        {{quant_tiles_kernel<CE_DT_F32, false>, quant_tiles_kernel<CE_DT_F32, true>},
         {quant_tiles_kernel<CE_DT_BF16, false>, quant_tiles_kernel<CE_DT_BF16, true>},
         {quant_tiles_kernel<CE_DT_F16, false>, quant_tiles_kernel<CE_DT_F16, true>}}};
    void *args[] = {&a};
    const int tall = block_rows == 1 ? 0 : 1;
    const cudaError_t e = cudaLaunchKernel(
        reinterpret_cast<const void *>(fns[tall][dtype][vec_rows(x, ld_x, esz, rows) ? 1 : 0]),
        dim3(static_cast<unsigned>(up * a.parts)), dim3(tall ? kTileThreads : kRowQuantThreads), args, 0,
        reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

}  // extern "C"
