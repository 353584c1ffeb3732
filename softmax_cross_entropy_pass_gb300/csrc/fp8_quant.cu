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

__device__ inline float block_scale(float amax) { return max_nan(amax / kE4m3Max, kFp8MinScale); }

// The fp32 quotients y / scale; a byte is the nearest e4m3 of that. (y times the rounded
// reciprocal misses ties, of which 16-bit inputs meet one in 2000 bytes.) The reciprocal
// is taken in two parts: hi, the hardware's (off by 2^-22 at most) and not above it, and
// lo = (1 - hi scale) hi, by a fused multiply-add. y hi + y lo is 2^-42 off the quotient
// before its one rounding (2^-31 for scales above 2^103, whose lo is below the normal
// range). No quotient of 16-bit blocks lies within 2^-42 of where its rounding takes or
// leaves a tie; one of an fp32 y does in some 2^37. (lo >= 0: a zero y keeps its sign. An
// infinite scale leaves y 0.) No slower than the product with one rounded reciprocal; the
// correctly rounded reciprocal and remainder: 8192 x 4096 bf16 norm 43.2 us against 41.6.
struct Quotient {
    F2 hi, lo;
    __device__ inline explicit Quotient(float scale) {
        float h;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(scale));
        if (fmaf(-h, scale, 1.f) < 0.f) h = __uint_as_float(__float_as_uint(h) - 2u);
        const float l = scale < INFINITY ? fmaf(-h, scale, 1.f) * h : 0.f;
        hi = f2(h, h);
        lo = f2(l, l);
    }
    __device__ inline void operator()(float &a, float &b) const {
        const F2 v = f2(a, b);
        f2_split(f2_fma(v, hi, f2_mul(v, lo)), a, b);
    }
};

__device__ inline uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Eight consecutive elements of a row as they lie in memory.
template <int DT> struct Raw8 {
    uint4 v[DT == CE_DT_F32 ? 2 : 1];
    __device__ inline void unpack(float (&x)[8]) const {
        Fmt<DT>::unpack(v[0], x);
        if constexpr (DT == CE_DT_F32) Fmt<DT>::unpack(v[1], x + 4);
    }
    __device__ inline void pack(const float (&x)[8]) {
        v[0] = Fmt<DT>::pack(x);
        if constexpr (DT == CE_DT_F32) v[1] = Fmt<DT>::pack(x + 4);
    }
    // what was unpacked before is not kept in registers for an unpack() behind this
    __device__ inline void again() {
#pragma unroll
        for (uint4 &w : v) asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
    }
};

// ... from column c on, zeros past the last. VEC: the row starts on a 16-byte
// boundary (c is a multiple of 8).
template <int DT, bool VEC>
__device__ inline Raw8<DT> load8(const void *row, int c, int cols) {
    Raw8<DT> r;
    if (VEC && c + 8 <= cols) {
        const char *p = reinterpret_cast<const char *>(row) + static_cast<int64_t>(c) * Fmt<DT>::kBytes;
        r.v[0] = ld_stream(p);
        if constexpr (DT == CE_DT_F32) r.v[1] = ld_stream(p + 16);
    } else {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = c + j < cols ? Fmt<DT>::load1(row, c + j) : 0.f;
        r.pack(x);
    }
    return r;
}
template <int DT, bool VEC>
__device__ inline void store8(void *row, int c, int cols, const float (&x)[8]) {
    if (VEC && c + 8 <= cols) {
        uint4 *p = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(row) + static_cast<int64_t>(c) * Fmt<DT>::kBytes);
        p[0] = Fmt<DT>::pack(x);
        if (DT == CE_DT_F32) p[1] = Fmt<DT>::pack(x + 4);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < cols) Fmt<DT>::store1(row, c + j, x[j]);
    }
}
// the rows of q start on 16-byte boundaries, whatever the input's do
__device__ inline void store_q8(uint8_t *row, int c, int cols, float (&y)[8], const Quotient &over) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) over(y[j], y[j + 1]);
    const uint32_t lo = e4m3x4(y[0], y[1], y[2], y[3]), hi = e4m3x4(y[4], y[5], y[6], y[7]);
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

// eight weights, read for every row: kept in L1
template <int DT>
__device__ inline void load_weight(const void *w, int c, int cols, float (&x)[8]) {
    if (c + 8 <= cols) {
        const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(w) + static_cast<int64_t>(c) * Fmt<DT>::kBytes);
        Fmt<DT>::unpack(__ldg(p), x);
        if constexpr (DT == CE_DT_F32) Fmt<DT>::unpack(__ldg(p + 1), x + 4);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = c + j < cols ? Fmt<DT>::load1(w, c + j) : 0.f;
    }
}

struct NormArgs {
    const void *x, *residual, *weight;
    void *residual_out;
    uint8_t *q;
    float *scale;
    int64_t n_rows, ld_x, ld_res, ld_out, ld_q, blocks;
    int cols, weight_f32;
    float eps;
};

// How a row is split: a warp of 8 in a CTA, or a CTA of up to 256, 512 or 1024
// threads; the registers are held to what lets 1024 threads of an SM run (512
// with four vectors a thread, or two of fp32). Rows above 16384 columns take a CTA of 1024
// threads with four vectors each, whose 64 registers spill (300 to 950 bytes): 4096 x 16384
// bf16 96 us, 4096 x 16392 202.
enum { NORM_WARP = 0, NORM_256 = 1, NORM_512 = 2, NORM_1024 = 3 };
__host__ __device__ constexpr int norm_threads(int mode) { return mode < NORM_512 ? 256 : (mode == NORM_512 ? 512 : 1024); }
__host__ __device__ constexpr int norm_resident(int dtype, int vpt) { return vpt * (dtype == CE_DT_F32 ? 2 : 1) >= 4 ? 512 : 1024; }
__host__ __device__ constexpr int norm_ctas(int dtype, int mode, int vpt) {
    return mode == NORM_1024 ? 1 : norm_resident(dtype, vpt) / norm_threads(mode);
}

// A row by one warp or by a CTA's W; thread t of a row's holds the vectors of 8 columns t, t + 32 W, ... (16 neighbouring
// lanes hold a block). Rows are dealt out round robin, and the next row's loads
// are under way while the reductions of this one wait for one another (not above
// 16384 columns, whose registers are all taken): a row at a time left HBM at 65%.
// 8192 x 4096 bf16 with a residual, 236 MB: 41.6 us, 84% of the copy rate; 4 rows 2.7 us,
// a launch and one row's chain of loads, two reductions and stores.
template <int DT, bool VEC, int VPT, int MODE>
__global__ void __launch_bounds__(norm_threads(MODE), norm_ctas(DT, MODE, VPT)) norm_fp8_kernel(NormArgs a) {
    constexpr bool WARP = MODE == NORM_WARP, AHEAD = MODE != NORM_1024;
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31, nwarps = WARP ? 1 : blockDim.x >> 5, warp = WARP ? 0 : threadIdx.x >> 5;
    const int tid = WARP ? lane : threadIdx.x, step = 8 * 32 * nwarps;
    const int64_t stride = WARP ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
    int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    Raw8<DT> x[VPT], r[VPT];
    const auto fetch = [&](int64_t i) {
        const char *px = reinterpret_cast<const char *>(a.x) + i * a.ld_x * Fmt<DT>::kBytes;
        const char *pr = reinterpret_cast<const char *>(a.residual) + i * a.ld_res * Fmt<DT>::kBytes;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            x[v] = load8<DT, VEC>(px, tid * 8 + v * step, a.cols);
            if (a.residual) r[v] = load8<DT, VEC>(pr, tid * 8 + v * step, a.cols);
        }
    };
    int turn = 0;
    // sum over the row of (h f)^2, the same in every thread
    const auto squares = [&](const float (&h)[VPT][8], float f) {
        float t = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) t = fmaf(h[v][j] * f, h[v][j] * f, t);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        if (!WARP) {
            // two buffers in turn: nobody writes one that a warp may still read
            if (lane == 0) part[turn][warp] = t;
            __syncthreads();
            t = lane < nwarps ? part[turn][lane] : 0.f;
            turn ^= 1;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        }
        return t;
    };
    if (row < a.n_rows) fetch(row);
    for (; row < a.n_rows; row += stride) {
        float h[VPT][8];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            x[v].unpack(h[v]);
            if (a.residual) {
                float b[8];
                r[v].unpack(b);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[v][j] += b[j];
            }
        }
        if (AHEAD && row + stride < a.n_rows) fetch(row + stride);
        if (a.residual_out) {
            char *o = reinterpret_cast<char *>(a.residual_out) + row * a.ld_out * Fmt<DT>::kBytes;
#pragma unroll
            for (int v = 0; v < VPT; ++v) store8<DT, VEC>(o, tid * 8 + v * step, a.cols, h[v]);
        }
        // squares past fp32's range, or under it beside an eps that small, are taken of h 2^-80 or h 2^80
        float f = 1.f, ss = squares(h, 1.f);
        if (ss == INFINITY) f = 0x1p-80f;
        else if (ss < 1e-28f && a.eps < 1e-28f) f = 0x1p80f;
        if (f != 1.f) ss = squares(h, f);
        const float rstd = f / sqrtf(ss / static_cast<float>(a.cols) + a.eps * f * f);
        uint8_t *q = a.q + row * a.ld_q;
        float *scales = a.scale + row * a.blocks;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = tid * 8 + v * step;
            float w[8];
            if (a.weight_f32) load_weight<CE_DT_F32>(a.weight, c, a.cols, w);
            else load_weight<DT>(a.weight, c, a.cols, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[v][j] = h[v][j] * rstd * w[j];
            const float scale = block_scale(block_amax(h[v]));
            if (c < a.cols) {
                store_q8(q, c, a.cols, h[v], Quotient(scale));
                if ((lane & 15) == 0) scales[c / kFp8Block] = scale;
            }
        }
        if (!AHEAD && row + stride < a.n_rows) fetch(row + stride);
    }
}

struct QuantArgs {
    const void *x;
    uint8_t *q;
    float *scale;
    int64_t rows, ld, ld_q;
    int cols, blocks;
    int parts;  // CTAs of a row (of a row of blocks)
};

// 1 x 128: a half warp per block, kRowVecs vectors a thread (4096 x 8192 bf16, 102 MB: 16.4 us, 92% of the copy rate)
constexpr int kRowVecs = 4, kRowQuantThreads = 128;
template <int DT, bool VEC>
__global__ void __launch_bounds__(kRowQuantThreads) quant_rows_kernel(QuantArgs a) {
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts;
    const char *x = reinterpret_cast<const char *>(a.x) + row * a.ld * Fmt<DT>::kBytes;
    Raw8<DT> raw[kRowVecs];
    const int c0 = (part * kRowVecs * kRowQuantThreads + threadIdx.x) * 8;
#pragma unroll
    for (int v = 0; v < kRowVecs; ++v) raw[v] = load8<DT, VEC>(x, c0 + v * kRowQuantThreads * 8, a.cols);
#pragma unroll
    for (int v = 0; v < kRowVecs; ++v) {
        const int c = c0 + v * kRowQuantThreads * 8;
        float y[8];
        raw[v].unpack(y);
        const float scale = block_scale(block_amax(y));
        if (c < a.cols) {
            store_q8(a.q + row * a.ld_q, c, a.cols, y, Quotient(scale));
            if ((threadIdx.x & 15) == 0) a.scale[row * a.blocks + c / kFp8Block] = scale;
        }
    }
}

// 128 x 128: a CTA per block at a time, half a warp per row, 4 rows a half warp.
// The block stays in registers as it was read, and the next one's loads are under
// way while this one's maximum is found and its bytes written: a CTA per block
// without that left HBM at 72% (128256 x 4096 bf16, 1.6 GB: 325 us, 253 now, 92% of the copy rate; 315 us
// where the compiler keeps unpacked values over the barrier, and spills).
constexpr int kTileThreads = 512, kTileRows = kFp8Block / (kTileThreads / 16);
template <int DT, bool VEC>
__global__ void __launch_bounds__(kTileThreads, DT == CE_DT_F32 ? 1 : 2) quant_tiles_kernel(QuantArgs a) {
    __shared__ float part[2][kTileThreads / 32];
    const int64_t tiles = (a.rows + kFp8Block - 1) / kFp8Block * a.blocks;
    Raw8<DT> next[kTileRows];
    const auto fetch = [&](int64_t tile) {
        const int64_t r0 = tile / a.blocks * kFp8Block + (threadIdx.x >> 4);
        const int c = static_cast<int>(tile % a.blocks) * kFp8Block + (threadIdx.x & 15) * 8;
#pragma unroll
        for (int v = 0; v < kTileRows; ++v) {
            const int64_t r = r0 + v * (kTileThreads / 16);
            const char *x = reinterpret_cast<const char *>(a.x) + r * a.ld * Fmt<DT>::kBytes;
            next[v] = load8<DT, VEC>(x, c, r < a.rows ? a.cols : 0);
        }
    };
    int64_t tile = blockIdx.x;
    int turn = 0;
    if (tile < tiles) fetch(tile);
    for (; tile < tiles; tile += gridDim.x, turn ^= 1) {
        Raw8<DT> raw[kTileRows];
        float amax = 0.f;
#pragma unroll
        for (int v = 0; v < kTileRows; ++v) {
            raw[v] = next[v];
            float y[8];
            raw[v].unpack(y);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(y[j]));
        }
        if (tile + gridDim.x < tiles) fetch(tile + gridDim.x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        // two buffers in turn: nobody writes one that a warp may still read
        if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = amax;
        __syncthreads();
        amax = part[turn][threadIdx.x & (kTileThreads / 32 - 1)];
#pragma unroll
        for (int off = kTileThreads / 64; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const float scale = block_scale(amax);
        const Quotient over(scale);
        if (threadIdx.x == 0) a.scale[tile] = scale;
        const int64_t r0 = tile / a.blocks * kFp8Block + (threadIdx.x >> 4);
        const int c = static_cast<int>(tile % a.blocks) * kFp8Block + (threadIdx.x & 15) * 8;
#pragma unroll
        for (int v = 0; v < kTileRows; ++v) {
            const int64_t r = r0 + v * (kTileThreads / 16);
            float y[8];
            raw[v].again();
            raw[v].unpack(y);
            if (r < a.rows && c < a.cols) store_q8(a.q + r * a.ld_q, c, a.cols, y, over);
        }
    }
}

// A warp a row up to 256 columns; above, a CTA a row, with one vector of 8 columns
// a thread while the rows are few (latency) or short, two or four otherwise.
// A warp / a CTA a row (us, bf16 with a residual): 256 columns 2.05 / 2.20 (1 row) and
// 2.7 / 3.1 (2000 rows), 512 columns 2.8 / 2.3 and 3.9 / 3.7. One vector / two: 4096 columns
// 2.5 / 3.2 (8 rows), 4.0 / 4.5 (300), 5.4 / 5.2 (400) and 45.8 / 41.0 (8192), 2048 columns
// 8.3 / 8.5 (2000), 23.8 / 22.7 (8192) and 87 / 79 (32768).
cudaError_t launch_norm(const NormArgs &a, int dtype, bool vec, cudaStream_t s) {
    const int vecs = (a.cols + 7) / 8;
    using Fn = void (*)(NormArgs);
#define CE_NORM(DT, V) {norm_fp8_kernel<DT, V, 1, NORM_WARP>, norm_fp8_kernel<DT, V, 1, NORM_256>, \
                        norm_fp8_kernel<DT, V, 2, NORM_256>, norm_fp8_kernel<DT, V, 1, NORM_512>, \
                        norm_fp8_kernel<DT, V, 2, NORM_512>, norm_fp8_kernel<DT, V, 4, NORM_512>, \
                        norm_fp8_kernel<DT, V, 4, NORM_1024>}
    static const Fn fns[3][2][7] = {{CE_NORM(CE_DT_F32, false), CE_NORM(CE_DT_F32, true)},
                                    {CE_NORM(CE_DT_BF16, false), CE_NORM(CE_DT_BF16, true)},
                                    {CE_NORM(CE_DT_F16, false), CE_NORM(CE_DT_F16, true)}};
#undef CE_NORM
    constexpr int kSms = 152;
    NormArgs b = a;
    void *args[] = {&b};
    int which, threads, per_sm;
    int64_t grid;
    if (vecs <= 32) {
        which = 0;
        threads = 256;
        grid = (a.n_rows + 7) / 8;
        per_sm = norm_resident(dtype, 1) / threads;
    } else {
        const bool two = vecs > 512 || (vecs > 256 && a.n_rows > 2 * kSms) || (vecs > 128 && a.n_rows > 26 * kSms);
        const int vpt = vecs > 1024 ? 4 : (two ? 2 : 1);
        threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
        which = threads > 512 ? 6 : (threads > 256 || vpt == 4 ? 3 : 1) + (vpt >> 1);
        grid = a.n_rows;
        per_sm = threads > 512 ? 1 : norm_resident(dtype, vpt) / threads;
    }
    if (grid > static_cast<int64_t>(kSms) * per_sm) grid = static_cast<int64_t>(kSms) * per_sm;
    return cudaLaunchKernel(reinterpret_cast<const void *>(fns[dtype][vec ? 1 : 0][which]),
                            dim3(static_cast<unsigned>(grid)), dim3(threads), args, 0, s);
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
    a.n_rows = n; a.cols = static_cast<int>(p->cols);
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
    if (rows > kMaxRows || cols > kMaxRows - 8192) return CE_ERR_UNSUPPORTED;  // column indices are 32-bit
    a.rows = rows; a.cols = static_cast<int>(cols); a.ld = ld_x; a.ld_q = ld_q;
    a.blocks = static_cast<int>((cols + kFp8Block - 1) / kFp8Block);
    const int64_t up = block_rows == 1 ? rows : (rows + kFp8Block - 1) / kFp8Block;
    constexpr int64_t per = kRowVecs * kRowQuantThreads * 8;
    a.parts = block_rows == 1 ? static_cast<int>((cols + per - 1) / per) : a.blocks;
    if (up > kMaxRows / a.parts) return CE_ERR_UNSUPPORTED;
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
    int64_t grid = up * a.parts;
    if (tall && grid > 152 * 2) grid = 152 * 2;
    const cudaError_t e = cudaLaunchKernel(
        reinterpret_cast<const void *>(fns[tall][dtype][vec_rows(x, ld_x, esz, rows) ? 1 : 0]),
        dim3(static_cast<unsigned>(grid)), dim3(tall ? kTileThreads : kRowQuantThreads), args, 0,
        reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}

}  // extern "C"
