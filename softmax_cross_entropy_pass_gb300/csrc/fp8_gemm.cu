// fp8_gemm.cu -- matrix product of e4m3 operands with a scale for every block
// of 128 along K (and of 128 rows of the weight):
//
//   D[m, n] = sum_b sa[m, b] sb[n / 128, b] sum_{k in block b} A[m, k] B[n, k] (+ bias[n])
//
// The tensor core (tcgen05.mma kind::f8f6f4, K = 32 an instruction) forms the
// inner sum of one block; the scales are fp32 numbers of any value, so the
// partial sum of every block leaves tensor memory and is scaled and added up by
// the epilogue warps in fp32 registers. (The tensor core's long sums truncate;
// over 128 products that is below the registers' own rounding.)
//
// fp8_few_kernel: the weight's rows are the tensor core's M side, so that few
// rows of A cost no more than reading the weights: a CTA multiplies tiles of 128
// weight rows by NT rows of A and owns a contiguous share of the weight's rows,
// cut at multiples of 16.
#include <atomic>

#include "ce_device.cuh"
#include "ce_kernels.h"
#include "fp8.h"
#include "tc_device.cuh"

namespace ce {

namespace {


struct Fp8Args {
    int m, n, K;              // rows of A, rows of B
    int kblocks;
    const float *a_scale;     // [m, kblocks]
    const float *b_scale;     // [ceil(n / 128), kblocks]
    const float *bias;        // [n] or NULL
    void *out;
    int64_t ldo;
    int shares;               // CTAs along the weight's rows
    int stages;
};

template <int DT>
__device__ inline void store_out(void *out, int64_t i, float v) { Fmt<DT>::store1(out, i, v); }

constexpr int kFewM = 128;                    // weight rows of a tile
constexpr int kFewWBytes = kFewM * kFp8Block; // 16 KB of weights a stage
constexpr int kFewBox = 16;                   // rows of the small boxes, the unit of the shares
constexpr int kFewMaxStages = 12;
constexpr int kFewSmem = 218 * 1024;
constexpr int kScaleBlocks = 32;              // K blocks whose scales of A are in shared memory at a time

// NT rows of A a tile, COLS of them an epilogue thread
template <int NT> struct Few {
    static constexpr int kCols = NT <= 64 ? 16 : 32;
    static constexpr int kSets = NT / kCols;
    static constexpr int kThreads = 64 + 128 * kSets;
    static constexpr int kAcc = NT <= 64 ? 8 : 4;  // accumulators in tensor memory
    static constexpr uint32_t kTmemCols = kAcc * NT;
    static constexpr int kStageBytes = kFewWBytes + NT * kFp8Block;
    static constexpr int kScaleBytes = kScaleBlocks * NT * 4;
    static constexpr int kStages = (kFewSmem - 1024 - kScaleBytes) / kStageBytes < kFewMaxStages
                                       ? (kFewSmem - 1024 - kScaleBytes) / kStageBytes : kFewMaxStages;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kScaleBytes;
};

template <int C>
__device__ inline void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[C]) {
    if constexpr (C == 16) tmem_ld_32x32b_x16(taddr, v);
    else tmem_ld_32x32b_x32(taddr, v);
}

template <int NT, int DT>
__global__ void __launch_bounds__(Few<NT>::kThreads, 1)
fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWs,
               const __grid_constant__ CUtensorMap tmA, Fp8Args g) {
    using F = Few<NT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[F::kStages], empty[F::kStages], tfull[F::kAcc], tempty[F::kAcc];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, drain_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;  // 128-byte swizzle atoms
    float *scales = reinterpret_cast<float *>(smem_raw + (base - raw) + F::kStages * F::kStageBytes);  // [kScaleBlocks][NT]
    volatile int *abort = &abort_flag;
    const int share = blockIdx.x % g.shares, m0 = (blockIdx.x / g.shares) * NT;
    const int64_t units = (g.n + kFewBox - 1) / kFewBox;
    const int v_lo = static_cast<int>(units * share / g.shares) * kFewBox;
    const int v_end = static_cast<int>(units * (share + 1) / g.shares) * kFewBox;
    const int v_hi = v_end < g.n ? v_end : g.n;
    const int ntiles = (v_hi - v_lo + kFewM - 1) / kFewM;

    if (tid == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < F::kAcc; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 4 * F::kSets);
        }
        abort_flag = drain_abort = 0;
        fence_mbar_init_cluster();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmWs);
        tma_prefetch_desc(&tmA);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), F::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            uint32_t s = 0, round = 0;
            for (int tile = 0; tile < ntiles; ++tile) {
                const int v0 = v_lo + tile * kFewM;
                const int boxes = (min(kFewM, v_hi - v0) + kFewBox - 1) / kFewBox;
                const uint32_t bytes = boxes * kFewBox * kFp8Block + NT * kFp8Block;
                for (int kb = 0; kb < g.kblocks; ++kb) {
                    const uint32_t fb = smem_u32(&full[s]), dst = base + s * F::kStageBytes;
                    if (round > 0) mbar_wait_bounded<false>(smem_u32(&empty[s]), (round - 1) & 1u, abort);
                    mbar_expect_tx(fb, bytes);
                    if (boxes == kFewM / kFewBox) {
                        tma_load_2d(dst, &tmW, kb * kFp8Block, v0, fb);
                    } else {
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(dst + b * kFewBox * kFp8Block, &tmWs, kb * kFp8Block, v0 + b * kFewBox, fb);
                    }
                    tma_load_2d(dst + kFewWBytes, &tmA, kb * kFp8Block, m0, fb);
                    if (++s == F::kStages) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // the copies in flight, with a limit of their own where another wait gave up
            const uint32_t used = round > 0 ? F::kStages : s;
            for (uint32_t i = 0; i < used; ++i) {
                const uint32_t uses = round + (i < s ? 1u : 0u);
                mbar_wait_bounded<false>(smem_u32(&full[i]), (uses - 1) & 1u, &drain_abort);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------ MMA issuer: one accumulator a K block
            const uint32_t idesc = idesc_e4m3_f32(kFewM, NT);
            uint32_t s = 0, phase = 0, unit = 0;
            for (int tile = 0; tile < ntiles; ++tile)
                for (int kb = 0; kb < g.kblocks; ++kb, ++unit) {
                    const uint32_t acc = unit % F::kAcc, u = unit / F::kAcc;
                    if (u > 0) mbar_wait_bounded<false>(smem_u32(&tempty[acc]), (u - 1) & 1u, abort);
                    mbar_wait_bounded<false>(smem_u32(&full[s]), phase, abort);
                    tc_fence_after();
                    const uint32_t a = base + s * F::kStageBytes, b = a + kFewWBytes;
#pragma unroll
                    for (int kk = 0; kk < kFp8Block / 32; ++kk)
                        mma_e4m3(tmem + acc * NT, smem_desc_sw128(a + kk * 32, 16, 1024),
                                 smem_desc_sw128(b + kk * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
                    mma_commit(smem_u32(&empty[s]));
                    mma_commit(smem_u32(&tfull[acc]));
                    if (++s == F::kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
        }
    } else {
        // ---------------------------------------------------- epilogue: 4 warps for every kCols rows of A
        constexpr int C = F::kCols;
        const int q = warp & 3, set = (warp - 2) >> 2;  // tensor memory lanes, rows of A
        const int et = tid - 64;
        const uint32_t taddr0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + set * C;
        uint32_t unit = 0;
        for (int tile = 0; tile < ntiles; ++tile) {
            const int row = v_lo + tile * kFewM + q * 32 + lane;
            const float *sb = g.b_scale + static_cast<int64_t>(min(row, g.n - 1) / kFp8Block) * g.kblocks;
            float acc[C];
#pragma unroll
            for (int j = 0; j < C; ++j) acc[j] = 0.f;
            float next = __ldg(sb);
            for (int kb = 0; kb < g.kblocks; ++kb, ++unit) {
                const int k0 = kb % kScaleBlocks;
                if (k0 == 0 && (tile == 0 || g.kblocks > kScaleBlocks)) {
                    // the next blocks' scales of A, columns of the tile side by side
                    const int nb = min(kScaleBlocks, g.kblocks - kb);
                    asm volatile("bar.sync 1, %0;" ::"r"(128 * F::kSets) : "memory");
                    for (int i = et; i < nb * NT; i += 128 * F::kSets) {
                        const int r = i / nb, b = i % nb;
                        scales[b * NT + r] = m0 + r < g.m ? __ldg(g.a_scale + static_cast<int64_t>(m0 + r) * g.kblocks + kb + b) : 0.f;
                    }
                    asm volatile("bar.sync 1, %0;" ::"r"(128 * F::kSets) : "memory");
                }
                const float w = next;
                if (kb + 1 < g.kblocks) next = __ldg(sb + kb + 1);
                const uint32_t a = unit % F::kAcc, u = unit / F::kAcc;
                mbar_wait_bounded<false>(smem_u32(&tfull[a]), u & 1u, abort);
                tc_fence_after();
                uint32_t v[C];
                tmem_ld_cols<C>(taddr0 + a * NT, v);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&tempty[a]));
                const float4 *sa = reinterpret_cast<const float4 *>(scales + k0 * NT + set * C);
#pragma unroll
                for (int j = 0; j < C / 4; ++j) {
                    const float4 s4 = sa[j];
                    acc[4 * j] = fmaf(s4.x * w, __uint_as_float(v[4 * j]), acc[4 * j]);
                    acc[4 * j + 1] = fmaf(s4.y * w, __uint_as_float(v[4 * j + 1]), acc[4 * j + 1]);
                    acc[4 * j + 2] = fmaf(s4.z * w, __uint_as_float(v[4 * j + 2]), acc[4 * j + 2]);
                    acc[4 * j + 3] = fmaf(s4.w * w, __uint_as_float(v[4 * j + 3]), acc[4 * j + 3]);
                }
            }
            if (row < v_hi) {
                // a wait that gave up leaves no result: NaN
                const float bias = *abort ? NAN : (g.bias ? __ldg(g.bias + row) : 0.f);
                const bool add = g.bias || *abort;
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const int r = m0 + set * C + j;
                    if (r < g.m) store_out<DT>(g.out, static_cast<int64_t>(r) * g.ldo + row, add ? acc[j] + bias : acc[j]);
                }
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, F::kTmemCols);
    }
}

template <typename Fn>
cudaError_t allow_smem(Fn fn, int bytes, std::atomic<uint64_t> &done) {
    // the shared-memory limit is a per-device attribute: set once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit && (done.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

constexpr int kSms = 152;  // of a full GB300; fewer only cost a second wave

template <int NT, int DT>
cudaError_t launch_few_t(const CUtensorMap &tw, const CUtensorMap &tws, const CUtensorMap &ta, const Fp8Args &g, int grid,
                         cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const void *fn = reinterpret_cast<const void *>(&fp8_few_kernel<NT, DT>);
    cudaError_t e = allow_smem(fn, Few<NT>::kSmem, done);
    if (e != cudaSuccess) return e;
    void *args[] = {const_cast<CUtensorMap *>(&tw), const_cast<CUtensorMap *>(&tws), const_cast<CUtensorMap *>(&ta),
                    const_cast<Fp8Args *>(&g)};
    return cudaLaunchKernel(fn, dim3(grid), dim3(Few<NT>::kThreads), args, Few<NT>::kSmem, s);
}
template <int NT>
cudaError_t launch_few(const void *A, int64_t lda, const void *B, int64_t ldb, Fp8Args g, int dtype, cudaStream_t s) {
    const int mt = (g.m + NT - 1) / NT, units = (g.n + kFewBox - 1) / kFewBox;
    int shares = kSms / mt > 0 ? kSms / mt : 1;
    if (shares > units) shares = units;
    g.shares = shares;
    CUtensorMap tw, tws, ta;  // weight boxes of a whole tile, and of 16 rows for a share's last one
    cudaError_t e = make_tmap_bytes(&tw, B, g.n, g.K, ldb, kFewM);
    if (e == cudaSuccess) e = make_tmap_bytes(&tws, B, g.n, g.K, ldb, kFewBox);
    if (e == cudaSuccess) e = make_tmap_bytes(&ta, A, g.m, g.K, lda, NT);
    if (e != cudaSuccess) return e;
    const int grid = shares * mt;
    if (dtype == CE_DT_BF16) return launch_few_t<NT, CE_DT_BF16>(tw, tws, ta, g, grid, s);
    if (dtype == CE_DT_F16) return launch_few_t<NT, CE_DT_F16>(tw, tws, ta, g, grid, s);
    return launch_few_t<NT, CE_DT_F32>(tw, tws, ta, g, grid, s);
}

cudaError_t fp8_gemm(const void *A, int64_t lda, const void *B, int64_t ldb, const Fp8Args &g, int dtype, cudaStream_t s) {
    if (g.m <= 16) return launch_few<16>(A, lda, B, ldb, g, dtype, s);
    if (g.m <= 32) return launch_few<32>(A, lda, B, ldb, g, dtype, s);
    if (g.m <= 64) return launch_few<64>(A, lda, B, ldb, g, dtype, s);
    return launch_few<128>(A, lda, B, ldb, g, dtype, s);
}

}  // namespace

}  // namespace ce

using namespace ce;

extern "C" ce_status ce_gemm_fp8(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const float *a_scale,
                                 const void *B, int64_t ldb, const float *b_scale, const float *bias, int32_t dtype,
                                 void *D, int64_t ldd, void *stream) {
    if (M < 0 || N < 0 || K < 1 || !fp8_dtype_ok(dtype)) return CE_ERR_INVALID_ARG;
    if (lda < K || ldb < K || ldd < N || lda % 16 || ldb % 16) return CE_ERR_INVALID_ARG;
    // tile origins and counters are 32-bit
    constexpr int64_t kMost = (int64_t(1) << 31) - 1024;
    if (M > kMost || N > kMost || K > kMost) return CE_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return CE_OK;
    if (!A || !B || !D || !a_scale || !b_scale) return CE_ERR_INVALID_ARG;
    if (!fp8_on(A, 16) || !fp8_on(B, 16) || !fp8_on(D, fp8_elem(dtype)) || !fp8_on(a_scale, 4) || !fp8_on(b_scale, 4) ||
        !fp8_on(bias, 4))
        return CE_ERR_INVALID_ARG;
    Fp8Args g{};
    g.m = static_cast<int>(M);
    g.n = static_cast<int>(N);
    g.K = static_cast<int>(K);
    g.kblocks = static_cast<int>((K + kFp8Block - 1) / kFp8Block);
    const int64_t db = ((M - 1) * ldd + N) * fp8_elem(dtype);
    if (!fp8_apart(D, db, A, (M - 1) * lda + K) || !fp8_apart(D, db, B, (N - 1) * ldb + K) ||
        !fp8_apart(D, db, a_scale, M * g.kblocks * 4) || !fp8_apart(D, db, b_scale, (N + 127) / 128 * g.kblocks * 4) ||
        (bias && !fp8_apart(D, db, bias, N * 4)))
        return CE_ERR_INVALID_ARG;
    g.a_scale = a_scale;
    g.b_scale = b_scale;
    g.bias = bias;
    g.out = D;
    g.ldo = ldd;
    const cudaError_t e = fp8_gemm(A, lda, B, ldb, g, dtype, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CE_OK : cuda_fail(e);
}
