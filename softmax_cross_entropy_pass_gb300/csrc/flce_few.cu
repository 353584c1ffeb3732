// flce_few.cu -- log-probability statistics of a linear head for few rows (up
// to 64: single tokens, a decoding batch). Bound by reading the weights once:
// 128256 x 4096 bf16 are 1.05 GB, 155 us at the measured copy rate.
//
// The vocabulary is the tensor core's M side: a CTA multiplies tiles of 128
// weight rows with all hidden rows (N = 16, 32 or 64) and owns a contiguous
// share of the vocabulary cut at multiples of 16 rows, so that one CTA per SM
// ends with the others (whole 256-column tiles leave the last of four waves a
// third full). Weights go through a ring of 16 KB stages by TMA; a share's last
// tile loads only the rows it has. Partial products of 256 K
// columns go to their own accumulator in tensor memory and are added up by the
// epilogue in registers (the tensor core's long sums truncate). Every epilogue
// thread keeps the running statistics of its weight rows for 16 hidden rows;
// they meet across lanes once, at the end.
#include <atomic>

#include "ce_device.cuh"
#include "flce.h"
#include "lp_device.cuh"
#include "tc_device.cuh"

namespace ce {

constexpr int kFewM = 128, kFewK = 64;
constexpr int kFewWBytes = kFewM * kFewK * 2;   // 16 KB of weights a stage
constexpr int kFewBoxRows = 16;                 // the unit of the shares
constexpr int kFewBoxBytes = kFewBoxRows * kFewK * 2;
constexpr int kFewPartSteps = 4;                // K steps of one accumulator
constexpr int kFewAcc = 8;                      // accumulators in flight
constexpr int kFewMaxStages = 12;
constexpr int kFewSmem = 222 * 1024;

struct FewArgs {
    int n, V, H, N;          // N: hidden rows of a tile (16, 32 or 64)
    int stages;
    const float *bias;
    const void *target;
    int tgt32;
    int64_t ignore_index;
    float k;
    int entropy;
    float4 *part;
    float *xy;
    unsigned int *status;
};

// one value into a row's statistics
template <bool ENT>
__device__ inline void few_add(LpState &st, float x, float k) {
    if (x > st.m) lp_rebase<ENT>(st, x, k);
    if (st.m == -INFINITY) {
        if (x != x) st.s = x;
        return;
    }
    const float a = lp_clamp((x - st.m) * k), e = ex2_hw(a);
    st.s += e;
    if (ENT) st.u = fmaf(e, a, st.u);
}

__global__ void __launch_bounds__(64 + 128 * 4, 1)
flce_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWs,
                const __grid_constant__ CUtensorMap tmH, FewArgs g) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kFewMaxStages], empty[kFewMaxStages], tfull[kFewAcc], tempty[kFewAcc];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, drain_abort;
    __shared__ int tgt[kFewMaxRows];
    __shared__ float red_mem[kFewMaxRows * 4 * 3];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nsets = g.N / 16;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // 128-byte swizzle atoms
    const uint32_t stage_bytes = kFewWBytes + g.N * kFewK * 2;
    volatile int *abort = &abort_flag;
    // this CTA's share of the vocabulary, in units of kFewBoxRows rows
    const int64_t units = (g.V + kFewBoxRows - 1) / kFewBoxRows;
    const int v_lo = static_cast<int>(units * blockIdx.x / gridDim.x) * kFewBoxRows;
    const int v_end = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x) * kFewBoxRows;
    const int v_hi = v_end < g.V ? v_end : g.V;
    const int ntiles = (v_hi - v_lo + kFewM - 1) / kFewM;
    const int ksteps = (g.H + kFewK - 1) / kFewK;
    const int nparts = (ksteps + kFewPartSteps - 1) / kFewPartSteps;
    const uint32_t tmem_cols = kFewAcc * g.N;

    if (tid == 0) {
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < kFewAcc; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 4 * nsets);
        }
        abort_flag = drain_abort = 0;
        if (blockIdx.x == 0) *g.status = 0u;  // no wait can have given up yet (they run for 2 s)
        fence_mbar_init_cluster();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmWs);
        tma_prefetch_desc(&tmH);
    }
    for (int r = tid; r < kFewMaxRows; r += blockDim.x) {
        int64_t t = r < g.n ? load_target(g.target, g.tgt32, r) : -1;
        tgt[r] = r < g.n && target_valid(t, g.ignore_index, g.V) ? static_cast<int>(t) : -1;
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            // (stage and round are counted, not divided out: one thread issues every copy)
            uint32_t s = 0, round = 0;
            for (int tile = 0; tile < ntiles; ++tile) {
                const int v0 = v_lo + tile * kFewM;
                const int boxes = (min(kFewM, v_hi - v0) + kFewBoxRows - 1) / kFewBoxRows;
                const uint32_t bytes = boxes * kFewBoxBytes + g.N * kFewK * 2;
                for (int ks = 0; ks < ksteps; ++ks) {
                    const uint32_t fb = smem_u32(&full[s]), dst = base + s * stage_bytes;
                    if (round > 0) mbar_wait_bounded<false>(smem_u32(&empty[s]), (round - 1) & 1u, abort);
                    mbar_expect_tx(fb, bytes);
                    if (boxes == kFewM / kFewBoxRows) {
                        tma_load_2d(dst, &tmW, ks * kFewK, v0, fb);
                    } else {
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(dst + b * kFewBoxBytes, &tmWs, ks * kFewK, v0 + b * kFewBoxRows, fb);
                    }
                    tma_load_2d(dst + kFewWBytes, &tmH, ks * kFewK, 0, fb);
                    if (++s == static_cast<uint32_t>(g.stages)) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // the copies in flight, with a limit of their own where another wait gave up
            const uint32_t used = round > 0 ? static_cast<uint32_t>(g.stages) : s;
            for (uint32_t i = 0; i < used; ++i) {
                const uint32_t uses = round + (i < s ? 1u : 0u);  // of stage i
                mbar_wait_bounded<false>(smem_u32(&full[i]), (uses - 1) & 1u, &drain_abort);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------ MMA issuer
            const uint32_t idesc = idesc_bf16_f32(kFewM, g.N, 0, 0);
            uint32_t s = 0, phase = 0, unit = 0;
            for (int tile = 0; tile < ntiles; ++tile)
                for (int pt = 0; pt < nparts; ++pt, ++unit) {
                    const uint32_t acc = unit % kFewAcc, u = unit / kFewAcc;
                    if (u > 0) mbar_wait_bounded<false>(smem_u32(&tempty[acc]), (u - 1) & 1u, abort);
                    tc_fence_after();
                    const int kb = pt * kFewPartSteps, ke = min(ksteps, kb + kFewPartSteps);
                    for (int ks = kb; ks < ke; ++ks) {
                        mbar_wait_bounded<false>(smem_u32(&full[s]), phase, abort);
                        tc_fence_after();
                        const uint32_t a = base + s * stage_bytes, b = a + kFewWBytes;
#pragma unroll
                        for (int kk = 0; kk < kFewK / 16; ++kk)
                            mma_bf16(tmem + acc * g.N, smem_desc_sw128(a + kk * 32, 16, 1024),
                                     smem_desc_sw128(b + kk * 32, 16, 1024), idesc, (ks > kb || kk > 0) ? 1u : 0u);
                        mma_commit(smem_u32(&empty[s]));
                        if (++s == static_cast<uint32_t>(g.stages)) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
                    mma_commit(smem_u32(&tfull[acc]));
                }
        }
    } else if (warp - 2 < 4 * nsets) {
        // ---------------------------------------------------- epilogue: 4 warps for every 16 hidden rows
        const int q = warp & 3, set = (warp - 2) >> 2;  // tensor memory lanes, hidden rows
        const float k = g.k;
        LpState st[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) st[j] = lp_empty();
        uint32_t unit = 0;
        for (int tile = 0; tile < ntiles; ++tile) {
            float acc[16];
            for (int pt = 0; pt < nparts; ++pt, ++unit) {
                const uint32_t a = unit % kFewAcc, u = unit / kFewAcc;
                mbar_wait_bounded<false>(smem_u32(&tfull[a]), u & 1u, abort);
                tc_fence_after();
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + a * g.N + set * 16, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[j] = pt == 0 ? __uint_as_float(v[j]) : acc[j] + __uint_as_float(v[j]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&tempty[a]));
            }
            const int col = v_lo + tile * kFewM + q * 32 + lane;
            if (col < v_hi) {
                const float bias = g.bias ? __ldg(g.bias + col) : 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int row = set * 16 + j;
                    if (row < g.n) {
                        const float x = acc[j] + bias;
                        if (tgt[row] == col) g.xy[row] = x;
                        else if (g.entropy) few_add<true>(st[j], x, k);
                        else few_add<false>(st[j], x, k);
                    }
                }
            }
        }
        // the lanes' statistics, row by row, then those of the four warps of a row set
        LpState(*red)[4] = reinterpret_cast<LpState(*)[4]>(red_mem);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const LpState m = lp_warp_merge<true>(st[j], k);
            if (lane == 0) red[set * 16 + j][q] = m;
        }
        asm volatile("bar.sync 1, %0;" ::"r"(128 * nsets) : "memory");
        const int row = tid - 64;
        if (row < g.n) {
            LpState m = red[row][0];
            for (int i = 1; i < 4; ++i) m = lp_merge<true>(m, red[row][i], k);
            g.part[static_cast<int64_t>(row) * gridDim.x + blockIdx.x] = make_float4(m.m, m.s, m.u, 0.f);
        }
    }
    pdl_launch_dependents();  // the kernel that merges the parts may be set up meanwhile
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tmem_cols);
    }
    if (tid == 0 && abort_flag) atomicOr(g.status, CE_FLAG_WAIT_TIMEOUT);
}

// One CTA per SM of a full GB300, fixed so that the workspace is a function of
// the sizes alone; fewer where the vocabulary has fewer units of 16 rows.
static int few_blocks(int64_t V) {
    const int64_t units = (V + kFewBoxRows - 1) / kFewBoxRows;
    return static_cast<int>(units < 152 ? units : 152);
}
int flce_few_parts(int64_t V) { return few_blocks(V); }

cudaError_t flce_few(int n, int V, int H, const void *hidden, const void *weight, const float *bias, const void *target,
                     int tgt32, int64_t ignore_index, float k, int entropy, float4 *part, float *xy, unsigned int *status,
                     cudaStream_t s) {
    FewArgs g{};
    g.n = n; g.V = V; g.H = H;
    g.N = n <= 16 ? 16 : (n <= 32 ? 32 : 64);
    const int stage = kFewWBytes + g.N * kFewK * 2;
    g.stages = (kFewSmem - 1024) / stage;
    if (g.stages > kFewMaxStages) g.stages = kFewMaxStages;
    g.bias = bias; g.target = target; g.tgt32 = tgt32; g.ignore_index = ignore_index;
    g.k = k; g.entropy = entropy; g.part = part; g.xy = xy; g.status = status;
    CUtensorMap tw, tws, th;  // weight boxes of a whole tile, and of 16 rows for a share's last one
    cudaError_t e = make_tmap(&tw, weight, V, H, H, kFewK, kFewM);
    if (e == cudaSuccess) e = make_tmap(&tws, weight, V, H, H, kFewK, kFewBoxRows);
    if (e == cudaSuccess) e = make_tmap(&th, hidden, n, H, H, kFewK, g.N);
    if (e != cudaSuccess) return e;
    // the shared-memory limit is a per-device attribute: set once per device
    static std::atomic<uint64_t> attr_set{0};
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (!bit || !(attr_set.load() & bit)) {
        e = cudaFuncSetAttribute(flce_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit);
    }
    void *args[] = {&tw, &tws, &th, &g};
    return cudaLaunchKernel(reinterpret_cast<const void *>(&flce_few_kernel), dim3(few_blocks(V)),
                            dim3(64 + 128 * (g.N / 16)), args, 1024 + g.stages * stage, s);
}

}  // namespace ce
