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
// weight rows by NT rows of A. Either it owns a contiguous share of the weight's
// rows, cut at multiples of 16, so that one CTA per SM ends with the others; or,
// where that share would be less than half a tile, a cluster of up to eight CTAs
// takes one tile, each a part of K, and adds the parts up through distributed
// shared memory, in the order of the ranks (a K block's copies, MMAs and epilogue
// follow one another in 0.3 us whatever the rows: 64 x 4096 x 4096 took 14.9 us in
// 32 such steps, 11.1 in a cluster's 8).
#include <atomic>
#include <type_traits>

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
    int shares;               // CTAs (clusters) along the weight's rows
    int ksplit;               // CTAs of a cluster, each a part of K
};

// A block's sum v counts v sa sb. Where sa sb is a normal fp32 number that is one
// product with it, and the addition. Scales may be others, though: below 2^-126 their
// product has few bits or none while v (up to 2^24.6) lifts the result back, above fp32's
// range it is infinite while v may be 0, or 2^-18.
// Few rows: an epilogue warp looks whether a product of its scales over a chunk of K
// blocks leaves the normal range, and has a loop of its own for such chunks, in which v is
// multiplied by pre, the product 2^64 nearer to 1, and post = 2^-64 or 2^64 brings the result
// back in the addition. Pairs have no registers for a second loop (beside one the ordinary
// loop took 17% longer): there the sums are kept 2^(ea + eb) times what they stand for
// where the scales lie far from 1, ea a row's and eb the columns', which is exact.
// Scales of 2^-126, the least that quantising gives (blocks of zeros, and those with nothing
// above 5.3e-36), do not count.
struct Scaled {
    float pre, post;
};
__device__ inline Scaled scaled(float sa, float sb) {
    const float w = sa * sb;
    const bool numbers = fabsf(sa) < INFINITY && fabsf(sb) < INFINITY && sa != 0.f && sb != 0.f;
    const bool plain = (fabsf(w) >= 0x1p-126f && fabsf(w) < INFINITY) || !numbers, low = fabsf(w) < 1.f;
    const float far = sa * (low ? 0x1p64f : 0x1p-64f) * sb;
    // (past the largest number the result is infinite, or 0 where v is)
    const float pre = copysignf(fminf(fabsf(far), 3.402823466e38f), far);
    return Scaled{plain ? 1.f : pre, plain ? w : (low ? 0x1p-64f : 0x1p64f)};
}
// no product of two such leaves the normal range (or counts)
__device__ inline bool scale_ordinary(float v) { return (v >= 0x1p-50f && v <= 0x1p50f) || v == kFp8MinScale; }
// the ends of a set of magnitudes, but zeros, infinities, NaN and the least scale
struct Ends {
    float least = INFINITY, most = 0.f;
    __device__ inline void take(float v) {
        v = fabsf(v);
        const bool counts = v != 0.f && v != kFp8MinScale && v < INFINITY;
        least = fminf(least, counts ? v : INFINITY);
        most = fmaxf(most, counts ? v : 0.f);
    }
    __device__ inline void join(const Ends &o) {
        least = fminf(least, o.least);
        most = fmaxf(most, o.most);
    }
    // whether a product of the two sets leaves the normal range
    __device__ inline bool leave(const Ends &o) const {
        return most > 0.f && o.most > 0.f && (least * o.least < 0x1p-126f || most * o.most > 3.402823466e38f);
    }
};

template <int DT>
__device__ inline void store_out(void *out, int64_t i, float v) { Fmt<DT>::store1(out, i, v); }

constexpr int kFewM = 128;                    // weight rows of a tile
constexpr int kFewWBytes = kFewM * kFp8Block; // 16 KB of weights a stage
constexpr int kFewBox = 16;                   // rows of the small boxes, the unit of the shares
constexpr int kFewMaxStages = 12;
constexpr int kFewSmem = 218 * 1024;
constexpr int kScaleBlocks = 32;              // K blocks whose scales of A are in shared memory at a time

// NT rows of A a tile, kCols of them an epilogue thread
template <int NT> struct Few {
    static constexpr int kCols = NT < 32 ? NT : 32;
    static constexpr int kSets = NT / kCols;
    static constexpr int kThreads = 64 + 128 * kSets;
    static constexpr int kAcc = 8;  // accumulators in tensor memory
    static constexpr uint32_t kTmemCols = kAcc * NT;
    static constexpr int kStageBytes = kFewWBytes + NT * kFp8Block;
    static constexpr int kScaleBytes = kScaleBlocks * NT * 4;
    static constexpr int kStages = (kFewSmem - 1024 - kScaleBytes) / kStageBytes < kFewMaxStages
                                       ? (kFewSmem - 1024 - kScaleBytes) / kStageBytes : kFewMaxStages;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kScaleBytes;
    static_assert(kStages * kStageBytes >= NT * kFewM * 4, "a cluster's partial tiles take the stages' place");
};

template <int C>
__device__ inline void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[C]) {
    if constexpr (C == 16) tmem_ld_32x32b_x16(taddr, v);
    else tmem_ld_32x32b_x32(taddr, v);
}
__device__ inline float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int NT, int DT>
__global__ void __launch_bounds__(Few<NT>::kThreads, 1)
fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWs,
               const __grid_constant__ CUtensorMap tmA, Fp8Args g) {
    using F = Few<NT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[F::kStages], empty[F::kStages], tfull[F::kAcc], tempty[F::kAcc], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, drain_abort[2];
    __shared__ int ordinary[4 * F::kSets];  // whether all scales of A that an epilogue warp has put into shared memory are
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;  // 128-byte swizzle atoms
    float *parts = reinterpret_cast<float *>(smem_raw + (base - raw));  // [NT][kFewM], once the stages are done with
    float *scales = reinterpret_cast<float *>(smem_raw + (base - raw) + F::kStages * F::kStageBytes);  // [kScaleBlocks][NT]
    volatile int *abort = &abort_flag;
    const int split = g.ksplit, rank = static_cast<int>(blockIdx.x) % split, work = static_cast<int>(blockIdx.x) / split;
    const int share = work % g.shares, m0 = work / g.shares * NT;
    const int64_t units = (g.n + kFewBox - 1) / kFewBox;
    // split: shares are tiles
    const int v_lo = split > 1 ? share * kFewM : static_cast<int>(units * share / g.shares) * kFewBox;
    const int v_end = split > 1 ? v_lo + kFewM : static_cast<int>(units * (share + 1) / g.shares) * kFewBox;
    const int v_hi = v_end < g.n ? v_end : g.n;
    const int ntiles = (v_hi - v_lo + kFewM - 1) / kFewM;
    const int kb0 = static_cast<int>(static_cast<int64_t>(g.kblocks) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(g.kblocks) * (rank + 1) / split);

    if (tid == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < F::kAcc; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 4 * F::kSets);
        }
        mbar_init(smem_u32(&done), 1);
        abort_flag = drain_abort[0] = drain_abort[1] = 0;
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
        if (elect_one()) {
            // ------------------------------------------------ TMA producer
            uint32_t s = 0, round = 0;
            for (int tile = 0; tile < ntiles; ++tile) {
                const int v0 = v_lo + tile * kFewM;
                const int boxes = (min(kFewM, v_hi - v0) + kFewBox - 1) / kFewBox;
                const uint32_t bytes = boxes * kFewBox * kFp8Block + NT * kFp8Block;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const uint32_t fb = smem_u32(&full[s]), dst = base + s * F::kStageBytes;
                    if (round > 0) mbar_wait_polled(smem_u32(&empty[s]), (round - 1) & 1u, abort);
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
                mbar_wait_polled(smem_u32(&full[i]), (uses - 1) & 1u, &drain_abort[0]);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ------------------------------------------------ MMA issuer: one accumulator a K block
            const uint32_t idesc = idesc_e4m3_f32(kFewM, NT);
            uint32_t s = 0, phase = 0, unit = 0;
            for (int tile = 0; tile < ntiles; ++tile)
                for (int kb = kb0; kb < kb1; ++kb, ++unit) {
                    const uint32_t acc = unit % F::kAcc, u = unit / F::kAcc;
                    if (u > 0) mbar_wait_polled(smem_u32(&tempty[acc]), (u - 1) & 1u, abort);
                    mbar_wait_polled(smem_u32(&full[s]), phase, abort);
                    tc_fence_after();
                    const uint32_t a = base + s * F::kStageBytes, b = a + kFewWBytes;
#pragma unroll
                    for (int kk = 0; kk < kFp8Block / 32; ++kk)
                        mma_e4m3(tmem + acc * NT, smem_desc_sw128(a + kk * 32, 16, 1024),
                                 smem_desc_sw128(b + kk * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
                    mma_commit(smem_u32(&tfull[acc]));
                    mma_commit(smem_u32(&empty[s]));
                    if (++s == F::kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            // the MMAs in flight end before tensor memory is given back, whatever the epilogue waited for
            mma_commit(smem_u32(&done));
            mbar_wait_polled(smem_u32(&done), 0, &drain_abort[1]);
        }
    } else {
        // ---------------------------------------------------- epilogue: 4 warps for every kCols rows of A
        constexpr int C = F::kCols;
        const int q = warp & 3, set = (warp - 2) >> 2;  // tensor memory lanes, rows of A
        const int et = tid - 64;
        const uint32_t taddr0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + set * C;
        uint32_t unit = 0;
        bool a_in = true;  // all scales of A in shared memory are ordinary
        for (int tile = 0; tile < ntiles; ++tile) {
            const int row = v_lo + tile * kFewM + q * 32 + lane;
            const bool live = v_lo + tile * kFewM + q * 32 < v_hi;  // any row of this warp's
            const float *sb = g.b_scale + static_cast<int64_t>(min(row, g.n - 1) / kFp8Block) * g.kblocks;
            F2 acc[C / 2];
#pragma unroll
            for (int j = 0; j < C / 2; ++j) acc[j] = f2(0.f, 0.f);
            float next = __ldg(sb + kb0);
            // K blocks c0 .. c1 - 1, whose scales of A are in shared memory
            const auto blocks = [&](auto far, int c0, int c1) {
                for (int kb = c0; kb < c1; ++kb, ++unit) {
                    const int k0 = kb - c0;
                    const float sb1 = next;
                    const F2 w = f2(next, next);
                    if (kb + 1 < kb1) next = __ldg(sb + kb + 1);
                    const uint32_t a = unit % F::kAcc, u = unit / F::kAcc;
                    mbar_wait_polled(smem_u32(&tfull[a]), u & 1u, abort);
                    if (live) {
                        tc_fence_after();
                        uint32_t v[C];
                        tmem_ld_cols<C>(taddr0 + a * NT, v);
                        tmem_ld_wait(v);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&tempty[a]));
                        const float4 *sa = reinterpret_cast<const float4 *>(scales + k0 * NT + set * C);
#pragma unroll
                        for (int j = 0; j < C / 4; ++j) {
                            const float4 s4 = sa[j];
                            if constexpr (decltype(far)::value) {
                                const Scaled p0 = scaled(s4.x, sb1), p1 = scaled(s4.y, sb1), p2 = scaled(s4.z, sb1), p3 = scaled(s4.w, sb1);
                                acc[2 * j] = f2_fma(f2(p0.post, p1.post), f2_mul(f2(p0.pre, p1.pre), f2(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]))), acc[2 * j]);
                                acc[2 * j + 1] = f2_fma(f2(p2.post, p3.post), f2_mul(f2(p2.pre, p3.pre), f2(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]))), acc[2 * j + 1]);
                            } else {
                                acc[2 * j] = f2_fma(f2_mul(f2(s4.x, s4.y), w), f2(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])), acc[2 * j]);
                                acc[2 * j + 1] = f2_fma(f2_mul(f2(s4.z, s4.w), w), f2(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])), acc[2 * j + 1]);
                            }
                        }
                    } else if (lane == 0) {
                        mbar_arrive(smem_u32(&tempty[a]));
                    }
                }
            };
            for (int c0 = kb0; c0 < kb1; c0 += kScaleBlocks) {
                const int nb = min(kScaleBlocks, kb1 - c0);
                // the weight's scales of K block `lane` of the chunk, for the warp's first row and its last (32 rows are in two blocks at most)
                const int row0 = v_lo + tile * kFewM + q * 32;
                const float first = lane < nb ? __ldg(g.b_scale + static_cast<int64_t>(min(row0, g.n - 1) / kFp8Block) * g.kblocks + c0 + lane) : 1.f;
                const float last = lane < nb ? __ldg(g.b_scale + static_cast<int64_t>(min(row0 + 31, g.n - 1) / kFp8Block) * g.kblocks + c0 + lane) : 1.f;
                if (tile == 0 || kb1 - kb0 > kScaleBlocks) {
                    // the next blocks' scales of A, rows of the tile side by side
                    asm volatile("bar.sync 1, %0;" ::"r"(128 * F::kSets) : "memory");
                    bool in = true;
                    for (int i = et; i < kScaleBlocks * NT; i += 128 * F::kSets) {
                        const int r = i / kScaleBlocks, b = i % kScaleBlocks;
                        if (b < nb) {
                            const float v = m0 + r < g.m ? __ldg(g.a_scale + static_cast<int64_t>(m0 + r) * g.kblocks + c0 + b) : 1.f;
                            scales[b * NT + r] = v;
                            in = in && scale_ordinary(v);
                        }
                    }
                    in = __all_sync(0xffffffffu, in);
                    if (lane == 0) ordinary[warp - 2] = in ? 1 : 0;
                    asm volatile("bar.sync 1, %0;" ::"r"(128 * F::kSets) : "memory");
                    a_in = true;
#pragma unroll
                    for (int i = 0; i < 4 * F::kSets; ++i) a_in = a_in && ordinary[i] != 0;
                }
                bool far = false;
                if (!__all_sync(0xffffffffu, a_in && scale_ordinary(first) && scale_ordinary(last))) {
                    Ends a_ends, b_ends;
                    b_ends.take(first);
                    b_ends.take(last);
                    for (int i = 0; i < NT && lane < nb; ++i) a_ends.take(scales[lane * NT + (i + lane) % NT]);  // (a bank a lane)
                    far = __any_sync(0xffffffffu, a_ends.leave(b_ends));
                }
                if (far) blocks(std::true_type(), c0, c0 + nb);
                else blocks(std::false_type(), c0, c0 + nb);
            }
            float x[C];
#pragma unroll
            for (int j = 0; j < C / 2; ++j) f2_split(acc[j], x[2 * j], x[2 * j + 1]);
            const bool bad = *abort != 0;  // a wait that gave up leaves no result
            if (split > 1) {
                // every copy of this CTA has landed and every MMA has read it
#pragma unroll
                for (int j = 0; j < C; ++j) parts[(set * C + j) * kFewM + q * 32 + lane] = bad ? NAN : x[j];
            } else if (row < v_hi) {
                const float bias = g.bias ? __ldg(g.bias + row) : 0.f;
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const int r = m0 + set * C + j;
                    if (r < g.m) store_out<DT>(g.out, static_cast<int64_t>(r) * g.ldo + row, bad ? NAN : (g.bias ? x[j] + bias : x[j]));
                }
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, F::kTmemCols);
    }
    if (split > 1) {
        // this rank's share of the rows of A: the parts' sums
        cluster_sync_all();
        const int c0 = NT * rank / split, c1 = min(NT * (rank + 1) / split, g.m - m0);
        const uint32_t mine = smem_u32(parts);
        for (int i = tid; i < (c1 - c0) * kFewM; i += F::kThreads) {
            const int c = c0 + i / kFewM, r = i % kFewM, row = v_lo + r;
            if (row >= v_hi) continue;
            float v = 0.f;
            for (int k = 0; k < split; ++k) v += ld_cluster_f32(mapa_shared(mine + (c * kFewM + r) * 4, k));
            if (g.bias) v += __ldg(g.bias + row);
            store_out<DT>(g.out, static_cast<int64_t>(m0 + c) * g.ldo + row, v);
        }
        cluster_sync_all();  // no CTA leaves while another reads its part
    }
}

// ------------------------------------------------------------------ CTA pairs
// fp8_pair_kernel: many rows of A. A pair of CTAs (a cluster of 2, one CTA per
// SM) per tile of 256 rows of A and 256 of the weight: the even CTA issues
// tcgen05.mma.cta_group::2, each CTA loads its 128 rows of either operand a K
// block (32 KB) and holds its 128 rows of the accumulator, 256 of the 512 columns
// of tensor memory. Every K block's sums have to leave tensor memory before it is
// used again, so the time from the end of a K block's MMAs to its accumulator's
// return shows wherever it is longer than the next block's MMAs. Eight
// epilogue warps a CTA scale and add a row and 128 columns a thread, with one scale
// of A (through shared memory, copied half a chunk ahead) and one of the weight.
// 4096 x 128256 x 4096: 1740 to 1780 us (GPUs differ), 2.4 PFLOP/s. At 2048 rows, on a GPU
// with 833 us: without the adds 699, with them but without the loads 719: each hides behind
// the MMAs, the two one after the other in a warp do not. Slower there: tiles of 224, 192,
// 160 (three accumulators) and 128 columns (four), a thread's share loaded whole and given
// back before it is added, 894, 950, 1046 and 1036 us; sixteen epilogue warps 952; no change:
// sums that leave through shared memory behind the next tile's, 820.
// Barriers as in the bf16 product: `full` in the even CTA counts both CTAs'
// bytes, `empty` and `tfull` are signalled by multicast commits, `tempty` in the
// even CTA collects the 16 epilogue warps of the pair (each arrival from the other
// CTA takes 6 ns: sixteen warps a CTA with half the columns were slower).
constexpr int kPairM = 256, kPairN = 256, kPairAcc = 2;
constexpr int kPairHalf = 128 * kFp8Block;  // 16 KB: this CTA's half of an operand's stage
constexpr int kPairEpi = 256;
// four warps for the copies and the MMAs (two of them idle), so that warpgroups
// can trade registers: launched with 168 a thread, the epilogue's two
// warpgroups take 232 and the first keeps 40 (2 x 128 x 232 + 128 x 40 = 384 x 168)
constexpr int kPairThreads = 128 + kPairEpi;
constexpr int kPairLaunchRegs = 168, kPairEpiRegs = 232, kPairFirstRegs = 40;
static_assert(kPairEpi == kPairN, "a column's bias a thread");
static_assert(kPairEpi * kPairEpiRegs + 128 * kPairFirstRegs <= kPairThreads * kPairLaunchRegs, "registers of the launch");
constexpr int kPairChunk = 32;              // K blocks whose scales of A are in shared memory
constexpr int kPairRow = 129;               // floats of one K block's scales: another bank for each block
constexpr int kPairStage = 32 * 33;         // floats: 32 x 32 sums of an epilogue warp on their way out
constexpr int kPairStages = 5;
constexpr int pair_smem(bool staged) {
    return 1024 + kPairStages * 2 * kPairHalf + 2 * kPairChunk * kPairRow * 4 +
           (staged ? kPairEpi / 32 * kPairStage : kPairN) * 4;
}
constexpr uint32_t kPairTmemCols = 512;

// 32 bytes to a 32-byte aligned address: a whole sector a lane (rows lie apart)
__device__ inline void st_sector(void *p, const uint4 &a, const uint4 &b) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
}

// 16 consecutive columns of one row from column c on; rows start on whole sectors
template <int DT>
__device__ inline void store_cols(const Fp8Args &g, int row, int c, float (&x)[16], const float *bias, bool bad) {
    if (g.bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 b = *reinterpret_cast<const float4 *>(bias + 4 * j);
            x[4 * j] += b.x; x[4 * j + 1] += b.y; x[4 * j + 2] += b.z; x[4 * j + 3] += b.w;
        }
    }
    if (bad) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = NAN;
    }
    const int64_t at = static_cast<int64_t>(row) * g.ldo + c;
    if (c + 16 <= g.n) {
        char *o = reinterpret_cast<char *>(g.out) + at * Fmt<DT>::kBytes;
        st_sector(o, Fmt<DT>::pack(x), Fmt<DT>::pack(x + Fmt<DT>::kVec));
        if (DT == CE_DT_F32) st_sector(o + 32, Fmt<DT>::pack(x + 8), Fmt<DT>::pack(x + 12));
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (c + j < g.n) store_out<DT>(g.out, at + j, x[j]);
    }
}

// 32 rows (a lane's each) of 32 columns from column c on through a warp's shared
// memory, so that lanes store neighbouring columns: for rows that start anywhere
// (a lane storing its own row would touch 32 sectors a store). 300 x 50257 x 2048 in
// fp32: 75 us, 64 where rows start on sectors.
template <int DT>
__device__ inline void store_staged(const Fp8Args &g, int row0, int c, const F2 *acc, float *stage, bool bad) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 16; ++j) f2_split(acc[j], stage[lane * 33 + 2 * j], stage[lane * 33 + 2 * j + 1]);
    __syncwarp();
    const int col = c + lane;
    if (col < g.n) {
        const float bias = g.bias ? __ldg(g.bias + col) : 0.f;
        const int64_t at = static_cast<int64_t>(row0) * g.ldo + col;
        if (row0 + 32 <= g.m && !bad) {
#pragma unroll 4
            for (int r = 0; r < 32; ++r) store_out<DT>(g.out, at + r * g.ldo, g.bias ? stage[r * 33 + lane] + bias : stage[r * 33 + lane]);
        } else {
            for (int r = 0; r < min(32, g.m - row0); ++r)
                store_out<DT>(g.out, at + r * g.ldo, bad ? NAN : (g.bias ? stage[r * 33 + lane] + bias : stage[r * 33 + lane]));
        }
    }
    __syncwarp();
}

// 2^e, e in [-126, 127]
__device__ inline float pow2(int e) { return __int_as_float((e + 127) << 23); }
// the power of 2 that brings scales whose largest is `most` (0: none) up to 2^30
__device__ inline int lift(float most) {
    const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;  // -127 below the normal range
    return most > 0.f ? max(-126, min(126, 30 - e)) : 0;
}
// 128 sums times 2^d, in steps that fp32 holds
__device__ inline void rescale(F2 (&sums)[64], int d) {
    const int step = d >> 2;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const float f = pow2(i < 3 ? step : d - 3 * step);
#pragma unroll
        for (int j = 0; j < 64; ++j) sums[j] = f2_mul(sums[j], f2(f, f));
    }
}

// STAGED: the output's rows do not all start on sectors
template <int DT, bool STAGED>
__global__ void __launch_bounds__(kPairThreads, 1)
fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Fp8Args g) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kPairStages], empty[kPairStages], tfull[kPairAcc], tempty[kPairAcc], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, drain_abort[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int cid = static_cast<int>(cluster_id_x()), ncl = static_cast<int>(nclusters_x());
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;  // the same offsets in both CTAs of the pair
    float *scales = reinterpret_cast<float *>(smem_raw + (base - raw) + kPairStages * 2 * kPairHalf);
    float *extra = scales + 2 * kPairChunk * kPairRow;  // the bias of this tile's columns; STAGED: the warps' sums on their way out
    const uint32_t sA = base, sB = base + kPairStages * kPairHalf;
    const int tiles_m = (g.m + kPairM - 1) / kPairM;
    const int tiles = tiles_m * ((g.n + kPairN - 1) / kPairN);

    if (tid == 0) {
        for (int st = 0; st < kPairStages; ++st) {
            mbar_init(smem_u32(&full[st]), 1);
            mbar_init(smem_u32(&empty[st]), 1);
        }
        for (int a = 0; a < kPairAcc; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 2 * kPairEpi / 32);
        }
        mbar_init(smem_u32(&done), 1);
        abort_flag = drain_abort[0] = drain_abort[1] = 0;
        fence_mbar_init_cluster();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any remote arrive or copy
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&tmem_slot), kPairTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairFirstRegs));
        if (warp == 0 && elect_one()) {
            // ------------------------------------------------ TMA producer (both CTAs)
            uint32_t s = 0, round = 0;
            for (int t = cid; t < tiles; t += ncl) {
                const int row0 = t % tiles_m * kPairM + static_cast<int>(rank) * 128;
                const int col0 = t / tiles_m * kPairN + static_cast<int>(rank) * 128;
                for (int kb = 0; kb < g.kblocks; ++kb) {
                    if (round > 0) mbar_wait_pair(smem_u32(&empty[s]), (round - 1) & 1u, &abort_flag);
                    const uint32_t fb = mapa_shared(smem_u32(&full[s]), 0);  // the even CTA's barrier
                    if (rank == 0) mbar_expect_tx(smem_u32(&full[s]), 4 * kPairHalf);
                    tma_load_2d_pair(sA + s * kPairHalf, &tmA, kb * kFp8Block, row0, fb);
                    tma_load_2d_pair(sB + s * kPairHalf, &tmB, kb * kFp8Block, col0, fb);
                    if (++s == kPairStages) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // the copies in flight, with a limit of their own where another wait gave up
            if (rank == 0) {
                const uint32_t used = round > 0 ? kPairStages : s;
                for (uint32_t i = 0; i < used; ++i) {
                    const uint32_t uses = round + (i < s ? 1u : 0u);
                    mbar_wait_polled(smem_u32(&full[i]), (uses - 1) & 1u, &drain_abort[0]);
                }
            }
        }
        if (warp == 1 && rank == 0 && elect_one()) {
            // ------------------------------------------------ MMA issuer (even CTA): one accumulator a K block
            const uint32_t idesc = idesc_e4m3_f32(kPairM, kPairN);
            uint32_t s = 0, phase = 0, unit = 0;
            for (int t = cid; t < tiles; t += ncl)
                for (int kb = 0; kb < g.kblocks; ++kb, ++unit) {
                    const uint32_t acc = unit & 1u, u = unit >> 1;
                    mbar_wait_pair(smem_u32(&full[s]), phase, &abort_flag);
                    if (u > 0) mbar_wait_pair(smem_u32(&tempty[acc]), (u - 1) & 1u, &abort_flag);
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kFp8Block / 32; ++kk)
                        mma_e4m3_pair(tmem + acc * kPairN, smem_desc_sw128(sA + s * kPairHalf + kk * 32, 16, 1024),
                                      smem_desc_sw128(sB + s * kPairHalf + kk * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
                    mma_commit_pair_mc(smem_u32(&tfull[acc]), 0x3);
                    mma_commit_pair_mc(smem_u32(&empty[s]), 0x3);
                    if (++s == kPairStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            // the MMAs in flight end before tensor memory is given back, whatever the epilogue waited for
            mma_commit_pair_mc(smem_u32(&done), 0x1);
            mbar_wait_polled(smem_u32(&done), 0, &drain_abort[1]);
        }
    } else {
        // ---------------------------------------------------- epilogue (warps 4..11, both CTAs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairEpiRegs));
        const int q = warp & 3, half = (warp - 4) >> 2;
        const int et = tid - 128;
        const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
        // scales of A of this CTA's 128 rows of tile t, K blocks k0 .. k0 + 31, into buffer `buf` (rows past the last: its)
        const auto fetch = [&](int t, int k0, int buf) {
            const int row0 = t % tiles_m * kPairM + static_cast<int>(rank) * 128;
            const int nb = min(kPairChunk, g.kblocks - k0), kb = et & 31;
            const uint32_t dst = smem_u32(scales + buf * kPairChunk * kPairRow + kb * kPairRow);
            if (kb < nb) {
#pragma unroll
                for (int r = et >> 5; r < 128; r += kPairEpi / 32) {
                    const float *src = g.a_scale + static_cast<int64_t>(min(row0 + r, g.m - 1)) * g.kblocks + k0 + kb;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + r * 4), "l"(src) : "memory");
                }
            }
        };
        uint32_t unit = 0, chunk = 0;  // K blocks and chunks of scales so far
        if (cid < tiles) fetch(cid, 0, 0);
        for (int t = cid; t < tiles; t += ncl) {
            const int row = t % tiles_m * kPairM + static_cast<int>(rank) * 128 + q * 32 + lane;
            const int col0 = t / tiles_m * kPairN + half * 128;
            // columns past the last are multiplied like it, and not stored
            const float *sb = g.b_scale + static_cast<int64_t>(min(col0, g.n - 1) / kFp8Block) * g.kblocks;
            F2 acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = f2(0.f, 0.f);
            float sb1 = 0.f;  // the weight's scale of K block `lane` of the chunk, times 2^eb
            // the sums are 2^(ea + eb) times what they stand for: the row's and the columns' part (fa = 2^ea); the largest
            // scales so far, b_most a lane's
            float fa = 1.f;
            struct {
                float a_most, b_most;
                int ea, eb;
            } dom = {0.f, 0.f, 0, 0};
            // halfway: the next chunk's scales, of this tile or the next
            const auto ahead = [&](int c0) {
                const int k1 = c0 + kPairChunk;
                if (k1 < g.kblocks) fetch(t, k1, chunk & 1u);
                else if (t < tiles - ncl) fetch(t + ncl, 0, chunk & 1u);
            };
            // K blocks c0 .. c1 - 1, whose scales of A are in shared memory
            const auto blocks = [&](int c0, int c1) {
                for (int kb = c0; kb < c1; ++kb, ++unit) {
                    const int k0 = kb - c0;
                    if (k0 == (c1 - c0) / 2) ahead(c0);
                    const float w1 = scales[((chunk - 1) & 1u) * kPairChunk * kPairRow + k0 * kPairRow + q * 32 + lane] * fa * __shfl_sync(0xffffffffu, sb1, k0);
                    const F2 w = f2(w1, w1);
                    const uint32_t a = unit & 1u;
                    mbar_wait_pair(smem_u32(&tfull[a]), (unit >> 1) & 1u, &abort_flag);
                    tc_fence_after();
                    const uint32_t taddr = lane_addr + a * kPairN;
                    const auto add = [&](const uint32_t *x, int n, int at) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j < n / 2)
                                acc[at / 2 + j] = f2_fma(f2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), w, acc[at / 2 + j]);
                    };
                    const auto give_back = [&] {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_relaxed(tempty0 + a * 8u);
                    };
                    // As many columns at once as fit beside the sums (all 128 do not), the others while those are added.
                    // With 96 at once registers spill (4096 x 128256 x 4096: 2091 us against 1809); without the row's
                    // factor they do not, 1726.
                    uint32_t v0[32], v1[32], v2[16];
                    tmem_ld_32x32b_x32(taddr, v0);
                    tmem_ld_32x32b_x16(taddr + 32, v2);
                    tmem_ld_32x32b_x32(taddr + 48, v1);
                    tmem_ld_wait(v0);
                    tmem_ld_wait(v1);
                    tmem_ld_wait(v2);
                    add(v0, 32, 0);
                    tmem_ld_32x32b_x32(taddr + 80, v0);
                    add(v2, 16, 32);
                    tmem_ld_32x32b_x16(taddr + 112, v2);
                    tmem_ld_wait(v0);
                    tmem_ld_wait(v2);
                    give_back();
                    add(v1, 32, 48);
                    add(v0, 32, 80);
                    add(v2, 16, 112);
                }
            };
            for (int c0 = 0; c0 < g.kblocks; c0 += kPairChunk) {
                const int nb = min(kPairChunk, g.kblocks - c0);
                // this chunk's scales have arrived, and no warp reads the chunk before last any more
                asm volatile("cp.async.wait_all;" ::: "memory");
                asm volatile("bar.sync 1, %0;" ::"n"(kPairEpi) : "memory");
                ++chunk;
                // the tile's bias, for its end (all warps have added the last one's)
                const int c = t / tiles_m * kPairN + et;
                if (!STAGED && c0 == 0 && g.bias && c < g.n)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(extra + et)), "l"(g.bias + c) : "memory");
                // the scales of this thread's row, and the weight's, a K block a lane: whether all lie within 2^-50 and 2^50
                const float *sa = scales + ((chunk - 1) & 1u) * kPairChunk * kPairRow + q * 32 + lane;
                float least = INFINITY, most = 0.f;
#pragma unroll 8
                for (int kb = 0; kb < nb; ++kb) {
                    const float v = sa[kb * kPairRow];
                    least = fminf(least, v);
                    most = fmaxf(most, v);
                }
                int eb = dom.eb;
                sb1 = lane < nb ? __ldg(sb + c0 + lane) : 0.f;
                const float fb = pow2(eb), sbf = sb1 * fb;
                const bool in = least * fa >= 0x1p-50f && most * fa <= 0x1p50f && (lane >= nb || (sbf >= 0x1p-50f && sbf <= 0x1p50f));
                if (!__all_sync(0xffffffffu, in)) {
                    Ends a_ends, b_ends;
                    for (int kb = 0; kb < nb; ++kb) a_ends.take(sa[kb * kPairRow]);
                    b_ends.take(sb1);
                    most = a_ends.most;
                    dom.b_most = fmaxf(dom.b_most, b_ends.most);
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
                        b_ends.join(Ends{__shfl_xor_sync(0xffffffffu, b_ends.least, off), __shfl_xor_sync(0xffffffffu, b_ends.most, off)});
                    const bool leave = most > 0.f && b_ends.most > 0.f &&
                                       !((a_ends.least * fa) * (b_ends.least * fb) >= 0x1p-100f && (most * fa) * (b_ends.most * fb) <= 0x1p100f);
                    if (__any_sync(0xffffffffu, leave)) {
                        float b_most = dom.b_most;
#pragma unroll
                        for (int off = 16; off > 0; off >>= 1) b_most = fmaxf(b_most, __shfl_xor_sync(0xffffffffu, b_most, off));
                        const int was = dom.ea + eb, ea = lift(fmaxf(dom.a_most, most));
                        eb = lift(b_most);
                        fa = pow2(ea);
                        dom.ea = ea;
                        dom.eb = eb;
                        rescale(acc, ea + eb - was);
                    }
                } else {
                    dom.b_most = fmaxf(dom.b_most, sb1);
                }
                dom.a_most = fmaxf(dom.a_most, most);
                sb1 *= pow2(eb);
                blocks(c0, c0 + nb);
            }
            const int e = dom.ea + dom.eb;
            if (__any_sync(0xffffffffu, e != 0)) rescale(acc, -e);
            if (!STAGED && g.bias) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                asm volatile("bar.sync 1, %0;" ::"n"(kPairEpi) : "memory");
            }
            const bool bad = *const_cast<volatile int *>(&abort_flag) != 0;  // a wait of the pair that gave up leaves no result
            if (!STAGED) {
                if (row < g.m) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float x[16];
#pragma unroll
                        for (int j = 0; j < 8; ++j) f2_split(acc[c * 8 + j], x[2 * j], x[2 * j + 1]);
                        if (col0 + c * 16 < g.n) store_cols<DT>(g, row, col0 + c * 16, x, extra + half * 128 + c * 16, bad);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (col0 + c * 32 < g.n && row - lane < g.m)
                        store_staged<DT>(g, row - lane, col0 + c * 32, acc + c * 16, extra + (warp - 4) * kPairStage, bad);
            }
        }
    }
    __syncthreads();
    cluster_sync_all();  // every MMA of the pair has completed and both CTAs have read their accumulators
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kPairTmemCols);
    }
    cluster_sync_all();  // no CTA leaves while its peer may still signal one of its barriers
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(Few<NT>::kThreads);
    cfg.dynamicSmemBytes = Few<NT>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(g.ksplit);
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}
template <int NT>
cudaError_t launch_few(const void *A, int64_t lda, const void *B, int64_t ldb, Fp8Args g, int dtype, cudaStream_t s) {
    const int mt = (g.m + NT - 1) / NT, units = (g.n + kFewBox - 1) / kFewBox, tiles = (g.n + kFewM - 1) / kFewM;
    const int64_t all = static_cast<int64_t>(tiles) * mt;
    g.ksplit = 1;
    while (g.ksplit < 8 && all * g.ksplit * 2 <= kSms && g.ksplit * 4 <= g.kblocks) g.ksplit *= 2;
    int shares = kSms / mt > 0 ? kSms / mt : 1;
    if (shares > units) shares = units;
    g.shares = g.ksplit > 1 ? tiles : shares;
    if (static_cast<int64_t>(g.shares) * mt * g.ksplit > INT32_MAX) return cudaErrorInvalidValue;
    CUtensorMap tw, tws, ta;  // weight boxes of a whole tile, and of 16 rows for a share's last one
    cudaError_t e = make_tmap_bytes(&tw, B, g.n, g.K, ldb, kFewM);
    if (e == cudaSuccess) e = make_tmap_bytes(&tws, B, g.n, g.K, ldb, kFewBox);
    if (e == cudaSuccess) e = make_tmap_bytes(&ta, A, g.m, g.K, lda, NT);
    if (e != cudaSuccess) return e;
    const int grid = g.shares * mt * g.ksplit;
    if (dtype == CE_DT_BF16) return launch_few_t<NT, CE_DT_BF16>(tw, tws, ta, g, grid, s);
    if (dtype == CE_DT_F16) return launch_few_t<NT, CE_DT_F16>(tw, tws, ta, g, grid, s);
    return launch_few_t<NT, CE_DT_F32>(tw, tws, ta, g, grid, s);
}

// Resident CTA pairs of the pair kernel on a device (0 if unknown), asked once.
int pair_clusters(const void *fn, bool staged, int dev) {
    constexpr int kDevs = 64;
    static std::atomic<int> known[kDevs];  // both variants fill an SM's shared memory
    int n = 0;
    if (dev < kDevs && (n = known[dev].load()) > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 128);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = pair_smem(staged);
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) n = 0;
    (void)cudaGetLastError();
    if (dev < kDevs && n > 0) known[dev].store(n);
    return n;
}

template <int DT, bool STAGED>
cudaError_t launch_pair(const void *A, int64_t lda, const void *B, int64_t ldb, Fp8Args g, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const void *fn = reinterpret_cast<const void *>(&fp8_pair_kernel<DT, STAGED>);
    CUtensorMap ta, tb;
    cudaError_t e = make_tmap_bytes(&ta, A, g.m, g.K, lda, 128);
    if (e == cudaSuccess) e = make_tmap_bytes(&tb, B, g.n, g.K, ldb, 128);
    if (e == cudaSuccess && done.load() == 0) {
        // a share above what the launch brings would wait for ever
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, fn);
        if (e == cudaSuccess && at.numRegs != kPairLaunchRegs) e = cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess) e = allow_smem(fn, pair_smem(STAGED), done);
    int dev = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int clusters = pair_clusters(fn, STAGED, dev);
    if (clusters < 1) clusters = kSms / 2;
    const int64_t tiles = static_cast<int64_t>((g.m + kPairM - 1) / kPairM) * ((g.n + kPairN - 1) / kPairN);
    if (tiles > INT32_MAX - 1024) return cudaErrorInvalidValue;
    if (clusters > tiles) clusters = static_cast<int>(tiles);
    void *args[] = {&ta, &tb, &g};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = pair_smem(STAGED);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Which kernel: up to 64 rows of A the weights are read at HBM's rate by the first.
// Above, pairs of CTAs, except where the first kernel's tiles of 128 x 64 fill at
// most half the SMs, so that clusters can split K. First / pairs (us, with a cold
// L2): 65 x 128256 x 4096 182 / 119, 129 x 14336 x 4096 47 / 27, 300 x 4096 x 4096
// 35 / 24, 65 x 4096 x 4096 23 / 23, 300 x 1024 x 8192 27 / 35, 1024 x 1024 x 8192 37 / 35.
bool fp8_takes_pairs(int m, int n) {
    return m > 64 && static_cast<int64_t>((n + kFewM - 1) / kFewM) * ((m + 63) / 64) * 2 > kSms;
}

cudaError_t fp8_gemm(const void *A, int64_t lda, const void *B, int64_t ldb, const Fp8Args &g, int dtype, cudaStream_t s) {
    if (fp8_takes_pairs(g.m, g.n)) {
        const int esz = fp8_elem(dtype);
        const bool staged = ((reinterpret_cast<uintptr_t>(g.out) | static_cast<uintptr_t>(g.m > 1 ? g.ldo * esz : 0)) & 31u) != 0;
        using Fn = cudaError_t (*)(const void *, int64_t, const void *, int64_t, Fp8Args, cudaStream_t);
        static const Fn fns[3][2] = {{launch_pair<CE_DT_F32, false>, launch_pair<CE_DT_F32, true>},
                                     {launch_pair<CE_DT_BF16, false>, launch_pair<CE_DT_BF16, true>},
                                     {launch_pair<CE_DT_F16, false>, launch_pair<CE_DT_F16, true>}};
        return fns[dtype][staged ? 1 : 0](A, lda, B, ldb, g, s);
    }
    if (g.m <= 16) return launch_few<16>(A, lda, B, ldb, g, dtype, s);
    if (g.m <= 32) return launch_few<32>(A, lda, B, ldb, g, dtype, s);
    return launch_few<64>(A, lda, B, ldb, g, dtype, s);
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
