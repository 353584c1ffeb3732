// A cluster of two CTAs, each with an mbarrier and a flag. In CTA `who` (none: 2) a
// thread waits for a phase that nothing completes, for a millisecond; in both a
// thread waits for one that completes. Prints the two flags for every `who`.
#include <cstdio>

#include "tc_device.cuh"

using namespace ce;

__global__ void __cluster_dims__(2, 1, 1) pair_wait(int *out, int who) {
    __shared__ uint64_t never, soon;
    __shared__ int flag;
    const int rank = static_cast<int>(cluster_ctarank());
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&never), 1);
        mbar_init(smem_u32(&soon), 1);
        flag = 0;
        fence_mbar_init_cluster();
    }
    __syncthreads();
    cluster_sync_all();
    if (threadIdx.x == 32) mbar_arrive(smem_u32(&soon));
    if (threadIdx.x == 0) {
        if (!mbar_wait_pair(smem_u32(&soon), 0, &flag)) flag = 2;
        if (rank == who && mbar_wait_pair(smem_u32(&never), 0, &flag, 1000000)) flag = 3;
    }
    __syncthreads();
    cluster_sync_all();
    if (threadIdx.x == 0) out[rank] = flag;
}

int main() {
    int *out, got[2];
    if (cudaMalloc(&out, sizeof got) != cudaSuccess) return 1;
    for (int who = 0; who < 3; ++who) {
        pair_wait<<<2, 64>>>(out, who);
        if (cudaMemcpy(got, out, sizeof got, cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
        std::printf("%d %d\n", got[0], got[1]);
    }
    return 0;
}
