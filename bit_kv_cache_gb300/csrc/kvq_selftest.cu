// kvq_selftest.cu -- self-tests of the kernels' bounded waits (kvq_selftest_wait_timeout and
// kvq_selftest_roles_timeout, declared in include/kvq.h).  They have no counterpart on the pages: they let a test make
// a wait run out on a GPU without faulting, hanging or trapping it.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_device.cuh"
#include "kvq_tcgen05.cuh"

namespace {

// One warp waits on an mbarrier that nothing completes, through the same bounded wait
// the decode kernels use (mbar_wait, kWaitLimitCycles): it runs out, ORs the timeout
// bit into *status and returns.
__global__ void wait_selftest_kernel(int32_t *status) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        kvq::mbar_init(&bar, 1);
        kvq::fence_barrier_init();
    }
    __syncwarp();
    kvq::mbar_wait(&bar, 0u, status);
}

// A block of eight warps in the way of the chunk attention's: each waits on three barriers in
// turn, by warp_await with a flag that the block shares, and none is ever completed.  The first
// wait to run out sets the bit and the flag; all others return then.  left[w]: the waits that
// warp w has come through.
__global__ void roles_selftest_kernel(int32_t *status, int32_t *left) {
    __shared__ uint64_t bar[3];
    __shared__ int stop;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; i++) kvq::mbar_init(&bar[i], 1);
        stop = 0;
        kvq::fence_barrier_init();
    }
    __syncthreads();
    for (int i = 0; i < 3; i++) {
        kvq::warp_await(&bar[i], 0u, &stop, status);
        if ((threadIdx.x & 31) == 0) left[threadIdx.x >> 5] = i + 1;
    }
    __syncthreads();
}

}  // namespace

extern "C" int kvq_selftest_wait_timeout(int32_t *status, void *stream) {
    if (!status || ((uintptr_t)status & 3)) return KVQ_ERR_INVALID_ARG;
    wait_selftest_kernel<<<1, 32, 0, (cudaStream_t)stream>>>(status);
    return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

extern "C" int kvq_selftest_roles_timeout(int32_t *status, int32_t *left, void *stream) {
    if (!status || ((uintptr_t)status & 3) || !left || ((uintptr_t)left & 3)) return KVQ_ERR_INVALID_ARG;
    roles_selftest_kernel<<<1, 256, 0, (cudaStream_t)stream>>>(status, left);
    return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
