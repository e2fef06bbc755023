// kvq_chunk_attn.cu -- the chunk attention kernel over min-max codes.
#include "kvq_chunk_attn_kernel.cuh"

namespace kvq {

cudaError_t launch_chunk_combine(const ChunkAttnParams &p, cudaStream_t st);

cudaError_t launch_chunk_attn(const ChunkAttnParams &p, cudaStream_t st) {
    const cudaError_t e = launch_chunk_kernel<kMinMax>(p, st);
    return e == cudaSuccess && p.cut ? launch_chunk_combine(p, st) : e;
}

}  // namespace kvq
