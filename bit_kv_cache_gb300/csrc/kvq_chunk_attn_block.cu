// kvq_chunk_attn_block.cu -- the chunk attention kernel over 8-bit codes with one scale per page
// and head.
#include "kvq_chunk_attn_kernel.cuh"

namespace kvq {

cudaError_t launch_chunk_combine(const ChunkAttnParams &p, cudaStream_t st);

cudaError_t launch_chunk_attn_block(const ChunkAttnParams &p, bool e4m3, cudaStream_t st) {
    const cudaError_t e = e4m3 ? launch_chunk_kernel<kE4m3>(p, st) : launch_chunk_kernel<kInt8>(p, st);
    return e == cudaSuccess && p.cut ? launch_chunk_combine(p, st) : e;
}

}  // namespace kvq
