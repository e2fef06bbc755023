// kvq_chunk_combine.cu -- joins the partial results of the chunk attention's ranges.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_chunk_attn.cuh"

namespace kvq {

namespace {

// Joins the partials of the unit that the boundary before range c cuts, if it is the first
// boundary inside the unit: 8 rows per CTA, a warp each.  Ranges are joined in order, so
// the result does not depend on timing.
__global__ void __launch_bounds__(256) chunk_combine_kernel(const __grid_constant__ ChunkAttnParams p) {
    const int c = blockIdx.x + 1, cut = range_begin(p, c);
    if (cut >= p.cost) return;
    const Item it = find_item(p, cut);
    const int begin = range_begin(p, c - 1);
    if (it.first == cut || it.first < begin) return;
    const int end = it.first + it.n * it.w;
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= min(it.rows, it.s.n_new * p.g - it.t * it.rows)) return;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // slot of a range's partial: its first segment's, or of a unit that starts later its last's
    size_t s = 2 * (size_t)(c - 1) + (it.first == begin ? 0 : 1);
    for (int k = c, next = cut;; k++) {
        const float2 ml = p.part_ml[s * kWideRows + row];
        const float4 v = reinterpret_cast<const float4 *>(p.part_o + (s * kWideRows + row) * kD)[lane];
        const float mn = fmaxf(m, ml.x);
        const float a = m == mn ? 1.f : exp2f(m - mn), b = ml.x == mn ? 1.f : exp2f(ml.x - mn);
        m = mn;
        l = a * l + b * ml.y;
        o.x = a * o.x + b * v.x;
        o.y = a * o.y + b * v.y;
        o.z = a * o.z + b * v.z;
        o.w = a * o.w + b * v.w;
        int at = next;
        while (at < end && (next = range_begin(p, k + 1)) == at) k++;  // a range without items
        if (at >= end) break;
        s = 2 * (size_t)k;
    }
    const float inv = 1.0f / l;
    const int r = it.t * it.rows + row;
    uint16_t *dst = p.out + ((int64_t)(it.s.cu + r / p.g) * p.H_kv * p.g + it.h * p.g + r % p.g) * kD;
    reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(pack_half2(o.x * inv, o.y * inv), pack_half2(o.z * inv, o.w * inv));
}

}  // namespace

cudaError_t launch_chunk_combine(const ChunkAttnParams &p, cudaStream_t st) {
    if (p.C > 1) chunk_combine_kernel<<<dim3((unsigned)(p.C - 1), kWideRows / 8), 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace kvq
