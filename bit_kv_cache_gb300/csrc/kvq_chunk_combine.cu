// kvq_chunk_combine.cu -- joins the partial results of the chunk attention's ranges, always in
// range order, so that the result does not depend on timing.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_chunk_attn.cuh"

namespace kvq {

namespace {

// A row's state: (maximum, sum) and four channels of its output per lane.
struct Part {
    float m, l;
    float4 o;
};
__device__ __forceinline__ void join(Part &a, const Part &b) {
    const float m = fmaxf(a.m, b.m);
    const float x = a.m == m ? 1.f : exp2f(a.m - m), y = b.m == m ? 1.f : exp2f(b.m - m);
    a.m = m;
    a.l = x * a.l + y * b.l;
    a.o.x = x * a.o.x + y * b.o.x;
    a.o.y = x * a.o.y + y * b.o.y;
    a.o.z = x * a.o.z + y * b.o.z;
    a.o.w = x * a.o.w + y * b.o.w;
}
__device__ __forceinline__ Part load_part(const ChunkAttnParams &p, size_t row, int lane) {
    const float2 ml = p.part_ml[row];
    return {ml.x, ml.y, reinterpret_cast<const float4 *>(p.part_o + row * kD)[lane]};
}
__device__ __forceinline__ void store_row(const ChunkAttnParams &p, const Item &it, int row, const Part &a, int lane) {
    const float inv = 1.0f / a.l;
    const int r = it.t * it.rows + row;
    uint16_t *dst = p.out + ((int64_t)(it.s.cu + r / p.g) * p.H_kv * p.g + it.h * p.g + r % p.g) * kD;
    reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(pack_half2(a.o.x * inv, a.o.y * inv), pack_half2(a.o.z * inv, a.o.w * inv));
}
constexpr Part kNone = {-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};

static_assert(kMaxRanges <= 256, "a thread per range");

// Narrow units: CTA (head, slot, z) joins rows z, z + gridDim.z, ... of one, its eight warps
// every eighth partial each (a range leaves as many as the unit has copies of its rows).
__global__ void __launch_bounds__(256) combine_narrow_kernel(const __grid_constant__ ChunkAttnParams p) {
    __shared__ int s_slot[256], s_n[8];
    __shared__ Part s_part[8][32];
    griddep_wait();
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    Item it = make_item(p, blockIdx.y);
    const int valid = it.s.n_new * p.g;
    if (valid == 0 || it.rows != kNarrowRows || (int)blockIdx.z >= valid) return;
    it.h = blockIdx.x;
    it.t = 0;
    it.n = chunk_tiles(it.s, 0, it.rows, p.g);
    it.first = p.cost0[it.b] + it.h * ((p.cost0[it.b + 1] - p.cost0[it.b]) / p.H_kv);
    const int rep = chunk_copies(valid), R = 128 / rep, last = it.end();
    // the partials' slots: a range's first segment has slot 2 c, one that starts later 2 c + 1
    const int a = tid < p.C ? p.begin[tid] : p.cost, b = tid < p.C ? p.begin[tid + 1] : p.cost;
    const bool in = a < last && b > it.first && b > a;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_n[w] = __popc(m);
    __syncthreads();
    int at = __popc(m & ((1u << lane) - 1)), parts = 0;
    for (int i = 0; i < 8; i++) {
        if (i < w) at += s_n[i];
        parts += s_n[i];
    }
    if (in) s_slot[at] = 2 * tid + (a < it.first ? 1 : 0);
    __syncthreads();
    if (parts == 1) return;  // written by its range
    for (int row = blockIdx.z; row < valid; row += gridDim.z) {
        Part acc = kNone;
        for (int i = w; i < parts * rep; i += 8) {
            const int k = i / rep;
            join(acc, load_part(p, (size_t)s_slot[k] * kWideRows + (i - k * rep) * R + row, lane));
        }
        s_part[w][lane] = acc;
        __syncthreads();
        if (w == 0) {
            for (int i = 1; i < min(8, parts * rep); i++) join(acc, s_part[i][lane]);
            store_row(p, it, row, acc, lane);
        }
        __syncthreads();
    }
}

// Wide units: the CTAs of boundary c join the unit that it cuts, if it is the first boundary
// inside the unit: 32 rows each, a warp per row.
__global__ void __launch_bounds__(256) combine_wide_kernel(const __grid_constant__ ChunkAttnParams p) {
    griddep_wait();
    const int c = blockIdx.x + 1, cut = p.begin[c];
    if (cut >= p.cost) return;
    const Item it = find_item(p, cut);
    const int begin = p.begin[c - 1], lane = threadIdx.x & 31;
    if (it.rows != kWideRows || it.first == cut || it.first < begin) return;
    const int valid = min(it.rows, it.s.n_new * p.g - it.t * it.rows), end = it.end();
    for (int row = blockIdx.y * 32 + (threadIdx.x >> 5); row < min(valid, (int)blockIdx.y * 32 + 32); row += 8) {
        Part acc = load_part(p, (2 * (size_t)(c - 1) + (it.first == begin ? 0 : 1)) * kWideRows + row, lane);
        for (int k = c, at = cut; at < end; k++) {
            const int next = p.begin[k + 1];
            if (next > at) join(acc, load_part(p, 2 * (size_t)k * kWideRows + row, lane));
            at = next;
        }
        store_row(p, it, row, acc, lane);
    }
}

}  // namespace

cudaError_t launch_chunk_combine(const ChunkAttnParams &p, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.wide && p.C > 1) e = launch_dependent(combine_wide_kernel, dim3((unsigned)(p.C - 1), kWideRows / 32), 256, 0, st, p);
    if (e == cudaSuccess && p.narrow)
        e = launch_dependent(combine_narrow_kernel, dim3((unsigned)p.H_kv, (unsigned)p.B, (unsigned)(p.narrow < 16 ? p.narrow : 16)), 256, 0, st, p);
    return e;
}

}  // namespace kvq
