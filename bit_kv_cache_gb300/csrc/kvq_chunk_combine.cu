// kvq_chunk_combine.cu -- joins the partial results of the chunk attention's ranges, always in
// range order, so that the result does not depend on timing.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_chunk_attn.cuh"

namespace kvq {

namespace {

// A row's state: (reference, sum) and four channels of its output per lane.
struct Part {
    float m, l;
    float4 o;
};
// The factor of a part below the maximum; positive, as an infinite value in it stays infinite
// (2^-126 of a finite part is far below the other's smallest step).
__device__ __forceinline__ float factor(float m, float top) { return m == top ? 1.f : fmaxf(exp2f((m - top) * kScale), 0x1p-126f); }
__device__ __forceinline__ void join(Part &a, const Part &b) {
    const float m = fmaxf(a.m, b.m), x = factor(a.m, m), y = factor(b.m, m);
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

// Narrow units: CTA (head, slot, z of nz) joins rows z, z + nz, ... of one, its eight warps
// every eighth partial each (a range leaves as many as the unit has copies of its rows).
__device__ __forceinline__ void combine_narrow(const ChunkAttnParams &p, int h, int b, int z, int nz) {
    __shared__ int s_slot[256], s_n[8];
    __shared__ Part s_part[8][32];
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    Item it = make_item(p, b);
    const int valid = it.s.n_new * p.g;
    if (valid == 0 || it.rows != kNarrowRows || z >= valid) return;
    it.h = h;
    it.t = 0;
    it.n = chunk_tiles(it.s, 0, it.rows, p.g);
    it.first = p.cost0[it.b] + it.h * ((p.cost0[it.b + 1] - p.cost0[it.b]) / p.H_kv);
    const int rep = chunk_copies(valid), R = 128 / rep, last = it.end();
    // the partials' slots: a range's first segment has slot 2 c, one that starts later 2 c + 1
    const int a = tid < p.C ? p.begin[tid] : p.cost, e = tid < p.C ? p.begin[tid + 1] : p.cost;
    const bool in = a < last && e > it.first && e > a;
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
    for (int row = z; row < valid; row += nz) {
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
// inside the unit: 32 rows each, four rows per warp at once.
constexpr int kCombineRows = 4;
__device__ __forceinline__ void combine_wide(const ChunkAttnParams &p, int c, int row0) {
    const int cut = p.begin[c];
    if (cut >= p.cost) return;
    const Item it = find_item(p, cut, p.first[c], p.tile[c]);
    const int begin = p.begin[c - 1], lane = threadIdx.x & 31;
    if (it.rows != kWideRows || it.first == cut || it.first < begin) return;
    const int valid = min(it.rows, it.s.n_new * p.g - it.t * it.rows), end = it.end();
    const int row = row0 + kCombineRows * (threadIdx.x >> 5);
    if (row >= valid) return;
    Part acc[kCombineRows], x[kCombineRows];
    auto load = [&](Part (&y)[kCombineRows], size_t slot) {  // a partial has all rows of the tile
#pragma unroll
        for (int i = 0; i < kCombineRows; i++) y[i] = load_part(p, slot * kWideRows + min(row + i, valid - 1), lane);
    };
    load(acc, 2 * (size_t)(c - 1) + (it.first == begin ? 0 : 1));
    for (int k = c, at = cut; at < end; k++) {
        const int next = p.begin[k + 1];
        if (next > at) {
            load(x, 2 * (size_t)k);
#pragma unroll
            for (int i = 0; i < kCombineRows; i++) join(acc[i], x[i]);
        }
        at = next;
    }
#pragma unroll
    for (int i = 0; i < kCombineRows; i++)
        if (row + i < valid) store_row(p, it, row + i, acc[i], lane);
}

// One launch: n_wide CTAs (boundary, 32 rows), then (head, slot, z).
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ ChunkAttnParams p, int n_wide, int nz) {
    griddep_wait();
    int x = blockIdx.x;
    if (x < n_wide) {
        combine_wide(p, x / (kWideRows / 32) + 1, x % (kWideRows / 32) * 32);
    } else {
        x -= n_wide;
        const int z = x % nz, u = x / nz;
        combine_narrow(p, u % p.H_kv, u / p.H_kv, z, nz);
    }
}

}  // namespace

cudaError_t launch_chunk_combine(const ChunkAttnParams &p, cudaStream_t st) {
    const int n_wide = p.wide ? (p.C - 1) * (kWideRows / 32) : 0, nz = p.narrow < 16 ? p.narrow : 16;
    const int grid = n_wide + nz * p.H_kv * p.B;
    if (grid == 0) return cudaSuccess;
    return launch_dependent(combine_kernel, dim3((unsigned)grid), 256, 0, st, p, n_wide, nz > 0 ? nz : 1);
}

}  // namespace kvq
