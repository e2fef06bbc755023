// kvq_chunk_attn.cuh -- device helpers shared by the chunk attention kernels: items and
// ranges (see ChunkAttnParams), fp16 rows and pages of a slot.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_chunk.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

constexpr int kD = 128;
constexpr float kLog2e = 1.4426950408889634f;

// Where an item lies: slot, key head, row tile, key tile, and the unit's item range.
struct Item {
    ChunkSlot s;
    int b, h, t;
    int first, n;          // first item of the unit, its number of items
};

__device__ __forceinline__ ChunkSlot load_slot(const int32_t *desc, int b) {
    const int4 *d = reinterpret_cast<const int4 *>(desc) + 2 * b;
    const int4 x = d[0], y = d[1];
    return {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

__device__ __forceinline__ Item find_item(const ChunkAttnParams &p, int it, int rows) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.item0[mid + 1] > it) hi = mid;
        else lo = mid + 1;
    }
    Item r;
    r.b = lo;
    r.s = load_slot(p.desc, lo);
    const int per = (p.item0[lo + 1] - p.item0[lo]) / p.H_kv;  // items of one head
    int x = it - p.item0[lo];
    r.h = x / per;
    x -= r.h * per;
    int t = 0, a = 0;
    for (;; t++) {
        const int n = chunk_tiles(r.s, t, rows, p.g);
        if (x < a + n) {
            r.n = n;
            break;
        }
        a += n;
    }
    r.t = t;
    r.first = p.item0[lo] + r.h * per + a;
    return r;
}

// CTA whose range holds item x: ranges [c N / C, (c + 1) N / C).
__host__ __device__ __forceinline__ int range_begin(int c, int N, int C) { return (int)((int64_t)c * N / C); }
__device__ __forceinline__ int range_of(int x, int N, int C) {
    int c = (int)(((int64_t)x * C) / N);
    while (c + 1 < C && range_begin(c + 1, N, C) <= x) c++;
    while (range_begin(c, N, C) > x) c--;
    return c;
}

// Row of fp16 token x of [sink | residual | chunk].
__device__ __forceinline__ const uint16_t *tail_row(const ChunkAttnParams &p, const Item &it, int x, bool value) {
    const size_t u = (size_t)it.b * p.H_kv + it.h;
    if (x < it.s.ns) return (value ? p.v_sink : p.k_sink) + (u * p.S + x) * kD;
    x -= it.s.ns;
    if (x < it.s.nr) return (value ? p.v_res : p.k_res) + (u * p.R + x) * kD;
    x -= it.s.nr;
    return value ? p.v_new + (int64_t)(it.s.cu + x) * p.v_stride + it.h * kD
                 : p.k_new + (int64_t)(it.s.cu + x) * p.k_stride + it.h * kD;
}

__device__ __forceinline__ int64_t page_of(const ChunkAttnParams &p, const Item &it, int tile) {
    int64_t e = p.ptab[(size_t)it.b * p.ptab_stride + (int64_t)tile * kChunkKeys / p.G];
    if (e < 0 || e >= p.n_pages) {
        report(p.status, KVQ_DEV_BAD_STATE);
        e = 0;
    }
    return e * p.H_kv + it.h;
}

}  // namespace kvq
