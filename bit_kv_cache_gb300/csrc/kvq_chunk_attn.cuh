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
constexpr float kScale = kLog2e * 0.08838834764831845f;  // log2(e) / sqrt(128)

// A unit: slot, key head, row tile; its first position, number of items, the cost of each,
// query rows.  Item 0 lies at the unit's first position, item j > 0 at first + (kUnitItems + j) w.
struct Item {
    ChunkSlot s;
    int b, h, t;
    int first, n, w, rows;
    __device__ __forceinline__ int end() const { return first + (n + kUnitItems) * w; }
    // the item at a position where one lies, or n at the unit's end or behind it
    __device__ __forceinline__ int at(int pos) const { return pos >= end() ? n : pos == first ? 0 : (pos - first) / w - kUnitItems; }
};

__device__ __forceinline__ ChunkSlot load_slot(const int32_t *desc, int b) {
    const int4 *d = reinterpret_cast<const int4 *>(desc) + 2 * b;
    const int4 x = d[0], y = d[1];
    return {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

__device__ __forceinline__ int slot_of(const ChunkAttnParams &p, int pos) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.cost0[mid + 1] > pos) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Unit (slot, head, row tile) without its position in the slot's row tiles.
__device__ __forceinline__ Item make_item(const ChunkAttnParams &p, int b) {
    Item r;
    r.b = b;
    r.s = load_slot(p.desc, b);
    const bool narrow = chunk_narrow(r.s.n_new, p.g);
    r.rows = narrow ? kNarrowRows : kWideRows;
    r.w = narrow ? kNarrowCost : kWideCost;
    return r;
}

// The unit at a position, given one of the same slot and head at or before it (first
// position, row tile), or any before.
__device__ __forceinline__ Item find_item(const ChunkAttnParams &p, int pos, int first, int tile) {
    Item r = make_item(p, slot_of(p, pos));
    const int per = (p.cost0[r.b + 1] - p.cost0[r.b]) / p.H_kv;  // cost of one head
    r.h = (pos - p.cost0[r.b]) / per;
    const int head = p.cost0[r.b] + r.h * per;
    const bool near = first > head;
    r.t = near ? tile : 0;
    r.first = near ? first : head;
    for (;; r.t++) {
        r.n = chunk_tiles(r.s, r.t, r.rows, p.g);
        if (pos < r.end()) break;
        r.first = r.end();
    }
    return r;
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

// The page index that a page-table entry stands for.
__device__ __forceinline__ int64_t page_index(const ChunkAttnParams &p, const Item &it, int32_t entry) {
    if (entry < 0 || entry >= p.n_pages) {
        report(p.status, KVQ_DEV_BAD_STATE);
        entry = 0;
    }
    return (int64_t)entry * p.H_kv + it.h;
}

}  // namespace kvq
