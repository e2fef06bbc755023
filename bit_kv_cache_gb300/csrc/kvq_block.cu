// kvq_block.cu -- pages of 8-bit codes with one scale per page and head: new tokens' pages
// (kvq_paged_extend), a prompt's (kvq_paged_prefill) and full residuals' (kvq_paged_flush).
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_block.cuh"
#include "kvq_block.h"

namespace kvq {

namespace {

struct Sides {
    uint8_t *codes;
    float4 *scales;
    const uint16_t *res, *src;
    int64_t stride;
};
__device__ __forceinline__ Sides sides(const PackParams &p, bool value) {
    return {reinterpret_cast<uint8_t *>(value ? p.v_codes : p.k_codes), reinterpret_cast<float4 *>(value ? p.v_meta : p.k_meta),
            value ? p.v_res : p.k_res, value ? p.v_new : p.k_new, value ? p.v_stride : p.k_stride};
}

// The page index of a page-table entry; -1 (reported) if it is no page.
__device__ __forceinline__ int64_t page_of(const PackParams &p, int entry, int h) {
    if (entry >= 0 && entry < p.n_pages) return (int64_t)entry * p.H_kv + h;
    if (threadIdx.x == 0) report(p.status, KVQ_DEV_BAD_STATE);
    return -1;
}

// Pages of a planned chunk, then the slots' fp16 rows.  CTA i: head i % H of one side of page (slot)
// i / (2 H): the heads of a token are neighbours in memory, and are read at about the same time
// (pages next to each other first: four long prompts 55 us against 53 at 256 threads a CTA).
template <bool E4M3, int G>
__global__ void __launch_bounds__(4 * G, kPackCtas<G>) block_extend_kernel(const __grid_constant__ BlockExtendParams p) {
    const int x = blockIdx.x / p.H_kv, h = blockIdx.x - x * p.H_kv, side = x & 1, i = x >> 1;
    griddep_wait();
    if (i >= p.n_pack) {
        extend_slot(p, i - p.n_pack, h, side, 0, 1);
        return;
    }
    int lo = 0, hi = p.B - 1;  // the slot: the first one whose pages end behind page i
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.page0[mid + 1] > i) hi = mid;
        else lo = mid + 1;
    }
    const int b = lo, j = i - p.page0[b], t0 = j * G, nr = p.nr[b];
    const Sides s = sides(p, side);
    const int entry = p.ptab[(size_t)b * p.ptab_stride + p.lp0[b] + j];
    const uint16_t *res = s.res + (((size_t)b * p.H_kv + h) * p.R + t0) * 128, *src = s.src + (int64_t)(p.row0[b] + t0) * s.stride + h * 128;
    // residual rows are read by ordinary loads: a CTA of the slot writes over them
    pack_block<E4M3, G>(res, nr - t0, src, s.stride, [&] { return page_of(p, entry, h); }, side, s.codes, s.scales);
    // a slot that packs has a page for each G rows of its residual: the CTA that has read the old rows
    // (the barrier inside the packing) writes the new ones
    if (t0 < p.R) {
        const int4 *d = reinterpret_cast<const int4 *>(p.desc) + 2 * b;
        keep_rows(p, d[0], d[1], b, h, side, false, true, threadIdx.x, 4 * G, t0, t0 + G);
    }
}

// Pages of listed slots.  A prefill of 12345 tokens of 8 heads (76 MB), with the copies of its last
// rows, takes 26 us (e4m3; int8 27, min-max codes of 4 bits 36); a flush of 256 full residuals (201 MB),
// with setting the lengths back, 38 (39, 53).
template <bool E4M3, int G>
__global__ void __launch_bounds__(4 * G, kPackCtas<G>) block_list_kernel(const __grid_constant__ BlockListParams p) {
    const int h = blockIdx.y, side = blockIdx.z, k = blockIdx.x / p.per, j = blockIdx.x - k * p.per, b = p.seq[k];
    griddep_wait();
    const Sides s = sides(p, side);
    const int entry = p.ptab[(size_t)b * p.ptab_stride + p.lp0[k] + j];
    const uint16_t *src = p.residual ? s.res + (((size_t)b * p.H_kv + h) * p.R + j * G) * 128
                                     : s.src + h * p.h_stride + (int64_t)(p.row0 + j * G) * s.stride;
    pack_block<E4M3, G>(nullptr, 0, src, p.residual ? 128 : s.stride, [&] { return page_of(p, entry, h); }, side, s.codes, s.scales);
    if (p.residual && j == 0 && h == 0 && side == 0 && threadIdx.x == 0) {
        p.lens[4 * b + 1] += p.R;
        p.lens[4 * b + 2] = 0;
    }
}

template <typename F>
cudaError_t by_form(int G, bool e4m3, F f) {
    auto g = [&](auto form) {
        return G == 64 ? f(form, std::integral_constant<int, 64>()) : G == 128 ? f(form, std::integral_constant<int, 128>())
                                                                                : f(form, std::integral_constant<int, 256>());
    };
    return e4m3 ? g(std::true_type()) : g(std::false_type());
}

}  // namespace

cudaError_t launch_block_extend(const ExtendParams &x, const ChunkSlot *slots, bool e4m3, cudaStream_t st) {
    if (x.n_pack == 0) return launch_extend_tail(x, st);
    BlockExtendParams p;
    static_cast<ExtendParams &>(p) = x;
    for (int b = 0; b < x.B; b++) {
        p.nr[b] = slots[b].nr;
        p.row0[b] = slots[b].cu + slots[b].to_sink - slots[b].nr;
        p.lp0[b] = slots[b].T / x.G;
    }
    const int64_t ctas = ((int64_t)p.n_pack + p.B) * 2 * p.H_kv;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas);
    return by_form(p.G, e4m3, [&](auto form, auto g) {
        return launch_dependent(block_extend_kernel<decltype(form)::value, decltype(g)::value>, grid, 4 * decltype(g)::value, 0, st, p);
    });
}

cudaError_t launch_block_list(const BlockListParams &p, bool e4m3, cudaStream_t st) {
    const dim3 grid((unsigned)p.n_pack, (unsigned)p.H_kv, 2);
    return by_form(p.G, e4m3, [&](auto form, auto g) {
        return launch_dependent(block_list_kernel<decltype(form)::value, decltype(g)::value>, grid, 4 * decltype(g)::value, 0, st, p);
    });
}

}  // namespace kvq
