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

// Page blockIdx.x of a planned chunk, or, behind them, a slot's fp16 rows.
template <bool E4M3, int G>
__global__ void __launch_bounds__(256, G == 256 ? 2 : 4) block_extend_kernel(const __grid_constant__ ExtendParams p) {
    const int h = blockIdx.y, side = blockIdx.z;
    griddep_wait();
    if (blockIdx.x >= p.n_pack) {
        extend_slot(p, blockIdx.x - p.n_pack, h, side, 0, 1);
        return;
    }
    const PageJob jb = find_page(p, blockIdx.x);
    const Sides s = sides(p, side);
    pack_block<E4M3, G>([&](int t) { return stream_row(p, jb, s.res, s.src, s.stride, h, jb.t0 + t); }, [&] { return jb.page(p, h); },
                        side, s.codes, s.scales);
    if (p.once && jb.t0 == 0) {  // every thread has read its rows (the barrier inside the packing)
        const int4 *d = reinterpret_cast<const int4 *>(p.desc) + 2 * jb.b;
        keep_rows(p, d[0], d[1], jb.b, h, side, false, true, threadIdx.x, 256);
    }
}

template <bool E4M3, int G>
__global__ void __launch_bounds__(256, G == 256 ? 2 : 4) block_list_kernel(const __grid_constant__ BlockListParams p) {
    const int h = blockIdx.y, side = blockIdx.z, k = blockIdx.x / p.per, j = blockIdx.x - k * p.per, b = p.seq[k];
    griddep_wait();
    const Sides s = sides(p, side);
    const uint16_t *res = s.res + ((size_t)b * p.H_kv + h) * p.R * 128, *src = s.src + h * p.h_stride;
    const int entry = p.ptab[(size_t)b * p.ptab_stride + p.lp0[k] + j];
    auto row = [&](int t) {
        t += j * G;
        return t < p.nr ? res + (size_t)t * 128 : src + (int64_t)(p.row0 + t - p.nr) * s.stride;
    };
    auto page = [&]() -> int64_t {
        if (entry >= 0 && entry < p.n_pages) return (int64_t)entry * p.H_kv + h;
        if (threadIdx.x == 0) report(p.status, KVQ_DEV_BAD_STATE);
        return -1;
    };
    pack_block<E4M3, G>(row, page, side, s.codes, s.scales);
    if (p.commit && j == 0 && h == 0 && side == 0 && threadIdx.x == 0) {
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

cudaError_t launch_block_extend(const ExtendParams &p, bool e4m3, cudaStream_t st) {
    const bool once = p.once && p.n_pack > 0;
    if (p.n_pack > 0) {
        const dim3 grid((unsigned)(p.n_pack + (once ? p.B : 0)), (unsigned)p.H_kv, 2);
        const cudaError_t e = by_form(p.G, e4m3, [&](auto form, auto g) {
            return launch_dependent(block_extend_kernel<decltype(form)::value, decltype(g)::value>, grid, 256, 0, st, p);
        });
        if (e != cudaSuccess || once) return e;
    }
    return launch_extend_tail(p, st);
}

cudaError_t launch_block_list(const BlockListParams &p, bool e4m3, cudaStream_t st) {
    const dim3 grid((unsigned)p.n_pack, (unsigned)p.H_kv, 2);
    return by_form(p.G, e4m3, [&](auto form, auto g) {
        return launch_dependent(block_list_kernel<decltype(form)::value, decltype(g)::value>, grid, 256, 0, st, p);
    });
}

}  // namespace kvq
