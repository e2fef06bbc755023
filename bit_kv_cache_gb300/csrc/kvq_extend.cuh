// kvq_extend.cuh -- device pieces of the calls that pack pages from [residual | new rows]:
// pages of a call, their rows, the min-max codes of keys and values, the rows that stay fp16
// (kvq_chunk.cu, kvq_block.cu, kvq_append_rope.cu).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_chunk.h"
#include "kvq_internal.h"
#include "kvq_quantizer.cuh"

namespace kvq {

struct PageJob {
    ChunkSlot s;
    int b;
    int entry;             // of the page table; read early, checked and used by page() at the end
    int t0;                // first stream token
    // -1: no page, nothing may be stored
    __device__ __forceinline__ int64_t page(const PackParams &p, int h) const {
        if (entry < 0 || entry >= p.n_pages) {
            if (threadIdx.x == 0) report(p.status, KVQ_DEV_BAD_STATE);
            return -1;
        }
        return (int64_t)entry * p.H_kv + h;
    }
};

// Page i of the call; its slot is the first one whose pages end behind it.
__device__ __forceinline__ PageJob find_page(const ExtendParams &p, int i) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.page0[mid + 1] > i) hi = mid;
        else lo = mid + 1;
    }
    const int4 *d = reinterpret_cast<const int4 *>(p.desc) + 2 * lo;
    const int4 x = d[0], y = d[1];
    PageJob j;
    j.s = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    j.b = lo;
    const int k = i - p.page0[lo];
    j.t0 = k * p.G;
    j.entry = p.ptab[(size_t)lo * p.ptab_stride + x.y / p.G + k];
    return j;
}

// Row t of a page's stream.  Residual rows are read by ordinary loads: where one launch does the
// call, keep_rows writes over them.
__device__ __forceinline__ const uint16_t *stream_row(const PackParams &p, const PageJob &j, const uint16_t *res,
                                                      const uint16_t *src, int64_t stride, int h, int t) {
    return t < j.s.nr ? res + (((size_t)j.b * p.H_kv + h) * p.R + t) * 128
                      : src + (int64_t)(j.s.cu + j.s.to_sink + t - j.s.nr) * stride + h * 128;
}

// Keys of one page: TPW tokens per warp, lane l holds channels 4 l .. 4 l + 3 of them.
template <int BITS, int TPW>
__device__ __forceinline__ void extend_keys(const PackParams &p, const PageJob &jb, int h, unsigned char *smem) {
    constexpr int D = 128, FPI = 32 / BITS, NWR = TPW / FPI, MAXI = (1 << BITS) - 1;
    uint16_t(*s_lo)[D] = reinterpret_cast<uint16_t(*)[D]>(smem);
    uint16_t(*s_hi)[D] = s_lo + 8;
    float *s_mn = reinterpret_cast<float *>(smem + 16 * D * 2), *s_inv = s_mn + D;
    uint32_t *s_meta = reinterpret_cast<uint32_t *>(s_inv + D);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    uint2 x[TPW];
#pragma unroll
    for (int j = 0; j < TPW; j++)
        x[j] = reinterpret_cast<const uint2 *>(stream_row(p, jb, p.k_res, p.k_new, p.k_stride, h, jb.t0 + w * TPW + j))[lane];
    __half2 lo0 = *reinterpret_cast<const __half2 *>(&x[0].x), hi0 = lo0;
    __half2 lo1 = *reinterpret_cast<const __half2 *>(&x[0].y), hi1 = lo1;
#pragma unroll
    for (int j = 1; j < TPW; j++) {
        const __half2 a = *reinterpret_cast<const __half2 *>(&x[j].x), c = *reinterpret_cast<const __half2 *>(&x[j].y);
        lo0 = __hmin2(lo0, a);
        hi0 = __hmax2(hi0, a);
        lo1 = __hmin2(lo1, c);
        hi1 = __hmax2(hi1, c);
    }
    reinterpret_cast<uint2 *>(&s_lo[w][0])[lane] =
        make_uint2(*reinterpret_cast<uint32_t *>(&lo0), *reinterpret_cast<uint32_t *>(&lo1));
    reinterpret_cast<uint2 *>(&s_hi[w][0])[lane] =
        make_uint2(*reinterpret_cast<uint32_t *>(&hi0), *reinterpret_cast<uint32_t *>(&hi1));
    __syncthreads();
    const int64_t page = jb.page(p, h);
    if (page < 0) return;
    if (tid < D) {
        float mn = h2f(s_lo[0][tid]), mx = h2f(s_hi[0][tid]);
#pragma unroll
        for (int ww = 1; ww < 8; ww++) {
            mn = fminf(mn, h2f(s_lo[ww][tid]));
            mx = fmaxf(mx, h2f(s_hi[ww][tid]));
        }
        const GroupQ g = make_group(mn, mx, MAXI);
        s_mn[tid] = g.mn;
        s_inv[tid] = g.inv;
        const uint32_t m = (uint32_t)g.s16 | ((uint32_t)g.mn16 << 16);
        s_meta[tid] = m;
        reinterpret_cast<uint32_t *>(p.k_meta + (size_t)page * D * 2)[tid] = m;
    }
    __syncthreads();
    const float4 mn4 = reinterpret_cast<const float4 *>(s_mn)[lane], in4 = reinterpret_cast<const float4 *>(s_inv)[lane];
    const uint64_t mn01 = pk2(mn4.x, mn4.y), mn23 = pk2(mn4.z, mn4.w);
    const uint64_t in01 = pk2(in4.x, in4.y), in23 = pk2(in4.z, in4.w);
    constexpr uint32_t lim = kMagicBits + MAXI;
    const int64_t row0 = page * (8 * TPW / FPI) + w * NWR;
#pragma unroll
    for (int r = 0; r < NWR; r++) {
        uint32_t wd[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < FPI; k++) {
            const uint2 v = x[r * FPI + k];
            uint32_t a0, a1, a2, a3;
            float em = 0.f;
            qbits2(v.x, mn01, in01, lim, a0, a1, em);
            qbits2(v.y, mn23, in23, lim, a2, a3, em);
            if (em > kTieMargin) {
                const uint4 e = exact_codes4(v, reinterpret_cast<const uint4 *>(s_meta)[lane], MAXI);
                a0 = kMagicBits + e.x;
                a1 = kMagicBits + e.y;
                a2 = kMagicBits + e.z;
                a3 = kMagicBits + e.w;
            }
            const uint32_t m = 1u << (BITS * k);
            wd[0] += a0 * m;
            wd[1] += a1 * m;
            wd[2] += a2 * m;
            wd[3] += a3 * m;
        }
        const uint32_t off = magic_sum(BITS, FPI);
        *reinterpret_cast<uint4 *>(p.k_codes + (size_t)(row0 + r) * D + kword_pos(4 * lane, w * NWR + r)) =
            make_uint4(wd[0] - off, wd[1] - off, wd[2] - off, wd[3] - off);
    }
}

// The exact codes of eight channels of one group (m: its (scale, min)), packed: one word of
// 2- or 4-bit codes, two of 8-bit ones.  Out of line, as exact_codes4: the unrolled loop
// around the rare call has to fit the instruction cache.
static __device__ __noinline__ uint2 exact_codes8(uint4 x, uint32_t m, int bits) {
    const GroupQ g = group_from_meta(m, (1 << bits) - 1);
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    uint64_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float2 f = unpack_half2(u[k]);
        w |= (uint64_t)quant_code(f.x, g) << (bits * 2 * k);
        w |= (uint64_t)quant_code(f.y, g) << (bits * (2 * k + 1));
    }
    return make_uint2((uint32_t)w, (uint32_t)(w >> 32));
}

// 128 value tokens of one page (block vb of it): 16 tokens per warp, lane (tq, c) holds
// tokens 8 g + tq and of each the 8-channel chunks c, c + 4, c + 8, c + 12.
template <int BITS>
__device__ __forceinline__ void extend_values(const PackParams &p, const PageJob &jb, int h, int vb, unsigned char *smem) {
    constexpr int D = 128, FPI = 32 / BITS, NWORD = D / FPI;
    uint32_t(*s_codes)[128] = reinterpret_cast<uint32_t(*)[128]>(smem);
    uint32_t *s_meta = reinterpret_cast<uint32_t *>(smem + NWORD * 512);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, tq = lane >> 2, c = lane & 3;
    uint4 x[2][4];
#pragma unroll
    for (int g = 0; g < 2; g++) {
        const uint4 *row = reinterpret_cast<const uint4 *>(
            stream_row(p, jb, p.v_res, p.v_new, p.v_stride, h, jb.t0 + vb * 128 + 16 * w + 8 * g + tq));
#pragma unroll
        for (int i = 0; i < 4; i++) x[g][i] = row[c + 4 * i];
    }
    constexpr uint32_t lim = kMagicBits + (1u << BITS) - 1;
#pragma unroll
    for (int g = 0; g < 2; g++) {
        const int tt = 16 * w + 8 * g + tq;
        __half2 lo = *reinterpret_cast<const __half2 *>(&x[g][0].x), hi = lo;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int k = (i == 0 ? 1 : 0); k < 4; k++) {
                const uint32_t wk = (&x[g][i].x)[k];
                const __half2 v = *reinterpret_cast<const __half2 *>(&wk);
                lo = __hmin2(lo, v);
                hi = __hmax2(hi, v);
            }
        float a = fminf(__low2float(lo), __high2float(lo)), b = fmaxf(__low2float(hi), __high2float(hi));
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            a = fminf(a, __shfl_xor_sync(0xffffffffu, a, o));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
        const GroupQ gr = make_group(a, b, (1 << BITS) - 1);
        if (c == 0) s_meta[tt] = (uint32_t)gr.s16 | ((uint32_t)gr.mn16 << 16);
        const uint64_t mn2 = pk2(gr.mn, gr.mn), inv2 = pk2(gr.inv, gr.inv);
#pragma unroll
        for (int i = 0; i < 4; i++) {  // chunk c + 4 i: channels 8 (c + 4 i) .. + 7
            constexpr int NP = BITS == 8 ? 2 : 1, PER = 8 / NP;  // words of a chunk, codes in each
            uint32_t part[NP];
            float emax = 0.f;
#pragma unroll
            for (int n = 0; n < NP; n++) {
                part[n] = 0;
#pragma unroll
                for (int k = 0; k < PER / 2; k++) {
                    uint32_t c0, c1;
                    qbits2((&x[g][i].x)[n * (PER / 2) + k], mn2, inv2, lim, c0, c1, emax);
                    part[n] += c0 * (1u << (BITS * (2 * k)));
                    part[n] += c1 * (1u << (BITS * (2 * k + 1)));
                }
                part[n] -= magic_sum(BITS, PER);
            }
            if (emax > kTieMargin) {  // near a half-integer in this chunk: the exact path
                const uint2 w = exact_codes8(x[g][i], (uint32_t)gr.s16 | ((uint32_t)gr.mn16 << 16), BITS);
                part[0] = w.x;
                if (NP == 2) part[NP - 1] = w.y;
            }
            if (BITS == 2) {  // 16 channels per word: chunks 2m (lane c even) and 2m + 1
                const uint32_t nb = __shfl_xor_sync(0xffffffffu, part[0], 1);
                if ((c & 1) == 0) s_codes[(c + 4 * i) >> 1][tt] = part[0] | (nb << 16);
            } else {
#pragma unroll
                for (int n = 0; n < NP; n++) s_codes[NP * (c + 4 * i) + n][tt] = part[n];
            }
        }
    }
    __syncthreads();
    const int64_t page = jb.page(p, h);
    if (page < 0) return;
    const int TV = p.TV;
    for (int i = tid; i < NWORD * 32; i += 256) {
        const int m = i >> 5, tt = vb * 128 + 4 * (i & 31), tile = tt / TV, j = tt - tile * TV;
        *reinterpret_cast<uint4 *>(p.v_codes + (size_t)page * NWORD * p.G + ((size_t)tile * NWORD + m) * TV + vword_pos(j, m, TV)) =
            *reinterpret_cast<const uint4 *>(&s_codes[m][4 * (i & 31)]);
    }
    if (tid < 32)
        reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(p.v_meta) + (size_t)page * p.G + vb * 128)[tid] =
            *reinterpret_cast<const uint4 *>(&s_meta[4 * tid]);
}

// Rows of a slot that stay fp16: its new sink rows and, from row lo on, its residual's new
// rows up to hi, which are the chunk's last tokens (a slot that packs nothing keeps its old
// rows, one that packs takes all of them), of these rows from .. to - 1.  Sixteen threads per row,
// thread t of n.
__device__ __forceinline__ void keep_rows(const ExtendParams &p, const int4 &x, const int4 &y, int b, int h, int side, bool sink,
                                          bool residual, int t, int n, int from = 0, int to = INT32_MAX) {
    const int to_sink = sink ? y.y : 0, pk = y.z, lo = max(from, pk ? 0 : x.z), hi = residual ? min(to, x.z + x.w - y.y - pk) : lo;
    const int64_t stride = side ? p.v_stride : p.k_stride;
    const uint16_t *src = (side ? p.v_new : p.k_new) + h * 128;
    const size_t u = (size_t)b * p.H_kv + h;
    uint16_t *sk = side ? p.v_sink : p.k_sink, *res = side ? p.v_res : p.k_res;
    const int rows = to_sink + max(hi - lo, 0), c = t & 15;
    for (int i = t >> 4; i < rows; i += n >> 4) {
        const int r = i - to_sink + lo;
        const int tok = i < to_sink ? i : y.y + pk + r - x.z;
        uint16_t *dst = i < to_sink ? sk + (u * p.S + x.x + i) * 128 : res + (u * p.R + r) * 128;
        reinterpret_cast<uint4 *>(dst)[c] = __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)(y.x + tok) * stride) + c);
    }
}

// Slot b's fp16 rows and lengths; slice z of nz.
__device__ __forceinline__ void extend_slot(const ExtendParams &p, int b, int h, int side, int z, int nz) {
    const int4 *d = reinterpret_cast<const int4 *>(p.desc);
    const int4 x = d[2 * b], y = d[2 * b + 1];
    if (!x.w) return;
    keep_rows(p, x, y, b, h, side, true, !(p.once && y.z), z * blockDim.x + threadIdx.x, nz * blockDim.x);
    if (h == 0 && side == 0 && z == 0 && threadIdx.x == 0)
        reinterpret_cast<int4 *>(p.lens)[b] = make_int4(x.x + y.y, x.y + y.z, x.z + x.w - y.y - y.z, 1);
}

}  // namespace kvq
