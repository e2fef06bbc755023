// kvq_block.cuh -- device pieces of the 8-bit caches with one scale per page and head: the codes
// of a page, and codes as fp16 operands.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_extend.cuh"

namespace kvq {

// Two codes of a word (bytes 0 and 1, or 2 and 3) as the fp16 values they are.  int8: a code
// with its sign bit flipped is an unsigned byte u; under the exponent of 1024 it makes 1024 + u,
// and 1152 less is the code.
template <bool E4M3>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (E4M3) {
        lo = e4m3x2_to_f16x2(w);
        hi = e4m3x2_to_f16x2(w >> 16);
    } else {
        w ^= 0x80808080u;
        const uint32_t a = prmt(w, 0x64646464u, 0x4140), b = prmt(w, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off), y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    }
}

// A page's scale as attention reads it: an infinite one, of a page with an infinite value, is NaN, as
// int8 codes hold no NaN: keys of one would be infinite scores, of either sign.
__device__ __forceinline__ float page_scale(float s) { return fmaf(s, 0.f, s); }

// Four fp16 values to codes (the low half of x in the low byte): the fp32 product with inv, rounded
// to nearest even.
template <bool E4M3>
__device__ __forceinline__ uint32_t to_codes(uint32_t x, uint32_t y, uint64_t inv2) {
    const float2 a = unpack_half2(x), b = unpack_half2(y);
    const float2 c = up2(mul_x2(pk2(a.x, a.y), inv2)), d = up2(mul_x2(pk2(b.x, b.y), inv2));
    if (E4M3) {
        uint32_t r;
        asm("{.reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};}"
            : "=r"(r) : "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
        return r;
    }
    // 1.5 * 2^23 more, the low byte is the integer (at most 127: x * (127 / amax) <= 127 (1 + 2^-23)).
    // The additions are scalar: a pair's product and sum were joined to one rounding
    const float m = 12582912.f;
    const uint32_t i = __float_as_uint(__fadd_rn(c.x, m)), j = __float_as_uint(__fadd_rn(c.y, m));
    const uint32_t k = __float_as_uint(__fadd_rn(d.x, m)), l = __float_as_uint(__fadd_rn(d.y, m));
    return prmt(prmt(i, j, 0x0040), prmt(k, l, 0x0040), 0x5410);
}

// The larger magnitudes of two pairs, NaN if one is.
__device__ __forceinline__ __half2 max_abs2(__half2 m, uint32_t x) { return __hmax2_nan(m, __habs2(*reinterpret_cast<const __half2 *>(&x))); }

// One side of a page of G tokens by a CTA of 4 G threads:
//   scale = amax / M, code = rn(x (M / amax)),  M = 448 (e4m3) or 127 (int8); 1 and 0 of zeros.
// Token t's 128 fp16 channels lie at res + 128 t for t < nr, behind that at src + t stride (nr <= 0:
// all there, the common case, which has loads of its own: one addition for an address); page(): the
// page's index, asked for once the rows are in registers (-1: nothing is stored).  A page that holds
// an infinity or NaN gets an infinite or NaN scale, so that all its values count as NaN.
// Bound by the latency of its loads: half the stalls of a warp wait for them.  So a thread holds no
// more than four rows of 8 channels, in 32 registers, and an SM's 2048 threads 128 KB (256 residuals
// of 128 tokens: 44 us with 256 threads of eight rows, 43 with 512 of four; four long prompts 52.7
// and 51.8, one short prompt 14.8 and 15.2).  Tried and dropped: persistent CTAs that load a page
// while they pack the one before (four long prompts 72 us against 55: fewer loads on their way).
// Keys: thread (tid / 16, tid % 16) holds 8 channels of every G/4-th row, so that loads and stores
// are whole rows.  Values are stored with tokens contiguous: a thread holds four neighbouring
// tokens of 8 channels and turns their bytes in registers (16 lanes store 64 contiguous bytes; no
// staging in shared memory, no second barrier).
template <bool E4M3, int G, typename Page>
__device__ __forceinline__ void pack_block(const uint16_t *res, int nr, const uint16_t *src, int64_t stride, Page page, bool value,
                                           uint8_t *codes, float4 *scales) {
    constexpr int N = 4, Q = G / 4, kWarps = G / 8;  // rows of a thread, threads along the tokens
    __shared__ uint32_t s_max[kWarps];
    const int tid = threadIdx.x;
    const int cg = value ? tid / Q : tid & 15;        // eight channels
    const int first = value ? 4 * (tid % Q) : tid >> 4, step = value ? 1 : Q;
    uint4 x[N];
    if (nr <= 0) {
        const uint16_t *at = src + first * stride + 8 * cg;
#pragma unroll
        for (int i = 0; i < N; i++) x[i] = *reinterpret_cast<const uint4 *>(at + i * step * stride);
    } else {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int t = first + i * step;
            x[i] = *reinterpret_cast<const uint4 *>((t < nr ? res + t * 128 : src + t * stride) + 8 * cg);
        }
    }
    __half2 m2 = __half2half2(__ushort_as_half(0));
#pragma unroll
    for (int i = 0; i < N; i++) m2 = max_abs2(max_abs2(max_abs2(max_abs2(m2, x[i].x), x[i].y), x[i].z), x[i].w);
    // magnitudes as integers: NaN (0x7fff) is above infinity
    const uint32_t mm = *reinterpret_cast<const uint32_t *>(&m2);
    uint32_t m = __reduce_max_sync(0xffffffffu, max(mm & 0x7fffu, mm >> 16 & 0x7fffu));
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
    const int64_t pg = page();
    if (pg < 0) return;
    m = __reduce_max_sync(0xffffffffu, s_max[tid & (kWarps - 1)]);
    const float amax = h2f((uint16_t)m), top = E4M3 ? 448.f : 127.f;
    const float inv = m ? __fdiv_rn(top, amax) : 0.f;
    const uint64_t inv2 = pk2(inv, inv);
    if (tid == 0) scales[pg] = make_float4(m ? __fdiv_rn(amax, top) : 1.f, 0.f, 0.f, 0.f);
    uint8_t *dst = codes + (size_t)pg * (G * 128);
    uint32_t c[N][2];
#pragma unroll
    for (int i = 0; i < N; i++) {
        c[i][0] = to_codes<E4M3>(x[i].x, x[i].y, inv2);
        c[i][1] = to_codes<E4M3>(x[i].z, x[i].w, inv2);
    }
    if (!value) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int t = first + i * Q, pos = (cg >> 1) ^ ((t & 1) << 2);
            *reinterpret_cast<uint2 *>(dst + t * 128 + pos * 16 + (cg & 1) * 8) = make_uint2(c[i][0], c[i][1]);
        }
        return;
    }
    uint8_t *at = dst + (first >> 6) * 8192 + cg * 512 + (first & 63);
#pragma unroll
    for (int k = 0; k < 2; k++) {  // the bytes of four tokens by four channels, transposed
        const uint32_t a = prmt(c[0][k], c[1][k], 0x5140), b = prmt(c[2][k], c[3][k], 0x5140);
        const uint32_t e = prmt(c[0][k], c[1][k], 0x7362), f = prmt(c[2][k], c[3][k], 0x7362);
        *reinterpret_cast<uint32_t *>(at + (4 * k) * 64) = prmt(a, b, 0x5410);
        *reinterpret_cast<uint32_t *>(at + (4 * k + 1) * 64) = prmt(a, b, 0x7632);
        *reinterpret_cast<uint32_t *>(at + (4 * k + 2) * 64) = prmt(e, f, 0x5410);
        *reinterpret_cast<uint32_t *>(at + (4 * k + 3) * 64) = prmt(e, f, 0x7632);
    }
}
// CTAs per SM: all its threads.
template <int G>
constexpr int kPackCtas = 2048 / (4 * G);

}  // namespace kvq
