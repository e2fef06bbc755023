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

// Four values to codes (a in the low byte): the fp32 product with inv, rounded to nearest even.
template <bool E4M3>
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d, float inv) {
    a = __fmul_rn(a, inv);
    b = __fmul_rn(b, inv);
    c = __fmul_rn(c, inv);
    d = __fmul_rn(d, inv);
    if (E4M3) {
        uint16_t x, y;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(x) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(d), "f"(c));
        return (uint32_t)x | ((uint32_t)y << 16);
    }
    // 1.5 * 2^23 more, the low byte is the integer (at most 127: x * (127 / amax) <= 127 (1 + 2^-23))
    const float m = 12582912.f;
    const uint32_t i = __float_as_uint(__fadd_rn(a, m)), j = __float_as_uint(__fadd_rn(b, m));
    const uint32_t k = __float_as_uint(__fadd_rn(c, m)), l = __float_as_uint(__fadd_rn(d, m));
    return prmt(prmt(i, j, 0x0040), prmt(k, l, 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) { return __vmaxu2(m, x & 0x7fff7fffu); }

// One side of a page of G tokens by a CTA of 256 threads:
//   scale = amax / M, code = rn(x (M / amax)),  M = 448 (e4m3) or 127 (int8); 1 and 0 of zeros.
// row(t): address of token t's 128 fp16 channels; page(): the page's index, asked for once the
// rows are in registers (-1: nothing is stored).  Largest magnitudes are compared as integers, in
// which NaN is above infinity: a page that holds one gets an infinite or NaN scale, so that all
// its values count as NaN.
// Keys: thread (tid / 16, tid % 16) holds 8 channels of every 16th row, so that loads and stores
// are whole rows.  Values are stored with tokens contiguous: a thread holds four neighbouring
// tokens of 8 channels and turns their bytes in registers (16 lanes store 64 contiguous bytes; no
// staging in shared memory, no second barrier).
template <bool E4M3, int G, typename Row, typename Page>
__device__ __forceinline__ void pack_block(Row row, Page page, bool value, uint8_t *codes, float4 *scales) {
    constexpr int N = G / 16;
    __shared__ uint32_t s_max[8];
    const int tid = threadIdx.x, lo = tid & 15, hi = tid >> 4;
    const int cg = value ? hi : lo;  // eight channels
    uint4 x[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int t = value ? 64 * (i >> 2) + 4 * lo + (i & 3) : 16 * i + hi;
        x[i] = reinterpret_cast<const uint4 *>(row(t))[cg];
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; i++) m = max_abs2(max_abs2(max_abs2(max_abs2(m, x[i].x), x[i].y), x[i].z), x[i].w);
    m = max(m & 0xffffu, m >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
    const int64_t pg = page();
    if (pg < 0) return;
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, s_max[i]);
    const float amax = h2f((uint16_t)m), top = E4M3 ? 448.f : 127.f;
    const float inv = m ? __fdiv_rn(top, amax) : 0.f;
    if (tid == 0) scales[pg] = make_float4(m ? __fdiv_rn(amax, top) : 1.f, 0.f, 0.f, 0.f);
    uint8_t *dst = codes + (size_t)pg * (G * 128);
    uint32_t c[N][2];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float2 a = unpack_half2(x[i].x), b = unpack_half2(x[i].y), e = unpack_half2(x[i].z), f = unpack_half2(x[i].w);
        c[i][0] = to_codes<E4M3>(a.x, a.y, b.x, b.y, inv);
        c[i][1] = to_codes<E4M3>(e.x, e.y, f.x, f.y, inv);
    }
    if (!value) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int t = 16 * i + hi, pos = (cg >> 1) ^ ((t & 1) << 2);
            *reinterpret_cast<uint2 *>(dst + t * 128 + pos * 16 + (cg & 1) * 8) = make_uint2(c[i][0], c[i][1]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        uint8_t *at = dst + (i >> 2) * 8192 + cg * 512 + 4 * lo;
#pragma unroll
        for (int k = 0; k < 2; k++) {  // the bytes of four tokens by four channels, transposed
            const uint32_t a = prmt(c[i][k], c[i + 1][k], 0x5140), b = prmt(c[i + 2][k], c[i + 3][k], 0x5140);
            const uint32_t e = prmt(c[i][k], c[i + 1][k], 0x7362), f = prmt(c[i + 2][k], c[i + 3][k], 0x7362);
            *reinterpret_cast<uint32_t *>(at + (4 * k) * 64) = prmt(a, b, 0x5410);
            *reinterpret_cast<uint32_t *>(at + (4 * k + 1) * 64) = prmt(a, b, 0x7632);
            *reinterpret_cast<uint32_t *>(at + (4 * k + 2) * 64) = prmt(e, f, 0x5410);
            *reinterpret_cast<uint32_t *>(at + (4 * k + 3) * 64) = prmt(e, f, 0x7632);
        }
    }
}

}  // namespace kvq
