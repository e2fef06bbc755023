// kvq_quantizer.cuh -- the min-max quantizer of the quant/pack kernels (see kvq_quant.cu
// for the definition it follows): group parameters, exact codes, and the division-free
// fp32-pair form.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_device.cuh"

namespace kvq {

// Group parameters from exact fp16 min/max (as fp32 values).
struct GroupQ {
    float mn, s, inv, maxf;
    uint16_t s16, mn16;
    bool zero;
};

__device__ __forceinline__ GroupQ make_group(float mn, float mx, int max_int) {
    GroupQ g;
    if (mn == 0.0f) mn = 0.0f;  // -0 -> +0
    if (mx == 0.0f) mx = 0.0f;
    float range = __fsub_rn(mx, mn);
    float s32 = __fdiv_rn(range, (float)max_int);
    __half sh = __float2half_rn(s32);
    g.s16 = __half_as_ushort(sh);
    g.mn16 = __half_as_ushort(__float2half_rn(mn));  // exact: mn is an fp16 value
    g.mn = mn;
    g.s = __half2float(sh);
    g.zero = (g.s == 0.0f);
    g.inv = g.zero ? 0.0f : __frcp_rn(g.s);
    g.maxf = (float)max_int;
    return g;
}

__device__ __forceinline__ uint32_t quant_code(float x, const GroupQ &g) {
    float d = __fsub_rn(x, g.mn);  // >= 0
    float r = __fmul_rn(d, g.inv);
    float k = rintf(r);
    if (fabsf(__fsub_rn(r, k)) > 0.5f - 0x1p-11f) k = rintf(__fdiv_rn(d, g.s));
    k = fminf(k, g.maxf);
    return g.zero ? 0u : (uint32_t)k;
}

// |x| * 2^24 of an fp16 value as an exact integer.
__device__ __forceinline__ unsigned long long abs_units(uint32_t h) {
    uint32_t e = (h >> 10) & 0x1fu, m = h & 0x3ffu;
    if (e == 0) return m;
    return (unsigned long long)(m | 0x400u) << (e - 1);
}

// ------------------------------------------------------------------------------
// Fast quantizer.  r = (x - mn) * rcp(s) in fp32 (x - mn is exact: both are fp16
// values); t = r + 1.5 * 2^23 rounds r to the nearest integer, ties to even, into
// the low mantissa bits (0 <= r < 2^22): its bits are 0x4B400000 + rint(r), clamped
// to 0x4B400000 + max_int as integers.  A zero scale has rcp 0, so every code is 0.
// Each thread tracks max |r - rint(r)|; one that comes within 2^-14 of a
// half-integer redoes its block with quant_code (IEEE division), so the codes are
// those of the plain definition: |r - q| <= 1.5 * 2^-23 * q for the correctly
// rounded quotient q, below 2^-14 for q < 128, and larger quotients are clamped to
// max_int by both.  A word accumulates t * 2^(b pos) by integer multiply-add and
// subtracts 0x4B400000 * sum 2^(b pos) once (mod 2^32), which leaves the packed codes.
// ------------------------------------------------------------------------------
constexpr uint32_t kMagicBits = 0x4B400000u;  // 1.5 * 2^23
constexpr float kTieMargin = 0.5f - 0x1p-14f;

// fp32 pairs (Blackwell's f32x2 arithmetic): each lane of the pair rounds exactly as
// the scalar operation, so the pair forms give the same bits, in half the instructions.
__device__ __forceinline__ uint64_t pk2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 up2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t sub_x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul_x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add_x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t fma_x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// qbits for two elements at once: h is a half2 of two fp16 values whose groups have
// (min, rcp(scale)) = mn2, inv2.  Returns the two clamped magic-biased codes; em
// tracks the largest distance to a rounding tie.
__device__ __forceinline__ void qbits2(uint32_t h, uint64_t mn2, uint64_t inv2, uint32_t lim, uint32_t &c0,
                                       uint32_t &c1, float &em) {
    const uint64_t mg2 = 0x4B4000004B400000ull;  // (1.5 * 2^23, 1.5 * 2^23)
    const float2 f = unpack_half2(h);
    const uint64_t r = mul_x2(sub_x2(pk2(f.x, f.y), mn2), inv2);
    const uint64_t t = add_x2(r, mg2);
    const float2 e = up2(sub_x2(r, sub_x2(t, mg2)));
    em = fmaxf(em, fmaxf(fabsf(e.x), fabsf(e.y)));
    const float2 tf = up2(t);
    c0 = min(__float_as_uint(tf.x), lim);
    c1 = min(__float_as_uint(tf.y), lim);
}

// 0x4B400000 * sum_{j < n} 2^(b j)  (mod 2^32): the offset a word of n codes picks up.
__host__ __device__ constexpr uint32_t magic_sum(int b, int n) {
    uint32_t s = 0;
    for (int j = 0; j < n; j++) s += kMagicBits << (b * j);
    return s;
}

__device__ __forceinline__ GroupQ group_from_meta(uint32_t m, int max_int) {
    GroupQ g;
    g.s16 = (uint16_t)(m & 0xffffu);
    g.mn16 = (uint16_t)(m >> 16);
    g.mn = h2f(g.mn16);
    g.s = h2f(g.s16);
    g.zero = (g.s == 0.0f);
    g.inv = g.zero ? 0.0f : __frcp_rn(g.s);
    g.maxf = (float)max_int;
    return g;
}

// The exact codes of one token's four channels (x: two half2 words; m: their
// (scale, min) words).  Out of line: the rare near-tie path stays out of the unrolled
// loop, whose code would otherwise outgrow the instruction cache.
static __device__ __noinline__ uint4 exact_codes4(uint2 x, uint4 m, int max_int) {
    const float2 f01 = unpack_half2(x.x), f23 = unpack_half2(x.y);
    return make_uint4(quant_code(f01.x, group_from_meta(m.x, max_int)), quant_code(f01.y, group_from_meta(m.y, max_int)),
                      quant_code(f23.x, group_from_meta(m.z, max_int)), quant_code(f23.y, group_from_meta(m.w, max_int)));
}

}  // namespace kvq
