// kvq_rope.h -- host side of the rotary embedding: angles in 64-bit fixed point, argument checks.
// Not part of the public ABI.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "kvq.h"

namespace kvq {
namespace host {

// A positive number m 2^(e - 64), 2^63 <= m.
struct Mantissa {
    uint64_t m;
    int e;
};
inline Mantissa mantissa(double x) {
    int e;
    const double f = frexp(x, &e);
    return {(uint64_t)ldexp(f, 64), e};
}
inline Mantissa operator*(Mantissa a, Mantissa b) {
    unsigned __int128 p = (unsigned __int128)a.m * b.m;
    int e = a.e + b.e;
    if (!(p >> 127)) p <<= 1, e--;
    return {(uint64_t)(p >> 64), e};
}

// base^(-1/m) for base > 1 in units of 2^-64, off by a few of them: the double root y and one
// Newton step, y (1 - (y^m base - 1) / m), whose residual is formed with 64-bit mantissas
// (a long double power, emulated in software on Arm, took 1.2 us more of the call's 11).
inline uint64_t inverse_root(double base, int m) {
    const Mantissa y = mantissa(std::min(pow(base, -1.0 / m), 1.0 - 0x1p-53));
    Mantissa z = mantissa(base), sq = y;
    for (int i = m; i; i >>= 1, sq = sq * sq)
        if (i & 1) z = z * sq;
    // z = 1 + d 2^-64
    const int64_t d = z.e == 1 ? (int64_t)((z.m - (1ull << 63)) << 1) : (int64_t)z.m;
    const uint64_t f = y.m >> -y.e;
    return f - (uint64_t)(int64_t)((double)f * ((double)d * 0x1p-64) / m);
}

// Steps of pairs j < n / 2 at one position, base^(-2j/n) / (2 pi), in units of 2^-64 turns.
inline void turns_of_base(float rope_base, int n, uint64_t *out) {
    const double base = rope_base > 0.f ? (double)rope_base : 10000.0;
    // turn[j] = base^(-2j/n) / (2 pi) in 64-bit fixed point: one root, then integer products
    // (a call's host time is a small part of that of a power per pair).  The root's error and the
    // products' truncations add up: a step is off by n/4 + 1 units of 2^-64 at most (64.3 for
    // n = 256 and bases next to 1, 9 for a base of 10000, against 80 digits), so an angle by
    // 2^-27 of a turn at positions below 2^31
    if (base > 1.0) {
        const uint64_t f = inverse_root(base, n / 2);
        uint64_t turn = 0x28be60db9391054aull;  // 2^64 / (2 pi)
        for (int j = 0; j < n / 2; j++, turn = (uint64_t)(((unsigned __int128)turn * f) >> 64)) out[j] = turn;
    } else {
        const long double step = powl((long double)base, -2.0L / n);
        long double turn = 0.159154943091895335768883763372514362L;
        for (int j = 0; j < n / 2; j++, turn *= step) out[j] = (uint64_t)ldexpl(turn - floorl(turn), 64);
    }
}

// The same of given frequencies, in radians per position: whole turns drop out.  A frequency below
// 2 pi is off by a unit of 2^-64 turns at most, besides its own rounding.
inline void turns_of_freq(const double *freq, int n, uint64_t *out) {
    const Mantissa inv2pi = {0xa2f9836e4e441529ull, -2};  // 1 / (2 pi)
    for (int j = 0; j < n / 2; j++) {
        out[j] = 0;
        if (!(freq[j] > 0)) continue;
        const Mantissa t = mantissa(freq[j]) * inv2pi;
        if (t.e <= -64) continue;
        out[j] = t.e < 0 ? t.m >> -t.e : t.e < 64 ? t.m << t.e : 0;
    }
}

// Head dim, channels, norm and angles of a kvq_qk_config; freq: may be null.
inline int rope_check(const kvq_qk_config *c, const double *freq, float amp) {
    if (c->D != 64 && c->D != 128 && c->D != 256) return KVQ_ERR_UNSUPPORTED;
    if (c->rotary_dim < 0 || c->rotary_dim > c->D || (c->halves & ~1) || (c->rotate & ~3)) return KVQ_ERR_INVALID_ARG;
    if (c->rotary_dim % 16) return KVQ_ERR_UNSUPPORTED;
    if (!(c->eps >= 0.f) || !std::isfinite(c->eps) || !(c->rope_base >= 0.f) || !std::isfinite(c->rope_base) || !std::isfinite(amp))
        return KVQ_ERR_INVALID_ARG;
    for (int j = 0; freq && j < c->rotary_dim / 2; j++)
        if (!(freq[j] >= 0) || freq[j] > 0x1p31) return KVQ_ERR_INVALID_ARG;
    return KVQ_OK;
}

}  // namespace host
}  // namespace kvq
