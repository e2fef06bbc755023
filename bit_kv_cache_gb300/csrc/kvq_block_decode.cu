// kvq_block_decode.cu -- attention of one token per slot over an 8-bit cache with one scale per
// page and head (kvq_paged_decode_attn), and of a few new tokens per slot (kvq_paged_chunk_attn).
//
// For a row (query head of a key head's group, token) and cached token x of tile i, with the page's
// scales s_K and s_V,
//   y_x = (q . code_x) s_K log2(e) / sqrt(D),   w_x = 2^(y_x - t_i),   t_i near the tile's largest y,
//   O = sum_i 2^(t_i - m) s_V sum_x w_x code_x,   l = sum_i 2^(t_i - m) sum_x w_x,   out = O / l:
// both products have exact operands (codes in fp16) but for w, which is rounded to fp16 once.  A tile's
// product is counted into the state by an fp32 factor that holds the value scale and the distance of
// the tile's reference from the state's, so that a weight's bits do not depend on other tiles: beside a
// token that takes most of the attention (an fp16 sink, a page of zeros, whose scale is 1), and beside
// pages of other scales, a weight has fp16's 11 bits as long as it is 2^-29 of its tile's largest.
// (With the scale in the exponent and one reference for all tiles, which cost 1 us less of
// chunk_verify's 31 and nothing elsewhere, weights of pages of small values fell below fp16's normal
// numbers: outputs off by up to 20 times what roundings make.)  Sums, m and l are fp32.
//
// Bound by memory: 8 slots of 17K to 56K tokens (561 MB) take 88 us, 6.4 TB/s, 0.94 of a plain copy's
// rate.  Each warp has a ring of its own and works alone until its part ends: no barriers, 192 KB on
// their way per SM.  Three CTAs of two 8 KB pieces a warp: 88 us, 128 slots of 8 to 4001 tokens 40
// (two CTAs of three pieces: 90.8 and 41; six CTAs of two warps: 90 and 56, the longest slots end
// last; plain loads into registers: 119 and 70).  One slot of 131K tokens takes 47 us, of which joining
// its 57 parts takes 5.  Long slots first: 128 slots 51 -> 41 us.  More parts than run at once: 46 to
// 52 us there, as joining costs a launch.  Letting the kernel behind start early: 44 us there
// (from the end of the loop on: no change, nor in joining).
// Rows of a chunk: up to 8 (16, 32) in one (two, four) operand tiles of 8.  8 slots as above with 4
// tokens and heads each take 90 us; with 8 tokens 126 (int8 132), bound by the tensor core's issue at
// two CTAs per SM (255 registers; 520 to 640 bytes of a thread spilled, of tiles between products).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "kvq_block.cuh"
#include "kvq_block.h"
#include "kvq_host.h"
#include "kvq_tcgen05.cuh"

namespace kvq {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStages = 2, kPiece = 8192;                // of a warp's ring: keys or values of a packed tile
constexpr int kTokens = 64, kTailTokens = 16;            // of an item: packed, fp16
constexpr int kLeast = 16;                               // items of a part, if the slot has as many
constexpr float kUp = 15.f, kLag = 16.f;                 // log2: a tile's largest weight; the state's reference lags by so much at most
static_assert(kFewRows == 32, "row tiles of the largest form");

// A warp's state for NT tiles of 8 rows: lane (r, c) = (lane / 4, lane % 4) has rows 2 c, 2 c + 1 of
// each (columns of the products) and, of the output, channels of rows r and r + 8 of eight 16-row
// tiles.
template <int NT>
struct State {
    float m[NT][2], l[NT][2];   // reference (-inf: none yet), sum in units of 2^m, the lane's own share
    float o[NT][8][4];          // in the same units
};

// Query operands: rows of tile n, step i, of a lane.  One tile stays in registers, more in shared
// memory.
template <int NT>
struct Queries {
    const uint2 *sm;
    __device__ __forceinline__ uint2 get(int i, int n, int lane) const { return sm[(i * NT + n) * 32 + lane]; }
};
template <>
struct Queries<1> {
    uint2 x[8];
    __device__ __forceinline__ uint2 get(int i, int, int) const { return x[i]; }
};

// The channel of output row r (hi: r + 8) of tile i.
__device__ __forceinline__ int out_channel(int i, int r, int hi) { return 32 * (i >> 1) + 8 * (r >> 1) + 4 * (i & 1) + 2 * hi + (r & 1); }

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Scores of 16 N tokens (x[s]: tokens r and r + 8 of group s, rows 2 c, 2 c + 1 of row tile n) to
// weights 2^(y - t), y = x a, as B operands of the value product; t is kUp below the tile's largest y
// of a row.  u: 2^(t - m), what the product counts in the state.
template <int N, int NT>
__device__ __forceinline__ void weights(State<NT> &st, int n, float (&x)[N][4], float a, float (&u)[2], uint32_t (*b)[2]) {
#pragma unroll
    for (int s = 0; s < N; s++)
#pragma unroll
        for (int e = 0; e < 4; e++) x[s][e] = __fmul_rn(x[s][e], a);  // (not joined with the difference to t, which has its rounding)
    float top[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
        top[e] = fmaxf(x[0][e], x[0][2 + e]);
#pragma unroll
        for (int s = 1; s < N; s++) top[e] = fmaxf(top[e], fmaxf(x[s][e], x[s][2 + e]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
    }
    if (__any_sync(0xffffffffu, top[0] - st.m[n][0] > kLag || top[1] - st.m[n][1] > kLag)) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const float m = fmaxf(st.m[n][e], top[e]), f = m == st.m[n][e] ? 1.f : ex2(st.m[n][e] - m);
            st.m[n][e] = m;
            st.l[n][e] *= f;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                st.o[n][i][e] *= f;
                st.o[n][i][2 + e] *= f;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; e++) {
        // t itself beyond 2^22, where exponents are 0.5 and more apart and kUp less would be rounded
        if (fabsf(top[e]) < 0x1p22f) top[e] -= kUp;
        u[e] = top[e] == -INFINITY ? 0.f : ex2(top[e] - st.m[n][e]);
        if (top[e] == -INFINITY) top[e] = 0.f;
    }
    const uint64_t less = pk2(-top[0], -top[1]);
    uint64_t sum = 0;
#pragma unroll
    for (int s = 0; s < N; s++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            float2 w = up2(add_x2(pk2(x[s][2 * e], x[s][2 * e + 1]), less));
            w.x = ex2(w.x);
            w.y = ex2(w.y);
            sum = add_x2(sum, pk2(w.x, w.y));
            b[s][e] = transpose8(pack_half2(w.x, w.y));
        }
    const float2 add = up2(sum);
    st.l[n][0] = fmaf(add.x, u[0], st.l[n][0]);
    st.l[n][1] = fmaf(add.y, u[1], st.l[n][1]);
}

// o += p u, of rows 2 c and 2 c + 1 for two channels.
__device__ __forceinline__ void count(float (&o)[4], const float (&p)[4], uint64_t u) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const float2 y = up2(fma_x2(pk2(p[e], p[e + 1]), u, pk2(o[e], o[e + 1])));
        o[e] = y.x;
        o[e + 1] = y.y;
    }
}

// A packed tile.  The order of the contracted dimension is free as long as both operands share
// it.  Keys: lane c's words of a row are its 16-byte chunks c and c + 4, so a word (four
// neighbouring channels) is one step's operand; q is held in that order.  Values: a lane's 16 bytes
// are 16 neighbouring tokens of a channel, word s those of step s: step s takes tokens 16 c + 4 s
// .. + 3 of every c, and the score rows are arranged so.
template <bool E4M3, int NT>
__device__ __forceinline__ void key_tile(const Queries<NT> &q, const uint8_t *k, float (&x)[NT][4][4], int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int s = 0; s < 4; s++) {
        const uint8_t *row = k + (16 * (r >> 1) + 4 * s + (r & 1)) * 128 + c * 16;
        const int near = (r & 1) << 6, far = 64 - near;
        uint4 w[2][2];
        w[0][0] = *reinterpret_cast<const uint4 *>(row + near);
        w[0][1] = *reinterpret_cast<const uint4 *>(row + far);
        w[1][0] = *reinterpret_cast<const uint4 *>(row + 256 + near);
        w[1][1] = *reinterpret_cast<const uint4 *>(row + 256 + far);
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) x[n][s][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            uint32_t a[4];
            code_pairs<E4M3>((&w[0][i >> 2].x)[i & 3], a[0], a[2]);
            code_pairs<E4M3>((&w[1][i >> 2].x)[i & 3], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const uint2 y = q.get(i, n, lane);
                mma_16816(x[n][s], a[0], a[1], a[2], a[3], y.x, y.y);
            }
        }
    }
}
template <bool E4M3, int NT>
__device__ __forceinline__ void value_tile(State<NT> &st, const uint8_t *v, const uint32_t (&b)[NT][4][2], const float (&u)[NT][2], float scale, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint4 lo = *reinterpret_cast<const uint4 *>(v + out_channel(i, r, 0) * 64 + c * 16);
        const uint4 hi = *reinterpret_cast<const uint4 *>(v + out_channel(i, r, 1) * 64 + c * 16);
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[n][e] = 0.f;
#pragma unroll
        for (int s = 0; s < 4; s++) {
            uint32_t a[4];
            code_pairs<E4M3>((&lo.x)[s], a[0], a[2]);
            code_pairs<E4M3>((&hi.x)[s], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NT; n++) mma_16816(o[n], a[0], a[1], a[2], a[3], b[n][s][0], b[n][s][1]);
        }
#pragma unroll
        for (int n = 0; n < NT; n++) count(st.o[n][i], o[n], pk2(u[n][0] * scale, u[n][1] * scale));
    }
}

// Infinite and NaN values of eight channels become 0 (a weight of 0 would make them NaN in rows
// that may not see them); true if there are any.
__device__ __forceinline__ bool drop_odd(uint4 &v) {
    bool odd = false;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        uint32_t &x = (&v.x)[e];
        if ((x & 0x7c00u) == 0x7c00u) x &= 0xffff0000u, odd = true;
        if ((x & 0x7c000000u) == 0x7c000000u) x &= 0xffffu, odd = true;
    }
    return odd;
}

// 16 fp16 tokens from x0 on: rows r and r + 8 (k0, k1, v0, v1), seen by a row if below its lim.  A
// value row's 8 channels 32 j + 8 c .. of lane c are turned into operand rows by 8 x 8 transposes.
// True if a value was infinite or NaN.
template <int NT>
__device__ __forceinline__ bool tail_tile(State<NT> &st, const Queries<NT> &q, const uint16_t *k0, const uint16_t *k1,
                                          const uint16_t *v0, const uint16_t *v1, int x0, int seen, const int (&lim)[NT][2], int lane) {
    const int r = lane >> 2, c = lane & 3;
    const bool on0 = x0 + r < seen, on1 = x0 + r + 8 < seen;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 k[4][2], v[4][2];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int ch = (i >> 1) * 64 + c * 16 + (i & 1) * 8;
        k[i][0] = on0 ? *reinterpret_cast<const uint4 *>(k0 + ch) : zero;
        k[i][1] = on1 ? *reinterpret_cast<const uint4 *>(k1 + ch) : zero;
    }
    auto load_values = [&] {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i][0] = on0 ? *reinterpret_cast<const uint4 *>(v0 + 32 * i + 8 * c) : zero;
            v[i][1] = on1 ? *reinterpret_cast<const uint4 *>(v1 + 32 * i + 8 * c) : zero;
        }
    };
    if (NT < 4) load_values();  // before the first use of the keys, if there are registers for both
    uint32_t b[NT][1][2];
    float u[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++) {
        float x[1][4] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint2 y = q.get(2 * i, n, lane), z = q.get(2 * i + 1, n, lane);
            mma_16816(x[0], k[i][0].x, k[i][1].x, k[i][0].y, k[i][1].y, y.x, y.y);
            mma_16816(x[0], k[i][0].z, k[i][1].z, k[i][0].w, k[i][1].w, z.x, z.y);
        }
#pragma unroll
        for (int e = 0; e < 2; e++) {
            if (x0 + r >= lim[n][e]) x[0][e] = -INFINITY;
            if (x0 + r + 8 >= lim[n][e]) x[0][2 + e] = -INFINITY;
        }
        weights<1, NT>(st, n, x, kScale, u[n], b[n]);
    }
    if (NT == 4) load_values();
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        odd |= drop_odd(v[j][0]);
        odd |= drop_odd(v[j][1]);
        const uint32_t a[8] = {transpose8(v[j][0].x), transpose8(v[j][0].y), transpose8(v[j][1].x), transpose8(v[j][1].y),
                               transpose8(v[j][0].z), transpose8(v[j][0].w), transpose8(v[j][1].z), transpose8(v[j][1].w)};
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float o[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            mma_16816(o[0], a[0], a[1], a[2], a[3], b[n][0][0], b[n][0][1]);
            mma_16816(o[1], a[4], a[5], a[6], a[7], b[n][0][0], b[n][0][1]);
            count(st.o[n][2 * j], o[0], pk2(u[n][0], u[n][1]));
            count(st.o[n][2 * j + 1], o[1], pk2(u[n][0], u[n][1]));
        }
    }
    return odd;
}

// Of a state below the largest reference: positive, so that an infinite value stays infinite
// (2^-126 of a finite one is far below the other's smallest step).
__device__ __forceinline__ float factor(float m, float top) { return m == top ? 1.f : fmaxf(ex2(m - top), 0x1p-126f); }

struct Bars {
    uint64_t full[kWarps][kStages];
    int stop, odd;
};
// Shared memory: rings (then the outputs of the warps' states), queries, references and sums, barriers.
constexpr int kRingBytes = kWarps * kStages * kPiece;
static_assert(kWarps * kFewRows * 128 * 4 <= kRingBytes, "shared memory");
template <int NT>
constexpr int kSmemBytes = kRingBytes + (NT > 1 ? NT * 2048 : 0) + kWarps * 8 * NT * 8 + (int)sizeof(Bars);

// Lengths of a slot: {sink, packed, residual, new tokens (decode: 0)}, the row of its first query.
struct Slot {
    int ns, T, nr, n_new;
    int64_t q0;
    bool on;
    __device__ __forceinline__ int seen() const { return ns + nr + n_new; }
};
__device__ __forceinline__ Slot slot_at(const BlockDecodeParams &p, int b) {
    if (p.desc) {
        const int4 x = reinterpret_cast<const int4 *>(p.desc)[2 * b];
        return {x.x, x.y, x.z, x.w, p.desc[8 * b + 4], x.w > 0};
    }
    const int4 x = reinterpret_cast<const int4 *>(p.lens)[b];
    return {x.x, x.y, x.z, 0, b, x.w && x.x + x.y + x.z > 0};
}
// Row x of a slot's [sink | residual | new tokens].
__device__ __forceinline__ const uint16_t *tail_at(const BlockDecodeParams &p, const Slot &s, size_t u, int h, int x, bool value) {
    if (x < s.ns) return (value ? p.v_sink : p.k_sink) + (u * p.S + x) * 128;
    x -= s.ns;
    if (x < s.nr) return (value ? p.v_res : p.k_res) + (u * p.R + x) * 128;
    x -= s.nr;
    return value ? p.v_new + (s.q0 + x) * p.v_stride + h * 128 : p.k_new + (s.q0 + x) * p.k_stride + h * 128;
}

template <bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) block_decode_kernel(const __grid_constant__ BlockDecodeParams p) {
    extern __shared__ __align__(128) unsigned char sm[];
    uint2 *s_q = reinterpret_cast<uint2 *>(sm + kRingBytes);
    Bars *bar = reinterpret_cast<Bars *>(sm + kSmemBytes<NT> - sizeof(Bars));
    const int h = blockIdx.x, w = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps; i++)
            for (int j = 0; j < kStages; j++) mbar_init(&bar->full[i][j], 1);
        bar->stop = bar->odd = 0;
        fence_barrier_init();
    }
    int lo = 0, hi = p.n_slots - 1;  // the slot
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.part0[mid + 1] > (int)blockIdx.y) hi = mid;
        else lo = mid + 1;
    }
    const int b = p.slot[lo], parts = p.part0[lo + 1] - p.part0[lo], part = blockIdx.y - p.part0[lo];
    const size_t u = (size_t)b * p.H_kv + h;
    const int32_t *row = p.ptab + (size_t)b * p.ptab_stride;
    griddep_wait();
    const Slot sl = slot_at(p, b);
    if (!sl.on) return;
    const int rows = max(sl.n_new, 1) * p.g;
    Queries<NT> q;
    auto operand = [&](int n, uint2 (&x)[8]) {  // rows behind the last one are zeros
        const int row = 8 * n + r;
        const uint16_t *src = p.q + (sl.q0 + row / p.g) * p.q_stride + (h * p.g + row % p.g) * 128;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint4 y = make_uint4(0, 0, 0, 0);
            if (row < rows) y = *reinterpret_cast<const uint4 *>(src + (i >> 1) * 64 + c * 16 + (i & 1) * 8);
            x[2 * i] = make_uint2(y.x, y.y);
            x[2 * i + 1] = make_uint2(y.z, y.w);
        }
    };
    if constexpr (NT == 1) {
        operand(0, q.x);
    } else {
        q.sm = s_q;
        if (w < NT) {
            uint2 x[8];
            operand(w, x);
#pragma unroll
            for (int i = 0; i < 8; i++) s_q[(i * NT + w) * 32 + lane] = x[i];
        }
    }
    __syncthreads();
    const int np = sl.T / kTokens, seen = sl.seen(), n = np + (seen + kTailTokens - 1) / kTailTokens;
    const int begin = (int)((int64_t)n * part / parts), end = (int)((int64_t)n * (part + 1) / parts);
    State<NT> st;
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
            st.m[t][e] = -INFINITY, st.l[t][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) st.o[t][i][e] = 0.f;
    }

    // Packed tiles begin + w, begin + w + kWarps, ...: their pieces, keys and values in turn, are
    // brought by bulk copies kStages ahead.  Lane j holds page and scales of tile j of 32.
    const int tiles = begin + w < min(end, np) ? (min(end, np) - begin - w + kWarps - 1) / kWarps : 0;
    unsigned char *ring = sm + w * kStages * kPiece;
    uint64_t *full = bar->full[w];
    int brought = 0;  // pieces
    for (int t0 = 0; t0 == 0 || t0 < tiles; t0 += 32) {
        const int m = min(32, tiles - t0);
        size_t at = 0;
        float sk = 0.f, sv = 0.f;
        if (lane < m) {
            const int tok = (begin + w + (t0 + lane) * kWarps) * kTokens;
            int page = row[tok >> p.g_shift];
            if (page < 0 || page >= p.n_pages) {
                report(p.status, KVQ_DEV_BAD_STATE);
                page = 0;
            }
            const size_t pg = (size_t)page * p.H_kv + h;
            at = ((pg << p.g_shift) + (tok & ((1 << p.g_shift) - 1))) * 128;
            sk = page_scale(p.k_scale[pg].x);
            sv = page_scale(p.v_scale[pg].x);
        }
        auto bring = [&](int i) {  // piece i of these tiles
            const size_t from = __shfl_sync(0xffffffffu, at, i >> 1);
            if (*(volatile int *)&bar->stop) return;  // a wait ran out: nothing more is asked for
            brought = 2 * t0 + i + 1;
            if (lane) return;
            const int stage = (2 * t0 + i) % kStages;
            mbar_arrive_expect_tx(&full[stage], kPiece);
            bulk_g2s(ring + stage * kPiece, (i & 1 ? p.v_codes : p.k_codes) + from, kPiece, &full[stage]);
        };
        for (int i = 0; i < min(kStages, 2 * m); i++) bring(i);
        // the warp's fp16 tiles, while the first pieces are on their way
        for (int i = t0 ? end : begin + w + (max(np - begin - w, 0) + kWarps - 1) / kWarps * kWarps; i < end; i += kWarps) {
            int lim[NT][2];  // fp16 tokens that a row may see
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int e = 0; e < 2; e++) lim[t][e] = sl.n_new ? sl.ns + sl.nr + min(8 * t + 2 * c + e, rows - 1) / p.g + 1 : seen;
            const int x = (i - np) * kTailTokens, x0 = min(x + r, seen - 1), x1 = min(x + r + 8, seen - 1);
            if (tail_tile<NT>(st, q, tail_at(p, sl, u, h, x0, false), tail_at(p, sl, u, h, x1, false), tail_at(p, sl, u, h, x0, true),
                              tail_at(p, sl, u, h, x1, true), x, seen, lim, lane))
                *(volatile int *)&bar->odd = 1;
        }
        for (int t = 0; t < m; t++) {
            uint32_t bp[NT][4][2];
            float u[NT][2];
            const int i = 2 * t, k = 2 * t0 + i;  // pieces: of these tiles, of all
            warp_await(&full[k % kStages], (k / kStages) & 1, &bar->stop, p.status);
            const float tk = kScale * __shfl_sync(0xffffffffu, sk, t), tv = __shfl_sync(0xffffffffu, sv, t);
            float x[NT][4][4];
            key_tile<E4M3, NT>(q, ring + k % kStages * kPiece, x, lane);
            __syncwarp();
            if (i + kStages < 2 * m) bring(i + kStages);
#pragma unroll
            for (int y = 0; y < NT; y++) weights<4, NT>(st, y, x[y], tk, u[y], bp[y]);
            warp_await(&full[(k + 1) % kStages], ((k + 1) / kStages) & 1, &bar->stop, p.status);
            value_tile<E4M3, NT>(st, ring + (k + 1) % kStages * kPiece, bp, u, tv, lane);
            __syncwarp();
            if (i + 1 + kStages < 2 * m) bring(i + 1 + kStages);
        }
    }
    // where a wait ran out, the copies on their way land (or are waited for once more) before the block ends
    if (*(volatile int *)&bar->stop)
        for (int k = max(brought - kStages, 0); k < brought; k++) mbar_wait(&full[k % kStages], (k / kStages) & 1, p.status);
    // the warps' states, joined in warp order: 8 NT rows of 128 channels each, in the rings
    constexpr int kRows = 8 * NT;
    float(*s_o)[kRows][128] = reinterpret_cast<float(*)[kRows][128]>(sm);
    float(*s_m)[kRows] = reinterpret_cast<float(*)[kRows]>(sm + kRingBytes + (NT > 1 ? NT * 2048 : 0)), (*s_l)[kRows] = s_m + kWarps;
    __syncthreads();  // every piece has arrived and been read
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int y = 8 * t + 2 * c + e;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) st.l[t][e] += __shfl_xor_sync(0xffffffffu, st.l[t][e], o);
            if (r == 0) {
                s_m[w][y] = st.m[t][e];
                s_l[w][y] = st.l[t][e];
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                s_o[w][y][out_channel(i, r, 0)] = st.o[t][i][e];
                s_o[w][y][out_channel(i, r, 1)] = st.o[t][i][2 + e];
            }
        }
    __syncthreads();
    const int odd = *(volatile int *)&bar->odd;
#pragma unroll 2
    for (int y = w; y < rows; y += kWarps) {  // a warp per row, four channels a lane
        float m = s_m[0][y], l = 0.f;
#pragma unroll
        for (int i = 1; i < kWarps; i++) m = fmaxf(m, s_m[i][y]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kWarps; i++) {
            const float f = factor(s_m[i][y], m);
            const float4 v = reinterpret_cast<const float4 *>(s_o[i][y])[lane];
            l = fmaf(f, s_l[i][y], l);
            o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
        }
        const int tok = y / p.g;
        if (odd) {  // infinite and NaN values of the part's fp16 tokens
            const int to = min(sl.n_new ? sl.ns + sl.nr + tok + 1 : seen, (end - np) * kTailTokens);
            for (int x = max(begin - np, 0) * kTailTokens; x < to; x++) {
                const uint2 v = reinterpret_cast<const uint2 *>(tail_at(p, sl, u, h, x, true))[lane];
                const float2 v0 = unpack_half2(v.x), v1 = unpack_half2(v.y);
                if (!isfinite(v0.x)) o.x += v0.x;
                if (!isfinite(v0.y)) o.y += v0.y;
                if (!isfinite(v1.x)) o.z += v1.x;
                if (!isfinite(v1.y)) o.w += v1.y;
            }
        }
        if (parts == 1) {
            const float inv = 1.f / l;
            uint16_t *dst = p.out + ((sl.q0 + tok) * p.H_kv * p.g + h * p.g + y - tok * p.g) * 128;
            reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(pack_half2(o.x * inv, o.y * inv), pack_half2(o.z * inv, o.w * inv));
        } else {
            const size_t at = ((size_t)blockIdx.y * p.H_kv + h) * p.most_rows + y;
            reinterpret_cast<float4 *>(p.part_o + at * 128)[lane] = o;
            if (lane == 0) p.part_ml[at] = make_float2(m, l);
        }
    }
}

// Slots in several parts: WARPS warps (1 or 8) per row of a key head, every WARPS-th part each, four
// at a time; then the warps' states in warp order.  Eight for slots in many parts (one slot of 131K
// tokens in 57, cold: 22 us with a CTA per row and one part after the other), one for at most eight.
constexpr int kJoinWarps = 8;
template <int WARPS>
__global__ void __launch_bounds__(32 * kJoinWarps) block_combine_kernel(const __grid_constant__ BlockDecodeParams p) {
    __shared__ float4 s_o[kJoinWarps][32];
    __shared__ float2 s_ml[kJoinWarps];
    const int w = WARPS == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31, at_slot = blockIdx.y;
    const int x = WARPS == 1 ? blockIdx.x * kJoinWarps + (threadIdx.x >> 5) : blockIdx.x, y = x % p.most_rows, h = x / p.most_rows;
    if (h >= p.H_kv) return;
    const int first = p.part0[at_slot], parts = p.part0[at_slot + 1] - first, b = p.slot[at_slot];
    if (parts < 2) return;
    griddep_wait();
    const Slot sl = slot_at(p, b);
    if (!sl.on || y >= max(sl.n_new, 1) * p.g) return;
    const size_t step = (size_t)p.H_kv * p.most_rows, at = ((size_t)first * p.H_kv + h) * p.most_rows + y;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto join = [&](const float2 &ml, const float4 &x) {
        const float top = fmaxf(m, ml.x), f0 = factor(m, top), f1 = factor(ml.x, top);
        m = top;
        l = fmaf(f0, l, f1 * ml.y);
        o.x = fmaf(f0, o.x, f1 * x.x);
        o.y = fmaf(f0, o.y, f1 * x.y);
        o.z = fmaf(f0, o.z, f1 * x.z);
        o.w = fmaf(f0, o.w, f1 * x.w);
    };
    for (int i0 = w; i0 < parts; i0 += 4 * WARPS) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const size_t z = at + min(i0 + k * WARPS, parts - 1) * step;
            ml[k] = p.part_ml[z];
            v[k] = reinterpret_cast<const float4 *>(p.part_o + z * 128)[lane];
        }
#pragma unroll
        for (int k = 0; k < 4; k++)
            if (i0 + k * WARPS < parts) join(ml[k], v[k]);
    }
    if (WARPS > 1) {
        s_o[w][lane] = o;
        if (lane == 0) s_ml[w] = make_float2(m, l);
        __syncthreads();
        if (w) return;
        for (int i = 1; i < min(WARPS, parts); i++) join(s_ml[i], s_o[i][lane]);
    }
    const float inv = 1.f / l;
    uint16_t *dst = p.out + ((sl.q0 + y / p.g) * p.H_kv * p.g + h * p.g + y % p.g) * 128;
    reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(pack_half2(o.x * inv, o.y * inv), pack_half2(o.z * inv, o.w * inv));
}

template <bool E4M3, int NT>
cudaError_t launch(dim3 grid, const BlockDecodeParams &p, cudaStream_t st) {
    static bool ready[64];  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        e = cudaFuncSetAttribute(block_decode_kernel<E4M3, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<NT>);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    return launch_dependent(block_decode_kernel<E4M3, NT>, grid, kThreads, kSmemBytes<NT>, st, p);
}

// CTAs that run at once; parts of the slots that are cut (none where there are as many slots as
// that).
int resident(int tiles) { return (tiles == 1 ? 3 : 2) * host::num_sms(); }
int64_t most_parts(const kvq_config *c) { return host::cdiv(resident(1), c->H_kv); }

// Cuts the slots (items each, 0: not part of the call) into parts and launches.
cudaError_t run(const kvq_config *c, const int *items, BlockDecodeParams &p, cudaStream_t st) {
    const int tiles = p.most_rows <= 8 ? 1 : p.most_rows <= 16 ? 2 : 4;
    int count[64] = {0}, longest = 0, active = 0;
    for (int b = 0; b < c->B; b++) {
        longest = std::max(longest, items[b]);
        active += items[b] > 0;
    }
    // slots of more items first (64 classes), so that what runs last is short
    auto size_class = [&](int n) { return 63 - (int)((int64_t)n * 63 / longest); };
    for (int b = 0; b < c->B; b++)
        if (items[b]) count[size_class(items[b])]++;
    for (int i = 0, at = 0; i < 64; i++) {
        const int n = count[i];
        count[i] = at;
        at += n;
    }
    for (int b = 0; b < c->B; b++)
        if (items[b]) p.slot[count[size_class(items[b])]++] = (int16_t)b;
    // parts of at most X items, the smallest X whose parts are all resident at once
    const int64_t room = std::max<int64_t>(active, host::cdiv(resident(tiles), c->H_kv));
    int lo = std::min(longest, kLeast), hi = longest;
    while (lo < hi) {
        const int X = (lo + hi) / 2;
        int64_t parts = 0;
        for (int i = 0; i < active; i++) parts += (items[p.slot[i]] + X - 1) / X;
        if (parts <= room) hi = X;
        else lo = X + 1;
    }
    int parts = 0, cut = 0;  // cut: the slots before it are in several parts
    for (int i = 0; i < active; i++) {
        p.part0[i] = parts;
        const int n = (items[p.slot[i]] + lo - 1) / lo;
        if (n > 1) cut = i + 1;
        parts += n;
    }
    p.n_slots = active;
    p.part0[active] = parts;
    const dim3 grid((unsigned)c->H_kv, (unsigned)parts);
    auto go = [&](auto form) {
        constexpr bool F = decltype(form)::value;
        return tiles == 1 ? launch<F, 1>(grid, p, st) : tiles == 2 ? launch<F, 2>(grid, p, st) : launch<F, 4>(grid, p, st);
    };
    const cudaError_t e = c->mode == KVQ_MODE_E4M3 ? go(std::true_type()) : go(std::false_type());
    if (e != cudaSuccess || !cut) return e;
    const int64_t joined = (int64_t)p.most_rows * c->H_kv;
    if (p.part0[1] > kJoinWarps)  // the longest slot's parts
        return launch_dependent(block_combine_kernel<kJoinWarps>, dim3((unsigned)joined, (unsigned)cut), 32 * kJoinWarps, 0, st, p);
    return launch_dependent(block_combine_kernel<1>, dim3((unsigned)host::cdiv(joined, kJoinWarps), (unsigned)cut), 32 * kJoinWarps, 0, st, p);
}

// What both calls read of the cache.
void fill(const kvq_config *c, const kvq_paged *pc, BlockDecodeParams &p) {
    memset(&p, 0, sizeof(p));
    p.k_codes = reinterpret_cast<const uint8_t *>(pc->k_codes);
    p.v_codes = reinterpret_cast<const uint8_t *>(pc->v_codes);
    p.k_scale = reinterpret_cast<const float4 *>(pc->k_meta);
    p.v_scale = reinterpret_cast<const float4 *>(pc->v_meta);
    p.k_sink = pc->k_sink;
    p.v_sink = pc->v_sink;
    p.k_res = pc->k_res;
    p.v_res = pc->v_res;
    p.ptab = pc->page_table;
    p.n_pages = pc->n_pages;
    p.H_kv = c->H_kv;
    p.g = c->H_q / c->H_kv;
    p.g_shift = c->G == 64 ? 6 : c->G == 128 ? 7 : 8;
    p.S = c->S;
    p.R = c->R;
    p.ptab_stride = (int)(c->max_T / c->G);
}

int items_of(int ns, int T, int nr, int n_new) { return T / kTokens + (ns + nr + n_new + kTailTokens - 1) / kTailTokens; }

size_t ml_bytes(const kvq_config *c) { return (size_t)host::cdiv(most_parts(c) * c->H_q * 8, 256) * 256; }

}  // namespace

size_t block_decode_ws_bytes(const kvq_config *c) { return 256 + ml_bytes(c) + (size_t)most_parts(c) * c->H_q * 128 * 4; }

int block_decode(const kvq_config *c, const kvq_paged *pc, const uint16_t *q, uint16_t *out, void *ws, size_t ws_bytes,
                 cudaStream_t st) {
    const size_t rows = (size_t)c->B * c->H_q * c->D * 2;
    if (out != q && host::overlap(out, rows, q, rows)) return KVQ_ERR_INVALID_ARG;  // a row's own place: read before it is written
    if (!ws || !host::aligned16(ws) || ws_bytes < block_decode_ws_bytes(c)) return KVQ_ERR_WORKSPACE;
    BlockDecodeParams p;
    fill(c, pc, p);
    char *w = static_cast<char *>(ws);
    p.status = reinterpret_cast<int32_t *>(w);
    p.part_ml = reinterpret_cast<float2 *>(w + 256);
    p.part_o = reinterpret_cast<float *>(w + 256 + ml_bytes(c));
    p.q = q;
    p.q_stride = (int64_t)c->H_q * c->D;
    p.out = out;
    p.lens = pc->lens;
    p.most_rows = p.g;
    int items[KVQ_PAGED_MAX_B];
    bool any = false;
    for (int b = 0; b < c->B; b++) {
        const int32_t *l = pc->lens_host + 4 * b;
        items[b] = l[3] ? items_of(l[0], l[1], l[2], 0) : 0;
        if (l[3] && l[1] && pc->n_pages < 1) return KVQ_ERR_INVALID_ARG;  // page 0 stands in for bad entries
        any |= items[b] > 0;
    }
    return any ? host::status_of(run(c, items, p, st)) : KVQ_OK;
}

int block_chunk_few(const kvq_config *c, const kvq_paged *pc, const ChunkSlot *slots, const bool *few, const ChunkAttnParams &a,
                    cudaStream_t st) {
    BlockDecodeParams p;
    fill(c, pc, p);
    p.desc = a.desc;
    p.status = a.status;
    p.part_ml = a.part_ml;
    p.part_o = a.part_o;
    p.q = a.q;
    p.k_new = a.k_new;
    p.v_new = a.v_new;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.out = a.out;
    int items[KVQ_PAGED_MAX_B];
    for (int b = 0; b < c->B; b++) {
        const ChunkSlot &s = slots[b];
        items[b] = few[b] ? items_of(s.ns, s.T, s.nr, s.n_new) : 0;
        if (few[b]) p.most_rows = std::max(p.most_rows, s.n_new * p.g);
    }
    return host::status_of(run(c, items, p, st));
}

}  // namespace kvq
