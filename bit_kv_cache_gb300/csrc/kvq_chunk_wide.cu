// kvq_chunk_wide.cu -- chunk attention for many query rows per slot: 256 rows per unit on
// the 5th-generation tensor cores.
//
// One CTA per SM, sixteen warps in four groups of four:
//   groups 0, 1  softmax of query tile m = 0, 1 (128 rows each, a thread per row): reads
//                the scores S_m from tensor memory, keeps the row's running maximum and sum
//                in registers, writes the weights P_m over S_m as fp16, rescales O_m when
//                the maximum has grown by more than 2^8;
//   group 2      makes the key and value tiles: packed pages arrive by bulk copies and are
//                dequantized into fp16 tiles in shared memory, fp16 rows are gathered;
//   warp 12      issues the products S_m = Q_m K^T and O_m += P_m V.
// The two query tiles alternate on the tensor core: while one's scores are in softmax, the
// other's products run; a key tile is dequantized once for both.  Tensor memory holds S_0,
// S_1, O_0, O_1 (128 columns each).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_chunk_attn.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

namespace {

constexpr int kRows = 256, kThreads = 512;
constexpr int kTileBytes = kChunkKeys * kD * 2;          // an fp16 key or value tile: 32 KB
constexpr int kRing = 2;                                 // tiles of each kind
constexpr int kRawBytes = 2 * (16384 + 512);             // packed tiles: codes and (scale, min)
constexpr int kMaxRaw = 4;
constexpr int kOffQ = 0, kOffK = 2 * kTileBytes, kOffV = kOffK + kRing * kTileBytes, kOffRaw = kOffV + kRing * kTileBytes,
              kOffBar = kOffRaw + kRawBytes;
constexpr float kScale = kLog2e * 0.08838834764831845f;  // log2(e) / sqrt(128)
// Weights are 2^(s - m + kUp): the running maximum may lag by kLag, so they stay below
// 2^(kUp + kLag) < 65504, and small ones keep kUp more bits above fp16's smallest step.
constexpr float kUp = 6.f, kLag = 8.f;
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
static_assert(256 * kRegsSoftmax + 256 * kRegsOther <= 65536 && kThreads * 128 == 65536, "register split");

struct Bars {
    uint64_t q_full, q_empty, k_full[kRing], k_empty[kRing], v_full[kRing], v_empty[kRing];
    uint64_t s_full[2], p_full[2], o_full[2], drain;
    uint64_t rawk[kMaxRaw], rawv[kMaxRaw];            // packed tile arrived
    uint64_t readk[kMaxRaw], readv[kMaxRaw];          // packed tile read by all producers
    uint32_t tmem;
    int stop;
    int odd[4];              // segment (+ 1) whose tail values are not all finite, by segment mod 4
};
constexpr int kSmemBytes = kOffBar + (int)sizeof(Bars) + 1024;  // + alignment
static_assert(kSmemBytes <= 232448, "shared memory");

// Segment: the items of one unit inside the CTA's range.
struct Seg {
    Item it;
    int k0, k1, np, valid, first;
};
__device__ __forceinline__ Seg next_seg(const ChunkAttnParams &p, int at, int end) {
    Seg s;
    s.it = find_item(p, at, kRows);
    s.k0 = at - s.it.first;
    s.k1 = min(s.it.n, end - s.it.first);
    s.np = s.it.s.T / kChunkKeys;
    s.valid = min(kRows, s.it.s.n_new * p.g - s.it.t * kRows);
    s.first = s.it.first;
    return s;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// Two codes in place (bits sh .. sh + BITS - 1 of each half) -> code * scale + min.  With
// the exponent of 1024 above them the halves are 1024 + code 2^sh; one fused step makes the
// exact code of it, another the value, rounded once.
template <int SH, uint32_t MASK>
__device__ __forceinline__ uint32_t deq2(uint32_t w, uint32_t s2, uint32_t m2) {
    const uint32_t v = (w & (MASK << SH)) | 0x64006400u;
    constexpr uint32_t mul = (uint32_t)(0x3c00 - (SH << 10)) * 0x10001u;            // 2^-SH
    constexpr uint32_t sub = (uint32_t)(0xe400 - (SH << 10)) * 0x10001u;            // -1024 2^-SH
    return hfma2(hfma2(v, mul, sub), s2, m2);
}
// The codes of one word as half2 pairs (j, j + n/2), n = 32 / BITS codes.
template <int BITS>
__device__ __forceinline__ void deq_word(uint32_t w, uint32_t s2, uint32_t m2, uint32_t *h) {
    if (BITS == 2) {
        h[0] = deq2<0, 0x00030003u>(w, s2, m2);
        h[1] = deq2<2, 0x00030003u>(w, s2, m2);
        h[2] = deq2<4, 0x00030003u>(w, s2, m2);
        h[3] = deq2<6, 0x00030003u>(w, s2, m2);
        h[4] = deq2<8, 0x00030003u>(w, s2, m2);
        w >>= 10;
        h[5] = deq2<0, 0x00030003u>(w, s2, m2);
        h[6] = deq2<2, 0x00030003u>(w, s2, m2);
        h[7] = deq2<4, 0x00030003u>(w, s2, m2);
    } else if (BITS == 4) {
        h[0] = deq2<0, 0x000f000fu>(w, s2, m2);
        h[1] = deq2<4, 0x000f000fu>(w, s2, m2);
        w >>= 8;
        h[2] = deq2<0, 0x000f000fu>(w, s2, m2);
        h[3] = deq2<4, 0x000f000fu>(w, s2, m2);
    } else {
        h[0] = deq2<0, 0x00ff00ffu>(w, s2, m2);
        w >>= 8;
        h[1] = deq2<0, 0x00ff00ffu>(w, s2, m2);
    }
}
// Position of token t within a packed tile: the pairs (j, j + n/2) of a key word side by side.
__device__ __forceinline__ int token_at(int pos, int kbits) {  // its inverse
    const int n = 32 / kbits, i = pos & (n - 1);
    return (pos & ~(n - 1)) + (i >> 1) + (n >> 1) * (i & 1);
}

// Keys: thread d dequantizes channel d.  Tile: rows are channels, tokens contiguous (two
// blocks of 64 tokens), so that a word's tokens are one or two 16-byte stores.
template <int BITS>
__device__ __forceinline__ void make_keys(const unsigned char *raw, unsigned char *tile, int d) {
    const uint32_t *cw = reinterpret_cast<const uint32_t *>(raw);
    const uint32_t sm = cw[512 * BITS + d];
    const uint32_t s2 = prmt(sm, sm, 0x1010), m2 = prmt(sm, sm, 0x3232);
    unsigned char *row = tile + d * 128;
    constexpr int NR = 4 * BITS;  // word rows of a tile
#pragma unroll 8
    for (int r = 0; r < NR; r += (BITS == 8 ? 2 : 1)) {
        uint32_t h[8];
        deq_word<BITS>(cw[r * kD + (d ^ ((r & 7) << 2))], s2, m2, h);
        if (BITS == 2) {
            unsigned char *b = row + (r >> 2) * 16384;
            const int c = 2 * (r & 3);
            *reinterpret_cast<uint4 *>(b + ((c ^ (d & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(b + (((c + 1) ^ (d & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
        } else if (BITS == 4) {
            *reinterpret_cast<uint4 *>(row + (r >> 3) * 16384 + (((r & 7) ^ (d & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
            deq_word<BITS>(cw[(r + 1) * kD + (d ^ (((r + 1) & 7) << 2))], s2, m2, h + 2);
            *reinterpret_cast<uint4 *>(row + (r >> 4) * 16384 + ((((r >> 1) & 7) ^ (d & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
}

// Values: thread p dequantizes the token at position p.  Tile: rows are token positions,
// channels contiguous (two blocks of 64 channels), in their natural order.
template <int BITS>
__device__ __forceinline__ void make_values(const unsigned char *raw, unsigned char *tile, int p, int kbits) {
    const uint32_t *cw = reinterpret_cast<const uint32_t *>(raw);
    const int t = token_at(p, kbits), TV = 256 / kbits, j = t & (TV - 1);
    constexpr int NR = 4 * BITS;  // word rows of a token
    const uint32_t sm = cw[512 * BITS + t];
    const uint32_t s2 = prmt(sm, sm, 0x1010), m2 = prmt(sm, sm, 0x3232);
    cw += (t - j) * NR;           // value tile of the token: [NR][TV]
    unsigned char *row = tile + p * 128;
#pragma unroll 8
    for (int m = 0; m < NR; m += (BITS == 8 ? 2 : 1)) {
        uint32_t h[8];
        deq_word<BITS>(cw[m * TV + (j ^ ((m & 7) << 2))], s2, m2, h);
        if (BITS == 2) {
            unsigned char *b = row + (m >> 2) * 16384;
            const int c = 2 * (m & 3);
            *reinterpret_cast<uint4 *>(b + ((c ^ (p & 7)) << 4)) = make_uint4(prmt(h[0], h[1], 0x5410), prmt(h[2], h[3], 0x5410),
                                                                            prmt(h[4], h[5], 0x5410), prmt(h[6], h[7], 0x5410));
            *reinterpret_cast<uint4 *>(b + (((c + 1) ^ (p & 7)) << 4)) = make_uint4(
                prmt(h[0], h[1], 0x7632), prmt(h[2], h[3], 0x7632), prmt(h[4], h[5], 0x7632), prmt(h[6], h[7], 0x7632));
        } else if (BITS == 4) {
            *reinterpret_cast<uint4 *>(row + (m >> 3) * 16384 + (((m & 7) ^ (p & 7)) << 4)) =
                make_uint4(prmt(h[0], h[1], 0x5410), prmt(h[2], h[3], 0x5410), prmt(h[0], h[1], 0x7632), prmt(h[2], h[3], 0x7632));
        } else {
            deq_word<BITS>(cw[(m + 1) * TV + (j ^ (((m + 1) & 7) << 2))], s2, m2, h + 2);
            *reinterpret_cast<uint4 *>(row + (m >> 4) * 16384 + ((((m >> 1) & 7) ^ (p & 7)) << 4)) =
                make_uint4(prmt(h[0], h[1], 0x5410), prmt(h[0], h[1], 0x7632), prmt(h[2], h[3], 0x5410), prmt(h[2], h[3], 0x7632));
        }
    }
}

// fp16 rows x0 .. x0 + 127 of [sink | residual | chunk]: row = token, 16-byte chunk c of a
// row at block c / 8, position c ^ row within it (the layout of both tail operands: key
// rows run along the tokens, value rows along the channels).  True if a value is not finite.
__device__ __forceinline__ bool make_tail(const ChunkAttnParams &p, const Seg &s, int x0, bool value, unsigned char *tile, int tid) {
    const int ntail = s.it.s.ns + s.it.s.nr + s.it.s.n_new, c = tid & 15;
    bool bad = false;
#pragma unroll 4
    for (int r = tid >> 4; r < kChunkKeys; r += 8) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (x0 + r < ntail) {
            a = __ldg(reinterpret_cast<const uint4 *>(tail_row(p, s.it, x0 + r, value)) + c);
            if (value) {
                uint32_t *v = reinterpret_cast<uint32_t *>(&a);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if ((v[e] & 0x7c00u) == 0x7c00u) v[e] &= 0xffff0000u, bad = true;
                    if ((v[e] & 0x7c000000u) == 0x7c000000u) v[e] &= 0xffffu, bad = true;
                }
            }
        }
        *reinterpret_cast<uint4 *>(tile + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = a;
    }
    return bad;
}

// ---------------------------------------------------------------- group 2: tiles ------
__device__ __forceinline__ void produce(const ChunkAttnParams &p, unsigned char *sm, Bars *bar, int begin, int end) {
    const int tid = threadIdx.x & 127;
    const int kraw = 2048 * p.kbits + 512, vraw = 2048 * p.vbits + 512;
    const uint32_t slots = min(kMaxRaw, kRawBytes / (kraw + vraw));
    unsigned char *raw_k = sm + kOffRaw, *raw_v = raw_k + slots * kraw;
    uint32_t nk = 0, nv = 0;              // tiles made
    uint32_t ck = 0, cv = 0, ik = 0, iv = 0;  // packed tiles consumed, copies issued (of keys, values)
    uint32_t nq = 0;
    // the copies of packed tile kt (thread 0)
    auto copy_k = [&](const Seg &s, int kt) {
        const int64_t page = page_of(p, s.it, kt);
        const int t0 = kt * kChunkKeys & (p.G - 1), sl = ik % slots;
        unsigned char *dst = raw_k + sl * kraw;
        mbar_arrive_expect_tx(&bar->rawk[sl], kraw);
        bulk_g2s(dst, p.k_codes + ((size_t)page * p.G + t0) * (kD * p.kbits / 32), 2048 * p.kbits, &bar->rawk[sl]);
        bulk_g2s(dst + 2048 * p.kbits, p.k_meta + (size_t)page * kD * 2, 512, &bar->rawk[sl]);
        ik++;
    };
    auto copy_v = [&](const Seg &s, int kt) {
        const int64_t page = page_of(p, s.it, kt);
        const int t0 = kt * kChunkKeys & (p.G - 1), sl = iv % slots;
        unsigned char *dst = raw_v + sl * vraw;
        mbar_arrive_expect_tx(&bar->rawv[sl], vraw);
        bulk_g2s(dst, p.v_codes + ((size_t)page * p.G + t0) * (kD * p.vbits / 32), 2048 * p.vbits, &bar->rawv[sl]);
        bulk_g2s(dst + 2048 * p.vbits, p.v_meta + ((size_t)page * p.G + t0) * 2, 512, &bar->rawv[sl]);
        iv++;
    };
    auto run = [&]() {
        int seg = 0;
        for (int at = begin; at < end; seg++) {
            const Seg s = next_seg(p, at, end);
            const int npk = min(s.k1, s.np);
            if (tid == 0)
                for (int kt = s.k0; kt < min(npk, s.k0 + (int)slots); kt++) {
                    // the slots' last readers were in the segment before
                    if (ik >= slots && !wait_or_stop(&bar->readk[ik % slots], (ik / slots - 1) & 1, &bar->stop, p.status)) return;
                    copy_k(s, kt);
                    if (iv >= slots && !wait_or_stop(&bar->readv[iv % slots], (iv / slots - 1) & 1, &bar->stop, p.status)) return;
                    copy_v(s, kt);
                }
            // queries: 128-row tiles, rows of tokens' heads; rows behind the last one repeat it
            if (!wait_or_stop(&bar->q_empty, (nq & 1) ^ 1, &bar->stop, p.status)) return;
            nq++;
            {
                const int c = tid & 15, rows = s.valid > 128 ? 256 : 128;
#pragma unroll 4
                for (int r = tid >> 4; r < rows; r += 8) {
                    const int x = s.it.t * kRows + min(r, s.valid - 1);
                    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p.q + (int64_t)(s.it.s.cu + x / p.g) * p.q_stride +
                                                                          (s.it.h * p.g + x % p.g) * kD) + c);
                    *reinterpret_cast<uint4 *>(sm + kOffQ + (r >> 7) * kTileBytes + (c >> 3) * 16384 + (r & 127) * 128 +
                                               (((c & 7) ^ (r & 7)) << 4)) = a;
                }
                fence_proxy_async();
                mbar_arrive(&bar->q_full);
            }
            for (int kt = s.k0; kt < s.k1; kt++) {
                const int ks = nk % kRing, vs = nv % kRing;
                unsigned char *kt_ = sm + kOffK + ks * kTileBytes, *vt_ = sm + kOffV + vs * kTileBytes;
                if (!wait_or_stop(&bar->k_empty[ks], ((nk / kRing) & 1) ^ 1, &bar->stop, p.status)) return;
                nk++;
                if (kt < s.np) {
                    const int sl = ck % slots;
                    if (!wait_or_stop(&bar->rawk[sl], (ck / slots) & 1, &bar->stop, p.status)) return;
                    ck++;
                    const unsigned char *raw = raw_k + sl * kraw;
                    if (p.kbits == 2) make_keys<2>(raw, kt_, tid);
                    else if (p.kbits == 4) make_keys<4>(raw, kt_, tid);
                    else make_keys<8>(raw, kt_, tid);
                } else {
                    make_tail(p, s, (kt - s.np) * kChunkKeys, false, kt_, tid);
                }
                fence_proxy_async();
                mbar_arrive(&bar->k_full[ks]);
                if (kt < s.np) {
                    const int sl = (ck - 1) % slots;
                    mbar_arrive(&bar->readk[sl]);
                    if (tid == 0 && kt + (int)slots < npk) {  // the next copy into this slot
                        if (!wait_or_stop(&bar->readk[sl], ((ck - 1) / slots) & 1, &bar->stop, p.status)) return;
                        copy_k(s, kt + (int)slots);
                    }
                }
                if (!wait_or_stop(&bar->v_empty[vs], ((nv / kRing) & 1) ^ 1, &bar->stop, p.status)) return;
                nv++;
                if (kt < s.np) {
                    const int sl = cv % slots;
                    if (!wait_or_stop(&bar->rawv[sl], (cv / slots) & 1, &bar->stop, p.status)) return;
                    cv++;
                    const unsigned char *raw = raw_v + sl * vraw;
                    if (p.vbits == 2) make_values<2>(raw, vt_, tid, p.kbits);
                    else if (p.vbits == 4) make_values<4>(raw, vt_, tid, p.kbits);
                    else make_values<8>(raw, vt_, tid, p.kbits);
                } else if (make_tail(p, s, (kt - s.np) * kChunkKeys, true, vt_, tid)) {
                    // infinite and NaN values enter the product as 0 (0 weights of rows that may
                    // not see them would spread them) and are added to their rows at the end
                    *(volatile int *)&bar->odd[seg & 3] = seg + 1;
                }
                fence_proxy_async();
                mbar_arrive(&bar->v_full[vs]);
                if (kt < s.np) {
                    const int sl = (cv - 1) % slots;
                    mbar_arrive(&bar->readv[sl]);
                    if (tid == 0 && kt + (int)slots < npk) {  // the next copy into this slot
                        if (!wait_or_stop(&bar->readv[sl], ((cv - 1) / slots) & 1, &bar->stop, p.status)) return;
                        copy_v(s, kt + (int)slots);
                    }
                }
            }
            at = s.first + s.k1;
        }
    };
    run();
    if (tid == 0) {  // copies still in flight after an early end
        for (; ck < ik; ck++) mbar_wait(&bar->rawk[ck % slots], (ck / slots) & 1, p.status);
        for (; cv < iv; cv++) mbar_wait(&bar->rawv[cv % slots], (cv / slots) & 1, p.status);
    }
}

// ---------------------------------------------------------------- warp 12: products ---
__device__ __forceinline__ void multiply(const ChunkAttnParams &p, unsigned char *sm, Bars *bar, uint32_t tm, int begin, int end) {
    const uint32_t base = smem_u32(sm);
    uint32_t nk = 0, nv = 0, nq = 0, np_[2] = {0, 0};
    auto scores = [&](int m, int ks, bool packed) {
        const uint64_t a0 = smem_desc(base + kOffQ + m * kTileBytes, 16, 1024);
        const uint32_t kb = base + kOffK + ks * kTileBytes;
        const uint64_t b0 = packed ? smem_desc(kb, 16384, 1024) : smem_desc(kb, 16, 1024);
        const uint32_t id = packed ? f16_idesc(128, 128, true) : f16_idesc(128, 128, false);
#pragma unroll
        for (int k = 0; k < 8; k++) {  // 16 channels each
            const uint64_t a = a0 + (((k >> 2) * 16384 + (k & 3) * 32) >> 4);
            const uint64_t b = b0 + (packed ? (k * 2048) >> 4 : ((k >> 2) * 16384 + (k & 3) * 32) >> 4);
            mma_ss(tm + m * 128, a, b, id, k > 0);
        }
        tc_commit(&bar->s_full[m]);
    };
    auto run = [&]() {
        for (int at = begin; at < end;) {
            const Seg s = next_seg(p, at, end);
            const int n = s.k1 - s.k0, M = s.valid > 128 ? 2 : 1;
            if (!wait_or_stop(&bar->q_full, nq & 1, &bar->stop, p.status)) return;
            nq++;
            if (!wait_or_stop(&bar->k_full[nk % kRing], (nk / kRing) & 1, &bar->stop, p.status)) return;
            tc_fence_after();
            for (int m = 0; m < M; m++) scores(m, nk % kRing, s.k0 < s.np);
            tc_commit(&bar->k_empty[nk % kRing]);
            nk++;
            if (n == 1) tc_commit(&bar->q_empty);
            for (int j = 0; j < n; j++) {
                const int vs = nv % kRing;
                if (!wait_or_stop(&bar->v_full[vs], (nv / kRing) & 1, &bar->stop, p.status)) return;
                for (int m = 0; m < M; m++) {
                    if (!wait_or_stop(&bar->p_full[m], np_[m] & 1, &bar->stop, p.status)) return;
                    np_[m]++;
                    tc_fence_after();
                    const uint64_t b0 = smem_desc(base + kOffV + vs * kTileBytes, 16384, 1024);
#pragma unroll
                    for (int k = 0; k < 8; k++)  // 16 tokens each
                        mma_ts(tm + 256 + m * 128, tm + m * 128 + 8 * k, b0 + ((k * 2048) >> 4), f16_idesc(128, 128, true), j > 0 || k > 0);
                    if (j + 1 < n) {
                        if (m == 0) {
                            if (!wait_or_stop(&bar->k_full[nk % kRing], (nk / kRing) & 1, &bar->stop, p.status)) return;
                            tc_fence_after();
                        }
                        scores(m, nk % kRing, s.k0 + j + 1 < s.np);
                    } else {
                        tc_commit(&bar->o_full[m]);
                    }
                }
                tc_commit(&bar->v_empty[vs]);
                nv++;
                if (j + 1 < n) {
                    tc_commit(&bar->k_empty[nk % kRing]);
                    nk++;
                    if (j + 2 == n) tc_commit(&bar->q_empty);
                }
            }
            at = s.first + s.k1;
        }
    };
    run();
    tc_commit(&bar->drain);  // every product has ended before the tensor memory is freed
    mbar_wait(&bar->drain, 0, p.status);
}

// ---------------------------------------------------------------- groups 0, 1 ---------
__device__ __forceinline__ void softmax(const ChunkAttnParams &p, Bars *bar, uint32_t tm, int m, int begin, int end) {
    const int lane = threadIdx.x & 31, row = 128 * m + (threadIdx.x & 127);
    const uint32_t lanes = (uint32_t)(threadIdx.x & 96) << 16;
    const uint32_t ts = tm + lanes + m * 128, to = tm + lanes + 256 + m * 128;
    uint32_t ns = 0, no = 0;
    int seg = 0;
    for (int at = begin; at < end; seg++) {
        const Seg s = next_seg(p, at, end);
        const bool last_first = s.k0 == 0 && at != begin;
        at = s.first + s.k1;
        if (128 * m >= s.valid) continue;
        const int r = s.it.t * kRows + min(row, s.valid - 1);
        const int lim = s.it.s.ns + s.it.s.nr + r / p.g + 1;  // fp16 tokens this row may see
        float mx = -INFINITY, l = 0.f;
        for (int kt = s.k0; kt < s.k1; kt++) {
            if (!warp_wait_or_stop(&bar->s_full[m], ns & 1, &bar->stop, p.status)) return;
            ns++;
            tc_fence_after();
            uint32_t x[128];
#pragma unroll
            for (int c = 0; c < 4; c++) tmem_ld32(x + 32 * c, ts + 32 * c);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 8; c++) tmem_tie16(x + 16 * c);
            float *f = reinterpret_cast<float *>(x);
            if (kt >= s.np) {
                const int y = lim - (kt - s.np) * kChunkKeys;
                if (y < kChunkKeys) {
#pragma unroll
                    for (int c = 0; c < 128; c++)
                        if (c >= y) f[c] = -INFINITY;
                }
            }
            float t0 = fmaxf(f[0], f[1]), t1 = fmaxf(f[2], f[3]), t2 = fmaxf(f[4], f[5]), t3 = fmaxf(f[6], f[7]);
#pragma unroll
            for (int c = 8; c < 128; c += 8) {
                t0 = fmaxf(t0, fmaxf(f[c], f[c + 1]));
                t1 = fmaxf(t1, fmaxf(f[c + 2], f[c + 3]));
                t2 = fmaxf(t2, fmaxf(f[c + 4], f[c + 5]));
                t3 = fmaxf(t3, fmaxf(f[c + 6], f[c + 7]));
            }
            const float cand = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * kScale;
            // S is complete, so the product before it, the last to write O, is too
            const bool grow = cand > mx + kLag || (mx == -INFINITY && cand > -INFINITY);
            if (__any_sync(0xffffffffu, grow)) {
                const float corr = grow ? ex2(mx - cand) : 1.f;
                if (grow) mx = cand;
                l *= corr;
                if (kt > s.k0) {
#pragma unroll 1
                    for (int c = 0; c < 8; c++) {
                        uint32_t o[16];
                        tmem_ld16(o, to + 16 * c);
                        tmem_wait_ld();
                        tmem_tie16(o);
#pragma unroll
                        for (int e = 0; e < 16; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                        tmem_st16(to + 16 * c, o);
                    }
                }
            }
            const float off = kUp - (mx == -INFINITY ? 0.f : mx);
            float l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int c = 0; c < 128; c += 2) {
                const float a = ex2(fmaf(f[c], kScale, off)), b = ex2(fmaf(f[c + 1], kScale, off));
                l0 += a;
                l1 += b;
                x[c >> 1] = pack_half2(a, b);
            }
            l += l0 + l1;
            tmem_st32(ts, x);
            tmem_st32(ts + 32, x + 32);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bar->p_full[m]);
        }
        if (!warp_wait_or_stop(&bar->o_full[m], no & 1, &bar->stop, p.status)) return;
        no++;
        tc_fence_after();
        const bool whole = s.k0 == 0 && s.k1 == s.it.n;
        const bool odd = *(volatile int *)&bar->odd[seg & 3] == seg + 1;
        const float inv = 1.f / l;
        // the range's first segment has slot 2 c, its last one (a unit that goes on) 2 c + 1
        const size_t slot = (2 * (size_t)blockIdx.x + (last_first ? 1 : 0)) * kRows + row;
        uint16_t *dst = p.out + ((int64_t)(s.it.s.cu + r / p.g) * p.H_kv * p.g + s.it.h * p.g + r % p.g) * kD;
        if (!whole && row < s.valid) p.part_ml[slot] = make_float2(mx, l);
#pragma unroll 1
        for (int c = 0; c < 8; c++) {
            uint32_t o[16];
            tmem_ld16(o, to + 16 * c);
            tmem_wait_ld();
            tmem_tie16(o);
            float *f = reinterpret_cast<float *>(o);
            if (odd)
                for (int x = max(0, s.k0 - s.np) * kChunkKeys; x < min(lim, (s.k1 - s.np) * kChunkKeys); x++) {
                    const uint16_t *v = tail_row(p, s.it, x, true) + 16 * c;
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        const float y = h2f(v[e]);
                        if (!isfinite(y)) f[e] += y;
                    }
                }
            if (row >= s.valid) continue;
            if (whole) {
                uint4 y[2];
                uint32_t *w = reinterpret_cast<uint32_t *>(y);
#pragma unroll
                for (int e = 0; e < 8; e++) w[e] = pack_half2(f[2 * e] * inv, f[2 * e + 1] * inv);
                reinterpret_cast<uint4 *>(dst)[2 * c] = y[0];
                reinterpret_cast<uint4 *>(dst)[2 * c + 1] = y[1];
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    reinterpret_cast<float4 *>(p.part_o + slot * kD)[4 * c + e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
            }
        }
        __syncwarp();
        tc_fence_before();
    }
    (void)lane;
}

__global__ void __launch_bounds__(kThreads, 1) chunk_wide_kernel(const __grid_constant__ ChunkAttnParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars *bar = reinterpret_cast<Bars *>(sm + kOffBar);
    const int w = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        mbar_init(&bar->q_full, 128);
        mbar_init(&bar->q_empty, 1);
        for (int i = 0; i < kRing; i++) {
            mbar_init(&bar->k_full[i], 128);
            mbar_init(&bar->k_empty[i], 1);
            mbar_init(&bar->v_full[i], 128);
            mbar_init(&bar->v_empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&bar->s_full[i], 1);
            mbar_init(&bar->p_full[i], 128);
            mbar_init(&bar->o_full[i], 1);
        }
        mbar_init(&bar->drain, 1);
        for (int i = 0; i < kMaxRaw; i++) {
            mbar_init(&bar->rawk[i], 1);
            mbar_init(&bar->rawv[i], 1);
            mbar_init(&bar->readk[i], 128);
            mbar_init(&bar->readv[i], 128);
        }
        bar->stop = 0;
        for (int i = 0; i < 4; i++) bar->odd[i] = 0;
        fence_barrier_init();
    }
    if (w == 12) tmem_alloc(&bar->tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar->tmem;
    const int begin = range_begin(blockIdx.x, p.n_items, p.C), end = range_begin(blockIdx.x + 1, p.n_items, p.C);
    if (w < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax(p, bar, tm, w >> 2, begin, end);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (w < 12) produce(p, sm, bar, begin, end);
        else if (threadIdx.x == 384) multiply(p, sm, bar, tm, begin, end);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 12) tmem_free(tm);
}

}  // namespace

cudaError_t launch_chunk_wide(const ChunkAttnParams &p, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(chunk_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    chunk_wide_kernel<<<p.C, kThreads, kSmemBytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace kvq
