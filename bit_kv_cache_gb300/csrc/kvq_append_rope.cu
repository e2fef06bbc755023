// kvq_append_rope.cu -- one token for every active slot of a paged cache, its query and key
// normalized and rotated on the way (kvq_paged_append_rope).
//
// One launch does what kvq_paged_flush, kvq_qk_norm_rope and kvq_paged_append do.  The CTAs of a
// page come first: each packs one side of a page of a full residual; the one that holds the
// residual's first row then writes the new token's row there, which no other CTA reads.  Behind
// them come the slots' own CTAs: 16 lanes hold a head's row, both channels of a
// pair in one thread, so that a row needs one reduction and no exchange; sines and cosines are
// formed once per CTA, while the rows arrive.  Positions and destinations come as a parameter, from
// the host's lengths: no CTA reads the lengths that another one advances.
// What bounds it.  Few slots: the host call (8 slots: 11.6 us through the binding, 5.3 of them in the
// C call; the kernel takes 4).  256 slots whose residuals are all full (208 MB): 43 us, 4.8 TB/s (in
// another loop 44, and 53 over min-max codes of 4 bits);
// the CTAs of the pages spend most of their time in the latency of their loads (kvq_block.cuh).
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "kvq.h"
#include "kvq_block.cuh"
#include "kvq_block.h"
#include "kvq_host.h"
#include "kvq_rope.h"

namespace kvq {

namespace {

constexpr int kMaxPages = 1024;          // packed by one launch
template <int FORM, int G>
constexpr int kThreads = FORM ? 4 * G : 256;  // a page's CTA; slots' rows by as many
constexpr int32_t kToSink = 1 << 30, kFull = 1 << 29, kNone = -1;

struct AppendRopeParams : PackParams {
    const uint16_t *q, *w_q, *w_k;       // k_new, v_new and their strides are PackParams'
    uint16_t *q_out;
    int32_t *table;
    int64_t q_stride;
    int H_q, rotary, halves, rotate;
    float eps, amp;
    int kbits, vbits;
    int b0, n_slots, parts;              // slots b0 .. of this launch, CTAs of each
    int n_pack, per, sides;              // pages to pack, of a slot, CTAs of each page and head
    int map;                             // whether pages[] goes into the page table (else the table has them)
    int32_t pos[KVQ_PAGED_MAX_B];        // of the new token
    int32_t dst[KVQ_PAGED_MAX_B];        // its row; kToSink: of the sink; kFull: a full residual, row 0; kNone: no sequence
    int32_t lp0[KVQ_PAGED_MAX_B];        // full slots, by their order: first logical page,
    int16_t seq[KVQ_PAGED_MAX_B];        // slot
    int32_t pages[kMaxPages];
    uint64_t turn[64];
};

// Cosine and sine of every pair at a position, times amp.
__device__ __forceinline__ void angles(const AppendRopeParams &p, int64_t pos, float2 *cs) {
    for (int j = threadIdx.x; j < p.rotary >> 1; j += blockDim.x) {
        const uint64_t a = (uint64_t)pos * p.turn[j];
        float s, c;
        sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &s, &c);
        cs[j] = make_float2(p.amp * c, p.amp * s);
    }
}

// One head's row by 16 lanes (all lanes of the warp call): norm, if there are weights w, and
// rotation, if turn; the arithmetic of kvq_qk_norm_rope, bit for bit.  Lane l has two pieces of
// four channels: of halves a piece of the first half and its partners, else neighbours.
struct HeadRow {
    uint2 v[2], w[2];
    int c0, c1;
    bool split;
    __device__ __forceinline__ HeadRow(const AppendRopeParams &p, const uint16_t *src, const uint16_t *wt) {
        const int l = threadIdx.x & 15, half = p.rotary >> 1;
        split = p.halves && 4 * l < half;
        c0 = split ? 4 * l : 8 * l, c1 = split ? c0 + half : c0 + 4;
        v[0] = v[1] = make_uint2(0, 0);
        w[0] = w[1] = make_uint2(0x3c003c00u, 0x3c003c00u);
        if (src) {
            v[0] = *reinterpret_cast<const uint2 *>(src + c0);
            v[1] = *reinterpret_cast<const uint2 *>(src + c1);
        }
        if (wt) {
            w[0] = __ldg(reinterpret_cast<const uint2 *>(wt + c0));
            w[1] = __ldg(reinterpret_cast<const uint2 *>(wt + c1));
        }
    }
    __device__ __forceinline__ void store(const AppendRopeParams &p, bool norm, bool rotate, uint16_t *dst, const float2 *cs) const {
        auto pairs = [&](const uint2 (&r)[2], float (&x)[4], float (&y)[4]) {
            const float2 f0 = unpack_half2(r[0].x), f1 = unpack_half2(r[0].y), f2 = unpack_half2(r[1].x), f3 = unpack_half2(r[1].y);
            if (p.halves) {
                x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y;
                y[0] = f2.x, y[1] = f2.y, y[2] = f3.x, y[3] = f3.y;
            } else {
                x[0] = f0.x, x[1] = f1.x, x[2] = f2.x, x[3] = f3.x;
                y[0] = f0.y, y[1] = f1.y, y[2] = f2.y, y[3] = f3.y;
            }
        };
        float x[4], y[4], w0[4], w1[4];
        pairs(v, x, y);
        pairs(w, w0, w1);
        const float a = fmaf(x[0], x[0], fmaf(x[2], x[2], fmaf(y[0], y[0], y[2] * y[2])));
        const float b = fmaf(x[1], x[1], fmaf(x[3], x[3], fmaf(y[1], y[1], y[3] * y[3])));
        float ss = a + b;
#pragma unroll
        for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float f = norm ? rsqrtf(ss * (1.0f / 128) + p.eps) : 1.f;
        const bool turn = rotate && (p.halves ? split : c0 < p.rotary);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float2 c = turn ? cs[(p.halves ? c0 : c0 >> 1) + e] : make_float2(1.f, 0.f);
            const float xx = w0[e] * c.x, xy = -w1[e] * c.y, yx = w0[e] * c.y, yy = w1[e] * c.x;
            const float x0 = turn ? fmaf(x[e], xx, __fmul_rn(y[e], xy)) : __fmul_rn(x[e], xx);
            const float y0 = turn ? fmaf(x[e], yx, __fmul_rn(y[e], yy)) : __fmul_rn(y[e], yy);
            x[e] = __fmul_rn(f, x0);
            y[e] = __fmul_rn(f, y0);
        }
        if (!dst) return;
        if (p.halves) {
            *reinterpret_cast<uint2 *>(dst + c0) = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
            *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
        } else {
            *reinterpret_cast<uint2 *>(dst + c0) = make_uint2(pack_half2(x[0], y[0]), pack_half2(x[1], y[1]));
            *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(pack_half2(x[2], y[2]), pack_half2(x[3], y[3]));
        }
    }
};

__device__ __forceinline__ void copy_row(const uint16_t *src, uint16_t *dst) {
    reinterpret_cast<uint4 *>(dst)[threadIdx.x & 15] = reinterpret_cast<const uint4 *>(src)[threadIdx.x & 15];
}

// Part `part` of a slot's heads, queries, keys, values, by 16 threads each.
__device__ __forceinline__ void slot_rows(const AppendRopeParams &p, int b, int part, float2 *cs) {
    const int dst = p.dst[b], row = dst & (kFull - 1), heads = p.H_q + 2 * p.H_kv;
    const int i = part * (blockDim.x >> 4) + (threadIdx.x >> 4), kind = i < p.H_q ? 0 : i < p.H_q + p.H_kv ? 1 : 2, h = kind ? i - p.H_q - (kind - 1) * p.H_kv : i;
    const uint16_t *src = nullptr;
    uint16_t *to = nullptr;
    if (kind == 0) {
        src = p.q + b * p.q_stride + h * 128;
        to = p.q_out + ((int64_t)b * p.H_q + h) * 128;
    } else if (i < heads && !(dst & kFull)) {
        const size_t u = (size_t)b * p.H_kv + h;
        src = kind == 1 ? p.k_new + b * p.k_stride + h * 128 : p.v_new + b * p.v_stride + h * 128;
        to = dst & kToSink ? (kind == 1 ? p.k_sink : p.v_sink) + (u * p.S + row) * 128 : (kind == 1 ? p.k_res : p.v_res) + (u * p.R + row) * 128;
    }
    const uint16_t *w = kind == 0 ? p.w_q : kind == 1 ? p.w_k : nullptr;
    const HeadRow r(p, src, w);
    angles(p, p.pos[b], cs);  // while the rows arrive
    __syncthreads();
    r.store(p, w, kind == 0 ? p.rotate & 1 : kind == 1 ? p.rotate & 2 : 0, to, cs);
    if (part == 0 && threadIdx.x == 0) {
        int32_t *l = p.lens + 4 * b;
        if (dst & kToSink) {
            l[0]++;
        } else if (dst & kFull) {
            l[1] += p.R;
            l[2] = 1;
        } else {
            l[2]++;
        }
    }
}

// FORM: 0 min-max codes, 1 e4m3, 2 int8; G tokens a page.
template <int FORM, int G>
__global__ void __launch_bounds__(kThreads<FORM, G>, FORM == 0 ? (G == 256 ? 2 : 4) : kPackCtas<G>) append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    __shared__ __align__(16) unsigned char smem[FORM ? 16 : 32 * 512 + 512];
    __shared__ float2 s_cs[64];
    griddep_wait();
    int i = blockIdx.x;
    const int n_page = p.n_pack * p.H_kv * p.sides;
    if (i >= n_page) {
        i -= n_page;
        const int b = p.b0 + i / p.parts;
        if (p.dst[b] == kNone) return;
        slot_rows(p, b, i % p.parts, s_cs);
        return;
    }
    const int side = p.sides - 1 - i / (p.n_pack * p.H_kv), j = i % (p.n_pack * p.H_kv) / p.H_kv, h = i % p.H_kv;
    const int k = j / p.per, b = p.seq[k], page = j - k * p.per;
    int32_t *at = p.table + (size_t)b * p.ptab_stride + p.lp0[k] + page;
    PageJob jb;
    jb.s = {0, 0, p.R, 0, 0, 0, 0, 0};
    jb.b = b;
    jb.t0 = page * G;
    jb.entry = p.map ? p.pages[j] : *at;
    if (p.map && h == 0 && side == 0 && threadIdx.x == 0) *at = jb.entry;
    const bool first = page == 0 && side < 2;  // this CTA reads row 0 of the residual
    if (first && side == 0) angles(p, p.pos[b], s_cs);  // (a barrier inside the packing)
    if (FORM == 0) {
        if (side == 0) {
            if (p.kbits == 2) extend_keys<2, G / 8>(p, jb, h, smem);
            else if (p.kbits == 4) extend_keys<4, G / 8>(p, jb, h, smem);
            else extend_keys<8, G / 8>(p, jb, h, smem);
        } else {
            if (p.vbits == 2) extend_values<2>(p, jb, h, side - 1, smem);
            else if (p.vbits == 4) extend_values<4>(p, jb, h, side - 1, smem);
            else extend_values<8>(p, jb, h, side - 1, smem);
        }
    } else {
        const uint16_t *src = (side ? p.v_res : p.k_res) + (((size_t)b * p.H_kv + h) * p.R + jb.t0) * 128;
        pack_block<FORM == 1, G>(nullptr, 0, src, 128, [&] { return jb.page(p, h); }, side, reinterpret_cast<uint8_t *>(side ? p.v_codes : p.k_codes),
                                 reinterpret_cast<float4 *>(side ? p.v_meta : p.k_meta));
    }
    if (!first || threadIdx.x >= 32) return;
    const size_t u = (size_t)b * p.H_kv + h;
    if (side == 0)
        HeadRow(p, p.k_new + b * p.k_stride + h * 128, p.w_k).store(p, p.w_k, p.rotate & 2, threadIdx.x < 16 ? p.k_res + u * p.R * 128 : nullptr, s_cs);
    else if (threadIdx.x < 16)
        copy_row(p.v_new + b * p.v_stride + h * 128, p.v_res + u * p.R * 128);
}

cudaError_t launch_append_rope(AppendRopeParams &p, int form, cudaStream_t st) {
    using std::integral_constant;
    auto go = [&](auto f, auto g) {
        constexpr int F = decltype(f)::value, G = decltype(g)::value, T = kThreads<F, G>;
        p.parts = (16 * (p.H_q + 2 * p.H_kv) + T - 1) / T;
        const dim3 grid((unsigned)((int64_t)p.n_pack * p.H_kv * p.sides + (int64_t)p.n_slots * p.parts));
        return launch_dependent(append_rope_kernel<F, G>, grid, T, 0, st, p);
    };
    auto pages = [&](auto f) {
        return p.G == 64 ? go(f, integral_constant<int, 64>()) : p.G == 128 ? go(f, integral_constant<int, 128>()) : go(f, integral_constant<int, 256>());
    };
    if (form) return form == 1 ? pages(integral_constant<int, 1>()) : pages(integral_constant<int, 2>());
    const integral_constant<int, 0> f;
    return p.G == 128 ? go(f, integral_constant<int, 128>()) : go(f, integral_constant<int, 256>());
}

}  // namespace

}  // namespace kvq

using namespace kvq;
using namespace kvq::host;

extern "C" int kvq_paged_append_rope(const kvq_config *c, kvq_paged *pc, const kvq_qk_config *qk, const double *freq, float amp,
                                     const uint16_t *q, const uint16_t *k, const uint16_t *v, int64_t v_stride, const uint16_t *w_q,
                                     const uint16_t *w_k, uint16_t *q_out, const int32_t *new_pages, int64_t n_new_pages,
                                     void *stream) {
    int e = check_paged(c, pc);
    if (e) return e;
    if (!qk || qk->H_q != c->H_q || qk->H_kv != c->H_kv || qk->D != c->D || n_new_pages < 0 || (!new_pages && n_new_pages))
        return KVQ_ERR_INVALID_ARG;
    if ((e = rope_check(qk, freq, amp))) return e;
    const int B = c->B, per = c->R / c->G;
    int full = 0, active = 0;
    for (int b = 0; b < B; b++) {
        const int32_t *l = pc->lens_host + 4 * b;
        if (!l[3]) continue;
        active++;
        if ((int64_t)l[0] + l[1] + l[2] >= INT32_MAX) return KVQ_ERR_CAPACITY;
        if (l[0] < c->S || l[2] < c->R) continue;
        if ((int64_t)l[1] + c->R > c->max_T) return KVQ_ERR_CAPACITY;
        full++;
    }
    if (full && (pc->n_pages < 1 || (new_pages && n_new_pages < (int64_t)full * per))) return KVQ_ERR_CAPACITY;
    for (int64_t i = 0; new_pages && i < (int64_t)full * per; i++)
        if (new_pages[i] < 0 || new_pages[i] >= pc->n_pages) return KVQ_ERR_INVALID_ARG;
    if (!rows_ok(q, qk->q_stride, c->H_q, c->D) || !rows_ok(k, qk->k_stride, c->H_kv, c->D) || !rows_ok(v, v_stride, c->H_kv, c->D) ||
        !q_out || !aligned16(q_out) || (w_q && !aligned16(w_q)) || (w_k && !aligned16(w_k)))
        return KVQ_ERR_INVALID_ARG;
    auto span = [&](int64_t stride, int64_t heads) { return ((size_t)(B - 1) * stride + heads * c->D) * 2; };
    const size_t no = (size_t)B * c->H_q * c->D * 2;
    const bool own = q_out == q && (qk->q_stride == (int64_t)c->H_q * c->D || B == 1);
    if ((!own && overlap(q_out, no, q, span(qk->q_stride, c->H_q))) || overlap(q_out, no, k, span(qk->k_stride, c->H_kv)) ||
        overlap(q_out, no, v, span(v_stride, c->H_kv)) || (w_q && overlap(q_out, no, w_q, c->D * 2)) || (w_k && overlap(q_out, no, w_k, c->D * 2)))
        return KVQ_ERR_INVALID_ARG;
    if (full && per > kMaxPages) return KVQ_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    if (capturing(st)) return KVQ_ERR_UNSUPPORTED;
    if (!active) return KVQ_OK;
    AppendRopeParams p;
    memset(static_cast<PackParams *>(&p), 0, sizeof(PackParams));
    p.lens = pc->lens;
    p.status = pc->status;
    p.k_new = k;
    p.v_new = v;
    p.k_stride = qk->k_stride;
    p.v_stride = v_stride;
    p.k_sink = pc->k_sink;
    p.v_sink = pc->v_sink;
    p.k_res = pc->k_res;
    p.v_res = pc->v_res;
    p.k_codes = pc->k_codes;
    p.v_codes = pc->v_codes;
    p.k_meta = pc->k_meta;
    p.v_meta = pc->v_meta;
    p.ptab = pc->page_table;
    p.n_pages = pc->n_pages;
    p.B = B;
    p.H_kv = c->H_kv;
    p.G = c->G;
    p.S = c->S;
    p.R = c->R;
    p.TV = block8(c) ? 0 : vtile_of(c);
    p.ptab_stride = (int)(c->max_T / c->G);
    p.q = q;
    p.w_q = w_q;
    p.w_k = w_k;
    p.q_out = q_out;
    p.table = const_cast<int32_t *>(pc->page_table);
    p.q_stride = qk->q_stride;
    p.H_q = c->H_q;
    p.rotary = qk->rotary_dim;
    p.halves = qk->halves;
    p.rotate = qk->rotary_dim ? qk->rotate : 0;
    p.eps = qk->eps;
    p.amp = amp;
    p.kbits = c->bits;
    p.vbits = vbits_of(c);
    p.per = per;
    p.sides = block8(c) ? 2 : 1 + c->G / 128;
    p.map = new_pages != nullptr;
    if (qk->rotary_dim && freq) turns_of_freq(freq, qk->rotary_dim, p.turn);
    else if (qk->rotary_dim) turns_of_base(qk->rope_base, qk->rotary_dim, p.turn);
    const int form = c->mode == KVQ_MODE_E4M3 ? 1 : c->mode == KVQ_MODE_INT8 ? 2 : 0;
    // a launch packs kMaxPages pages at most: one launch, but for hundreds of full residuals of several pages
    for (int b0 = 0; b0 < B;) {
        int b = b0, n = 0;
        p.n_pack = 0;
        for (; b < B; b++) {
            const int32_t *l = pc->lens_host + 4 * b;
            p.pos[b] = l[0] + l[1] + l[2];
            if (!l[3]) {
                p.dst[b] = kNone;
            } else if (l[0] < c->S) {
                p.dst[b] = l[0] | kToSink;
            } else if (l[2] < c->R) {
                p.dst[b] = l[2];
            } else {
                if (p.n_pack + per > kMaxPages) break;
                p.dst[b] = kFull;
                p.seq[n] = (int16_t)b;
                p.lp0[n++] = l[1] / c->G;
                for (int i = 0; p.map && i < per; i++) p.pages[p.n_pack + i] = *new_pages++;
                p.n_pack += per;
            }
        }
        p.b0 = b0;
        p.n_slots = b - b0;
        if (launch_append_rope(p, form, st) != cudaSuccess) return KVQ_ERR_CUDA;
        for (; b0 < b; b0++) {
            int32_t *l = pc->lens_host + 4 * b0;
            if (!l[3]) continue;
            if (l[0] < c->S) {
                l[0]++;
            } else if (l[2] < c->R) {
                l[2]++;
            } else {
                l[1] += c->R;
                l[2] = 1;
            }
        }
    }
    return KVQ_OK;
}
