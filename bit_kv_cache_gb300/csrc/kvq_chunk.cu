// kvq_chunk.cu -- chunks of new tokens over the paged cache: the C ABI of
// kvq_paged_plan, kvq_paged_chunk_attn, kvq_paged_extend and kvq_qk_norm_rope, and the
// kernels of all but the attention (kvq_chunk_attn.cu).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kvq.h"
#include "kvq_block.h"
#include "kvq_chunk.h"
#include "kvq_extend.cuh"
#include "kvq_host.h"
#include "kvq_rope.h"

using namespace kvq;
using namespace kvq::host;

namespace kvq {

// ------------------------------------------------------------------------------
// Plan.  Every CTA scans the slots (one thread each: rows and pages before the slot) and
// writes its share of the rows and page-table entries; CTA 0 also the per-slot arrays.  The
// scan is repeated rather than shared, so that one launch does all: at most 512 slots, 8 KB.
// Bound by latency: one read of the lengths, two scans over a block, a binary search.
// ------------------------------------------------------------------------------
constexpr int kPlanThreads = 512;
static_assert(kPlanThreads >= KVQ_PAGED_MAX_B, "one thread per slot");

// The slot holding index i: the first one whose end (exclusive prefix of the next) is above i.
__device__ __forceinline__ int find_slot(const int *start, int B, int i) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (start[mid + 1] > i) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ int s_row[kPlanThreads + 1], s_page[kPlanThreads + 1], s_pos[kPlanThreads], s_lp[kPlanThreads];
    __shared__ int2 s_warp[kPlanThreads / 32];
    const int b = threadIdx.x, lane = b & 31, w = b >> 5;
    griddep_wait();
    int4 ln = make_int4(0, 0, 0, 0);
    int n = 0, to_sink = 0, pk = 0;
    if (b < p.B) {
        ln = reinterpret_cast<const int4 *>(p.lens)[b];
        if (!ln.w) ln = make_int4(0, 0, 0, 0);
        n = p.n_new[b];
        to_sink = min(n, p.S - ln.x);
        pk = n ? (ln.z + n - to_sink) / p.R * p.R : 0;
    }
    // inclusive scans of (rows, pages) over the warp, then over the warps
    int r = n, g = pk / p.G;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, r, o), c = __shfl_up_sync(0xffffffffu, g, o);
        if (lane >= o) {
            r += a;
            g += c;
        }
    }
    if (lane == 31) s_warp[w] = make_int2(r, g);
    __syncthreads();
    for (int i = 0; i < w; i++) {
        r += s_warp[i].x;
        g += s_warp[i].y;
    }
    s_row[b + 1] = r;
    s_page[b + 1] = g;
    s_pos[b] = ln.x + ln.y + ln.z;
    s_lp[b] = ln.y / p.G;
    if (b == 0) s_row[0] = s_page[0] = 0;
    __syncthreads();
    if (blockIdx.x == 0 && b < p.B) {
        p.cu[b] = r - n;
        if (b == p.B - 1) p.cu[p.B] = r;
        int4 *d = reinterpret_cast<int4 *>(p.desc) + 2 * b;
        d[0] = make_int4(ln.x, ln.y, ln.z, n);
        d[1] = make_int4(r - n, to_sink, pk, s_page[b]);
    }
    const int stride = gridDim.x * kPlanThreads, t0 = blockIdx.x * kPlanThreads + threadIdx.x;
    // four rows per thread; a group of four that stays in one slot (most do) costs one search
    for (int64_t i = 4 * (int64_t)t0; i < p.n_tokens; i += 4 * (int64_t)stride) {
        int sl = find_slot(s_row, p.B, (int)i);
        int s4[4], q4[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int x = (int)i + k;
            while (sl < p.B - 1 && s_row[sl + 1] <= x) sl++;
            s4[k] = sl;
            q4[k] = s_pos[sl] + x - s_row[sl];
        }
        if (i + 4 <= p.n_tokens) {
            *reinterpret_cast<int4 *>(p.slot + i) = make_int4(s4[0], s4[1], s4[2], s4[3]);
            *reinterpret_cast<int4 *>(p.pos + i) = make_int4(q4[0], q4[1], q4[2], q4[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (i + k < p.n_tokens) {
                    p.slot[i + k] = s4[k];
                    p.pos[i + k] = q4[k];
                }
        }
    }
    if (!p.new_pages) return;
    const int pages = s_page[p.B];
    for (int i = t0; i < pages; i += stride) {
        const int sl = find_slot(s_page, p.B, i);
        p.table[(size_t)sl * p.table_stride + s_lp[sl] + i - s_page[sl]] = p.new_pages[i];
    }
}

cudaError_t launch_plan(const PlanParams &p, cudaStream_t st) {
    const int64_t per = 4 * kPlanThreads;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(64, (p.n_tokens + per - 1) / per));
    return launch_dependent(plan_kernel, dim3((unsigned)grid), kPlanThreads, 0, st, p);
}

// ------------------------------------------------------------------------------
// Extend.  The tokens that a slot packs are the stream [residual | chunk behind the sink];
// page j of the call holds its tokens j G .. j G + G - 1.  One CTA per (page, head, keys or
// 128 value tokens) gathers its rows from the two places and quantizes them as the prefill
// kernels do (kvq_quantizer.cuh), so codes and scales are theirs bit for bit.  Few pages are
// bound by their dependent reads (plan, rows; a page-table entry only at the end): 13 us for
// a chunk of 2048 tokens of 8 heads.  Many: four prompts of 2K to 12K tokens, 237 MB in two
// calls, take 69 us (3.4 TB/s) with nothing saturated (issue 0.60 a cycle, ALU 0.46): four CTAs
// per SM at 64 registers, and in each the chain of search, plan row and table entry before its
// loads; the prefill quantizers, with the same arithmetic and without that chain, reach 4.5
// TB/s.  The slots of the pages come as a parameter (found from the plan's arrays: 70 us).
// ------------------------------------------------------------------------------
// Page blockIdx.x of the call (G = 8 TPW tokens), or, behind them, a slot's fp16 rows.  The
// values, whose CTAs take longer, come first (four prompts of 2K to 12K tokens: 70 us against 71).
template <int TPW>
__global__ void __launch_bounds__(256, TPW == 16 ? 4 : 2) extend_pack_kernel(const __grid_constant__ ExtendParams p, int kbits, int vbits) {
    __shared__ __align__(16) unsigned char smem[32 * 512 + 512];
    __shared__ int s_first;  // the slot, if this is its first page
    const int h = blockIdx.y, side = gridDim.z - 1 - blockIdx.z;  // 0: keys, 1 + i: values 128 i ..
    griddep_wait();
    if (blockIdx.x >= p.n_pack) {
        extend_slot(p, blockIdx.x - p.n_pack, h, side, 0, 1);
        return;
    }
    const PageJob jb = find_page(p, blockIdx.x);
    if (threadIdx.x == 0) s_first = jb.t0 == 0 ? jb.b : -1;
    if (side == 0) {
        if (kbits == 2) extend_keys<2, TPW>(p, jb, h, smem);
        else if (kbits == 4) extend_keys<4, TPW>(p, jb, h, smem);
        else extend_keys<8, TPW>(p, jb, h, smem);
    } else {
        const int vb = side - 1;
        if (vbits == 2) extend_values<2>(p, jb, h, vb, smem);
        else if (vbits == 4) extend_values<4>(p, jb, h, vb, smem);
        else extend_values<8>(p, jb, h, vb, smem);
    }
    if (TPW == 16 && p.once && s_first >= 0) {  // every thread has read its rows (a barrier inside the packing)
        const int4 *d = reinterpret_cast<const int4 *>(p.desc) + 2 * s_first;
        keep_rows(p, d[0], d[1], s_first, h, side, false, true, threadIdx.x, 256);
    }
}

// Every slot's fp16 rows: after the pages, which read the old residual rows.
constexpr int kTailSlices = 4;
__global__ void __launch_bounds__(256) extend_tail_kernel(const __grid_constant__ ExtendParams p) {
    griddep_wait();
    extend_slot(p, blockIdx.x, blockIdx.y >> 1, blockIdx.y & 1, blockIdx.z, kTailSlices);
}

cudaError_t launch_extend(const ExtendParams &p, int kbits, int vbits, cudaStream_t st) {
    const bool once = p.once && p.n_pack > 0;
    if (p.n_pack > 0) {
        const dim3 grid((unsigned)(p.n_pack + (once ? p.B : 0)), (unsigned)p.H_kv, (unsigned)(1 + p.G / 128));
        cudaError_t e = cudaErrorInvalidValue;
        if (p.G == 128) e = launch_dependent(extend_pack_kernel<16>, grid, 256, 0, st, p, kbits, vbits);
        else if (p.G == 256) e = launch_dependent(extend_pack_kernel<32>, grid, 256, 0, st, p, kbits, vbits);
        if (e != cudaSuccess || once) return e;
    }
    return launch_extend_tail(p, st);
}
cudaError_t launch_extend_tail(const ExtendParams &p, cudaStream_t st) {
    return launch_dependent(extend_tail_kernel, dim3((unsigned)p.B, (unsigned)(2 * p.H_kv), kTailSlices), 256, 0, st, p);
}

// ------------------------------------------------------------------------------
// Norm and rotation of new queries and keys.  D / 8 lanes hold a head's row, four channel
// pairs each (both channels of a pair in one thread), a warp a token's heads or a part of
// them; a thread's channels are the same in all its rows, so that their weights, sines and
// cosines are formed once.  An angle pos * base^(-2j/n) is reduced in 64-bit fixed point:
// pos * turn[j] mod 2^64 is the fraction of a turn, exact but for turn[j]'s error of some
// tens of 2^-64 (times pos: below 2^-27), and its upper 32 bits go to sincospif.  8191 tokens of 32 + 8 heads of 128 channels, 168 MB, take 30 us (5.6 TB/s);
// bound by instructions before: 63 us with a CTA per token, a row per warp and a shuffle per
// channel, 45 us with both channels of a pair in one thread and fp32 pairs, 41 us with the
// weights folded into sine and cosine, 30 us with a warp per token, which forms them once
// for 20 passes of rows.
// ------------------------------------------------------------------------------
constexpr int kQkRows = 4;  // rows of a thread in flight

// ALL: every channel of every row rotates (8191 tokens as above: 34.0 us a call; choosing per
// channel 34.5).
template <int D, bool HALVES, bool ALL>
__global__ void __launch_bounds__(256) qk_kernel(const __grid_constant__ QkParams p, int heads, int parts) {
    constexpr int L = D / 8, PER = 32 / L;  // lanes per row, rows per pass of the warp
    __shared__ float2 s_all[8][D / 2];
    const int lane = threadIdx.x & 31, l = lane % L, half = p.rotary >> 1;
    float2 *s_cs = s_all[threadIdx.x >> 5];
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), i = item / parts;
    if (i >= p.n) return;
    // the warp's heads (queries, then keys) and the thread's first
    const int h0 = (int)(item - i * parts) * heads, h1 = min(p.H_q + p.H_kv, h0 + heads), first = h0 + lane / L;
    // the thread's channels: two pieces of four.  Halves: a piece of the first half and its
    // partners; interleaved, and behind the rotary channels: neighbours
    const bool split = HALVES && 4 * l < half;
    const int c0 = split ? 4 * l : HALVES ? p.rotary + 2 * (4 * l - half) : 8 * l, c1 = split ? c0 + half : c0 + 4;
    griddep_wait();
    uint2 v[kQkRows][2];
    auto load = [&](uint2 (&r)[2], int h) {
        const uint16_t *src = h >= p.H_q ? p.k + i * p.k_stride + (h - p.H_q) * D : p.q + i * p.q_stride + h * D;
        r[0] = __ldcs(reinterpret_cast<const uint2 *>(src + c0));
        r[1] = __ldcs(reinterpret_cast<const uint2 *>(src + c1));
    };
#pragma unroll
    for (int r = 0; r < kQkRows; r++)
        if (first + r * PER < h1) load(v[r], first + r * PER);
    const int64_t pos = p.pos[i];
    for (int j = lane; j < half; j += 32) {
        const uint64_t a = (uint64_t)pos * p.turn[j];
        float s, c;
        sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &s, &c);
        s_cs[j] = make_float2(p.amp * c, p.amp * s);
    }
    __syncwarp();
    // first and second channels of the four pairs of eight halves
    auto pairs = [&](const uint2 (&r)[2], float (&x)[4], float (&y)[4]) {
        const float2 f0 = unpack_half2(r[0].x), f1 = unpack_half2(r[0].y), f2 = unpack_half2(r[1].x), f3 = unpack_half2(r[1].y);
        if (HALVES) {
            x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y;
            y[0] = f2.x, y[1] = f2.y, y[2] = f3.x, y[3] = f3.y;
        } else {
            x[0] = f0.x, x[1] = f1.x, x[2] = f2.x, x[3] = f3.x;
            y[0] = f0.y, y[1] = f1.y, y[2] = f2.y, y[3] = f3.y;
        }
    };
    // (x, y) -> f (x xx + y xy, x yx + y yy), f the norm's factor: the weights are folded into
    // sine and cosine.  Channels that do not rotate take no part of their neighbours, which may
    // be infinite or NaN
    uint64_t xx[2], xy[2], yx[2], yy[2];
    int side = -1;
    bool turn = false;
    for (int h = first; __any_sync(0xffffffffu, h < h1); h += kQkRows * PER) {
#pragma unroll
        for (int r = 0; r < kQkRows; r++) {
            const int hh = h + r * PER, key = hh >= p.H_q;
            if (!__any_sync(0xffffffffu, hh < h1)) break;
            const uint16_t *wt = key ? p.w_k : p.w_q;
            if (key != side) {  // once for the queries, once for the keys
                side = key;
                float w0[4] = {1.f, 1.f, 1.f, 1.f}, w1[4] = {1.f, 1.f, 1.f, 1.f};
                if (wt) {
                    const uint2 u[2] = {__ldg(reinterpret_cast<const uint2 *>(wt + c0)), __ldg(reinterpret_cast<const uint2 *>(wt + c1))};
                    pairs(u, w0, w1);
                }
                turn = (HALVES ? split : c0 < p.rotary) && (p.rotate & (key ? 2 : 1));
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int j = (HALVES ? c0 : c0 >> 1) + 2 * e;
                    const float2 c = turn ? s_cs[j] : make_float2(1.f, 0.f), d = turn ? s_cs[j + 1] : make_float2(1.f, 0.f);
                    xx[e] = pk2(w0[2 * e] * c.x, w0[2 * e + 1] * d.x);
                    xy[e] = pk2(-w1[2 * e] * c.y, -w1[2 * e + 1] * d.y);
                    yx[e] = pk2(w0[2 * e] * c.y, w0[2 * e + 1] * d.y);
                    yy[e] = pk2(w1[2 * e] * c.x, w1[2 * e + 1] * d.x);
                }
            }
            float x[4], y[4];
            pairs(v[r], x, y);
            const uint64_t X[2] = {pk2(x[0], x[1]), pk2(x[2], x[3])}, Y[2] = {pk2(y[0], y[1]), pk2(y[2], y[3])};
            const float2 sq = up2(fma_x2(X[0], X[0], fma_x2(X[1], X[1], fma_x2(Y[0], Y[0], mul_x2(Y[1], Y[1])))));
            float ss = sq.x + sq.y;
#pragma unroll
            for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float f = wt ? rsqrtf(ss * (1.0f / D) + p.eps) : 1.f;
            const uint64_t f2 = pk2(f, f);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const uint64_t x0 = ALL || turn ? fma_x2(X[e], xx[e], mul_x2(Y[e], xy[e])) : mul_x2(X[e], xx[e]);
                const uint64_t y0 = ALL || turn ? fma_x2(X[e], yx[e], mul_x2(Y[e], yy[e])) : mul_x2(Y[e], yy[e]);
                const float2 a = up2(mul_x2(f2, x0)), b = up2(mul_x2(f2, y0));
                x[2 * e] = a.x, x[2 * e + 1] = a.y, y[2 * e] = b.x, y[2 * e + 1] = b.y;
            }
            if (hh < h1) {
                uint16_t *dst = key ? p.k_out + (i * p.H_kv + hh - p.H_q) * D : p.q_out + (i * p.H_q + hh) * D;
                uint2 o[2];
                if (HALVES) {
                    o[0] = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
                    o[1] = make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
                } else {
                    o[0] = make_uint2(pack_half2(x[0], y[0]), pack_half2(x[1], y[1]));
                    o[1] = make_uint2(pack_half2(x[2], y[2]), pack_half2(x[3], y[3]));
                }
                *reinterpret_cast<uint2 *>(dst + c0) = o[0];
                *reinterpret_cast<uint2 *>(dst + c1) = o[1];
            }
            if (hh + kQkRows * PER < h1) load(v[r], hh + kQkRows * PER);
        }
    }
}

cudaError_t launch_qk(const QkParams &p, int D, cudaStream_t st) {
    const int H = p.H_q + p.H_kv, pass = 32 / (D / 8);
    // a warp per token; of few tokens the heads go to several warps, one pass of rows at least each
    int parts = 1;
    while (p.n * parts < 16 * num_sms() && (H + parts - 1) / parts > pass) parts++;
    const int heads = (H + parts - 1) / parts;
    parts = (H + heads - 1) / heads;
    const dim3 grid((unsigned)((p.n * parts + 7) / 8));
    auto go = [&](auto kernel) { return launch_dependent(kernel, grid, 256, 0, st, p, heads, parts); };
    auto form = [&](auto halves, auto all) {
        constexpr bool H2 = decltype(halves)::value, A = decltype(all)::value;
        return D == 64 ? go(qk_kernel<64, H2, A>) : D == 128 ? go(qk_kernel<128, H2, A>) : go(qk_kernel<256, H2, A>);
    };
    const std::true_type yes;
    const std::false_type no;
    if (p.rotary == D && p.rotate == 3) return p.halves ? form(yes, yes) : form(no, yes);
    return p.halves ? form(yes, no) : form(no, no);
}

}  // namespace kvq

// ------------------------------------------------------------------------------
// C ABI
// ------------------------------------------------------------------------------
namespace {

int check_chunk(const kvq_chunk *ch) {
    if (!ch || !ch->host || ch->max_tokens < 0) return KVQ_ERR_INVALID_ARG;
    const void *need[] = {ch->cu, ch->slot, ch->pos, ch->desc};
    for (const void *p : need)
        if (!p || !aligned16(p)) return KVQ_ERR_INVALID_ARG;
    return KVQ_OK;
}

ChunkSlot *slots_of(const kvq_chunk *ch) { return reinterpret_cast<ChunkSlot *>(ch->host); }

// Whether the cache's host lengths are those that the plan was made for.
bool plan_holds(const kvq_config *c, const kvq_paged *pc, const kvq_chunk *ch) {
    const ChunkSlot *s = slots_of(ch);
    int64_t rows = 0;
    for (int b = 0; b < c->B; b++) {
        const int32_t *l = pc->lens_host + 4 * b;
        const bool on = l[3] != 0;
        if (s[b].ns != (on ? l[0] : 0) || s[b].T != (on ? l[1] : 0) || s[b].nr != (on ? l[2] : 0)) return false;
        if (s[b].n_new < 0 || s[b].cu != rows) return false;
        // what the plan derived, for this configuration
        const int to_sink = std::min(s[b].n_new, c->S - s[b].ns);
        const int64_t pk = s[b].n_new ? ((int64_t)s[b].nr + s[b].n_new - to_sink) / c->R * c->R : 0;
        if (s[b].to_sink != to_sink || s[b].pk != pk || s[b].T + pk > c->max_T) return false;
        rows += s[b].n_new;
    }
    return rows == ch->n_tokens;
}

// Partials of the attention: two segments' ends per CTA.
struct ChunkWs {
    size_t ml, o, total;
};
ChunkWs chunk_ws() {
    ChunkWs w;
    const size_t slots = (size_t)2 * std::min(num_sms(), kMaxRanges) * kWideRows;  // rows
    w.ml = 0;
    w.o = (slots * sizeof(float2) + 255) / 256 * 256;
    w.total = w.o + slots * 128 * sizeof(float);
    return w;
}

// f(slot, row tile, items, cost of an item) for the units of one head of each slot.
template <typename F>
void for_units(const kvq_config *c, const ChunkSlot *slots, int g, F f) {
    for (int b = 0; b < c->B; b++) {
        const ChunkSlot &s = slots[b];
        const bool narrow = chunk_narrow(s.n_new, g);
        const int rows = narrow ? kNarrowRows : kWideRows, w = narrow ? kNarrowCost : kWideCost;
        for (int t = 0; (int64_t)t * rows < (int64_t)s.n_new * g; t++) f(b, t, chunk_tiles(s, t, rows, g), w);
    }
}
// Parts of equal length of a unit of n items, each of a cost of at most X, or kPartItems items.
int unit_parts(int n, int w, int X) {
    const int m = std::max(kPartItems, X / w - kUnitItems);  // items of a part
    return (n + m - 1) / m;
}
// Few units (at most C): parts of a unit each, if the longest is no longer than a range of
// even cuts, most of which hold the end of one unit and the start of another (four slots of
// 100 to 900 tokens with a new one each: 15.4 us against 18.5 with even cuts; a prompt of 200
// tokens 17.1 against 21.5).  Units stay whole where that is no longer than parts and the
// combine kernel (three key tiles: 13.2 us against 14.5).  A part has two items at least, one
// for each softmax group (16 key tiles: 15.3 us against 17.4 with parts of one).
bool unit_ranges(const kvq_config *c, const ChunkSlot *slots, int64_t units, ChunkAttnParams &p) {
    if (units > p.C) return false;
    int whole = 0;
    for_units(c, slots, p.g, [&](int, int, int n, int w) { whole = std::max(whole, (n + kUnitItems) * w); });
    int lo = 0, hi = whole;  // the smallest X whose parts are C at most
    while (lo < hi) {
        const int X = (lo + hi) / 2;
        int64_t parts = 0;
        for_units(c, slots, p.g, [&](int, int, int n, int w) { parts += (int64_t)c->H_kv * unit_parts(n, w, X); });
        if (parts <= p.C) hi = X;
        else lo = X + 1;
    }
    int longest = 0;
    for_units(c, slots, p.g, [&](int, int, int n, int w) {
        const int parts = unit_parts(n, w, hi);
        longest = std::max(longest, ((n + parts - 1) / parts + kUnitItems) * w);
    });
    const int even = std::max(p.cost / p.C, kPartItems * kNarrowCost) + kUnitItems * kNarrowCost;
    const bool in_one = whole <= std::min(longest, even) + kCombineCost;
    if (!in_one && longest > even) return false;
    const int X = in_one ? whole : hi;
    int k = 0;
    for (int b = 0; b < c->B; b++) {
        const ChunkSlot &s = slots[b];
        if (s.n_new == 0) continue;
        const bool narrow = chunk_narrow(s.n_new, p.g);
        const int rows = narrow ? kNarrowRows : kWideRows, w = narrow ? kNarrowCost : kWideCost;
        int first = p.cost0[b];
        for (int h = 0; h < c->H_kv; h++)
            for (int t = 0; (int64_t)t * rows < (int64_t)s.n_new * p.g; t++) {
                const int n = chunk_tiles(s, t, rows, p.g), parts = unit_parts(n, w, X);
                for (int i = 0; i < parts; i++, k++) {
                    const int x = (int)((int64_t)n * i / parts);
                    p.begin[k] = i ? first + (kUnitItems + x) * w : first;
                    p.first[k] = first;
                    p.tile[k] = t;
                }
                if (parts > 1) p.cut = 1;
                first += (n + kUnitItems) * w;
            }
    }
    p.C = k;
    p.begin[k] = p.cost;
    return true;
}

// Otherwise each of the C ranges starts at the item behind its even share of the cost.  A
// unit whose start is no further before the even cut than its own fixed cost starts the range.
void even_ranges(const kvq_config *c, const ChunkSlot *slots, ChunkAttnParams &p) {
    int b = 0, t = 0;
    int64_t head = 0, first = 0;  // start of the current head's units, and of unit t
    for (int k = 0; k <= p.C; k++) {
        const int64_t pos = (int64_t)k * p.cost / p.C;
        if (pos >= p.cost) {
            p.begin[k] = p.cost;
            continue;
        }
        for (;;) {  // the unit that holds pos
            while (p.cost0[b + 1] <= pos) head = first = p.cost0[++b], t = 0;
            const ChunkSlot &s = slots[b];
            const bool narrow = chunk_narrow(s.n_new, p.g);
            const int rows = narrow ? kNarrowRows : kWideRows, w = narrow ? kNarrowCost : kWideCost;
            const int64_t per = (p.cost0[b + 1] - p.cost0[b]) / c->H_kv;
            if (pos >= head + per) {
                head += (pos - head) / per * per;
                first = head;
                t = 0;
            }
            const int n = chunk_tiles(s, t, rows, p.g);
            const int64_t end = first + (int64_t)(n + kUnitItems) * w;
            if (pos >= end) {
                first = end;
                t++;
                continue;
            }
            const int64_t x = (pos - first + w - 1) / w - kUnitItems;  // items before it, rounded up
            p.begin[k] = (int32_t)(x <= 0 ? first : first + (kUnitItems + x) * w);
            p.first[k] = (int32_t)first;
            p.tile[k] = t;
            if (x > 0 && x < n) p.cut = 1;
            break;
        }
    }
}

}  // namespace

extern "C" {

int kvq_paged_plan(const kvq_config *c, kvq_paged *pc, const int32_t *n_new, const int32_t *new_pages,
                   int64_t n_new_pages, kvq_chunk *ch, void *stream) {
    int e = check_paged(c, pc);
    if (e) return e;
    if ((e = check_chunk(ch))) return e;
    if (!n_new || n_new_pages < 0 || (reinterpret_cast<uintptr_t>(new_pages) & 3u)) return KVQ_ERR_INVALID_ARG;
    int64_t rows = 0, pages = 0;
    for (int b = 0; b < c->B; b++) {
        const int32_t *l = pc->lens_host + 4 * b;
        if (n_new[b] < 0) return KVQ_ERR_INVALID_ARG;
        const int64_t ns = l[3] ? l[0] : 0, T = l[3] ? l[1] : 0, nr = l[3] ? l[2] : 0;
        const int64_t to_sink = std::min<int64_t>(n_new[b], c->S - ns);
        const int64_t pk = n_new[b] ? (nr + n_new[b] - to_sink) / c->R * c->R : 0;
        if (T + pk > c->max_T || ns + T + nr + n_new[b] > INT32_MAX) return KVQ_ERR_CAPACITY;
        rows += n_new[b];
        pages += pk / c->G;
    }
    if (rows > ch->max_tokens || rows > INT32_MAX - 4096) return KVQ_ERR_CAPACITY;
    if (new_pages && pages > n_new_pages) return KVQ_ERR_CAPACITY;
    cudaStream_t st = (cudaStream_t)stream;
    if (ch->captured || capturing(st)) return KVQ_ERR_UNSUPPORTED;
    PlanParams p;
    p.cu = ch->cu;
    p.slot = ch->slot;
    p.pos = ch->pos;
    p.desc = ch->desc;
    p.table = const_cast<int32_t *>(pc->page_table);
    p.lens = pc->lens;
    p.new_pages = new_pages;
    p.B = c->B;
    p.S = c->S;
    p.R = c->R;
    p.G = c->G;
    p.table_stride = (int)(c->max_T / c->G);
    p.n_tokens = (int)rows;
    memcpy(p.n_new, n_new, (size_t)c->B * 4);
    if (launch_plan(p, st) != cudaSuccess) return KVQ_ERR_CUDA;
    int cu = 0, pg = 0;
    for (int b = 0; b < c->B; b++) {
        const int32_t *l = pc->lens_host + 4 * b;
        ChunkSlot &s = slots_of(ch)[b];
        s.ns = l[3] ? l[0] : 0;
        s.T = l[3] ? l[1] : 0;
        s.nr = l[3] ? l[2] : 0;
        s.n_new = n_new[b];
        s.cu = cu;
        s.to_sink = std::min(n_new[b], c->S - s.ns);
        s.pk = n_new[b] ? (s.nr + n_new[b] - s.to_sink) / c->R * c->R : 0;
        s.page0 = pg;
        cu += n_new[b];
        pg += s.pk / c->G;
    }
    ch->n_tokens = rows;
    return KVQ_OK;
}

size_t kvq_paged_chunk_workspace_bytes(const kvq_config *c) {
    return paged_cfg_check(c) == KVQ_OK ? chunk_ws().total : 0;
}

int kvq_paged_chunk_attn(const kvq_config *c, const kvq_paged *pc, kvq_chunk *ch, const uint16_t *q,
                         int64_t q_stride, const uint16_t *kn, int64_t k_stride, const uint16_t *vn, int64_t v_stride,
                         uint16_t *out, void *ws, size_t ws_bytes, void *stream) {
    int e = check_paged(c, pc);
    if (e) return e;
    if ((e = check_chunk(ch))) return e;
    if (!plan_holds(c, pc, ch)) return KVQ_ERR_INVALID_ARG;
    if (ch->n_tokens == 0) return KVQ_OK;
    if (!rows_ok(q, q_stride, c->H_q, c->D) || !rows_ok(kn, k_stride, c->H_kv, c->D) ||
        !rows_ok(vn, v_stride, c->H_kv, c->D) || !out || !aligned16(out))
        return KVQ_ERR_INVALID_ARG;
    // rows are written while others are still read
    const size_t no = (size_t)ch->n_tokens * c->H_q * c->D * 2;
    auto span = [&](int64_t stride, int64_t heads) { return ((size_t)(ch->n_tokens - 1) * stride + heads * c->D) * 2; };
    if (overlap(out, no, q, span(q_stride, c->H_q)) || overlap(out, no, kn, span(k_stride, c->H_kv)) ||
        overlap(out, no, vn, span(v_stride, c->H_kv)))
        return KVQ_ERR_INVALID_ARG;
    const ChunkWs wl = chunk_ws();
    if (!ws || !aligned16(ws) || ws_bytes < wl.total) return KVQ_ERR_WORKSPACE;
    ChunkAttnParams p;
    memset(&p, 0, sizeof(p));
    p.desc = ch->desc;
    p.ptab = pc->page_table;
    p.k_codes = pc->k_codes;
    p.v_codes = pc->v_codes;
    p.k_meta = pc->k_meta;
    p.v_meta = pc->v_meta;
    p.k_sink = pc->k_sink;
    p.v_sink = pc->v_sink;
    p.k_res = pc->k_res;
    p.v_res = pc->v_res;
    p.q = q;
    p.k_new = kn;
    p.v_new = vn;
    p.out = out;
    p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(ws) + wl.ml);
    p.part_o = reinterpret_cast<float *>(static_cast<char *>(ws) + wl.o);
    p.status = pc->status;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_pages = pc->n_pages;
    p.B = c->B;
    p.H_kv = c->H_kv;
    p.g = c->H_q / c->H_kv;
    p.G = c->G;
    p.kbits = c->bits;
    p.vbits = vbits_of(c);
    p.S = c->S;
    p.R = c->R;
    p.ptab_stride = (int)(c->max_T / c->G);
    // over 8-bit codes, slots of few rows have a kernel of their own, if all are such slots, or if it
    // gains more than its launches cost
    bool few[KVQ_PAGED_MAX_B], any_few = false, all_few = block8(c);
    ChunkSlot rest[KVQ_PAGED_MAX_B];
    const ChunkSlot *slots = slots_of(ch);
    if (block8(c)) {
        int64_t tiles = 0;
        int most = 0;  // rows of such a slot
        for (int b = 0; b < c->B; b++) {
            const ChunkSlot &s = slots[b];
            if (s.n_new && s.T && pc->n_pages < 1) return KVQ_ERR_INVALID_ARG;
            few[b] = s.n_new && (int64_t)s.n_new * p.g <= kFewRows;
            any_few |= few[b];
            all_few &= few[b] || !s.n_new;
            if (!few[b]) continue;
            tiles += (int64_t)p.H_kv * (s.T / kChunkKeys);
            most = std::max(most, s.n_new * p.g);
        }
        any_few &= all_few || tiles >= (most > 16 ? kFewTiles32 : kFewTiles);
        for (int b = 0; any_few && b < c->B; b++) {
            rest[b] = slots[b];
            if (few[b]) rest[b].n_new = 0;
        }
        if (any_few) slots = rest;
    }
    int64_t cost = 0, items = 0, units = 0;
    for (int b = 0; b < c->B; b++) {
        const ChunkSlot &s = slots[b];
        p.cost0[b] = (int32_t)cost;
        const bool narrow = chunk_narrow(s.n_new, p.g);
        const int rows = narrow ? kNarrowRows : kWideRows;
        int64_t per = 0;
        for (int64_t t = 0; t * rows < (int64_t)s.n_new * p.g; t++) {
            const int n = chunk_tiles(s, (int)t, rows, p.g);
            per += n + kUnitItems;
            items += (int64_t)n * p.H_kv;
            units += p.H_kv;
        }
        if (s.n_new && s.T && pc->n_pages < 1) return KVQ_ERR_INVALID_ARG;  // page 0 stands in for bad entries
        if (s.n_new && narrow) p.narrow = std::max(p.narrow, s.n_new * p.g);
        if (s.n_new && !narrow) p.wide = 1;
        cost += per * p.H_kv * (narrow ? kNarrowCost : kWideCost);
        if (cost >= (1LL << 30)) return KVQ_ERR_UNSUPPORTED;
    }
    for (int b = c->B; b <= KVQ_PAGED_MAX_B; b++) p.cost0[b] = (int32_t)cost;
    p.cost = (int)cost;
    p.C = (int)std::min<int64_t>(items, std::min(num_sms(), kMaxRanges));
    if (any_few && (e = block_chunk_few(c, pc, slots_of(ch), few, p, (cudaStream_t)stream))) return e;
    if (!all_few && !unit_ranges(c, slots, units, p)) even_ranges(c, slots, p);
    p.ref_unit = block8(c) ? 1.f : kScale;
    if (!all_few && (block8(c) ? launch_chunk_attn_block(p, c->mode == KVQ_MODE_E4M3, (cudaStream_t)stream)
                   : launch_chunk_attn(p, (cudaStream_t)stream)) != cudaSuccess)
        return KVQ_ERR_CUDA;
    if (!ch->captured && capturing((cudaStream_t)stream)) ch->captured = 1;
    return KVQ_OK;
}

int kvq_paged_extend(const kvq_config *c, kvq_paged *pc, const kvq_chunk *ch, const uint16_t *kn, int64_t k_stride,
                     const uint16_t *vn, int64_t v_stride, void *stream) {
    int e = check_paged(c, pc);
    if (e) return e;
    if ((e = check_chunk(ch))) return e;
    if (!plan_holds(c, pc, ch)) return KVQ_ERR_INVALID_ARG;
    if (ch->n_tokens == 0) return KVQ_OK;
    if (!rows_ok(kn, k_stride, c->H_kv, c->D) || !rows_ok(vn, v_stride, c->H_kv, c->D)) return KVQ_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (capturing(st)) return KVQ_ERR_UNSUPPORTED;
    ExtendParams p;
    memset(&p, 0, sizeof(p));
    p.desc = ch->desc;
    p.lens = pc->lens;
    p.status = pc->status;
    p.k_new = kn;
    p.v_new = vn;
    p.k_stride = k_stride;
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
    p.B = c->B;
    p.H_kv = c->H_kv;
    p.G = c->G;
    p.S = c->S;
    p.R = c->R;
    p.TV = vtile_of(c);
    p.ptab_stride = (int)(c->max_T / c->G);
    for (int b = 0; b < c->B; b++) {
        p.page0[b] = p.n_pack;
        p.n_pack += slots_of(ch)[b].pk / c->G;
    }
    p.page0[c->B] = p.n_pack;
    if (p.n_pack > 0 && pc->n_pages < 1) return KVQ_ERR_CAPACITY;
    p.once = block8(c) || (c->R == c->G && c->G == 128);
    if ((block8(c) ? launch_block_extend(p, slots_of(ch), c->mode == KVQ_MODE_E4M3, st) : launch_extend(p, c->bits, vbits_of(c), st)) != cudaSuccess)
        return KVQ_ERR_CUDA;
    for (int b = 0; b < c->B; b++) {
        const ChunkSlot &s = slots_of(ch)[b];
        if (!s.n_new) continue;
        int32_t *l = pc->lens_host + 4 * b;
        l[0] = s.ns + s.to_sink;
        l[1] = s.T + s.pk;
        l[2] = s.nr + s.n_new - s.to_sink - s.pk;
        l[3] = 1;
    }
    return KVQ_OK;
}

int kvq_qk_norm_rope(const kvq_qk_config *c, const uint16_t *q, const uint16_t *k, const uint16_t *w_q,
                     const uint16_t *w_k, const int32_t *pos, int64_t n, uint16_t *q_out, uint16_t *k_out,
                     void *stream) {
    return kvq_qk_norm_rope_freq(c, nullptr, 1.f, q, k, w_q, w_k, pos, n, q_out, k_out, stream);
}

int kvq_qk_norm_rope_freq(const kvq_qk_config *c, const double *freq, float amp, const uint16_t *q, const uint16_t *k,
                          const uint16_t *w_q, const uint16_t *w_k, const int32_t *pos, int64_t n, uint16_t *q_out,
                          uint16_t *k_out, void *stream) {
    if (!c || c->H_q < 0 || c->H_kv < 0 || c->H_q + (int64_t)c->H_kv < 1 || c->H_q > 65535 || c->H_kv > 65535 || n < 0)
        return KVQ_ERR_INVALID_ARG;
    const int e = rope_check(c, freq, amp);
    if (e) return e;
    if (n == 0) return KVQ_OK;
    if (n > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
    if (!pos || (reinterpret_cast<uintptr_t>(pos) & 3u)) return KVQ_ERR_INVALID_ARG;
    struct Side {
        const uint16_t *x, *w;
        uint16_t *y;
        int64_t stride, H;
    } side[2] = {{q, w_q, q_out, c->q_stride, c->H_q}, {k, w_k, k_out, c->k_stride, c->H_kv}};
    for (const Side &s : side) {
        if (!s.H) continue;
        if (!rows_ok(s.x, s.stride, s.H, c->D) || !s.y || !aligned16(s.y) || (s.w && !aligned16(s.w)))
            return KVQ_ERR_INVALID_ARG;
    }
    for (int a = 0; a < 2; a++) {
        if (!side[a].H) continue;
        const size_t ny = (size_t)n * side[a].H * c->D * 2;
        if (side[1 - a].H && a == 0 && overlap(side[0].y, ny, side[1].y, (size_t)n * side[1].H * c->D * 2))
            return KVQ_ERR_INVALID_ARG;
        for (int b = 0; b < 2; b++) {
            if (!side[b].H) continue;
            const size_t nx = ((size_t)(n - 1) * side[b].stride + side[b].H * c->D) * 2;
            const bool own = a == b && side[a].y == side[a].x && (side[a].stride == side[a].H * c->D || n == 1);
            if (!own && overlap(side[a].y, ny, side[b].x, nx)) return KVQ_ERR_INVALID_ARG;
        }
    }
    QkParams p;
    memset(&p, 0, sizeof(p));
    p.q = q;
    p.k = k;
    // (lanes behind the last head look up a weight as well)
    p.w_q = c->H_q ? w_q : nullptr;
    p.w_k = c->H_kv ? w_k : nullptr;
    p.pos = pos;
    p.q_out = q_out;
    p.k_out = k_out;
    p.n = n;
    p.q_stride = c->q_stride;
    p.k_stride = c->k_stride;
    p.H_q = c->H_q;
    p.H_kv = c->H_kv;
    p.rotary = c->rotary_dim;
    p.halves = c->halves;
    p.rotate = c->rotary_dim ? c->rotate : 0;
    p.eps = c->eps;
    p.amp = amp;
    if (c->rotary_dim && freq) turns_of_freq(freq, c->rotary_dim, p.turn);
    else if (c->rotary_dim) turns_of_base(c->rope_base, c->rotary_dim, p.turn);
    return status_of(launch_qk(p, c->D, (cudaStream_t)stream));
}

}  // extern "C"
