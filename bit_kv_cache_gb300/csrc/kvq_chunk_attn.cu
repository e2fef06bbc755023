// kvq_chunk_attn.cu -- the chunk attention kernel: softmax(q K^T) V of a unit's query rows
// over a range of its key tiles, on the 5th-generation tensor cores.
//
// For query row r of a unit (see ChunkAttnParams) and key t of its slot,
//   s_t = q . (code_t * scale + min) / sqrt(D),   out = sum_t softmax(s)_t v_t,
// in one pass over the keys with a running maximum and sum per row.  Sums, maxima and the
// output's accumulators are fp32.  Dequantized keys and values and the softmax weights are
// rounded once to fp16, the operand type of the products: outputs of unit-variance values are
// then off by 3.1e-4 to 5.6e-4 of their size.  Alone, the output's own rounding makes 2.1e-4 of
// it, the keys' 2.1e-4 (2-bit) to 4.1e-4 (8-bit, a few channels of five times the size), the
// values' 1.3e-4 to 2.2e-4, the weights' 1.2e-4 to 1.9e-4.  Exact operands would be codes with
// the scales folded into the other operand, which differ from page to page (keys: another Q
// tile per page) and would be rounded there instead, or a second operand for the remainders:
// a second product per key tile, and no room in shared memory for its tiles.
//
// What bounds it.  Wide units: the tensor core.  A product with M = 128 reads its operands
// from shared memory at 128 bytes a cycle: K = 16 takes 48 cycles at N = 64, 64 at N = 128, so
// a key tile of 256 rows takes 2478 cycles when nothing else runs.  2048 tokens of 32 heads
// over 32868 cached ones (2-bit; 1137 GFLOP): 865 to 903 us, 1.26 to 1.31 PFLOP/s, 0.68 to 0.71
// of the measured rate of a large library product; dequantization and softmax take issue slots
// and shared memory beside it.  Narrow units: issue slots.  Eight slots of 17K to 56K tokens
// with 1 to 8 new ones take 145 us, where their packed bytes take 24: 0.62 instructions a cycle
// and scheduler, the ALU half busy (5600 warp instructions per key tile: one AND and two fused
// products per two codes, the stores of the fp16 tiles, the softmax, waits), the tensor core
// 0.45.  The kernel keeps 48 bytes of a thread on the stack (104 stored, 144 loaded).
// Tried there and dropped, when these cases stood at 148 and 847 us: both groups of a side on
// one tile (162 us; 77 us against 84 with 8-bit codes, but 911 us in the case above), barriers
// per half tile (164 us), an early start of the kernel behind (166 us).
//
// One CTA per SM, eight groups of four warps:
//   groups 0, 1  softmax, a thread per row of 128: reads the scores S_m from tensor memory,
//                keeps a reference near the row's running maximum and the sum in registers,
//                writes the weights P_m over S_m as fp16, rescales O_m when the reference moves;
//   groups 2-5   make the key tiles (2, 3) and the value tiles (4, 5), every second one each:
//                packed pages arrive by bulk copies and are dequantized into fp16 tiles in
//                shared memory, fp16 rows are gathered;
//   groups 6, 7  warps 24 + m issue the products S_m = Q K^T, warps 26 + m O_m += P_m V: each
//                waits for its own operands while the others keep the tensor core busy (one
//                warp for all four: 1520 us against 1253; a wait that is over costs it about
//                100 cycles, and up to 3000 when its scheduler's other warps never stall);
//                warps 28, 29 bring the packed keys and values (issued by the producers
//                themselves: 1025 us against 990).
// In a wide unit (256 rows) m names the query tile: a key tile is dequantized once for both.
// In a narrow one (at most 128 rows) m is the parity of the key tile: the two groups keep
// softmax states of their own, joined at the end.  With at most 64 (32) rows, a part of a unit
// that is cut holds them twice (four times) in its query tile, and each copy's softmax takes
// half (a quarter) of a tile's keys: the tensor core's rows cost nothing, and a step of the
// softmax, which is what such a unit waits for, is as much shorter (the eight slots above:
// 148 us then, against 187 without).  The combine kernel joins the copies' partials like those of
// the ranges.
// A step is half a key tile (64 keys).  S_m has two buffers of 64 columns, so that the scores
// of the next step are made while the softmax of this one runs.  Tensor memory: S_0, S_1,
// O_0, O_1, 128 columns each.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_chunk_attn.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

namespace {

constexpr int kRows = kWideRows, kThreads = 1024;
constexpr int kTileBytes = kChunkKeys * kD * 2;          // an fp16 key or value tile: 32 KB
constexpr int kRing = 2;                                 // tiles of each kind
constexpr int kRawBytes = 4 * (8192 + 512);              // packed tiles: codes and (scale, min)
constexpr int kMaxRaw = 4;
constexpr int kOffQ = 0, kOffK = 2 * kTileBytes, kOffV = kOffK + kRing * kTileBytes, kOffRaw = kOffV + kRing * kTileBytes,
              kOffBar = kOffRaw + kRawBytes;
// Weights are 2^((x - r) kScale + kUp) of scores x = q . k, with a reference r (one of the row's
// scores) that may lag behind the maximum while 64 weights sum to kMostSum at most, below
// fp16's 65504; kUp more bits keep small weights above fp16's smallest step.  With |r| of at
// most kNear the exponent is one fused product, x kScale + (kUp - r kScale), whose constant is
// off by 2^-15 at most; beyond it (362 in units of the softmax's exponent) x - r, which is
// exact where it matters, is formed first in every step, as scaled values of 2^28 and more
// would differ from their products by more than fp16's range has room for.  (A 2048-token
// chunk: 867 us against 859 with scaled references alone.  The weights of such rows as a
// branch of their own, or one body of code for both: 900 to 940, the hot code grows or stalls.)
constexpr float kUp = 6.f, kMostSum = 16384.f, kNear = 4096.f;
// registers of a thread after the split; 64 at launch, times 1024 threads
constexpr int kRegsSoftmax = 112, kRegsTiles = 48, kRegsOther = 48;
static_assert(256 * kRegsSoftmax + 512 * kRegsTiles + 256 * kRegsOther <= kThreads * 64, "register split");

struct Bars {
    uint64_t q_full, q_empty, k_full[kRing], k_empty[kRing], v_full[kRing], v_empty[kRing];
    uint64_t s_full[2][2], p_full[2][2];              // of query tile m, step parity h
    // (a wait names a phase by its parity, so no barrier may run two phases ahead of a waiter)
    uint64_t pv_done[2][2], drain;
    uint64_t o1_full, o1_free;                        // narrow units: O_1 and its sums are final, have been read
    uint64_t rawk[2][kMaxRaw], rawv[2][kMaxRaw];      // packed tile arrived, by the tile's parity
    uint64_t readk[kMaxRaw], readv[kMaxRaw];          // packed tile read by all producers
    uint32_t tmem;
    int stop;
    int odd;                 // whether a tail value of any segment so far was not finite
};
constexpr int kSmemBytes = kOffBar + (int)sizeof(Bars);
static_assert(kSmemBytes <= 232448, "shared memory");

// Segment: the items of one unit inside the CTA's range; its steps.
struct Seg {
    Item it;
    int k0, k1, np, valid, steps, rep;  // rep: copies of a narrow unit's rows in its query tile
    bool narrow;
};
// A CTA's place in its range.
struct At {
    int pos, end, first, tile;  // first, tile: of the unit at pos, or of one before it
    __device__ __forceinline__ explicit At(const ChunkAttnParams &p)
        : pos(p.begin[blockIdx.x]), end(p.begin[blockIdx.x + 1]), first(p.first[blockIdx.x]), tile(p.tile[blockIdx.x]) {}
    __device__ __forceinline__ bool more() const { return pos < end; }
};
__device__ __forceinline__ Seg next_seg(const ChunkAttnParams &p, At &c) {
    Seg s;
    const int at = c.pos, end = c.end;
    s.it = find_item(p, at, c.first, c.tile);
    s.narrow = s.it.rows == kNarrowRows;
    s.k0 = s.it.at(at);
    s.k1 = s.it.at(end);
    c.pos = min(end, s.it.end());
    c.first = s.it.end();
    c.tile = s.it.t + 1;
    s.np = s.it.s.T / kChunkKeys;
    s.valid = min(s.it.rows, s.it.s.n_new * p.g - s.it.t * s.it.rows);
    s.rep = s.narrow && s.k1 - s.k0 < s.it.n ? chunk_copies(s.valid) : 1;  // partials: each copy leaves its own
    // a wide unit's last key tile may end in its first half
    const int last = min(s.it.s.n_new, ((s.it.t + 1) * s.it.rows - 1) / p.g + 1);
    const int seen = s.it.s.ns + s.it.s.nr + last - (s.it.n - s.np - 1) * kChunkKeys;
    s.steps = 2 * (s.k1 - s.k0) - (!s.narrow && s.k1 == s.it.n && seen <= 64 ? 1 : 0);
    return s;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// A code's bits under the exponent of 1024 make 1024 + code 2^sh; one fused step makes the
// exact code of it, another code * scale + min, rounded once.
// A packed tile becomes an fp16 operand whose rows run along the packed direction (keys: a
// row per token, channels contiguous; values: a row per channel, tokens contiguous).  A job
// is one word row m and eight neighbouring columns: words w of two columns are split into
// halves (the codes of the rows' first and second half, in pairs of columns), so that every
// row is four half2, one 16-byte store.  wd: the eight words; s2, m2: (scale, min) of the
// column pairs; dst: row 0 of the job at its 16-byte chunk, which row r xors with r mod 8.
template <int BITS>
__device__ __forceinline__ void deq_job(const uint32_t (&wd)[8], const uint32_t (&s2)[4], const uint32_t (&m2)[4], uint32_t dst) {
    constexpr int N = 32 / BITS;                       // rows
    constexpr uint32_t MASK = ((1u << BITS) - 1u) * 0x10001u;
    constexpr int FIT = BITS == 2 ? 5 : BITS == 4 ? 2 : 1;  // codes of a half below bit 10
#pragma unroll 1
    for (int hf = 0; hf < 2; hf++) {
        uint32_t x[4];
#pragma unroll
        for (int c = 0; c < 4; c++) x[c] = prmt(wd[2 * c], wd[2 * c + 1], hf ? 0x7632 : 0x5410);
#pragma unroll
        for (int j = 0; j < N / 2; j++) {
            uint32_t y[4];
#pragma unroll
            for (int c = 0; c < 4; c++) {
                if (j > 0 && j % FIT == 0) x[c] >>= FIT * BITS;
                const uint32_t v = (x[c] & (MASK << (j % FIT * BITS))) | 0x64006400u;
                const uint32_t mul = (uint32_t)(0x3c00 - ((j % FIT * BITS) << 10)) * 0x10001u;  // 2^-sh
                const uint32_t sub = (uint32_t)(0xe400 - ((j % FIT * BITS) << 10)) * 0x10001u;  // -1024 2^-sh
                y[c] = hfma2(hfma2(v, mul, sub), s2[c], m2[c]);
            }
            const uint32_t at = (dst ^ ((j & 7) << 4)) + j * 128;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
        }
        dst = (dst ^ ((N / 2 & 7) << 4)) + N / 2 * 128;  // the rows of the second half
    }
}

__device__ __forceinline__ void lds128(uint32_t *r, uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// raw: codes [4 BITS word rows][128 columns] (values: tiles of TV columns, [rows][TV] each),
// then 128 (scale, min).  Thread t takes columns 8 (t mod 16) .. + 7 of word rows t / 16 + 8 i.
template <int BITS>
__device__ __forceinline__ void make_tile(uint32_t raw, uint32_t tile, int t, int TV) {
    const int c0 = 8 * (t & 15), m0 = t >> 4;
    constexpr int N = 32 / BITS, NR = 4 * BITS;
    uint32_t mt[8], s2[4], m2[4];
    lds128(mt, raw + 4 * (512 * BITS + c0));
    lds128(mt + 4, raw + 4 * (512 * BITS + c0) + 16);
#pragma unroll
    for (int c = 0; c < 4; c++) {
        s2[c] = prmt(mt[2 * c], mt[2 * c + 1], 0x5410);
        m2[c] = prmt(mt[2 * c], mt[2 * c + 1], 0x7632);
    }
    const int j = c0 & (TV - 1);
    const uint32_t src = raw + 4 * ((c0 - j) * NR);
#pragma unroll 1
    for (int i = 0; i < NR / 8; i++) {
        const int m = m0 + 8 * i;
        uint32_t wd[8];  // the row's 16-byte chunks are permuted by xor with m mod 8
        lds128(wd, src + 4 * (m * TV + (j ^ ((m & 7) << 2))));
        lds128(wd + 4, src + 4 * (m * TV + ((j + 4) ^ ((m & 7) << 2))));
        // row N m; N is a multiple of 4: for 8-bit codes an odd word row starts inside an atom
        const uint32_t row = tile + (c0 >> 6) * 16384 + m * N * 128 + ((((c0 >> 3) & 7) ^ ((m * N) & 7)) << 4);
        deq_job<BITS>(wd, s2, m2, row);
    }
}

// 16 bytes from global to shared memory without registers (zeros if !ok).
__device__ __forceinline__ void copy16(void *dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// fp16 rows x0 .. x0 + 127 of [sink | residual | chunk]: row = token, 16-byte chunk c of a
// row at block c / 8, position c ^ row within it (the layout of both tail operands: key
// rows run along the tokens, value rows along the channels).  True if a value is not finite;
// it is replaced by 0.
__device__ __forceinline__ bool make_tail(const ChunkAttnParams &p, const Seg &s, int x0, bool value, unsigned char *tile, int tid) {
    const int ntail = s.it.s.ns + s.it.s.nr + s.it.s.n_new, c = tid & 15;
    unsigned char *col = tile + (c >> 3) * 16384;
#pragma unroll 1
    for (int r = tid >> 4; r < kChunkKeys; r += 8) {
        const int x = min(x0 + r, ntail - 1);
        copy16(col + r * 128 + (((c & 7) ^ (r & 7)) << 4), tail_row(p, s.it, x, value) + 8 * c, x0 + r < ntail);
    }
    copy16_wait();
    bool bad = false;
    if (value)
#pragma unroll 1
        for (int r = tid >> 4; r < kChunkKeys; r += 8) {
            uint4 *at = reinterpret_cast<uint4 *>(col + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            uint4 a = *at;
            uint32_t *v = reinterpret_cast<uint32_t *>(&a);
            bool here = false;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if ((v[e] & 0x7c00u) == 0x7c00u) v[e] &= 0xffff0000u, here = true;
                if ((v[e] & 0x7c000000u) == 0x7c000000u) v[e] &= 0xffffu, here = true;
            }
            if (here) *at = a;
            bad |= here;
        }
    return bad;
}

// A position in a ring of barriers: slot, and the parity of its next completion.
struct Ring {
    int i;
    uint32_t parity;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) i = 0, parity ^= 1;
    }
};

// Shared memory of the packed tiles of one side.
struct Raw {
    int slots, size, off;
    __device__ __forceinline__ Raw(const ChunkAttnParams &p, bool value) {
        const int kraw = 2048 * p.kbits + 512, vraw = 2048 * p.vbits + 512;
        slots = min(kMaxRaw, kRawBytes / (kraw + vraw));
        size = value ? vraw : kraw;
        off = kOffRaw + (value ? slots * kraw : 0);
    }
};

// ---------------------------------------------------------------- warps 28, 29: copies --
// One lane brings the packed tiles of the keys (values) into their ring, as far ahead as it
// has slots.  The page-table entry of a tile is read before the copy of the tile before it
// is waited for.
__device__ __forceinline__ void bring(const ChunkAttnParams &p, unsigned char *sm, Bars *bar, bool value) {
    const Raw raw(p, value);
    const int bits = value ? p.vbits : p.kbits;
    uint64_t(*arrived)[kMaxRaw] = value ? bar->rawv : bar->rawk, *read = value ? bar->readv : bar->readk;
    const int32_t *codes = value ? p.v_codes : p.k_codes;
    const uint16_t *meta = value ? p.v_meta : p.k_meta;
    const int gshift = p.G == kChunkKeys ? 0 : 1;  // key tiles per page: 1 or 2
    Ring cp = {0, 1};
    int n = 0;                 // tiles of the segments before
    uint32_t used = 0, parity = 0;  // per barrier (bit kMaxRaw par + slot): whether and how often used
    for (At at(p); at.more();) {
        const Seg s = next_seg(p, at);
        const int npk = min(s.k1, s.np), n0 = n - s.k0;
        n += s.k1 - s.k0;
        const int32_t *row = p.ptab + (size_t)s.it.b * p.ptab_stride;
        if (s.k0 >= npk) continue;
        int32_t entry = row[s.k0 >> gshift];
        for (int kt = s.k0; kt < npk; kt++) {
            const int32_t ahead = row[min(kt + 1, npk - 1) >> gshift];
            await(&read[cp.i], cp.parity, &bar->stop, p.status);
            if (*(volatile int *)&bar->stop) break;
            const int64_t page = page_index(p, s.it, entry);
            const int t0 = kt * kChunkKeys & (p.G - 1);
            unsigned char *dst = sm + raw.off + cp.i * raw.size;
            const int par = (n0 + kt) & 1, bit = 1 << (kMaxRaw * par + cp.i);
            uint64_t *b = &arrived[par][cp.i];
            mbar_arrive_expect_tx(b, raw.size);
            bulk_g2s(dst, codes + ((size_t)page * p.G + t0) * (kD * bits / 32), 2048 * bits, b);
            bulk_g2s(dst + 2048 * bits, meta + (value ? ((size_t)page * p.G + t0) * 2 : (size_t)page * kD * 2), 512, b);
            cp.next(raw.slots);
            used |= bit;
            parity ^= bit;
            entry = ahead;
        }
    }
    // the last copies land before the block ends, whether they are awaited there or not
    for (int i = 0; i < 2 * kMaxRaw; i++)
        if ((used >> i) & 1) mbar_wait(&arrived[i / kMaxRaw][i % kMaxRaw], ~(parity >> i) & 1, p.status);
}

// ---------------------------------------------------------------- groups 2-5: tiles ---
// All four run the same code, and its loops stay rolled: the roles share an SM's instruction
// cache (unrolled loops: 1672 us against 1107, half of all stalls for want of instructions).
// Every second tile each: a group that makes every tile of its side waits for the release of
// the tile before (979 us against 950).
__device__ __forceinline__ void produce(const ChunkAttnParams &p, unsigned char *sm, Bars *bar, bool value, int par) {
    const int tid = threadIdx.x & 127, bits = value ? p.vbits : p.kbits, TV = value ? 256 / p.kbits : kChunkKeys;
    const Raw raw(p, value);
    unsigned char *dst = sm + (value ? kOffV : kOffK) + par * kTileBytes;
    uint64_t *arrived = (value ? bar->rawv : bar->rawk)[par], *read = value ? bar->readv : bar->readk;
    uint64_t *full = (value ? bar->v_full : bar->k_full) + par, *empty = (value ? bar->v_empty : bar->k_empty) + par;
    int slot = 0;              // of the next packed tile, of either parity
    uint32_t landed = 0, free = 1, nq = 1;  // parities: of the slots' arrivals, of the tile's release
    int n = 0;                 // tiles of the segments before
    for (At at(p); at.more();) {
        const Seg s = next_seg(p, at);
        if (value && par == 0) {
            // queries: 128-row tiles, rows of tokens' heads; rows behind the last one repeat it
            await(&bar->q_empty, nq & 1, &bar->stop, p.status);
            nq++;
            const int ch = tid & 15, rows = s.rep > 1 ? 128 : (s.valid + 31) & ~31;  // whole warps of the softmax
            const int copy = s.rep > 1 ? 128 / s.rep - 1 : kRows - 1;
#pragma unroll 1
            for (int r = tid >> 4; r < rows; r += 8) {
                const int x = s.it.t * s.it.rows + min(r & copy, s.valid - 1), tok = x / p.g;
                copy16(sm + kOffQ + (r >> 7) * kTileBytes + (ch >> 3) * 16384 + (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4),
                       p.q + (int64_t)(s.it.s.cu + tok) * p.q_stride + (s.it.h * p.g + x - tok * p.g) * kD + 8 * ch, true);
            }
            copy16_wait();
            fence_proxy_async();
            mbar_arrive(&bar->q_full);
        }
        for (int kt = s.k0; kt < s.k1; kt++) {
            if (((n + kt - s.k0) & 1) != par) {
                if (kt < s.np && ++slot == raw.slots) slot = 0;
                continue;
            }
            if (kt < s.np) {
                await(&arrived[slot], (landed >> slot) & 1, &bar->stop, p.status);
                landed ^= 1u << slot;
                await(empty, free, &bar->stop, p.status);
                const uint32_t from = smem_u32(sm + raw.off + slot * raw.size), to = smem_u32(dst);
                if (bits == 2) make_tile<2>(from, to, tid, TV);
                else if (bits == 4) make_tile<4>(from, to, tid, TV);
                else make_tile<8>(from, to, tid, TV);
                mbar_arrive(&read[slot]);
                if (++slot == raw.slots) slot = 0;
            } else {
                await(empty, free, &bar->stop, p.status);
                if (make_tail(p, s, (kt - s.np) * kChunkKeys, value, dst, tid)) {
                    // infinite and NaN values enter the product as 0 (0 weights of rows that may
                    // not see them would spread them) and are added to their rows at the end
                    *(volatile int *)&bar->odd = 1;
                }
            }
            fence_proxy_async();
            mbar_arrive(full);
            free ^= 1;
        }
        n += s.k1 - s.k0;
    }
}

// ---------------------------------------------------------------- warps 24-27: products
// Rows along M and N (keys: tokens, packed values: channels): 16 of the contracted dimension
// are 32 bytes of a row; fp16 value rows run along the tokens: 16 are two atoms.

// Warp 24 + m: the scores S_m.  A buffer's next scores go over its old weights, once the
// product that reads those has ended.
__device__ __forceinline__ void issue_scores(const ChunkAttnParams &p, unsigned char *sm, Bars *bar, uint32_t tm, int m) {
    const uint32_t base = smem_u32(sm), lead = (threadIdx.x & 31) == 0;
    uint32_t n = 0, nq = 0;       // key tiles, query tiles
    uint32_t ph = 0, any = 0;     // per buffer h: parity of the products awaited, whether there was one
    auto wait = [&](uint64_t *b, uint32_t parity) { warp_await(b, parity & 1, &bar->stop, p.status); };
    auto ready = [&](int h) {     // buffer h may be written
        if ((any >> h) & 1) wait(&bar->pv_done[m][h], ph >> h);
        ph ^= ((any >> h) & 1) << h;
        any |= 1u << h;
    };
    auto scores = [&](int q, int h, uint32_t slot, uint32_t idesc) {
        tc_fence_after();
        const uint64_t a0 = smem_desc(base + kOffQ + q * kTileBytes, 16, 1024);
        const uint64_t b0 = smem_desc(base + kOffK + slot * kTileBytes + h * 8192, 16, 1024);
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
            mma_ss(tm + m * 128 + h * 64, a0 + off, b0 + off, idesc, k > 0, lead);
        }
        tc_commit(&bar->s_full[m][h], lead);
    };
    for (At at(p); at.more();) {
        const Seg s = next_seg(p, at);
        wait(&bar->q_full, nq);
        nq++;
        const int tiles = s.k1 - s.k0;
        for (int j = 0; j < tiles; j++) {
            const uint32_t slot = n % kRing;
            wait(&bar->k_full[slot], n / kRing);
            n++;
            if (s.narrow ? (j & 1) == m : 128 * m < s.valid) {
                if (s.narrow) {
                    ready(0);
                    ready(1);
                    scores(0, 0, slot, f16_idesc(128, 128, false));  // both buffers
                    tc_commit(&bar->s_full[m][1], lead);
                } else {
#pragma unroll 1
                    for (int h = 0; h < 2 && 2 * j + h < s.steps; h++) {
                        ready(h);
                        scores(m, h, slot, f16_idesc(128, 64, false));
                    }
                }
                tc_commit(&bar->k_empty[slot], lead);
            } else if (lead) {
                mbar_arrive(&bar->k_empty[slot]);
            }
            __syncwarp();
        }
        tc_commit(&bar->q_empty, lead);
    }
}

// Warp 26 + m: the products O_m += P_m V.
__device__ __forceinline__ void issue_values(const ChunkAttnParams &p, unsigned char *sm, Bars *bar, uint32_t tm, int m) {
    const uint32_t base = smem_u32(sm), lead = (threadIdx.x & 31) == 0;
    uint32_t n = 0, ph = 0;       // value tiles; per buffer h: parity of the weights awaited
    auto wait = [&](uint64_t *b, uint32_t parity) { warp_await(b, parity & 1, &bar->stop, p.status); };
    for (At at(p); at.more();) {
        const Seg s = next_seg(p, at);
        const int tiles = s.k1 - s.k0, steps = s.narrow ? 2 * tiles : s.steps;
        bool acc = false;
        for (int j = 0; j < tiles; j++) {
            const uint32_t slot = n % kRing, vb = base + kOffV + slot * kTileBytes;
            wait(&bar->v_full[slot], n / kRing);
            n++;
            if (s.narrow ? (j & 1) == m : 128 * m < s.valid) {
                const bool packed = s.k0 + j < s.np;
                const uint32_t id = packed ? f16_idesc(128, 128, false) : f16_idesc(128, 128, true);
                const uint64_t b0 = packed ? smem_desc(vb, 16, 1024) : smem_desc(vb, 16384, 1024);
                const uint32_t step = (packed ? 32 : 2048) >> 4, half = (packed ? 16384 : 8192) >> 4;
#pragma unroll 1
                for (int h = 0; h < 2 && 2 * j + h < steps; h++) {
                    wait(&bar->p_full[m][h], ph >> h);
                    ph ^= 1u << h;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        mma_ts(tm + 256 + m * 128, tm + m * 128 + h * 64 + 8 * k, b0 + (h * half + k * step), id, acc || k > 0, lead);
                    acc = true;
                    tc_commit(&bar->pv_done[m][h], lead);
                }
                tc_commit(&bar->v_empty[slot], lead);
            } else if (lead) {
                mbar_arrive(&bar->v_empty[slot]);
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- groups 0, 1 ---------
// Scores of N keys: those from the n-th on are not seen.
template <int N>
__device__ __forceinline__ void mask_keys(uint32_t *x, int n) {
#pragma unroll
    for (int c = 0; c < N; c++)
        if (c >= n) x[c] = 0xff800000u;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <int N>
__device__ __forceinline__ float max_of(const float *f) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; e++) t[e] = f[e];
#pragma unroll
    for (int c = 8; c + 16 <= N; c += 16)
#pragma unroll
        for (int e = 0; e < 8; e++) t[e] = max3(t[e], f[c + 2 * e], f[c + 2 * e + 1]);
#pragma unroll
    for (int e = 0; e < 8; e++) t[e] = fmaxf(t[e], f[N - 8 + e]);
    return fmaxf(max3(t[0], t[1], t[2]), max3(max3(t[3], t[4], t[5]), t[6], t[7]));
}
// Weights of N scores to reference r, as N / 2 half2 in place; returns their sum.  FAR: r may
// be beyond kNear.
template <int N, bool FAR>
__device__ __forceinline__ float weights(uint32_t *x, float r) {
    uint64_t l0 = 0, l1 = 0;
    const float off = FAR ? kUp : __fmaf_rn(-r, kScale, kUp);
    const uint64_t sc2 = pair_of(kScale, kScale), of2 = pair_of(off, off), nr2 = pair_of(-r, -r);
    const float *f = reinterpret_cast<const float *>(x);
    auto exponents = [&](float x0, float x1) {
        uint64_t y = pair_of(x0, x1);
        if (FAR) y = add_pair(y, nr2);
        return of_pair(fma_pair(y, sc2, of2));
    };
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        float2 a = exponents(f[c], f[c + 1]), b = exponents(f[c + 2], f[c + 3]);
        a.x = ex2(a.x);
        a.y = ex2(a.y);
        b.x = ex2(b.x);
        b.y = ex2(b.y);
        l0 = add_pair(l0, pair_of(a.x, a.y));
        l1 = add_pair(l1, pair_of(b.x, b.y));
        x[c >> 1] = pack_half2(a.x, a.y);
        x[(c >> 1) + 1] = pack_half2(b.x, b.y);
    }
    const float2 ls = of_pair(add_pair(l0, l1));
    return ls.x + ls.y;
}

// Parities of a softmax group's barriers and the row's state.
struct RowState {
    uint32_t ns, given, no1;  // per buffer h: parity of the weights given, any given; narrow units joined
    float r, l;               // reference (-inf: none yet), sum of the weights
};
// Whether weights of this sum, formed with a near reference, stand; the reference that weights
// are formed with in any case.
__device__ __forceinline__ bool stands(float sum, float r) { return sum <= kMostSum && fabsf(r) <= kNear; }
__device__ __forceinline__ float some_ref(float r) { return r == -INFINITY ? 0.f : r; }

// N scores from column ts on, those of unseen keys (from the y-th on) as -inf.
template <int N>
__device__ __forceinline__ void load_scores(uint32_t *x, uint32_t ts, int y) {
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld32(x + c, ts + c);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < N; c += 16) tmem_tie16(x + c);
    if (y < N) mask_keys<N>(x, y);
}

// The steps of one segment for query tile or key parity m; narrow units: every second key
// tile.  ts, to: tensor memory of S_m and O_m; lim: fp16 tokens the row may see; any: whether
// the warp has rows at all.  The weights are formed with a reference r that some earlier
// step's maximum gave: their sum tells whether one of them may be too large for fp16, and
// only then the maximum is looked for and the weights are formed again (a maximum in every
// step: 1253 us against 1175).
template <bool NARROW>
__device__ __forceinline__ void softmax_steps(const ChunkAttnParams &p, Bars *bar, const Seg &s, RowState &st, uint32_t ts, uint32_t to,
                                              int m, int lim, bool any) {
    const int steps = NARROW ? 2 * ((s.k1 - s.k0 - m + 1) >> 1) : s.steps;
    float r = -INFINITY, l = 0.f;
    for (int i = 0; i < steps; i++) {
        const int h = i & 1, kt = s.k0 + (NARROW ? 2 * (i >> 1) + m : i >> 1);
        warp_await(&bar->s_full[m][h], (st.ns >> h) & 1, &bar->stop, p.status);
        if (any) {
            tc_fence_after();
            const int y = kt >= s.np ? lim - (kt - s.np) * kChunkKeys - 64 * h : 64;  // keys it may see
            uint32_t x[64];
            load_scores<64>(x, ts + 64 * h, y);
            float add = weights<64, false>(x, r);  // infinite or NaN without a reference
            if (__any_sync(0xffffffffu, !stands(add, r))) {
                load_scores<64>(x, ts + 64 * h, y);
                const float cand = max_of<64>(reinterpret_cast<const float *>(x));
                const bool grow = cand > r;
                const float corr = grow ? ex2((r - cand) * kScale) : 1.f;
                if (grow) r = cand;
                l *= corr;
                if (i > 0) {
                    // the step before was the last to write O
                    warp_await(&bar->pv_done[m][h ^ 1], (~st.ns >> (h ^ 1)) & 1, &bar->stop, p.status);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 8; c++) {
                        tmem_ld16(x, to + 16 * c);
                        tmem_wait_ld();
                        tmem_tie16(x);
#pragma unroll
                        for (int e = 0; e < 16; e++) x[e] = __float_as_uint(__uint_as_float(x[e]) * corr);
                        tmem_st16(to + 16 * c, x);
                    }
                }
                if (i > 0) load_scores<64>(x, ts + 64 * h, y);
                add = weights<64, true>(x, some_ref(r));
            }
            tmem_st32(ts + 64 * h, x);  // over the scores
            l += add;
            tmem_wait_st();
        }
        // a segment's first weights let their product overwrite O_1: once it has been read
        if (m == 1 && i == 0 && st.no1 > 0) warp_await(&bar->o1_free, (st.no1 - 1) & 1, &bar->stop, p.status);
        tc_fence_before();
        mbar_arrive(&bar->p_full[m][h]);
        st.ns ^= 1u << h;
        st.given |= 1u << h;
    }
    st.r = r;
    st.l = l;
}

// The key tiles of one segment of a narrow unit that holds its rows REP times: the thread's
// copy takes keys KEYS c .. of every tile, the other keys' weights in its lane are 0.
template <int REP>
__device__ __forceinline__ void softmax_tiles(const ChunkAttnParams &p, Bars *bar, const Seg &s, RowState &st, uint32_t ts, uint32_t to,
                                              int m, int lim, int c) {
    constexpr int KEYS = 128 / REP;
    float r = -INFINITY, l = 0.f;
    for (int kt = s.k0 + m; kt < s.k1; kt += 2) {
        warp_await(&bar->s_full[m][0], st.ns & 1, &bar->stop, p.status);
        warp_await(&bar->s_full[m][1], (st.ns >> 1) & 1, &bar->stop, p.status);
        tc_fence_after();
        const int y = kt >= s.np ? lim - (kt - s.np) * kChunkKeys - KEYS * c : KEYS;  // keys it may see
        uint32_t x[KEYS];
        load_scores<KEYS>(x, ts + KEYS * c, y);
        float add = weights<KEYS, false>(x, r);  // infinite or NaN without a reference
        if (__any_sync(0xffffffffu, !stands(add, r))) {
            load_scores<KEYS>(x, ts + KEYS * c, y);
            const float cand = max_of<KEYS>(reinterpret_cast<const float *>(x));
            const bool grow = cand > r;
            const float corr = grow ? ex2((r - cand) * kScale) : 1.f;
            if (grow) r = cand;
            l *= corr;
            if (kt > s.k0 + m) {  // the products before these scores have ended
#pragma unroll 1
                for (int e0 = 0; e0 < 128; e0 += 16) {
                    tmem_ld16(x, to + e0);
                    tmem_wait_ld();
                    tmem_tie16(x);
#pragma unroll
                    for (int e = 0; e < 16; e++) x[e] = __float_as_uint(__uint_as_float(x[e]) * corr);
                    tmem_st16(to + e0, x);
                }
                load_scores<KEYS>(x, ts + KEYS * c, y);
            }
            add = weights<KEYS, true>(x, some_ref(r));
        }
        l += add;
        // weights of keys 64 h .. at columns 64 h .., two to a column
        uint32_t zero[16];
#pragma unroll
        for (int e = 0; e < 16; e++) zero[e] = 0;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const uint32_t at = ts + 64 * (q >> 1) + 16 * (q & 1);
            if (q / (4 / REP) == c) tmem_st16(at, x + (q % (4 / REP)) * 16);
            else tmem_st16(at, zero);
        }
        tmem_wait_st();
        if (m == 1 && kt == s.k0 + m && st.no1 > 0) warp_await(&bar->o1_free, (st.no1 - 1) & 1, &bar->stop, p.status);
        tc_fence_before();
        mbar_arrive(&bar->p_full[m][0]);
        mbar_arrive(&bar->p_full[m][1]);
        st.ns ^= 3;
        st.given = 3;
    }
    st.r = r;
    st.l = l;
}

__device__ __forceinline__ void softmax(const ChunkAttnParams &p, Bars *bar, uint32_t tm, int m) {
    const int lane_row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(threadIdx.x & 96) << 16;
    const uint32_t ts = tm + lanes + m * 128, to = tm + lanes + 256 + m * 128;
    RowState st = {0, 0, 0, 0.f, 0.f};
    for (At at(p); at.more();) {
        const Seg s = next_seg(p, at);
        const bool last_first = s.k0 == 0 && s.it.first != p.begin[blockIdx.x];
        const int base = s.narrow ? 0 : 128 * m, row = s.rep > 1 ? lane_row & (128 / s.rep - 1) : base + lane_row;
        const int n = s.k1 - s.k0;
        if (base >= s.valid || (s.narrow && m >= n)) continue;
        const bool any = s.rep > 1 || base + (lane_row & 96) < s.valid;
        const int r = s.it.t * s.it.rows + min(row, s.valid - 1);
        const int lim = s.it.s.ns + s.it.s.nr + r / p.g + 1;
        const bool join = s.narrow && n > 1;
        if (s.rep == 4) softmax_tiles<4>(p, bar, s, st, ts, to, m, lim, lane_row >> 5);
        else if (s.rep == 2) softmax_tiles<2>(p, bar, s, st, ts, to, m, lim, lane_row >> 6);
        else if (s.narrow) softmax_steps<true>(p, bar, s, st, ts, to, m, lim, any);
        else softmax_steps<false>(p, bar, s, st, ts, to, m, lim, any);
        float ref = st.r, l = st.l;
        for (int h = 0; h < 2; h++)  // the last products
            if ((st.given >> h) & 1) warp_await(&bar->pv_done[m][h], (~st.ns >> h) & 1, &bar->stop, p.status);
        tc_fence_after();
        float a0 = 1.f, a1 = 0.f;
        // the range's first segment has slot 2 c, its last one (a unit that goes on) 2 c + 1
        const size_t slot0 = (2 * (size_t)blockIdx.x + (last_first ? 1 : 0)) * kRows;
        if (join) {  // O_1's states reach group 0 through the partial rows that its result goes to
            float2 *state1 = p.part_ml + slot0;
            st.no1++;
            if (m == 1) {
                state1[lane_row] = make_float2(ref, l);
                tc_fence_before();
                mbar_arrive(&bar->o1_full);
                continue;
            }
            warp_await(&bar->o1_full, (st.no1 - 1) & 1, &bar->stop, p.status);
            tc_fence_after();
            const float2 other = state1[lane_row];
            const float top = fmaxf(ref, other.x);
            a0 = ref == top ? 1.f : ex2((ref - top) * kScale);
            a1 = other.x == top ? 1.f : ex2((other.x - top) * kScale);
            ref = top;
            l = a0 * l + a1 * other.y;
        }
        const bool whole = s.k0 == 0 && s.k1 == s.it.n;
        // set before the tile's products; it stays set, as a group that has no rows in the segments
        // between may run any number of them ahead of the other
        const bool odd = *(volatile int *)&bar->odd;
        const float inv = 1.f / l;
        const bool mine = s.rep > 1 || row < s.valid;
        const size_t slot = slot0 + (s.rep > 1 ? lane_row : row);
        uint16_t *dst = p.out + ((int64_t)(s.it.s.cu + r / p.g) * p.H_kv * p.g + s.it.h * p.g + r % p.g) * kD;
        if (any) {
            if (!whole && mine) p.part_ml[slot] = make_float2(ref, l);
#pragma unroll 1
            for (int c = 0; c < 8; c++) {
                uint32_t o[16];
                float *f = reinterpret_cast<float *>(o);
                tmem_ld16(o, to + 16 * c);
                tmem_wait_ld();
                tmem_tie16(o);
                if (join) {
                    uint32_t o1[16];
                    tmem_ld16(o1, to + 128 + 16 * c);
                    tmem_wait_ld();
                    tmem_tie16(o1);
#pragma unroll
                    for (int e = 0; e < 16; e++) f[e] = a0 * f[e] + a1 * __uint_as_float(o1[e]);
                }
                if (odd)
                    for (int x = max(0, s.k0 - s.np) * kChunkKeys; x < min(lim, (s.k1 - s.np) * kChunkKeys); x++) {
                        if (s.rep > 1 && (x & 127) / (128 / s.rep) != lane_row / (128 / s.rep)) continue;  // another copy's key
                        const uint16_t *v = tail_row(p, s.it, x, true) + 16 * c;
#pragma unroll
                        for (int e = 0; e < 16; e++) {
                            const float y = h2f(v[e]);
                            if (!isfinite(y)) f[e] += y;
                        }
                    }
                if (mine) {
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
                            reinterpret_cast<float4 *>(p.part_o + slot * kD)[4 * c + e] =
                                make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        if (join) mbar_arrive(&bar->o1_free);
    }
}

__global__ void __launch_bounds__(kThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkAttnParams p) {
    extern __shared__ __align__(1024) unsigned char sm[];  // swizzle atoms are 1024 bytes
    Bars *bar = reinterpret_cast<Bars *>(sm + kOffBar);
    const int w = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    if (threadIdx.x == 0) {
        mbar_init(&bar->q_full, 128);
        mbar_init(&bar->q_empty, 2);
        for (int i = 0; i < kRing; i++) {
            mbar_init(&bar->k_full[i], 128);
            mbar_init(&bar->k_empty[i], 2);
            mbar_init(&bar->v_full[i], 128);
            mbar_init(&bar->v_empty[i], 2);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(i ? &bar->o1_free : &bar->o1_full, 128);
            for (int h = 0; h < 2; h++) {
                mbar_init(&bar->s_full[i][h], 1);
                mbar_init(&bar->p_full[i][h], 128);
                mbar_init(&bar->pv_done[i][h], 1);
            }
        }
        mbar_init(&bar->drain, 4);
        for (int i = 0; i < kMaxRaw; i++) {
            for (int par = 0; par < 2; par++) {
                mbar_init(&bar->rawk[par][i], 1);
                mbar_init(&bar->rawv[par][i], 1);
            }
            mbar_init(&bar->readk[i], 128);
            mbar_init(&bar->readv[i], 128);
        }
        bar->stop = 0;
        bar->odd = 0;
        fence_barrier_init();
    }
    if (w == 24) tmem_alloc(&bar->tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar->tmem;
    griddep_wait();
    if (w < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax(p, bar, tm, w >> 2);
    } else if (w < 24) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsTiles));
        produce(p, sm, bar, w >= 16, (w >> 2) & 1);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (w < 28) {
            if (w < 26) issue_scores(p, sm, bar, tm, w & 1);
            else issue_values(p, sm, bar, tm, w & 1);
            __syncwarp();
            tc_commit(&bar->drain, (threadIdx.x & 31) == 0);
            mbar_wait(&bar->drain, 0, p.status);  // every product has ended before the tensor memory is freed
        } else if (w < 30 && (threadIdx.x & 31) == 0) {
            bring(p, sm, bar, w == 29);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 24) tmem_free(tm);
}

}  // namespace

cudaError_t launch_chunk_combine(const ChunkAttnParams &p, cudaStream_t st);

cudaError_t launch_chunk_attn(const ChunkAttnParams &p, cudaStream_t st) {
    static bool ready[64];  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        e = cudaFuncSetAttribute(chunk_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    if ((e = launch_dependent(chunk_attn_kernel, dim3((unsigned)p.C), kThreads, kSmemBytes, st, p)) != cudaSuccess) return e;
    return p.cut ? launch_chunk_combine(p, st) : cudaSuccess;
}

}  // namespace kvq
