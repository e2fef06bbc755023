// kvq_chunk.h -- parameter blocks and launchers of the chunk operators of the paged cache
// (kvq_chunk.cu, kvq_chunk_attn.cu); not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"

namespace kvq {

// One slot of a plan (kvq_chunk.desc).
struct ChunkSlot {
    int ns, T, nr, n_new;                // lengths before the chunk, new tokens
    int cu, to_sink, pk, page0;          // first row, tokens to the sink, tokens to pack, pages before
};

struct PlanParams {
    int32_t *cu, *slot, *pos, *desc, *table;
    const int32_t *lens, *new_pages;
    int B, S, R, G, table_stride;
    int n_tokens;
    int32_t n_new[KVQ_PAGED_MAX_B];
};

struct ExtendParams {
    const int32_t *desc;
    int32_t *lens, *status;
    const uint16_t *k_new, *v_new;
    int64_t k_stride, v_stride;
    uint16_t *k_sink, *v_sink, *k_res, *v_res;
    int32_t *k_codes, *v_codes;
    uint16_t *k_meta, *v_meta;
    const int32_t *ptab;
    int64_t n_pages;
    int B, H_kv, G, S, R, TV, ptab_stride;
    int n_pack;                          // pages to pack, over all slots
    int32_t page0[KVQ_PAGED_MAX_B + 1];  // of the slots before each
};

struct QkParams {
    const uint16_t *q, *k, *w_q, *w_k;
    const int32_t *pos;
    uint16_t *q_out, *k_out;
    int64_t n, q_stride, k_stride;
    int H_q, H_kv, rotary, halves, rotate;
    float eps;
    uint64_t turn[128];                  // base^(-2j/rotary) / (2 pi) in units of 2^-64 turns
};

constexpr int kNarrowRows = 128, kWideRows = 256, kNarrowCost = 3, kWideCost = 4, kUnitItems = 5, kCombineCost = 6, kPartItems = 2, kMaxRanges = 256;

// Chunk attention.  A unit is (slot, key head, tile of query rows): row r of a slot is its
// new token r / g under query head r % g of the key head's group.  Its items are key tiles
// of 128 tokens: the packed ones, then the fp16 tokens [sink | residual | chunk] up to the
// row tile's last query token.  A slot of at most kNarrowRows rows is one narrow unit per
// head, a slot of more consists of wide ones (kWideRows rows).  Positions count cost: an
// item's (kNarrowCost, kWideCost: a tile took 1.5 and 2.0 us) and, before a unit's first item,
// that of kUnitItems more (the start and the end of a unit).  Measured: a chunk of 517 tokens
// beside three decoding slots 131, 110, 98, 99 us with 0, 3, 5, 8 of them; a 2048-token chunk
// 915 us with equal costs of the items against 865, eight decoding slots 152 against 147.  All
// units, slot-major, then by head and row tile, are cut into C ranges, one per CTA: of equal
// cost, or, of few units, parts of one unit each.  A unit inside one range is finished there;
// of one that is cut, each range leaves fp32 partials, which the combine kernel joins in range
// order.
struct ChunkAttnParams {
    const int32_t *desc;
    const int32_t *ptab;
    const int32_t *k_codes, *v_codes;
    const uint16_t *k_meta, *v_meta;
    const uint16_t *k_sink, *v_sink, *k_res, *v_res;
    const uint16_t *q, *k_new, *v_new;
    uint16_t *out;
    float *part_o;                       // [2 C][kWideRows][128]
    float2 *part_ml;                     // [2 C][kWideRows] (reference: a score before the scale, sum)
    int32_t *status;
    int64_t q_stride, k_stride, v_stride, n_pages;
    int B, H_kv, g, G, kbits, vbits, S, R, ptab_stride;
    int cost, C, cut;                    // of all units; ranges; whether a unit lies in several
    int narrow, wide;                    // most rows of a narrow unit (0: there is none); whether there are wide units
    int32_t cost0[KVQ_PAGED_MAX_B + 1];  // position of each slot's first unit
    int32_t begin[kMaxRanges + 1];       // first position of each range, that of an item; begin[C] = cost
    int32_t first[kMaxRanges], tile[kMaxRanges];  // the unit it lies in: first position, row tile
};

cudaError_t launch_plan(const PlanParams &p, cudaStream_t st);
cudaError_t launch_extend(const ExtendParams &p, int kbits, int vbits, cudaStream_t st);
cudaError_t launch_qk(const QkParams &p, int D, cudaStream_t st);
cudaError_t launch_chunk_attn(const ChunkAttnParams &p, cudaStream_t st);

__host__ __device__ inline bool chunk_narrow(int n_new, int g) { return (int64_t)n_new * g <= kNarrowRows; }
// Copies of a narrow unit's rows in its query tile.
__host__ __device__ inline int chunk_copies(int rows) { return rows > 64 ? 1 : rows > 32 ? 2 : 4; }

// Launches a kernel that may start before the kernel before it in the stream has ended; it
// calls griddep_wait before it touches anything that one writes.
template <typename K, typename... A>
inline cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = (size_t)smem;
    lc.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, kernel, args...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

constexpr int kChunkKeys = 128;          // tokens per key tile

// Key tiles of row tile t of a slot (rows query rows per tile, g per token).
__host__ __device__ inline int chunk_tiles(const ChunkSlot &s, int t, int rows, int g) {
    const int last = ((t + 1) * rows - 1) / g + 1;                 // new tokens up to the tile's last
    const int seen = s.ns + s.nr + (last < s.n_new ? last : s.n_new);
    return s.T / kChunkKeys + (seen + kChunkKeys - 1) / kChunkKeys;
}

}  // namespace kvq
