// kvq_block.h -- parameter blocks and launchers of the 8-bit caches with one scale per page and
// head (kvq_block.cu, kvq_block_decode.cu); not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_chunk.h"

namespace kvq {

// A planned chunk's pages, with what a page's CTA has to know of its slot: residual tokens before the
// chunk, the chunk row behind them (as if the residual had come from the chunk), first logical page.
struct BlockExtendParams : ExtendParams {
    int32_t nr[KVQ_PAGED_MAX_B], row0[KVQ_PAGED_MAX_B], lp0[KVQ_PAGED_MAX_B];
};

// Pages of listed slots: page i of the call is page i % per of slot seq[i / per], and logical page
// lp0[i / per] + i % per there.  Its rows are the residual's, whose lengths then become T + R and 0
// (residual), or those of k_new, v_new from row row0 on; heads lie h_stride apart there.
struct BlockListParams : PackParams {
    int64_t h_stride;
    int n_pack, per, row0, residual;
    int16_t seq[KVQ_PAGED_MAX_B];
    int32_t lp0[KVQ_PAGED_MAX_B];
};

// Attention of at most kFewRows rows (new tokens times query heads) per key head of a slot.  A CTA
// is (key head, part of a slot): the slot's items, packed tiles of 64 tokens and then 16-token tiles
// of the fp16 tokens [sink | residual | new ones], are cut into equal parts.  8 slots of 17K to 56K
// tokens with 32 rows each take 126 us, with 36 rows, which go to the tensor-memory kernel, 188.
// Beside slots of more rows it runs as a launch of its own from a number of tiles, of 128 tokens and
// heads, on.  Us, with a launch of its own against one kernel for all, beside a slot of 40, of 517 and
// of 2000 new tokens (4 heads a key head):
//   slots of 4 rows:  2288 tiles (517 new tokens) 88 and 87; 5584 tiles 75 and 74, 107 and 114, 504 and
//                     500; 6632 tiles 78 and 86, 112 and 126, 236 and 261; 15984 tiles 122 and 170, 158
//                     and 215, 283 and 357 (16 rows: 4056 tiles, 517 tokens 101 and 89, else the same);
//   slots of 32 rows: 6632 tiles 97 and 88, 131 and 130, 256 and 268; 8688 tiles 108 and 110, 140 and
//                     154, 266 and 296; 15984 tiles 154 and 179, 186 and 224, 312 and 364.
constexpr int kFewRows = 32, kFewTiles = 5120, kFewTiles32 = 8192;  // kFewTiles32: of more than 16 rows
struct BlockDecodeParams {
    const uint16_t *q, *k_new, *v_new;   // new rows of a chunk (decode: none, the cache holds the token)
    int64_t q_stride, k_stride, v_stride;
    uint16_t *out;
    const uint8_t *k_codes, *v_codes;
    const float4 *k_scale, *v_scale;     // a page's scale in the first component
    const uint16_t *k_sink, *v_sink, *k_res, *v_res;
    const int32_t *ptab, *lens, *desc;   // desc: of a plan (null: lens, one row per query head)
    float *part_o;                       // [parts][H_kv][most_rows][128], of slots in several parts
    float2 *part_ml;                     // [parts][H_kv][most_rows]
    int32_t *status;
    int64_t n_pages;
    int H_kv, g, g_shift, S, R, ptab_stride;  // g_shift: log2(G)
    int most_rows;                       // of a slot
    int n_slots;                         // of the call
    int16_t slot[KVQ_PAGED_MAX_B];       // those
    int32_t part0[KVQ_PAGED_MAX_B + 1];  // parts of the ones before each
};

cudaError_t launch_block_extend(const ExtendParams &p, const ChunkSlot *slots, bool e4m3, cudaStream_t st);
cudaError_t launch_block_list(const BlockListParams &p, bool e4m3, cudaStream_t st);
size_t block_decode_ws_bytes(const kvq_config *c);
int block_decode(const kvq_config *c, const kvq_paged *pc, const uint16_t *q, uint16_t *out, void *ws, size_t ws_bytes,
                 cudaStream_t st);
// The chunk attention of the slots few[]; inputs, output and partials as of `a`.
int block_chunk_few(const kvq_config *c, const kvq_paged *pc, const ChunkSlot *slots, const bool *few, const ChunkAttnParams &a,
                    cudaStream_t st);

}  // namespace kvq
