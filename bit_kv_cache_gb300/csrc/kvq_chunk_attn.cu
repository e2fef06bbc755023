// kvq_chunk_attn.cu -- attention of a chunk of new tokens over the paged low-bit cache.
//
// For query row r of a unit (see ChunkAttnParams) and key t of its slot,
//   s_t = q . (code_t * scale + min) / sqrt(D),   out = sum_t softmax(s)_t v_t,
// in one pass over the keys with a running maximum and sum per row.  A CTA takes a range
// of the items of all units; each item is a tile of 128 keys, dequantized once into shared
// memory as fp16 (one rounding of code * scale + min) and used by all of the unit's rows.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_chunk_attn.cuh"

namespace kvq {

namespace {

// ------------------------------------------------------------------------------
// 64 query rows per CTA, 16 per warp; mma.sync on fp16 tiles in shared memory.
// ------------------------------------------------------------------------------
constexpr int kRows = 64, kPitch = kD + 8;  // halves per shared-memory row: ldmatrix without bank conflicts

__global__ void __launch_bounds__(128) chunk_attn_kernel(const __grid_constant__ ChunkAttnParams p) {
    extern __shared__ __align__(16) uint16_t smem[];
    uint16_t *ks = smem, *vs = smem + kChunkKeys * kPitch;
    __shared__ int s_odd;                     // the tile holds values that are not finite
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const float scale = kLog2e * 0.08838834764831845f;  // log2(e) / sqrt(128)
    const int begin = range_begin(blockIdx.x, p.n_items, p.C), end = range_begin(blockIdx.x + 1, p.n_items, p.C);
    for (int at = begin; at < end;) {
        const Item it = find_item(p, at, kRows);
        const int k0 = at - it.first, k1 = min(it.n, end - it.first);
        const int valid = min(kRows, it.s.n_new * p.g - it.t * kRows);
        const int np = it.s.T / kChunkKeys, ntail = it.s.ns + it.s.nr + it.s.n_new;
        int row[2], lim[2];                   // this thread's rows; fp16 tokens each may see
#pragma unroll
        for (int i = 0; i < 2; i++) {
            row[i] = 16 * w + (lane >> 2) + 8 * i;
            const int r = it.t * kRows + min(row[i], valid - 1);
            lim[i] = it.s.ns + it.s.nr + r / p.g + 1;
        }
        uint32_t qf[8][4];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int r = it.t * kRows + min(row[i], valid - 1);
            const uint16_t *src = p.q + (int64_t)(it.s.cu + r / p.g) * p.q_stride + (it.h * p.g + r % p.g) * kD + 2 * (lane & 3);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                qf[k][i] = *reinterpret_cast<const uint32_t *>(src + 16 * k);
                qf[k][2 + i] = *reinterpret_cast<const uint32_t *>(src + 16 * k + 8);
            }
        }
        float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < 16; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[n][e] = 0.f;
        bool odd = false;
        for (int kt = k0; kt < k1; kt++) {
            __syncthreads();
            if (kt < np) {
                const int64_t page = page_of(p, it, kt);
                const int t0 = kt * kChunkKeys % p.G;
                const int fk = 32 / p.kbits, fv = 32 / p.vbits, TV = 256 / p.kbits;
                {  // keys: thread = channel
                    const int32_t *src = p.k_codes + ((size_t)page * p.G + t0) / fk * kD;
                    const float2 sm = unpack_half2(reinterpret_cast<const uint32_t *>(p.k_meta)[(size_t)page * kD + tid]);
                    for (int r = 0; r < kChunkKeys / fk; r++) {
                        uint32_t wd = (uint32_t)src[(size_t)r * kD + kword_pos(tid, t0 / fk + r)];
                        for (int j = 0; j < fk; j++, wd >>= p.kbits)
                            ks[(r * fk + j) * kPitch + tid] =
                                __half_as_ushort(__float2half_rn(fmaf((float)(wd & ((1u << p.kbits) - 1)), sm.x, sm.y)));
                    }
                }
                {  // values: thread = token
                    const int tt = t0 + tid, j0 = tt % TV;
                    const int32_t *src = p.v_codes + (size_t)page * p.G * (kD / fv) + (size_t)(tt / TV) * (kD / fv) * TV;
                    const float2 sm = unpack_half2(reinterpret_cast<const uint32_t *>(p.v_meta)[(size_t)page * p.G + tt]);
                    for (int r = 0; r < kD / fv; r++) {
                        uint32_t wd = (uint32_t)src[r * TV + vword_pos(j0, r, TV)];
                        for (int j = 0; j < fv; j++, wd >>= p.vbits)
                            vs[tid * kPitch + r * fv + j] =
                                __half_as_ushort(__float2half_rn(fmaf((float)(wd & ((1u << p.vbits) - 1)), sm.x, sm.y)));
                    }
                }
                __syncthreads();
            } else {
                if (tid == 0) s_odd = 0;
                __syncthreads();
                bool bad = false;
                for (int i = tid; i < kChunkKeys * 16; i += 128) {
                    const int x = (kt - np) * kChunkKeys + (i >> 4), c = i & 15;
                    uint4 a = make_uint4(0, 0, 0, 0), b = a;
                    if (x < ntail) {
                        a = reinterpret_cast<const uint4 *>(tail_row(p, it, x, false))[c];
                        b = reinterpret_cast<const uint4 *>(tail_row(p, it, x, true))[c];
                        // a value that is not finite would reach rows that may not see it (0 * inf):
                        // it enters the product as 0 and is added to its rows at the end
                        uint32_t *v = reinterpret_cast<uint32_t *>(&b);
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            if ((v[e] & 0x7c00u) == 0x7c00u) v[e] &= 0xffff0000u, bad = true;
                            if ((v[e] & 0x7c000000u) == 0x7c000000u) v[e] &= 0xffffu, bad = true;
                        }
                    }
                    *reinterpret_cast<uint4 *>(ks + (i >> 4) * kPitch + 8 * c) = a;
                    *reinterpret_cast<uint4 *>(vs + (i >> 4) * kPitch + 8 * c) = b;
                }
                if (bad) s_odd = 1;
                __syncthreads();
                odd |= s_odd != 0;
            }
            // s = q k^T: 16 rows x 128 keys
            float s[16][4];
#pragma unroll
            for (int n = 0; n < 16; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) s[n][e] = 0.f;
#pragma unroll
            for (int n = 0; n < 16; n++)
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    uint32_t b[4];
                    ldmatrix_x4(b, smem_u32(ks + (8 * n + (lane & 7)) * kPitch + 16 * k + 8 * (lane >> 3)));
                    mma_16816(s[n], qf[k][0], qf[k][1], qf[k][2], qf[k][3], b[0], b[1]);
                    mma_16816(s[n], qf[k + 1][0], qf[k + 1][1], qf[k + 1][2], qf[k + 1][3], b[2], b[3]);
                }
            if (kt >= np) {
                const int x0 = (kt - np) * kChunkKeys + 2 * (lane & 3);
#pragma unroll
                for (int n = 0; n < 16; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (x0 + 8 * n + (e & 1) >= lim[e >> 1]) s[n][e] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                float mx = -INFINITY;
#pragma unroll
                for (int n = 0; n < 16; n++) mx = fmaxf(mx, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[i], mx * scale);
                const float base = mn == -INFINITY ? 0.f : mn;  // a row that sees nothing yet keeps sum 0
                const float corr = exp2f(m[i] - base);
                m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 16; n++)
#pragma unroll
                    for (int e = 2 * i; e < 2 * i + 2; e++) {
                        s[n][e] = exp2f(fmaf(s[n][e], scale, -base));
                        sum += s[n][e];
                    }
                l[i] = l[i] * corr + sum;
#pragma unroll
                for (int n = 0; n < 16; n++) {
                    o[n][2 * i] *= corr;
                    o[n][2 * i + 1] *= corr;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const uint32_t a0 = pack_half2(s[2 * k][0], s[2 * k][1]), a1 = pack_half2(s[2 * k][2], s[2 * k][3]);
                const uint32_t a2 = pack_half2(s[2 * k + 1][0], s[2 * k + 1][1]), a3 = pack_half2(s[2 * k + 1][2], s[2 * k + 1][3]);
#pragma unroll
                for (int n = 0; n < 16; n += 2) {
                    uint32_t b[4];
                    ldmatrix_x4_trans(b, smem_u32(vs + (16 * k + (lane & 15)) * kPitch + 8 * n + 8 * (lane >> 4)));
                    mma_16816(o[n], a0, a1, a2, a3, b[0], b[1]);
                    mma_16816(o[n + 1], a0, a1, a2, a3, b[2], b[3]);
                }
            }
        }
        const bool whole = k0 == 0 && k1 == it.n;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        if (odd) {  // values that are not finite, in the tail tiles of this range
            for (int i = 0; i < 2; i++)
                for (int x = max(0, k0 - np) * kChunkKeys; x < min(lim[i], (k1 - np) * kChunkKeys); x++) {
                    const uint16_t *v = tail_row(p, it, x, true);
#pragma unroll
                    for (int n = 0; n < 16; n++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const float f = h2f(v[8 * n + 2 * (lane & 3) + e]);
                            if (!isfinite(f)) o[n][2 * i + e] += f;
                        }
                }
        }
        // the range's first segment has slot 2 c, its last one (a unit that goes on) 2 c + 1
        const size_t slot = 2 * (size_t)blockIdx.x + (k0 == 0 && at != begin ? 1 : 0);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (row[i] >= valid) continue;
            if (whole) {
                const float inv = 1.0f / l[i];
                const int r = it.t * kRows + row[i];
                uint16_t *dst = p.out + ((int64_t)(it.s.cu + r / p.g) * p.H_kv * p.g + it.h * p.g + r % p.g) * kD + 2 * (lane & 3);
#pragma unroll
                for (int n = 0; n < 16; n++)
                    *reinterpret_cast<uint32_t *>(dst + 8 * n) = pack_half2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
            } else {
                if ((lane & 3) == 0) p.part_ml[slot * kRows + row[i]] = make_float2(m[i], l[i]);
                float *dst = p.part_o + (slot * kRows + row[i]) * kD + 2 * (lane & 3);
#pragma unroll
                for (int n = 0; n < 16; n++) *reinterpret_cast<float2 *>(dst + 8 * n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
            }
        }
        at = it.first + k1;
    }
}

// Joins the partials of the unit that boundary x between two ranges cuts, if it is the
// unit's first: 8 rows per CTA, a warp each.  Ranges are joined in order, so the result
// does not depend on timing.
__global__ void __launch_bounds__(256) chunk_combine_kernel(const __grid_constant__ ChunkAttnParams p, int rows) {
    const int c0 = blockIdx.x, cut = range_begin(c0 + 1, p.n_items, p.C), begin = range_begin(c0, p.n_items, p.C);
    const Item it = find_item(p, cut, rows);
    if (it.first == cut || (it.first < begin)) return;  // not cut here, or cut before
    const int c1 = range_of(it.first + it.n - 1, p.n_items, p.C);
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= min(rows, it.s.n_new * p.g - it.t * rows)) return;
    const size_t s0 = 2 * (size_t)c0 + (it.first == begin ? 0 : 1);
    float m = -INFINITY;
    for (int c = c0; c <= c1; c++) m = fmaxf(m, p.part_ml[(c == c0 ? s0 : 2 * (size_t)c) * rows + row].x);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; c++) {
        const size_t s = (c == c0 ? s0 : 2 * (size_t)c) * rows + row;
        const float2 ml = p.part_ml[s];
        const float wgt = ml.x == -INFINITY && m != -INFINITY ? 0.f : exp2f(ml.x - m);
        const float4 v = reinterpret_cast<const float4 *>(p.part_o + s * kD)[lane];
        l += wgt * ml.y;
        o.x += wgt * v.x;
        o.y += wgt * v.y;
        o.z += wgt * v.z;
        o.w += wgt * v.w;
    }
    const float inv = 1.0f / l;
    const int r = it.t * rows + row;
    uint16_t *dst = p.out + ((int64_t)(it.s.cu + r / p.g) * p.H_kv * p.g + it.h * p.g + r % p.g) * kD;
    reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(pack_half2(o.x * inv, o.y * inv), pack_half2(o.z * inv, o.w * inv));
}

}  // namespace

cudaError_t launch_chunk_attn(const ChunkAttnParams &p, int rows, cudaStream_t st) {
    cudaError_t e;
    if (rows == kWideRows) {
        if ((e = launch_chunk_wide(p, st)) != cudaSuccess) return e;
    } else {
        const int smem = 2 * kChunkKeys * kPitch * 2;
        e = cudaFuncSetAttribute(chunk_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        chunk_attn_kernel<<<p.C, 128, smem, st>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (p.C > 1) {
        chunk_combine_kernel<<<dim3((unsigned)(p.C - 1), (unsigned)(rows / 8)), 256, 0, st>>>(p, rows);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace kvq
