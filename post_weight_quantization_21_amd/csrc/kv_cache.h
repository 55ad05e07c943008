// A key/value cache held in 4 bits, as the kernels that fill it (kv_append.hip),
// read it (kv_attention.hip) and thin it out (kv_evict.hip) see it.
//
// A pool of pages; per page and kv head, D values a token in NG groups:
//   k  [page][D/8] words: word b D/32 + t holds dims 32 t + 8 b + e, dim e at bits
//      4 (e / 2 + 4 (e % 2)).  A lane of a matrix instruction's key operand (lane row b,
//      step t) then reads its words next to each other.
//   v  [page/8][D/4][8] 16-bit units: unit 16 u + m of token 8 i + r holds dims
//      64 u + 16 j + m at bits 4 j.  Sixteen bytes are the eight tokens that a lane of
//      the value operand multiplies, for four dims, and a token's bits are its own.
//   k_grid, v_grid  [NG][page] words: the scale s as bf16 above, 8 - z as fp16 below;
//      a value is s ((q - 8) + (8 - z)), and q - 8 needs no grid.
//   weight  [page] fp32, or NULL
#pragma once

#include "common.h"

namespace gptq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct KvPool {
    uint32_t *k;
    uint16_t *v;
    uint32_t *k_grid, *v_grid;
    float *weight;
    int32_t pages, heads, lg_page, groups;  // pages of the pool, kv heads, log2 of a page's tokens, groups of a head

    __device__ __forceinline__ int page() const { return 1 << lg_page; }
    // The first token of a head's share of a page, counted over the pool.
    __device__ __forceinline__ int64_t first(int page_id, int head) const {
        return ((int64_t)page_id * heads + head) << lg_page;
    }
};

// Pages of the sequences: `width` entries a row, lengths in tokens.
struct KvSeqs {
    const int32_t *table, *lens;
    int32_t n, width;
    int64_t capacity;  // tokens that a sequence can have: max_len, or the table's

    __device__ __forceinline__ int len(int b) const {
        const int l = lens[b];
        return l < 0 ? 0 : (l < capacity ? l : (int)capacity);
    }
    // The page of a row's token, or -1 where the entry names none.
    __device__ __forceinline__ int page_of(const KvPool &pool, const int32_t *row, int slot) const {
        const int id = row[slot >> pool.lg_page];
        return (uint32_t)id < (uint32_t)pool.pages ? id : -1;
    }
};

__device__ __forceinline__ float grid_scale_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The inclusive sum over the lanes up to this one, by DPP row shifts and broadcasts.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 into rows 2 and 3
    return v;
}

KvPool kv_pool(const gptq_kv_cache &c);

}  // namespace gptq
