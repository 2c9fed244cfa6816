// Arguments and launches of the decoding operators: the paged cache, attention over it, matrix-vector products.
#pragma once

#include "lowbit_internal.h"

namespace lowbit {

// The paged cache of keys and values (kv_cache.h says how it lies).
struct CacheArgs {
    unsigned char *k, *v, *k_scales, *v_scales;  // scales null at 16 bits
    int pages, page_shift, heads, head_dim, bits;
};
// Rows that go into it or come back (kv_cache.hip): [tokens, heads, head_dim], strides in elements.
struct CacheRows {
    const uint16_t *k, *v;    // written
    uint16_t *k_out, *v_out;  // read back
    const int32_t* slots;     // [tokens]: page * page_size + place in it; outside the cache: none
    int64_t tokens, k_token, k_head, v_token, v_head;
};
hipError_t launch_cache_rows(const CacheArgs& c, const CacheRows& r, bool write, hipStream_t stream);

// Attention over it (cache_attention.hip).
struct CacheAttnArgs {
    CacheArgs cache;
    const uint16_t* q;
    uint16_t* o;
    const int32_t* table;   // [batch, table_stride]: page of each page_size keys
    const int32_t* lens;    // [batch]: keys, the new tokens' among them
    const int32_t* q_lens;  // [batch], null: q_len
    const uint64_t* tree;   // [batch, q_len]: which new tokens each takes, null: those up to itself
    int64_t q_batch, q_token, q_head, o_batch, o_token, o_head, table_stride;
    int batch, q_len, kv_len, group;
    float scale_log2;  // scale * log2(e)
    // set by the launch
    int row_tiles, splits;
    uint32_t* counters;  // arrivals of the splits, zero between calls
    float* part;
};
struct CacheAttnPlan {
    bool share_tiles;  // tiles go through LDS, for several waves' rows ("many"); otherwise straight into registers ("few")
    int tile_rows;     // of a workgroup: 16 (few), 32, 64 or 128 (many)
    int row_tiles, splits;
    size_t bytes;  // of workspace (0: none)
};
CacheAttnPlan plan_cache_attention(const CacheAttnArgs& a, bool may_split = true);
hipError_t launch_cache_attention(CacheAttnArgs a, const CacheAttnPlan& plan, void* workspace, hipStream_t stream);

// Matrix-vector products with affine 4-bit weights (gemv_affine.hip), up to 16 rows.
constexpr int kGemvMaxRows = 16;
struct GemvArgs {
    const uint16_t* X;      // bf16 [M, K]
    const uint32_t* W;      // levels [N or 2N, K / 8]
    const uint16_t *S, *B;  // fp16 [N or 2N, K / g]
    const uint16_t* R;      // bf16 [M, N] residual, null: none
    uint16_t* Y;            // bf16 [M, N]
    int M, N, K;
};
hipError_t launch_gemv_affine(const GemvArgs& a, int g, bool swiglu, hipStream_t stream);

}  // namespace lowbit
