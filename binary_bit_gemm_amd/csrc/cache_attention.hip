// Attention over a paged cache: how a call is divided, and its launch (cache_attention.h holds the kernel).
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/lowbit.h"
#include "decode_internal.h"

namespace lowbit {

hipError_t launch_cache_attention_4(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);
hipError_t launch_cache_attention_8(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);
hipError_t launch_cache_attention_16(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);

namespace {

constexpr int kTileKeys = 32;
constexpr int64_t kMostSplits = 64;
// Split workgroups are at most one a compute unit, of 128 rows, or (4 bits) two of 16.
static_assert(LOWBIT_CACHE_ATTENTION_WORKSPACE_BYTES == kWorkspaceCounterBytes + kComputeUnits * 128 * (128 + 2) * 4, "the largest plan");

// Up to 16 rows: one workgroup per compute unit at most, of four tiles of 32 keys at least (a tile a wave; 16 bits, whose tiles are larger:
// two), and past 12 ranges (24) of eight (four), since a join costs about 2 us: none below 16 tiles.  Measured, one token, 8 kv heads of 128, 8 bits
// (us by ranges): 700 keys 1: 8.7, 6: 8.2; 1500 keys 3: 10.1, 12: 8.7, 16: 9.0; 3000 keys 7: 10.2, 12: 9.4, 32: 10.6; 16 bits 1500 keys 3: 12.3, 24: 9.4.
// Ranges come in whole numbers per unit, so past half as many groups as units keys are not split, and units are left over: with 8 kv heads 16 requests
// over 16,000 keys take 93 us in 8 bits (178 in 16, 54 in 4), 17 take 135 (202, 66), 32 take 175 (340, 109); over 4000 25, 29 and 40.
int64_t few_splits(int64_t groups, int64_t tiles, int bits) {
    if (tiles < 16) return 1;
    const int64_t least = bits == 16 ? 2 : 4, small = bits == 16 ? 24 : 12;
    int64_t splits = kComputeUnits / groups;
    // two on a unit at 4 bits, which keep vector units busier than memory, where ranges stay long and few: 16 requests of 6000 keys 30.1 us, 24.8
    // with two; 8 of 4000 15.8, 14.5; one of 40,000 19.2, 19.5; at 8 bits 16 of 6000 33.7, 35.2
    if (bits == 4 && splits <= 8 && tiles >= 28 * (splits < 1 ? 1 : splits)) splits = 2 * kComputeUnits / groups;
    splits = splits < tiles / least ? splits : tiles / least;
    const int64_t most = tiles / (2 * least) > small ? tiles / (2 * least) : small;
    return splits < most ? splits : most;
}

// Many rows: one workgroup per compute unit at most, of two tiles at least, where that takes eight tiles or more off each; otherwise the join (3.5 us
// and the parts' way through memory) costs more than it saves.  Measured, trees of 12 over 300 keys, 8 kv heads of 128, 8 bits, 64 rows (us by ranges) 1:
// 12.9, 5: 10.2; of 64 over 4000 keys 2: 46, 4: 28, 8: 19.9.  The same whole numbers: trees of 16 over 4000 keys, 64 rows a tile, 16 requests 50 us, 17 80.
int64_t many_splits(int64_t groups, int64_t tiles) {
    int64_t splits = kComputeUnits / groups;
    splits = splits < tiles / 2 ? splits : tiles / 2;
    splits = splits < kMostSplits ? splits : kMostSplits;
    return splits > 1 && tiles - tiles_of(tiles, splits) >= 8 ? splits : 1;
}

}  // namespace

// may_split false: no workspace to split with.
//   LOWBIT_CACHE_ATTENTION=few|many32|many64|many128 in the environment forces the kernel (A/B runs and tests).
CacheAttnPlan plan_cache_attention(const CacheAttnArgs& a, bool may_split) {
    CacheAttnPlan p{};
    const int64_t rows = int64_t(a.q_len) * a.group, heads = int64_t(a.batch) * a.cache.heads, tiles = tiles_of(a.kv_len, kTileKeys);
    const int64_t few_groups = heads * tiles_of(rows, 16);
    const int64_t few = may_split && few_groups > 0 ? few_splits(few_groups, tiles, a.cache.bits) : 1;
    // Up to 16 rows the kernel that feeds registers from memory starts and ends sooner and keeps more loads in flight; the one that shares tiles joins
    // many ranges of many rows faster (a workgroup per four rows, not one for all).  Measured (us, few / many with 32 rows), 8 kv heads of 128: 8 bits,
    // 4 rows over 16,000 keys 13.0 / 16.2, 32 requests of 4 rows over 4000 40 / 51; 16 bits, 4 rows over 1500 keys 9.3 / 10.9, over 40,000 30.6 / 32.0, 16
    // over 2000 13.6 / 12.0, 12 over 16,000 21.0 / 20.6.  At 8 bits the two are close with more than 8 rows: 16 over 2000 10.8 / 11.4, 12 over 16,000
    // 16.6 / 17.1.
    // Over short caches (32 tiles) it also takes more rows, 16 to a workgroup, up to two workgroups a unit: 64 rows over 300 keys 7.3 / 10.8, 256
    // rows 7.4 / 11.4; four requests of 108 rows over 1000 keys 10.8 / 15.7; 16 of 108 over 300, 896 workgroups, 17.2 / 13.8.  Past that the two are
    // within 10% of each other up to 2000 keys.
    p.share_tiles = rows > 16 ? tiles > 32 || few_groups > 2 * kComputeUnits : rows > 8 && few > 8;
    int only = 0;
    if (const char* force = std::getenv("LOWBIT_CACHE_ATTENTION")) {
        if (std::strcmp(force, "few") == 0) p.share_tiles = false;
        for (const int r : {32, 64, 128})
            if (std::strncmp(force, "many", 4) == 0 && std::atoi(force + 4) == r) {
                p.share_tiles = true;
                only = r;
            }
    }
    int64_t splits = 1;
    if (!p.share_tiles) {
        p.tile_rows = 16;
        splits = few;
    } else {
        // 128 rows of a workgroup read a tile from LDS for twice the rows; 64 start and end sooner: 128 where 64 would have more than 20 tiles.
        // Measured (64 / 128 rows, us; 8 kv heads of 128, 8 bits; in brackets tiles of a workgroup of 64): 64 tokens, one request of 4000 keys
        // [16] 19.9 / 21.5, four of 1000 [16] 22.8 / 24.3, four of 4000 [63] 50 / 43; 27 tokens in 4 bits, heads of 64, three of 8191 [26] 21.9 / 20.8.
        p.tile_rows = only == 32 || (only == 0 && rows <= 32) ? 32 : 64;
        const int64_t groups = heads * tiles_of(rows, p.tile_rows);
        splits = may_split && groups > 0 ? many_splits(groups, tiles) : 1;
        if (only != 0 ? only == 128 : rows > 64 && tiles_of(tiles, splits) > 20) {
            p.tile_rows = 128;
            splits = may_split && groups > 0 ? many_splits(heads * tiles_of(rows, 128), tiles) : 1;
        }
    }
    p.row_tiles = int(tiles_of(rows, p.tile_rows));
    p.splits = splits < 1 ? 1 : splits < kMostSplits ? int(splits) : int(kMostSplits);
    const int64_t parts = heads * p.row_tiles * p.splits * p.tile_rows;
    p.bytes = p.splits > 1 ? kWorkspaceCounterBytes + size_t(parts) * (size_t(a.cache.head_dim) + 2) * 4u : 0;
    return p;
}

hipError_t launch_cache_attention(CacheAttnArgs a, const CacheAttnPlan& plan, void* workspace, hipStream_t stream) {
    a.row_tiles = plan.row_tiles;
    a.splits = plan.splits;
    a.counters = static_cast<uint32_t*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kWorkspaceCounterBytes);
    const hipError_t e = a.cache.bits == 4   ? launch_cache_attention_4(a, plan, stream)
                         : a.cache.bits == 8 ? launch_cache_attention_8(a, plan, stream)
                                             : launch_cache_attention_16(a, plan, stream);
    if (e == hipSuccess && trace_enabled())
        std::fprintf(stderr, "lowbit: cache_attention %s rows=%d splits=%d grid=%lld block=%d problem=%dx%dx%dx%d kv_heads=%d dim=%d bits=%d page=%d%s\n",
                     plan.share_tiles ? "many" : "few", plan.tile_rows, a.splits,
                     (long long)(int64_t(a.row_tiles) * a.splits * a.cache.heads * a.batch), plan.share_tiles ? 512 : 256, a.batch, a.q_len, a.kv_len, a.cache.heads * a.group, a.cache.heads, a.cache.head_dim, a.cache.bits, 1 << a.cache.page_shift,
                     a.tree != nullptr ? " tree" : "");
    return e;
}

}  // namespace lowbit
