// Attention over a paged cache: how a call is divided, and its launch (cache_attention.h holds the kernel).
#include <cstdio>
#include <cstdlib>

#include "lowbit_internal.h"

namespace lowbit {

hipError_t launch_cache_attention_4(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);
hipError_t launch_cache_attention_8(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);
hipError_t launch_cache_attention_16(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);

namespace {
constexpr int kTileKeys = 32, kMostSplits = 64;
}

// may_split false: no workspace to split with.
CacheAttnPlan plan_cache_attention(const CacheAttnArgs& a, bool may_split) {
    CacheAttnPlan p{};
    const int64_t rows = int64_t(a.q_len) * a.group;
    p.share_tiles = rows > 32;
    p.tile_rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    if (getenv("CA_ROWS") && p.share_tiles) p.tile_rows = atoi(getenv("CA_ROWS"));
    p.row_tiles = int(tiles_of(rows, p.tile_rows));
    p.waves = p.share_tiles ? (p.tile_rows == 256 ? 8 : p.tile_rows == 64 ? 4 : getenv("CA_WAVES") ? atoi(getenv("CA_WAVES")) : 4) : getenv("CA_WAVES") ? atoi(getenv("CA_WAVES")) : 4;
    const int64_t groups = int64_t(a.batch) * a.cache.heads * p.row_tiles, tiles = tiles_of(a.kv_len, kTileKeys);
    int64_t splits = groups == 0 || !may_split ? 1 : kComputeUnits / groups;
    splits = splits < tiles / 12 ? splits : tiles / 12;
    splits = splits < kMostSplits ? splits : kMostSplits;
    p.splits = splits < 1 ? 1 : int(splits);
    if (getenv("CA_SPLITS") && may_split) { int v = atoi(getenv("CA_SPLITS")); if (v <= tiles) p.splits = v; }
    p.bytes = p.splits > 1 ? kWorkspaceCounterBytes + size_t(groups) * p.splits * p.tile_rows * (size_t(a.cache.head_dim) + 2) * 4u : 0;
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
                     (long long)(int64_t(a.row_tiles) * a.splits * a.cache.heads * a.batch), 64 * plan.waves, a.batch, a.q_len, a.kv_len, a.cache.heads * a.group, a.cache.heads, a.cache.head_dim, a.cache.bits, 1 << a.cache.page_shift,
                     a.tree != nullptr ? " tree" : "");
    return e;
}

}  // namespace lowbit
