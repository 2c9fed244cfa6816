// Attention over a paged cache: how a call is divided, and its launch (cache_attention.h holds the kernel).
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "lowbit_internal.h"

namespace lowbit {

hipError_t launch_cache_attention_4(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);
hipError_t launch_cache_attention_8(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);
hipError_t launch_cache_attention_16(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream);

namespace {

constexpr int kTileKeys = 32, kMostSplits = 64;

// Few rows (up to 32): one workgroup per compute unit at most, of four tiles of 32 keys at least (a tile a wave; 16 bits, whose tiles are larger:
// two), and past 12 ranges (24) of eight (four), since a join costs about 2 us: none below 16 tiles.  Measured, one token, 8 kv heads of 128, 8 bits
// (us by ranges): 300 keys 1: 7.1; 700 keys 1: 9.2, 6: 8.6; 1500 keys 3: 10.7, 12: 9.2, 16: 9.4; 3000 keys 7: 10.8, 12: 10.0, 32: 10.8; 16 bits 1500
// keys 3: 14.7, 24: 10.5.
int64_t few_splits(int64_t groups, int64_t tiles, int bits) {
    if (tiles < 16) return 1;
    const int64_t least = bits == 16 ? 2 : 4, small = bits == 16 ? 24 : 12;
    int64_t splits = kComputeUnits / groups;
    splits = splits < tiles / least ? splits : tiles / least;
    const int64_t most = tiles / (2 * least) > small ? tiles / (2 * least) : small;
    return splits < most ? splits : most;
}

// Many rows, `rows` of a workgroup: an estimate (us) fitted to trees of 12, 27 and 64 tokens over 300 to 4000 keys, one and four requests of 32 / 8
// heads: a start, a time per tile, and for ranges the join with its parts' way through memory.  It serves to choose: over those shapes the choice
// is within 10% of the best of the three.  Measured (64 / 128 / 256 rows, us): 64 tokens, heads of 128, 8 bits: one request of 300 keys 15 / 16 / 21,
// four of 1000 32 / 29 / 35, four of 4000 63 / 48 / 45.  More workgroups than compute units are not split further: two of 64 rows on one unit, 64
// tokens over 4000 keys in 16 ranges rather than 8, took 31 us for 27.
double many_us(int rows, int head_dim, int64_t groups, int64_t tiles, int64_t splits) {
    const bool wide = head_dim == 128;
    const double start = rows == 64 ? 7 : rows == 128 ? 11 : 16;
    const double tile = rows == 64 ? (wide ? 0.95 : 0.74) : rows == 128 ? (wide ? 1.0 : 0.84) : (wide ? 1.35 : 1.17);
    const double wgs = double(groups) * double(splits), turns = wgs / kComputeUnits;
    const double load = turns <= 1 ? 1 : rows == 64 ? 0.8 * turns : double(int64_t(turns + 0.999));  // two of 64 rows share a unit
    const double join = splits > 1 ? 3.5 + wgs * rows * (head_dim + 2) * 8 / 8e6 : 0;
    return start + double(tiles_of(tiles, splits)) * tile * (load < 1 ? 1 : load) + join;
}

}  // namespace

// may_split false: no workspace to split with.
//   LOWBIT_CACHE_ATTENTION=few|many64|many128|many256 in the environment forces the kernel (A/B runs and tests).
CacheAttnPlan plan_cache_attention(const CacheAttnArgs& a, bool may_split) {
    CacheAttnPlan p{};
    const int64_t rows = int64_t(a.q_len) * a.group, heads = int64_t(a.batch) * a.cache.heads, tiles = tiles_of(a.kv_len, kTileKeys);
    p.share_tiles = rows > 32;
    int only = 0;
    if (const char* force = std::getenv("LOWBIT_CACHE_ATTENTION")) {
        if (std::strcmp(force, "few") == 0) p.share_tiles = false;
        for (const int r : {64, 128, 256})
            if (std::strncmp(force, "many", 4) == 0 && std::atoi(force + 4) == r) {
                p.share_tiles = true;
                only = r;
            }
    }
    int64_t splits = 1;
    if (!p.share_tiles) {
        p.tile_rows = rows <= 16 ? 16 : 32;
        p.waves = 4;
        if (may_split && heads * tiles_of(rows, p.tile_rows) > 0) splits = few_splits(heads * tiles_of(rows, p.tile_rows), tiles, a.cache.bits);
    } else {
        double best = 0;
        for (const int r : {64, 128, 256}) {
            if (only != 0 ? r != only : r > 64 && rows <= r / 2) continue;
            const int64_t groups = heads * tiles_of(rows, r);
            for (const int64_t s : {1, 2, 3, 4, 6, 8, 10, 12, 16, 20, 24, 32, 40, 48, 64}) {
                if (s > 1 && (!may_split || s > tiles || groups * s > kComputeUnits)) break;
                const double us = many_us(r, a.cache.head_dim, groups, tiles, s);
                if (p.tile_rows == 0 || us < best) {
                    best = us;
                    p.tile_rows = r;
                    splits = s;
                }
            }
        }
        p.waves = p.tile_rows == 64 ? 4 : 8;
    }
    p.row_tiles = int(tiles_of(rows, p.tile_rows));
    p.splits = splits < 1 ? 1 : splits < kMostSplits ? int(splits) : kMostSplits;
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
                     (long long)(int64_t(a.row_tiles) * a.splits * a.cache.heads * a.batch), 64 * plan.waves, a.batch, a.q_len, a.kv_len, a.cache.heads * a.group, a.cache.heads, a.cache.head_dim, a.cache.bits, 1 << a.cache.page_shift,
                     a.tree != nullptr ? " tree" : "");
    return e;
}

}  // namespace lowbit
