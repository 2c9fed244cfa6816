// Attention of new or drafted tokens over a paged, quantised cache: O = softmax(scale * Q K^T over the allowed keys) V.
//
// Row r of a kv head's problem is new token r / G of its q head r % G (G q heads share a kv head).  A workgroup takes a tile of the rows
// and a range of the keys; its waves take tiles of 32 keys with their own running maximum and sums, joined at the
// end (in wave order, then the key ranges in order: results do not depend on timing).  Two kernels, chosen in cache_attention.hip:
//   up to 16 rows of a workgroup: codes go from memory straight into the registers that the matrix cores read;
//   more: tiles go through LDS, read by as many waves as have rows.
//
// The cache's layout (kv_cache.h) is the operands' layout.  The products are computed transposed, S^T = K Q^T and O^T = V^T P^T, on 16x16x32
// MFMAs: lane (q, l16) then holds scores of query row l16 for keys 4q .. 4q + 3 of each 16, and the probabilities
// are already the second product's operand for its own keys.
//   * A code is never converted: 8 or 4 bits between zeros are an fp16 subnormal, code * 2^-24 (or, 4 bits higher, 16 times
//     that), which the matrix cores take exactly.  That is a byte permute for two codes, or a shift and a mask for
//     up to four.  The other operand carries the 1/16 and, per row or at the end, the 2^24.
//   * Scales multiply the fp32 sums: a key's scale its scores, a value's scale its probability (before that is rounded to fp16).
//     8 bits, codes u = c + 128:  sum q c = sum q u - 128 sum q, the second term being where the sums start from;
//       sum p s c = sum p s u - 128 sum p s, with the same rounded p s (a product with ones).
//     4 bits, x = s u + b per group: s (q.u) + b sum q for the scores, sum p s u + sum p b for the values (the latter in fp32).
//   * Q is a power of two per row (2^14 over its largest exponent) times fp16: exact for bf16 elements down to 2^-28 of the largest (4 bits, every
//     other pair, which carries 1/16: 2^-24).  What takes it back, scale * log2(e) * 2^(E + 10) for a largest exponent E, is one fp32 factor: finite
//     while scale |q| is below 2^117, and with a key's scale while scale |q| |k| is.  A second factor for rows past that, behind a branch
//     that all rows of a wave share, cost every call 1% (a loop of its own for such waves 2 to 6%, in registers).
//   * Everything that a row sums (p, p s, p b) carries one factor 2^-e, which the division at the end takes out.  e is the largest score plus
//     the power of two of its value's scale when it was last set, so that the weights p s lie in fp16's range; it
//     stays as long as they are below 2^12 (which the tile's largest score and largest scale tell), and the sums with it.
// 16-bit caches take the same path with bf16 operands and no scales; what divides a row is the sum of its rounded probabilities (a product with
// ones), so that a row with one key, or one that outweighs all others, gives that key's value back.
//
// Rounding: p s to fp16 (2^-11 of each; 16 bits: p to bf16, 2^-8 of each) and O to bf16; all else is fp32.  fp16 holds 24 bits below its normal
// range: a weight is off by 2^-25 of the row's largest at least, which shows only where one group's scales are 2^12 below the other's.
// A 16-bit cache's values are bf16 and a matrix instruction takes both operands in one type, so p has bf16's 8 bits there, as in lowbit_attention: with
// the sum taken of the rounded ones O is off by 2^-8 sum p |v - O| at most, nothing where one key has the weight.  A
// second product with what that rounding leaves would double the value products.  Trees of 64 over 4 x 4099 keys: 0.0023 of O's norm off
// the formula in 64 bits, 0.0017 of it by the rounding of O; at 8 and 4 bits 0.0017 and 0.0018.
#pragma once

#include "kv_cache.h"
#include "decode_device.h"
#include "decode_internal.h"

namespace lowbit {
namespace {

typedef float f32x2_t __attribute__((__vector_size__(2 * sizeof(float))));
typedef _Float16 f16x8_t __attribute__((__vector_size__(8 * sizeof(_Float16))));

constexpr float kNegInf = -__builtin_inff();
constexpr int kCacheTile = 32;      // keys of a wave's tile
constexpr float kMostWeight = 0x1p12f;    // of p s 2^-e: past it e moves
constexpr float kMostProbability = 0x1p70f;   // of p 2^-e, which values of scale 0 do not bound: times their smallest value it stays in fp32
constexpr float kCodeUnit = 0x1p24f;    // 1 / the value of code 1 as an fp16

// What a lane has of a tile: per block of 16 keys its words of K (a quarter of key l16's row) and of V (piece l16 of keys 4q ..).
template <int D, int BITS>
struct TileShape {
    static constexpr int kWords = CacheFmt<D, BITS>::kRow / 16;     // of K, and of V, per block
    static constexpr int kScales = CacheFmt<D, BITS>::kScaleBytes;  // words that hold the scales of four keys
};
template <int W>
struct Words {
    uint32_t w[W];
};
// The scales (4 bits: and smallest values) of the lane's keys 4q .. of a tile's two blocks, of K or of V.
template <int D, int BITS>
struct KeyScales {
    static constexpr int kN = TileShape<D, BITS>::kScales > 0 ? TileShape<D, BITS>::kScales : 1;
    uint32_t w[2][kN];
};
// K or V of a tile.
template <int D, int BITS>
struct TileWords {
    Words<TileShape<D, BITS>::kWords> block[2];
};

// Running state of a wave for NB blocks of 16 rows.
template <int D, int BITS, int NB>
struct CacheRowsState {
    u32x4_t q[D / 32][NB];  // B operands (bf16, or fp16 times the row's power of two)
    f32x4_t o[D / 16][NB];  // O^T: lane (q, l16): row l16, columns column(j, 4q + i)
    f32x4_t sum[NB];        // 8 bits: the sum of the rounded p s; 16 bits: of the rounded p 2^-e
    float e[NB], l[NB];     // the row's exponent, the lane's own keys' sum of p 2^-e (8 and 4 bits)
    uint32_t seen[NB];      // 1: the row has taken a key (e is 0 before)
    float low[NB][2];       // 4 bits: the lane's own keys' sum of p b 2^-e
    float gain[NB];         // scores in powers of two per unit of (scale * sum)
    float start[NB];        // 8 bits: where sums of scores start from
    float qsum[NB][2];      // 4 bits: scale * log2(e) * the group's sum of q
};

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
    const f16x2_t v = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

template <int BITS>
__device__ __forceinline__ f32x4_t cache_mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
    if constexpr (BITS == 16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// The element of a row of which MFMA `ks` of the scores takes eight in lane quarter q.
template <int BITS>
__device__ __forceinline__ int q_element(int ks, int q) {
    return BITS == 16 ? 32 * ks + 8 * q : 64 * (ks / 2) + 16 * q + 8 * (ks % 2);
}
// The column of O in row m of O^T's block j.
template <int D, int BITS>
__device__ __forceinline__ int o_column(int j, int m) {
    return BITS == 4 ? 64 * (j / 4) + 4 * m + j % 4 : D / 16 * m + j;
}

// The score operand ks of a block from the lane's words: eight codes of key l16.
template <int D, int BITS>
__device__ __forceinline__ u32x4_t k_operand(const Words<TileShape<D, BITS>::kWords>& k, int ks) {
    if constexpr (BITS == 16) {
        return u32x4_t{k.w[4 * ks], k.w[4 * ks + 1], k.w[4 * ks + 2], k.w[4 * ks + 3]};
    } else if constexpr (BITS == 8) {
        const uint32_t a = k.w[2 * ks], b = k.w[2 * ks + 1];
        return u32x4_t{perm_b32(0, a, 0x0C010C00u), perm_b32(0, a, 0x0C030C02u), perm_b32(0, b, 0x0C010C00u), perm_b32(0, b, 0x0C030C02u)};
    } else {
        const uint32_t w = k.w[ks], h = w >> 8;  // the second and fourth pair come 16 times too large
        return u32x4_t{w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u};
    }
}

// Keys 2p and 2p + 1 of a block in column o_column(j, l16): half of a word of the value operand.  Odd columns of 4-bit codes come
// 16 times too large.
template <int D, int BITS>
__device__ __forceinline__ uint32_t v_pair(const Words<TileShape<D, BITS>::kWords>& v, int j, int p) {
    constexpr int kPiece = CacheFmt<D, BITS>::kPiece;
    if constexpr (BITS == 16) {
        const int at = kPiece / 4 * 2 * p + j / 2;
        return perm_b32(v.w[at + kPiece / 4], v.w[at], j % 2 ? 0x07060302u : 0x05040100u);
    } else if constexpr (BITS == 8) {
        const int at = kPiece / 4 * 2 * p + j / 4;
        return perm_b32(v.w[at + kPiece / 4], v.w[at], 0x0C040C00u + 0x00010001u * (j % 4));
    } else if constexpr (kPiece == 4) {
        const int byte = 2 * (j / 4) + j % 4 / 2;
        return perm_b32(v.w[2 * p + 1], v.w[2 * p], 0x0C040C00u + 0x00010001u * byte) & (j % 2 ? 0x00F000F0u : 0x000F000Fu);
    } else {
        return (j / 2 ? v.w[p] >> 8 : v.w[p]) & (j % 2 ? 0x00F000F0u : 0x000F000Fu);
    }
}

// A value of the lanes that share l16 (and so a row).
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// 2^n for n in [-126, 127].
__device__ __forceinline__ float power_of_two(int n) { return __uint_as_float(uint32_t(n + 127) << 23); }

// Where a workgroup's rows and keys lie.
struct CacheWork {
    int b, hk, row0, rows;  // rows: of this tile that exist
    int n, base;            // keys, and those before the new tokens (negative: more new tokens than keys)
};

// The lane's pieces of its rows of q as they lie (rows past the last read as zeros).
template <int D, int BITS, int NB>
struct RawQueries {
    u32x4_t w[D / 32][NB];
};
template <int D, int BITS, int NB>
__device__ __forceinline__ void load_queries(RawQueries<D, BITS, NB>& raw, const CacheAttnArgs& a, const CacheWork& at) {
    const int lane = int(threadIdx.x) & 63, q = lane >> 4, l16 = lane & 15;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const uint32_t row = uint32_t(at.row0 + 16 * nb + l16), group = uint32_t(a.group);
        const bool in = 16 * nb + l16 < at.rows;
        const uint32_t t = in ? row / group : 0u, g = in ? row - t * group : 0u;
        const uint16_t* src = a.q + int64_t(at.b) * a.q_batch + int64_t(t) * a.q_token + int64_t(at.hk * a.group + int(g)) * a.q_head;
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            raw.w[ks][nb] = u32x4_t{0, 0, 0, 0};
            if (in) raw.w[ks][nb] = *reinterpret_cast<const u32x4_t*>(src + q_element<BITS>(ks, q));
        }
    }
}

// Operands from them, and what goes with a row.
template <int D, int BITS, int NB>
__device__ __forceinline__ void start_rows(CacheRowsState<D, BITS, NB>& w, const RawQueries<D, BITS, NB>& raw, const CacheAttnArgs& a) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        w.gain[nb] = a.scale_log2;
        w.start[nb] = w.qsum[nb][0] = w.qsum[nb][1] = 0.f;
        if constexpr (BITS == 16) {
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) w.q[ks][nb] = raw.w[ks][nb];
        } else {
            uint32_t most = 0;  // the largest magnitude's bits
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e) most = max(max(most, raw.w[ks][nb][e] & 0x7FFF0000u), (raw.w[ks][nb][e] << 16) & 0x7FFF0000u);
            most = max(most, uint32_t(__shfl_xor(int(most), 16)));
            most = max(most, uint32_t(__shfl_xor(int(most), 32)));
            int up = 14 - (int(most >> 23) - 127);  // the largest element comes to lie in [2^14, 2^15)
            up = up > 126 ? 126 : up < -113 ? -113 : up;  // (infinite or NaN: they stay that)
            const float f = power_of_two(up);
            float sum[D / 64];
#pragma unroll
            for (int g64 = 0; g64 < D / 64; ++g64) sum[g64] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = bf16_low(raw.w[ks][nb][e]) * f, y = bf16_high(raw.w[ks][nb][e]) * f;
                    sum[ks / 2] += x + y;
                    const float share = BITS == 4 && e % 2 ? 0.0625f : 1.f;
                    w.q[ks][nb][e] = pack_f16(x * share, y * share);
                }
            }
            w.gain[nb] = a.scale_log2 * power_of_two(-up) * kCodeUnit;
            if constexpr (BITS == 8) {
                float all = 0.f;
#pragma unroll
                for (int g64 = 0; g64 < D / 64; ++g64) all += sum[g64];
                w.start[nb] = row_sum(all) * (-128.f / kCodeUnit);
            } else {
#pragma unroll
                for (int g64 = 0; g64 < D / 64; ++g64) w.qsum[nb][g64] = row_sum(sum[g64]) * (a.scale_log2 * power_of_two(-up));
            }
        }
        w.seen[nb] = 0;
        w.e[nb] = w.l[nb] = w.low[nb][0] = w.low[nb][1] = 0.f;
        w.sum[nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) w.o[j][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
}

// Where a tile's two blocks of 16 keys lie: (page * heads + head) * page_size + the place of the first in its page; somewhere in the first page's
// first head and not `ok` where there is no such page or key (what is read there is not used).
struct Places {
    uint64_t at0, at1;
    bool ok0, ok1;
    __device__ __forceinline__ uint64_t at(int kb) const { return kb == 0 ? at0 : at1; }
};
// A word that nothing writes meanwhile, at an address that the wave shares: a scalar load, whose wait leaves vector loads in flight.
__device__ __forceinline__ int scalar_word(const int32_t* p) {
    typedef const __attribute__((address_space(4))) int32_t* Constant;
    const uint64_t x = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(x)), hi = __builtin_amdgcn_readfirstlane(uint32_t(x >> 32));
    return *reinterpret_cast<Constant>((uint64_t(hi) << 32) | lo);
}

// `end` > 0: the keys that count; t may be past the last tile.
__device__ __forceinline__ Places tile_places(const CacheAttnArgs& a, const CacheWork& at, int t, int end) {
    Places p;
    auto block = [&](uint32_t key, uint64_t& place, bool& ok) __attribute__((always_inline)) {
        const bool in = key < uint32_t(end);
        const uint32_t last = in ? key : uint32_t(end) - 1u;
        const int page = scalar_word(a.table + int64_t(at.b) * a.table_stride + (last >> a.cache.page_shift));
        ok = in && uint32_t(page) < uint32_t(a.cache.pages);
        // (page * heads fits 31 bits)
        const uint32_t head = ok ? uint32_t(page) * uint32_t(a.cache.heads) + uint32_t(at.hk) : 0u;
        place = (uint64_t(head) << a.cache.page_shift) + (last & ((1u << a.cache.page_shift) - 16u));
    };
    const uint32_t key = uint32_t(kCacheTile) * uint32_t(t);  // below 2^32: t is at most 32 past 2^26
    block(key, p.at0, p.ok0);
    block(key + 16u, p.at1, p.ok1);
    return p;
}

// The resource of a block's rows of `size` bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t block_rows(const unsigned char* base, uint64_t at, int size) {
    return make_rsrc(base + at * size, 16u * uint32_t(size));
}

// 16 or 8 bytes of the lane at `offset` of a block's rows of `size` bytes: one scalar base, a 32-bit offset.
template <class T>
__device__ __forceinline__ T load_at(const unsigned char* base, uint64_t at, int size, uint32_t offset) {
    const uint64_t from = reinterpret_cast<uint64_t>(base) + at * uint32_t(size);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(from)), hi = __builtin_amdgcn_readfirstlane(uint32_t(from >> 32));
    typedef const __attribute__((address_space(1))) unsigned char* Global;
    const Global scalar = reinterpret_cast<Global>((uint64_t(hi) << 32) | lo);
    return *reinterpret_cast<const __attribute__((address_space(1))) T*>(scalar + offset);
}

// The lane's byte in a block of K or V for load i.
template <int D, int BITS>
__device__ __forceinline__ uint32_t unit_offset(bool is_v, int i) {
    using F = CacheFmt<D, BITS>;
    const uint32_t lane = threadIdx.x & 63u, q = lane >> 4, l16 = lane & 15u;
    constexpr uint32_t kT = F::kBlock;
    if constexpr (TileShape<D, BITS>::kWords >= 4)
        return is_v ? 4u * q / kT * (kT * F::kRow) + 16u * l16 + kT * F::kRow * i : l16 * F::kRow + 16u * q + 64u * i;
    else
        return (is_v ? q * (4u * F::kRow) + 8u * l16 : l16 * F::kRow + 8u * q) + 4u * i;
}

// K or V of a tile into registers.
template <int D, int BITS, bool IS_V>
__device__ __forceinline__ void load_words(TileWords<D, BITS>& t, const CacheAttnArgs& a, const Places& p) {
    constexpr int kW = TileShape<D, BITS>::kWords;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        const unsigned char* const base = IS_V ? a.cache.v : a.cache.k;
        if constexpr (kW >= 4) {
#pragma unroll
            for (int i = 0; i < kW / 4; ++i) {
                const u32x4_t x = load_at<u32x4_t>(base, p.at(kb), CacheFmt<D, BITS>::kRow, unit_offset<D, BITS>(IS_V, i));
#pragma unroll
                for (int e = 0; e < 4; ++e) t.block[kb].w[4 * i + e] = x[e];
            }
        } else {
            const u32x2_t x = load_at<u32x2_t>(base, p.at(kb), CacheFmt<D, BITS>::kRow, unit_offset<D, BITS>(IS_V, 0));
            t.block[kb].w[0] = x[0];
            t.block[kb].w[1] = x[1];
        }
    }
}

template <int D, int BITS, bool IS_V>
__device__ __forceinline__ void load_scales(KeyScales<D, BITS>& s, const CacheAttnArgs& a, const Places& p) {
    constexpr int kS = CacheFmt<D, BITS>::kScaleBytes;
    if constexpr (kS > 0) {
        const uint32_t q = (threadIdx.x & 63u) >> 4;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const unsigned char* const base = IS_V ? a.cache.v_scales : a.cache.k_scales;
            if constexpr (kS == 2) {
                const u32x2_t x = load_at<u32x2_t>(base, p.at(kb), kS, 8u * q);
                s.w[kb][0] = x[0];
                s.w[kb][1] = x[1];
            } else {
#pragma unroll
                for (int i = 0; i < kS / 4; ++i) {
                    const u32x4_t x = load_at<u32x4_t>(base, p.at(kb), kS, 4u * kS * q + 16u * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s.w[kb][4 * i + e] = x[e];
                }
            }
        }
    }
}

// A tile in LDS: its two blocks of K and two of V as they lie in memory, each row of K with its 16-byte chunk c at position c ^ swizzle(row), so
// that the 16 rows of an operand read fall into different banks; then the scales of K's blocks and of V's.
template <int D, int BITS>
struct LdsTile {
    static constexpr int kRow = CacheFmt<D, BITS>::kRow;
    static constexpr int kBlock = 16 * kRow;
    static constexpr int kSegment = 16 * CacheFmt<D, BITS>::kScaleBytes;
    static constexpr int kBytes = 4 * kBlock + 4 * kSegment;
    static constexpr int kCopy = kBlock < 1024 ? kBlock : 1024;  // bytes that one wave-wide copy brings, neighbouring lanes on neighbouring chunks
    static constexpr int kCopies = 4 * kBlock / kCopy;           // of a tile: K's blocks, then V's
    static constexpr int swizzle(int row) { return kRow == 256 ? row & 15 : kRow == 128 ? (row >> 1) & 7 : kRow == 64 ? (row >> 2) & 3 : 0; }
};

// Copy c of a tile (the same for the wave): `at` is its block's place.
template <int D, int BITS>
__device__ __forceinline__ void copy_words(unsigned char* tile, const CacheAttnArgs& a, int c, uint64_t at) {
    using L = LdsTile<D, BITS>;
    constexpr int kPer = L::kBlock / L::kCopy;  // copies of a block
    const bool is_v = c >= 2 * kPer;
    const auto rs = block_rows(is_v ? a.cache.v : a.cache.k, at, L::kRow);
    const int lane = int(threadIdx.x) & 63, chunk = c % kPer * (L::kCopy / 16) + lane;  // of the block, in LDS
    const int row = chunk / (L::kRow / 16);
    const int from = is_v ? chunk : chunk ^ L::swizzle(row);
    if (L::kCopy == 1024 || lane < L::kCopy / 16) dma16(rs, tile + c * L::kCopy, 16u * uint32_t(from), 0);
}
// Segment s of its scales: K's blocks 0 and 1, then V's.
template <int D, int BITS>
__device__ __forceinline__ void copy_scales(unsigned char* tile, const CacheAttnArgs& a, int s, uint64_t at) {
    using L = LdsTile<D, BITS>;
    constexpr int kBytes = BITS == 8 ? 4 : 16;  // of a lane
    const int lane = int(threadIdx.x) & 63;
    const auto rs = block_rows(s >= 2 ? a.cache.v_scales : a.cache.k_scales, at, CacheFmt<D, BITS>::kScaleBytes);
    unsigned char* const to = tile + 4 * L::kBlock + s * L::kSegment;
    if (lane < L::kSegment / kBytes) {
        if constexpr (kBytes == 4)
            dma4(rs, to, 4u * uint32_t(lane), 0);
        else
            dma16(rs, to, 16u * uint32_t(lane), 0);
    }
}

// K or V of a tile from there.
template <int D, int BITS, bool IS_V>
__device__ __forceinline__ void read_words(TileWords<D, BITS>& t, const unsigned char* tile) {
    using S = TileShape<D, BITS>;
    using L = LdsTile<D, BITS>;
    const int l16 = int(threadIdx.x) & 15;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        const unsigned char* const block = tile + ((IS_V ? 2 : 0) + kb) * L::kBlock;
        if constexpr (S::kWords >= 4) {
#pragma unroll
            for (int i = 0; i < S::kWords / 4; ++i) {
                const uint32_t from = unit_offset<D, BITS>(IS_V, i);  // within a row of K: an aligned chunk
                const u32x4_t x = *reinterpret_cast<const u32x4_t*>(block + (IS_V ? from : from ^ uint32_t(L::swizzle(l16) << 4)));
#pragma unroll
                for (int e = 0; e < 4; ++e) t.block[kb].w[4 * i + e] = x[e];
            }
        } else {
            const u32x2_t x = *reinterpret_cast<const u32x2_t*>(block + unit_offset<D, BITS>(IS_V, 0));
            t.block[kb].w[0] = x[0];
            t.block[kb].w[1] = x[1];
        }
    }
}
template <int D, int BITS, bool IS_V>
__device__ __forceinline__ void read_scales(KeyScales<D, BITS>& s, const unsigned char* tile) {
    using L = LdsTile<D, BITS>;
    constexpr int kS = CacheFmt<D, BITS>::kScaleBytes;
    if constexpr (kS > 0) {
        const unsigned char* const at = tile + 4 * L::kBlock + (IS_V ? 2 : 0) * L::kSegment + ((threadIdx.x & 63u) >> 4) * (4 * kS);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const unsigned char* const from = at + kb * L::kSegment;
            if constexpr (kS == 2) {
                const u32x2_t x = *reinterpret_cast<const u32x2_t*>(from);
                s.w[kb][0] = x[0];
                s.w[kb][1] = x[1];
            } else {
#pragma unroll
                for (int i = 0; i < kS / 4; ++i) {
                    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(from + 16 * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s.w[kb][4 * i + e] = x[e];
                }
            }
        }
    }
}

// The scale of the lane's key i of block kb, and (4 bits, group g) its smallest value.
template <int D, int BITS>
__device__ __forceinline__ float scale_at(const uint32_t* s, int i, int g) {
    if constexpr (BITS == 8)
        return i % 2 ? bf16_high(s[i / 2]) : bf16_low(s[i / 2]);
    else
        return bf16_low(s[i * CacheFmt<D, BITS>::kGroups + g]);
}
template <int D, int BITS>
__device__ __forceinline__ float low_at(const uint32_t* s, int i, int g) {
    return bf16_high(s[i * CacheFmt<D, BITS>::kGroups + g]);
}

// 16-bit values of a tile with keys that some row leaves out or that are not there.  Zero in a product does not silence an infinity or a NaN, so
// these become zeros, and what is there is added to the rows that take it.
template <int D, int NB>
__device__ __forceinline__ void clean_values(CacheRowsState<D, 16, NB>& w, TileWords<D, 16>& v, const CacheAttnArgs& a, const CacheWork& at, int t, int end,
                                             uint32_t live, const uint32_t (&allowed)[NB]) {
    using F = CacheFmt<D, 16>;
    constexpr int kW = TileShape<D, 16>::kWords;
    const uint32_t q = (threadIdx.x & 63u) >> 4;
    uint32_t odd = 0;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const uint32_t x = (live >> (16 * kb + 4 * q + i / (kW / 4))) & 1 ? v.block[kb].w[i] : 0u;
            const uint32_t y = (x & 0x7F80u) == 0x7F80u ? x & 0xFFFF0000u : x;
            const uint32_t z = (y & 0x7F800000u) == 0x7F800000u ? y & 0xFFFFu : y;
            odd |= x ^ z;
            v.block[kb].w[i] = z;
        }
    if (!__any(odd != 0)) return;
    const Places place = tile_places(a, at, t, end);
    for (int key = 0; key < kCacheTile; ++key) {
        const uint64_t p = place.at0 ^ ((place.at0 ^ place.at1) & (key < 16 ? uint64_t(0) : ~uint64_t(0)));
        bool some = false;  // (a key that is not there is allowed to no row)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) some = some || ((allowed[nb] >> key) & 1);
        if (!__any(some)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the lane's columns: pieces 4q + i
            const unsigned char* src = a.cache.v + p * F::kRow + F::v_offset(uint32_t(key & 15), 4u * q + i);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const uint32_t b = reinterpret_cast<const uint16_t*>(src)[j];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    if ((b & 0x7F80u) == 0x7F80u && ((allowed[nb] >> key) & 1)) w.o[j][nb][i] += bf16_low(b);
            }
        }
    }
}

// Scores of a tile, in powers of two above the row's e: [block][row block], keys 16 kb + 4q ..
template <int NB>
struct TileScores {
    f32x4_t s[2][NB];
};

template <int D, int BITS, int NB>
__device__ __forceinline__ void tile_scores(const CacheRowsState<D, BITS, NB>& w, const TileWords<D, BITS>& k, const KeyScales<D, BITS>& ks,
                                            TileScores<NB>& x) {
    constexpr int kGroups = CacheFmt<D, BITS>::kGroups;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        if constexpr (BITS == 4) {
            f32x4_t raw[kGroups][NB];
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) raw[g][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks32 = 0; ks32 < D / 32; ++ks32) {
                const u32x4_t op = k_operand<D, BITS>(k.block[kb], ks32);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) raw[ks32 / 2][nb] = cache_mfma<BITS>(op, w.q[ks32][nb], raw[ks32 / 2][nb]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float sum = raw[0][nb][i] * scale_at<D, BITS>(ks.w[kb], i, 0);
                    float low = __builtin_fmaf(w.qsum[nb][0], low_at<D, BITS>(ks.w[kb], i, 0), -w.e[nb]);
                    if constexpr (kGroups == 2) {
                        sum = __builtin_fmaf(raw[1][nb][i], scale_at<D, BITS>(ks.w[kb], i, 1), sum);
                        low = __builtin_fmaf(w.qsum[nb][1], low_at<D, BITS>(ks.w[kb], i, 1), low);
                    }
                    x.s[kb][nb][i] = __builtin_fmaf(sum, w.gain[nb], low);
                }
        } else {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) x.s[kb][nb] = f32x4_t{w.start[nb], w.start[nb], w.start[nb], w.start[nb]};
#pragma unroll
            for (int ks32 = 0; ks32 < D / 32; ++ks32) {
                const u32x4_t op = k_operand<D, BITS>(k.block[kb], ks32);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) x.s[kb][nb] = cache_mfma<BITS>(op, w.q[ks32][nb], x.s[kb][nb]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    x.s[kb][nb][i] = __builtin_fmaf(x.s[kb][nb][i], BITS == 16 ? w.gain[nb] : w.gain[nb] * scale_at<D, 8>(ks.w[kb], i, 0), -w.e[nb]);
        }
    }
}

// All ones or zeros: bit (kb, i) of the lane's keys (bits from the lane's quarter on).
__device__ __forceinline__ uint32_t taken_mask(uint32_t mine, int kb, int i) { return uint32_t(int32_t(mine << (31 - 16 * kb - i)) >> 31); }

// Row block nb's e to what its scores x and the values' scales need, and x and the sums with it.
template <int D, int BITS, int NB>
__device__ __forceinline__ void rebase(CacheRowsState<D, BITS, NB>& w, int nb, TileScores<NB>& x, const KeyScales<D, BITS>& vs, float top) {
    top = row_max(top);
    float up = BITS == 16 ? top : kNegInf;  // of the new e above the old one
    if constexpr (BITS != 16) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float most = 0.f;
#pragma unroll
                for (int g = 0; g < CacheFmt<D, BITS>::kGroups; ++g) most = fmaxf(most, scale_at<D, BITS>(vs.w[kb], i, g));
                up = fmaxf(up, x.s[kb][nb][i] + __builtin_amdgcn_logf(most));
            }
        up = fmaxf(row_max(up), top - 64.f);  // all scales 0, or nearly
    }
    // a row without a key stays as it is, one with its first key takes any e, others a larger one
    up = top > kNegInf && (up > 0.f || w.seen[nb] == 0) ? __builtin_ceilf(up) : 0.f;  // whole, so that e stays exact
    const float f = w.seen[nb] != 0 ? __builtin_amdgcn_exp2f(-up) : 1.f;  // (sums of nothing are zeros, or what clean_values put there)
    w.seen[nb] = top > kNegInf ? 1u : w.seen[nb];
    w.e[nb] += up;
    w.l[nb] *= f;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) x.s[kb][nb][i] -= up;
    w.low[nb][0] *= f;
    w.low[nb][1] *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) w.sum[nb][i] *= f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) w.o[j][nb][i] *= f;
}

template <int D, int BITS, int NB>
struct TileWeights {
    u32x4_t p[NB][CacheFmt<D, BITS>::kGroups];  // operands: p s (16 bits: p), keys 4q .. of block 0, then of block 1
};

// The probabilities of a tile's scores, times the values' scales.
template <int D, int BITS, int NB>
__device__ __forceinline__ void tile_weights(CacheRowsState<D, BITS, NB>& w, TileScores<NB>& x, const KeyScales<D, BITS>& vs,
                                             TileWeights<D, BITS, NB>& p) {
    constexpr int kGroups = CacheFmt<D, BITS>::kGroups;
    float most = 0.f;  // of the values' scales
    if constexpr (BITS != 16) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int g = 0; g < kGroups; ++g) most = fmaxf(most, scale_at<D, BITS>(vs.w[kb], i, g));
    }
    float top[NB];
    bool again = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        top[nb] = kNegInf;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                top[nb] = fmaxf(top[nb], x.s[kb][nb][i]);
            }
        const float p = __builtin_amdgcn_exp2f(top[nb]);
        // (a bound: the largest score and the largest scale need not be one key's)
        again = again || (w.seen[nb] == 0 && top[nb] > kNegInf) || p > kMostProbability || p * (BITS == 16 ? 1.f : most) > kMostWeight;
    }
    if (__any(again)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) rebase(w, nb, x, vs, top[nb]);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float y[2][4];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[kb][i] = __builtin_amdgcn_exp2f(x.s[kb][nb][i]);
                if constexpr (BITS != 16) w.l[nb] += y[kb][i];
            }
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    if constexpr (BITS == 16) {
                        p.p[nb][0][2 * kb + i / 2] = pack_bf16(y[kb][i], y[kb][i + 1]);
                    } else {
                        float z[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            z[e] = y[kb][i + e] * scale_at<D, BITS>(vs.w[kb], i + e, g);
                            if constexpr (BITS == 4)
                                w.low[nb][g] = __builtin_fmaf(y[kb][i + e], low_at<D, BITS>(vs.w[kb], i + e, g), w.low[nb][g]);
                        }
                        p.p[nb][g][2 * kb + i / 2] = pack_f16(z[0], z[1]);
                    }
                }
    }
}

// O += V^T P^T of a tile.
template <int D, int BITS, int NB>
__device__ __forceinline__ void tile_values(CacheRowsState<D, BITS, NB>& w, const TileWords<D, BITS>& v, const TileWeights<D, BITS, NB>& p) {
    if constexpr (BITS != 4) {
        constexpr uint32_t kOnes = BITS == 16 ? 0x3F803F80u : 0x3C003C00u;
        const u32x4_t ones = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) w.sum[nb] = cache_mfma<BITS>(ones, p.p[nb][0], w.sum[nb]);
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        u32x4_t op;
#pragma unroll
        for (int e = 0; e < 4; ++e) op[e] = v_pair<D, BITS>(v.block[e / 2], j, e % 2);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) w.o[j][nb] = cache_mfma<BITS>(op, p.p[nb][BITS == 4 ? j / 4 : 0], w.o[j][nb]);
    }
}

// Bits 0 .. rel (none for rel < 0) of 32.
__device__ __forceinline__ uint32_t first_bits(int64_t rel) { return rel < 0 ? 0u : rel >= 31 ? ~0u : (2u << int(rel)) - 1u; }

// The keys that a row takes of the 32 from key0 on; `own` is its token's tree, or the tokens up to itself.
__device__ __forceinline__ uint32_t taken(bool tree, uint64_t own, int token, int base, int key0) {
    const int64_t rel = int64_t(key0) - base;  // the new token that key0 is
    if (!tree) return first_bits(int64_t(token) - rel);
    if (rel >= 64) return 0u;
    if (rel >= 0) return uint32_t(own >> int(rel));
    if (rel <= -32) return ~0u;
    return uint32_t(own << int(-rel)) | first_bits(-rel - 1);
}

// Which rows and keys a workgroup has; false: none.
struct CacheRange {
    CacheWork at;
    int group_of;    // of the workgroups that share rows
    int split, end;  // keys that some row takes and this or an earlier range has: [0, end)
    int first;       // that every row takes: [0, first)
    int t0, t1;      // tiles
    bool tree;
};
__device__ __forceinline__ bool cache_range(CacheRange& r, const CacheAttnArgs& a, int rows_of_tile) {
    // row tiles of one range of keys next to each other on one XCD, then the ranges of one head
    uint32_t id = uint32_t(xcd_remap(int(blockIdx.x), int(gridDim.x)));
    uint32_t next = id / uint32_t(a.row_tiles);
    const int rt = int(id - next * uint32_t(a.row_tiles));
    id = next;
    next = id / uint32_t(a.splits);
    r.split = int(id - next * uint32_t(a.splits));
    r.at.b = int(next / uint32_t(a.cache.heads));
    r.at.hk = int(next - uint32_t(r.at.b) * uint32_t(a.cache.heads));
    r.group_of = (r.at.b * a.cache.heads + r.at.hk) * a.row_tiles + rt;
    int n = scalar_word(a.lens + r.at.b);
    n = n < 0 ? 0 : n < a.kv_len ? n : a.kv_len;
    int ql = a.q_len;
    if (a.q_lens != nullptr) {
        const int v = scalar_word(a.q_lens + r.at.b);
        ql = v < 0 ? 0 : v < ql ? v : ql;
    }
    r.at.n = n;
    r.at.base = n - ql;
    r.at.row0 = rt * rows_of_tile;
    const int64_t left = int64_t(ql) * a.group - r.at.row0;
    if (left <= 0) return false;  // rows past the request's last token, in every range of keys
    r.at.rows = left < rows_of_tile ? int(left) : rows_of_tile;
    r.tree = a.tree != nullptr;
    const int64_t last = r.tree ? n : int64_t(r.at.base) + uint32_t(r.at.row0 + r.at.rows - 1) / uint32_t(a.group) + 1;
    r.end = last < 0 ? 0 : last < n ? int(last) : n;
    const int64_t first = r.tree ? r.at.base : int64_t(r.at.base) + uint32_t(r.at.row0) / uint32_t(a.group) + 1;
    r.first = first < 0 ? 0 : first < n ? int(first) : n;
    const uint32_t tiles = uint32_t(r.end + kCacheTile - 1) / kCacheTile;  // below 2^26, and 64 ranges at most
    // the ranges share the keys there are, not the keys there could be
    r.t0 = int(tiles * uint32_t(r.split) / uint32_t(a.splits));
    r.t1 = int(tiles * uint32_t(r.split + 1) / uint32_t(a.splits));
    r.end = r.end < r.t1 * kCacheTile ? r.end : r.t1 * kCacheTile;
    return true;
}

// The token of each of the lane's rows (those past the last: the tile's first), and its tree.
template <int NB>
struct RowTokens {
    int token[NB];
    uint64_t own[NB];
};
template <int NB>
__device__ __forceinline__ RowTokens<NB> row_tokens(const CacheRange& r, const CacheAttnArgs& a, const CacheWork& at) {
    RowTokens<NB> k;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int in_tile = 16 * nb + (int(threadIdx.x) & 15);
        const int row = in_tile < at.rows ? at.row0 + in_tile : r.at.row0;
        k.token[nb] = int(uint32_t(row) / uint32_t(a.group));
        k.own[nb] = r.tree ? a.tree[int64_t(at.b) * a.q_len + k.token[nb]] : 0;
    }
    return k;
}

// Keys of tile t that are there, and those that each of the lane's rows takes.
template <int NB>
__device__ __forceinline__ uint32_t tile_keys(uint32_t (&allowed)[NB], const CacheRange& r, const RowTokens<NB>& k, uint32_t blocks, int t) {
    const int key0 = kCacheTile * t;
    const uint32_t live = first_bits(int64_t(r.at.n) - key0 - 1) & ((blocks & 1u ? 0xFFFFu : 0u) | (blocks & 2u ? 0xFFFF0000u : 0u));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) allowed[nb] = live & taken(r.tree, k.own[nb], k.token[nb], r.at.base, key0);
    return live;
}

// Every row takes every key of tile t, and they are there.
__device__ __forceinline__ bool whole_tile(const CacheRange& r, const Places& place, int t) {
    return kCacheTile * (t + 1) <= r.first && place.ok0 && place.ok1;
}

// A tile with keys that some row leaves out or that are not there: their scores to -inf.  Scales (and smallest values) of keys that are not there
// may be anything; those of the others may be NaN or infinite, which is for the rows that take the key alone, and zero in a product does not
// silence it: both become zeros, and the sums of those rows NaN.
template <int D, int BITS, int NB>
__device__ __forceinline__ void trim_tile(CacheRowsState<D, BITS, NB>& w, TileScores<NB>& x, KeyScales<D, BITS>& vs, uint32_t live,
                                          const uint32_t (&allowed)[NB]) {
    constexpr int kGroups = CacheFmt<D, BITS>::kGroups;
    const uint32_t shift = 4u * ((threadIdx.x & 63u) >> 4);
    const uint32_t there = live >> shift;
    uint32_t mine[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) mine[nb] = allowed[nb] >> shift;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint32_t all = taken_mask(mine[nb], kb, i);
                x.s[kb][nb][i] = __uint_as_float((__float_as_uint(x.s[kb][nb][i]) & all) | (0xFF800000u & ~all));
            }
            if constexpr (BITS != 16) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    uint32_t& word = vs.w[kb][BITS == 8 ? i / 2 : i * kGroups + g];
                    const int up = BITS == 8 && i % 2 ? 16 : 0;                       // the scale's half of the word
                    const uint32_t half = BITS == 4 ? ~0u : up != 0 ? 0xFFFF0000u : 0xFFFFu;  // what goes with it
                    bool no_number = (word & (0x7F80u << up)) == (0x7F80u << up);
                    if constexpr (BITS == 4) no_number = no_number || (word & 0x7F800000u) == 0x7F800000u;
                    const uint32_t odd = no_number ? ~0u : 0u;
                    word &= ~half | (taken_mask(there, kb, i) & ~odd);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float& to = BITS == 4 ? w.low[nb][g] : w.l[nb];
                        to = __uint_as_float(__float_as_uint(to) | (odd & taken_mask(mine[nb], kb, i) & 0x7FFFFFFFu));  // NaN, or as it was
                    }
                }
            }
        }
}

// The sum that divides the lane's row in block nb (all lanes of the row have it).
template <int D, int BITS, int NB>
__device__ __forceinline__ float total_weight(const CacheRowsState<D, BITS, NB>& w, int nb) {
    return BITS == 16 ? w.sum[nb][0] : row_sum(w.l[nb]);
}

// O of the lane's row in block nb: element [j][i], column o_column(j, 4q + i), as a number.
template <int D, int BITS, int NB, class F>
__device__ __forceinline__ void each_o(const CacheRowsState<D, BITS, NB>& w, int nb, F f) {
    float low[2] = {0.f, 0.f};
    if constexpr (BITS == 4) {
        low[0] = row_sum(w.low[nb][0]);
        low[1] = row_sum(w.low[nb][1]);
    }
    const float unit = BITS == 16 ? 1.f : kCodeUnit;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = w.o[j][nb][i] * (BITS == 4 && j % 2 ? unit * 0.0625f : unit);
            if constexpr (BITS == 8) v = __builtin_fmaf(-128.f, w.sum[nb][i], v);
            if constexpr (BITS == 4) v += low[j / 4];
            f(j, i, v);
        }
}

__device__ __forceinline__ uint16_t* o_row(const CacheAttnArgs& a, const CacheWork& at, int in_tile) {
    const uint32_t row = uint32_t(at.row0 + in_tile);
    const uint32_t tok = row / uint32_t(a.group);
    const int g = int(row - tok * uint32_t(a.group));
    return a.o + int64_t(at.b) * a.o_batch + int64_t(tok) * a.o_token + int64_t(at.hk * a.group + g) * a.o_head;
}

// 16 rows of a workgroup (decoded tokens, short caches): the waves take tiles in turn.
//
// Bound by the cache's bytes where there are many, one wave's chain of latencies where there are few: a start of 2.5 us (lengths, then the
// table, then the first tile, each waiting for the last), a microsecond a tile and wave, 3 to 5 us for the join of split ranges.  Page
// numbers come by scalar loads, so that waiting for one leaves the tiles' loads in flight; a vector load's wait drains them.  8 kv heads of 128 (us, kernel
// and launch, the cache from HBM): 61 requests of 1025 to 2050 keys, 8 bits, 40.9 (201 MB, 4.9 TB/s); one of 40,007 keys in 4 bits 20.1 (46 MB), half
// of them in the loop; four of 2050 to 4099 in 8 bits 13.3.  Replayed, with the cache or part of it left in the last-level cache: 34.6, 19.2 and 11.4;
// one of 77 keys 5.2.
template <int D, int BITS>
__global__ __launch_bounds__(256, 2) void cache_attention_kernel(CacheAttnArgs a) {
    constexpr int NB = 1, kWaves = 4, kRows = 16;
    constexpr int kPitch = D + 4;  // floats of a row: neighbouring rows 4 banks apart
    __shared__ __attribute__((aligned(16))) float lds_o[kWaves][kRows * kPitch];
    __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows];  // e (-inf: no key), and the sum
    __shared__ int last_split;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int q = lane >> 4, l16 = lane & 15;
    CacheRange r;
    if (!cache_range(r, a, kRows)) return;
    const CacheWork& at = r.at;
    const int group_of = r.group_of, split = r.split;

    CacheRowsState<D, BITS, NB> w;
    RawQueries<D, BITS, NB> raw;
    load_queries(raw, a, at);
    int t = r.t0 + wave;
    // A tile on its way or in work: its registers of keys (values) are loaded anew, for the wave's next tile, as soon as its scores (products) are
    // there.  A second such set, two tiles on their way, cost more in registers than it hid: 4 bits, 40,007 keys 20.5 us, here 19.6; 8
    // bits, 300 keys 7.1, here 6.7; 16 bits, whose tiles are larger and where it spilled, 1500 keys 10.6, here 9.4.
    struct Set {
        TileWords<D, BITS> k, v;
        KeyScales<D, BITS> ks, vs;
        Places at;
    };
    auto load_keys = [&](Set& s, const Places& p) __attribute__((always_inline)) {
        load_words<D, BITS, false>(s.k, a, p);
        load_scales<D, BITS, false>(s.ks, a, p);
    };
    auto load_values = [&](Set& s, const Places& p) __attribute__((always_inline)) {
        load_words<D, BITS, true>(s.v, a, p);
        load_scales<D, BITS, true>(s.vs, a, p);
    };
    if (t < r.t1) {
        auto places = [&](int tile) __attribute__((always_inline)) { return tile_places(a, at, tile, r.end); };  // past the range: none
        Set s;
        s.at = places(t);
        load_keys(s, s.at);
        load_values(s, s.at);
        Places ahead = places(t + kWaves);
        start_rows(w, raw, a);
        const RowTokens<NB> rows = row_tokens<NB>(r, a, at);
        do {
            TileScores<NB> x;
            TileWeights<D, BITS, NB> p;
            const bool whole = whole_tile(r, s.at, t);
            tile_scores(w, s.k, s.ks, x);
            load_keys(s, ahead);
            __builtin_amdgcn_sched_barrier(0);  // the loads stay where they are
            if (!whole) {
                uint32_t allowed[NB];
                const uint32_t live = tile_keys(allowed, r, rows, (s.at.ok0 ? 1u : 0u) | (s.at.ok1 ? 2u : 0u), t);
                trim_tile(w, x, s.vs, live, allowed);
                if constexpr (BITS == 16) clean_values(w, s.v, a, at, t, r.end, live, allowed);
            }
            tile_weights(w, x, s.vs, p);
            tile_values(w, s.v, p);
            load_values(s, ahead);
            __builtin_amdgcn_sched_barrier(0);
            s.at = ahead;
            t += kWaves;
            ahead = places(t + kWaves);
        } while (t < r.t1);
    } else {
        start_rows(w, raw, a);
    }

    // ---- the waves' results, as numbers: row by row in LDS ----
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        each_o(w, nb, [&](int j, int i, float v) __attribute__((always_inline)) {
            lds_o[wave][(16 * nb + l16) * kPitch + o_column<D, BITS>(j, 4 * q + i)] = v;
        });
        const float l = total_weight(w, nb);
        if (q == 0) {
            lds_m[wave][16 * nb + l16] = l != 0.f ? w.e[nb] : kNegInf;  // (a NaN goes along)
            lds_l[wave][16 * nb + l16] = l;
        }
    }
    __syncthreads();
    // O of a row of the tile, columns col .. col + 3, divided by the sum l (0: a row without keys)
    auto store4 = [&](int in_tile, int col, f32x4_t v, float l) {
        const float f = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<u32x2_t*>(o_row(a, at, in_tile) + col) = u32x2_t{pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f)};
    };
    constexpr int kSc1 = 16;  // through to the device-coherent level: other workgroups' caches are elsewhere
    constexpr uint32_t kPart = uint32_t(D + 2) * 4u;  // bytes of a row's partial result: O, then maximum and sum
    const auto part_rs = make_rsrc(a.part + int64_t(group_of) * a.splits * kRows * (D + 2), a.splits > 1 ? uint32_t(a.splits) * kRows * kPart : 0u);
    const int items = at.rows * (D / 4);
    for (int item = int(threadIdx.x); item < items; item += 64 * kWaves) {
        const int row = item / (D / 4), col = 4 * (item % (D / 4));
        float top = kNegInf, total = 0.f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) top = fmaxf(top, lds_m[i][row]);
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            if (lds_m[i][row] == kNegInf) continue;
            const float f = __builtin_amdgcn_exp2f(lds_m[i][row] - top);
            total += f * lds_l[i][row];
            const f32x4_t u = *reinterpret_cast<const f32x4_t*>(&lds_o[i][row * kPitch + col]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, u[e], v[e]);
        }
        if (a.splits == 1) {
            store4(row, col, v, total);
        } else {
            const uint32_t to = uint32_t(split * kRows + row) * kPart;
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), part_rs, to + 4u * uint32_t(col), 0, kSc1);
            if (col == 0) {
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(top), part_rs, to + 4u * D, 0, kSc1);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(total), part_rs, to + 4u * D + 4u, 0, kSc1);
            }
        }
    }
    if (a.splits == 1) return;

    // ---- the ranges' results: the last workgroup of the rows to arrive joins them ----
    wait_vmcnt<0>();  // the partial result is there before the arrival counts
    __syncthreads();
    if (threadIdx.x == 0)
        last_split = __hip_atomic_fetch_add(&a.counters[group_of], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == uint32_t(a.splits - 1);
    __syncthreads();
    if (!last_split) return;
    if (threadIdx.x == 0) __hip_atomic_store(&a.counters[group_of], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // (row, 4 columns) per thread, with the ranges shared out over `parts` threads where threads are left over, kAhead of a thread's on their way; every
    // thread works out its ranges' factors itself
    constexpr int kAhead = 16;
    int parts = 1;
    while (parts < 8 && 2 * parts * items <= 64 * kWaves) parts *= 2;
    const int span = (a.splits + parts - 1) / parts;
    const int first_item = int(threadIdx.x) % items, part = int(threadIdx.x) / items;  // (threads past items * parts have nothing)
    const int s_end = (part + 1) * span < a.splits ? (part + 1) * span : a.splits;
    f32x4_t* const sums = reinterpret_cast<f32x4_t*>(&lds_o[0][0]);             // [threads], then their (e, sum)
    f32x2_t* const stats = reinterpret_cast<f32x2_t*>(sums + 64 * kWaves);
    static_assert(6 * 64 <= kRows * kPitch, "they fit the waves' results");
    for (int item = first_item; item < items && part < parts; item += 64 * kWaves) {  // more than one turn only with one part
        const int row = item / (D / 4);
        const uint32_t from = uint32_t(row) * kPart, col = 16u * uint32_t(item % (D / 4));
        float top = kNegInf, l = 0.f;
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = part * span; s0 < s_end; s0 += kAhead) {
            f32x4_t u[kAhead];
            f32x2_t st[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {  // a range past the last reads as zeros
                const uint32_t at_range = s0 + i < s_end ? uint32_t((s0 + i) * kRows) * kPart + from : 0xFFFFFF00u - kPart;
                st[i] = __builtin_bit_cast(f32x2_t, __builtin_amdgcn_raw_buffer_load_b64(part_rs, at_range + 4u * D, 0, kSc1));
                u[i] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(part_rs, at_range + col, 0, kSc1));
            }
            float most = top;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                st[i][0] = s0 + i < s_end ? st[i][0] : kNegInf;
                most = fmaxf(most, st[i][0]);
            }
            const float old = top == kNegInf ? 0.f : __builtin_amdgcn_exp2f(top - most);
            l *= old;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= old;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float f = st[i][0] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(st[i][0] - most);
                l = __builtin_fmaf(f, st[i][1], l);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, u[i][e], v[e]);
            }
            top = most;
        }
        if (parts == 1) {
            store4(row, 4 * (item % (D / 4)), v, l);
        } else {
            sums[part * items + item] = v;
            stats[part * items + item] = f32x2_t{top, l};
        }
    }
    if (parts == 1) return;
    __syncthreads();
    if (int(threadIdx.x) < items) {
        float top = kNegInf, l = 0.f;
        for (int i = 0; i < parts; ++i) top = fmaxf(top, stats[i * items + first_item][0]);
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < parts; ++i) {
            const f32x2_t st = stats[i * items + first_item];
            const float f = st[0] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(st[0] - top);
            l = __builtin_fmaf(f, st[1], l);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, sums[i * items + first_item][e], v[e]);
        }
        store4(first_item / (D / 4), 4 * (first_item % (D / 4)), v, l);
    }
}

// Behind the ranges' sums of O [heads][ranges][rows][D]: [heads][ranges][rows] of (e, sum).
template <int D>
__device__ __forceinline__ f32x2_t* row_stats(const CacheAttnArgs& a, int rows_of_tile) {
    return reinterpret_cast<f32x2_t*>(a.part + int64_t(a.batch) * a.cache.heads * a.row_tiles * a.splits * rows_of_tile * D);
}

// Many rows (trees, chunks): tiles go through LDS.  Four waves take 16 NB rows each, and as many the same rows on every other tile, so that two
// waves work on a SIMD and a tile is read from LDS four times; what the two have is added at the end.  A turn is kTurn tiles; the copies
// of the next turn's are on their way meanwhile, each wave-wide copy of 1 KB with neighbouring lanes on neighbouring 16 bytes.
//
// Bound by vector instructions at 4 bits (a score costs five, a weight six beside the exponential; matrix cores under a third) and by one wave's
// chain through LDS, matrix cores and exponentials otherwise: two waves of a SIMD overlap about half of it.  Eight waves with rows of their own (128 or
// 256 rows) read each tile twice as often and wrote twice the parts: trees of 64 over 4 x 4099 keys in 16 bits 41.4 us, here 40; of 27 over
// 3 x 8191 in 4 bits 21.9, here 19.4; of 64 over 4000 in 8 bits 27.5, here 20.5.  Reading the next tile's keys before this tile's exponentials gained nothing.
template <int D, int BITS, int NB, int ROW_WAVES>
__global__ __launch_bounds__(512, 2) void cache_attention_rows_kernel(CacheAttnArgs a) {
    using L = LdsTile<D, BITS>;
    constexpr int kWaves = 8, kRowWaves = ROW_WAVES, kKeyWaves = kWaves / kRowWaves;
    constexpr int kRows = 16 * NB * kRowWaves;
    constexpr int kTurn = 4;
    constexpr int kPitch = D + 4;  // floats of a result's row: neighbouring rows 4 banks apart
    constexpr int kSlab = 16 * kPitch * 4;
    constexpr int kBytes = kTurn * L::kBytes > kWaves * kSlab ? kTurn * L::kBytes : kWaves * kSlab;
    // an array per buffer: the compiler then sees that a tile's reads do not depend on the copies landing in the other
    __shared__ __attribute__((aligned(1024))) unsigned char buf0[kBytes], buf1[kTurn * L::kBytes];
    __shared__ f32x2_t stats[kWaves][16];
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int q = lane >> 4, l16 = lane & 15;
    CacheRange r;
    if (!cache_range(r, a, kRows)) return;
    const int row_wave = wave % kRowWaves, key_wave = wave / kRowWaves;
    CacheWork at = r.at;  // of the wave's rows
    at.row0 += 16 * NB * row_wave;
    at.rows = at.rows - 16 * NB * row_wave;
    at.rows = at.rows < 0 ? 0 : at.rows < 16 * NB ? at.rows : 16 * NB;
    CacheRowsState<D, BITS, NB> w;
    RawQueries<D, BITS, NB> raw;
    load_queries(raw, a, at);
    int t = r.t0;
    if (t < r.t1) {
        // Lane b has the page of block b of a turn's 2 kTurn (those after repeat).  Fetched a turn before its copies are issued.
        const int32_t* const table = a.table + int64_t(at.b) * a.table_stride;
        auto key_of = [&](int tile) __attribute__((always_inline)) { return uint32_t(kCacheTile) * uint32_t(tile) + 16u * uint32_t(lane & (2 * kTurn - 1)); };
        auto fetch_pages = [&](int tile) __attribute__((always_inline)) {
            const uint32_t key = key_of(tile), last = key < uint32_t(r.end) ? key : uint32_t(r.end) - 1u;
            return table[last >> a.cache.page_shift];
        };
        auto there = [&](int page, int tile) __attribute__((always_inline)) {  // bit b: block b's keys are there
            return __ballot(key_of(tile) < uint32_t(r.end) && uint32_t(page) < uint32_t(a.cache.pages));
        };
        auto copy = [&](unsigned char* to, int page, uint64_t ok, int tile) __attribute__((always_inline)) {
            auto place = [&](int b) __attribute__((always_inline)) {  // (blocks that are not there: the first page's, and what comes is not used)
                const uint32_t head = (ok >> b) & 1 ? uint32_t(__builtin_amdgcn_readlane(page, b)) * uint32_t(a.cache.heads) + uint32_t(at.hk) : 0u;
                return (uint64_t(head) << a.cache.page_shift) + ((uint32_t(kCacheTile) * uint32_t(tile) + 16u * uint32_t(b)) & ((1u << a.cache.page_shift) - 16u));
            };
            constexpr int kAll = kTurn * L::kCopies;
#pragma unroll
            for (int j = 0; j < (kAll + kWaves - 1) / kWaves; ++j) {
                const int c = wave + j * kWaves, i = c / L::kCopies, in_tile = c % L::kCopies;
                if (kAll % kWaves == 0 || c < kAll) copy_words<D, BITS>(to + i * L::kBytes, a, in_tile, place(2 * i + in_tile / (L::kCopies / 4) % 2));
            }
            if constexpr (BITS != 16) {
#pragma unroll
                for (int j = 0; j < 4 * kTurn / kWaves; ++j) {
                    const int c = wave + j * kWaves, i = c / 4;
                    copy_scales<D, BITS>(to + i * L::kBytes, a, c % 4, place(2 * i + c % 2));
                }
            }
        };
        int page = fetch_pages(t);
        uint64_t ok = there(page, t);
        copy(buf0, page, ok, t);
        page = fetch_pages(t + kTurn);
        start_rows(w, raw, a);
        const RowTokens<NB> rows = row_tokens<NB>(r, a, at);
        // The turn in `cur`, with the copies of the next one to `other` under way meanwhile.
        auto turn = [&](unsigned char* cur, unsigned char* other) __attribute__((always_inline)) {
            wait_vmcnt<0>();
            __syncthreads();  // the tiles are there, and no wave reads `other` any more
            const uint64_t ok_next = there(page, t + kTurn);
            if (t + kTurn < r.t1) {
                const int of_next = page;
                page = fetch_pages(t + 2 * kTurn);
                copy(other, of_next, ok_next, t + kTurn);
            }
#pragma unroll 1
            for (int i = key_wave; i < kTurn; i += kKeyWaves) {
                if (t + i >= r.t1) break;
                const unsigned char* const tile = cur + i * L::kBytes;
                TileWords<D, BITS> words;
                KeyScales<D, BITS> sc;
                TileScores<NB> x;
                TileWeights<D, BITS, NB> p;
                const uint32_t blocks = uint32_t(ok >> (2 * i)) & 3u;
                const bool whole = blocks == 3u && kCacheTile * (t + i + 1) <= r.first;
                uint32_t allowed[NB], live = 0;
                read_words<D, BITS, false>(words, tile);
                read_scales<D, BITS, false>(sc, tile);
                tile_scores(w, words, sc, x);
                read_scales<D, BITS, true>(sc, tile);
                if (!whole) {
                    live = tile_keys(allowed, r, rows, blocks, t + i);
                    trim_tile(w, x, sc, live, allowed);
                }
                tile_weights(w, x, sc, p);
                read_words<D, BITS, true>(words, tile);
                if constexpr (BITS == 16) {
                    if (!whole) clean_values(w, words, a, at, t + i, r.end, live, allowed);
                }
                tile_values(w, words, p);
            }
            t += kTurn;
            ok = ok_next;
        };
        while (true) {
            turn(buf0, buf1);
            if (t >= r.t1) break;
            turn(buf1, buf0);
            if (t >= r.t1) break;
        }
    } else {
        start_rows(w, raw, a);
    }
    __syncthreads();  // the buffers have been read
    // 16 rows at a time through the wave's part of LDS, so that neighbouring lanes store neighbouring columns, and what the waves with other keys
    // of these rows have is added
    float* const slab = reinterpret_cast<float*>(buf0) + wave * (kSlab / 4);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const float l = total_weight(w, nb);
        each_o(w, nb, [&](int j, int i, float v) __attribute__((always_inline)) { slab[l16 * kPitch + o_column<D, BITS>(j, 4 * q + i)] = v; });
        if (q == 0) stats[wave][l16] = f32x2_t{l != 0.f ? w.e[nb] : kNegInf, l};  // (a NaN goes along)
        __syncthreads();
        const int64_t part_row = int64_t(r.group_of * a.splits + r.split) * kRows + 16 * NB * row_wave + 16 * nb;
        for (int item = 64 * key_wave + lane; item < 16 * (D / 4); item += 64 * kKeyWaves) {
            const int row = item / (D / 4), col = 4 * (item % (D / 4));
            if (16 * nb + row >= at.rows) break;  // rows only grow
            f32x2_t of[kKeyWaves];
            float e = kNegInf, sum = 0.f;
#pragma unroll
            for (int k = 0; k < kKeyWaves; ++k) {
                of[k] = stats[row_wave + k * kRowWaves][row];
                e = fmaxf(e, of[k][0]);
            }
            f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kKeyWaves; ++k) {
                const f32x4_t u = *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(buf0) + (row_wave + k * kRowWaves) * (kSlab / 4) + row * kPitch + col);
                const float f = of[k][0] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(of[k][0] - e);
                sum = __builtin_fmaf(f, of[k][1], sum);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(f, u[i], v[i]);
            }
            if (a.splits == 1) {
                const float f = sum == 0.f ? 0.f : 1.f / sum;
                *reinterpret_cast<u32x2_t*>(o_row(a, at, 16 * nb + row) + col) = u32x2_t{pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f)};
            } else {
                *reinterpret_cast<f32x4_t*>(a.part + (part_row + row) * D + col) = v;
                if (col == 0) row_stats<D>(a, kRows)[part_row + row] = f32x2_t{e, sum};
            }
        }
        if (nb + 1 < NB) __syncthreads();
    }
}

// Joins the ranges' results of a row, in a fixed order: a wave per row of the padded tiles, on the XCD whose cache the row's ranges were written
// through (a head's ranges lie on one, and the remapping is the same).
template <int D>
__global__ __launch_bounds__(256) void cache_join_kernel(CacheAttnArgs a, int rows_of_tile) {
    const int lane = int(threadIdx.x) & 63;
    const int64_t id = int64_t(xcd_remap(int(blockIdx.x), int(gridDim.x))) * 4 + (threadIdx.x >> 6);
    const int64_t groups = int64_t(a.batch) * a.cache.heads * a.row_tiles;
    if (id >= groups * rows_of_tile) return;
    const int64_t group_of = id / rows_of_tile;
    const int in_tile = int(id - group_of * rows_of_tile);
    CacheWork at;
    at.row0 = int(group_of % a.row_tiles) * rows_of_tile;
    const int64_t bh = group_of / a.row_tiles;
    at.hk = int(bh % a.cache.heads);
    at.b = int(bh / a.cache.heads);
    int ql = a.q_len;
    if (a.q_lens != nullptr) ql = min(max(a.q_lens[at.b], 0), ql);
    if (int64_t(at.row0) + in_tile >= int64_t(ql) * a.group) return;
    const int64_t part_row = group_of * a.splits * rows_of_tile + in_tile;
    const float* const part = a.part + part_row * D;
    const int64_t step = int64_t(rows_of_tile) * D;
    // Four columns a lane, the ranges shared out over kParts groups of lanes, kAhead of a lane's on their way.  Every lane works out its ranges' factors
    // itself: a maximum and a sum over the wave, and only then the factors, took 0.4 us more (and eight on their way, with fewer waves resident, up to 1.5).
    constexpr int kLanes = D / 4, kParts = 64 / kLanes, kAhead = 4;
    const int col = 4 * (lane % kLanes), first = lane / kLanes;
    const f32x2_t* const stats = row_stats<D>(a, rows_of_tile) + part_row;
    float top = kNegInf, l = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = first; s0 < a.splits; s0 += kAhead * kParts) {
        f32x4_t u[kAhead];
        f32x2_t st[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int s = s0 + i * kParts;
            st[i] = f32x2_t{kNegInf, 0.f};
            u[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            if (s < a.splits) {
                st[i] = stats[int64_t(s) * rows_of_tile];
                u[i] = *reinterpret_cast<const f32x4_t*>(part + s * step + col);
            }
        }
        float most = top;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) most = fmaxf(most, st[i][0]);
        const float old = top == kNegInf ? 0.f : __builtin_amdgcn_exp2f(top - most);
        l *= old;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= old;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float f = st[i][0] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(st[i][0] - most);
            l = __builtin_fmaf(f, st[i][1], l);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(f, u[i][e], o[e]);
        }
        top = most;
    }
#pragma unroll
    for (int d = kLanes; d < 64; d *= 2) {  // (lanes below d have what is stored: its order is fixed)
        const float theirs = __shfl_xor(top, d), most = fmaxf(top, theirs);
        const float f = top == kNegInf ? 0.f : __builtin_amdgcn_exp2f(top - most);
        const float g = theirs == kNegInf ? 0.f : __builtin_amdgcn_exp2f(theirs - most);
        l = __builtin_fmaf(g, __shfl_xor(l, d), f * l);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(g, __shfl_xor(o[e], d), f * o[e]);
        top = most;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (first == 0)
        *reinterpret_cast<u32x2_t*>(o_row(a, at, in_tile) + col) = u32x2_t{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
}

template <int D, int BITS>
hipError_t launch_cache_attention_as(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream) {
    const unsigned grid = unsigned(a.row_tiles) * unsigned(a.splits) * unsigned(a.cache.heads) * unsigned(a.batch);
    if (!plan.share_tiles) {
        hipLaunchKernelGGL((cache_attention_kernel<D, BITS>), dim3(grid), dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    if (plan.tile_rows == 32)
        hipLaunchKernelGGL((cache_attention_rows_kernel<D, BITS, 1, 2>), dim3(grid), dim3(512), 0, stream, a);
    else if (plan.tile_rows == 64)
        hipLaunchKernelGGL((cache_attention_rows_kernel<D, BITS, 1, 4>), dim3(grid), dim3(512), 0, stream, a);
    else
        hipLaunchKernelGGL((cache_attention_rows_kernel<D, BITS, 2, 4>), dim3(grid), dim3(512), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t rows = int64_t(a.batch) * a.cache.heads * a.row_tiles * plan.tile_rows;
    hipLaunchKernelGGL((cache_join_kernel<D>), dim3(unsigned((rows + 3) / 4)), dim3(256), 0, stream, a, plan.tile_rows);
    return hipGetLastError();
}

}  // namespace
}  // namespace lowbit
