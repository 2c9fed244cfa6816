// Attention of new or drafted tokens over a paged, quantised cache: O = softmax(scale * Q K^T over the allowed keys) V.
//
// Row r of a kv head's problem is new token r / G of its q head r % G (G q heads share a kv head).  A workgroup takes 16 NB
// rows and a range of the keys; its four waves take tiles of 32 keys in turn, each with its own running maximum and sums, joined at the
// end (in wave order, then the key ranges in order: results do not depend on timing).
//
// Codes go from memory straight into the registers that the matrix cores read, without LDS: the cache's layout
// (kv_cache.h) is the operands' layout.  The products are computed transposed, S^T = K Q^T and O^T = V^T P^T, on 16x16x32
// MFMAs: lane (q, l16) then holds scores of query row l16 for keys 4q .. 4q + 3 of each 16, and the probabilities
// are already the second product's operand for its own keys.
//   * A code is never converted: 8 or 4 bits between zeros are an fp16 subnormal, code * 2^-24 (or, 4 bits higher, 16 times
//     that), which the matrix cores take exactly.  That is a byte permute for two codes, or a shift and a mask for
//     up to four.  The other operand carries the 1/16 and, per row or at the end, the 2^24.
//   * Scales multiply the fp32 sums: a key's scale its scores, a value's scale its probability (before that is rounded to fp16).
//     8 bits, codes u = c + 128:  sum q c = sum q u - 128 sum q, the second term being where the sums start from;
//       sum p s c = sum p s u - 128 sum p s, with the same rounded p s (a product with ones).
//     4 bits, x = s u + b per group: s (q.u) + b sum q for the scores, sum p s u + sum p b for the values (the latter in fp32).
//   * Q is a power of two per row (2^14 over its largest exponent) times fp16: exact for bf16 elements down to 2^-28 of the largest.
//   * p s is kept in fp16's range by a power of two per row, moved only when p s passes 2^12; p by the maximum, moved
//     only when a score passes it by 2^8.
// 16-bit caches take the same path with bf16 operands and no scales.
//
// Rounding: p s to fp16 (2^-11 of each; 16 bits: p to bf16, 2^-8 of each) and O to bf16; all else is fp32.
#pragma once

#include <cstdio>

#include "kv_cache.h"
#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {
namespace {

typedef _Float16 f16x8_t __attribute__((__vector_size__(8 * sizeof(_Float16))));

constexpr float kNegInf = -__builtin_inff();
constexpr int kCacheTile = 32;      // keys of a wave's tile
constexpr int kMaxCacheSplits = 64;  // a lane per split in the join
constexpr float kRise = 8.f;        // powers of two that a score may lie above the maximum in use
constexpr float kMostWeight = 0x1p12f;  // of p s: past it the row's factor moves
constexpr float kFirstFactor = 0x1p120f;  // of a row before its first keys: they set it
constexpr float kCodeUnit = 0x1p24f;    // 1 / the value of code 1 as an fp16

// A wave's tile as it comes from memory: per block of 16 keys the lane's words of K and V, and the scales of its four keys.
template <int D, int BITS>
struct CacheTile {
    static constexpr int kWords = CacheFmt<D, BITS>::kRow / 16;  // of K (a quarter of a row), and of V (a piece of four rows)
    static constexpr int kScales = CacheFmt<D, BITS>::kScaleBytes;  // words of four keys
    uint32_t k[2][kWords], v[2][kWords];
    uint32_t ks[2][kScales > 0 ? kScales : 1], vs[2][kScales > 0 ? kScales : 1];
};

// Running state of a wave for NB blocks of 16 rows.
template <int D, int BITS, int NB>
struct CacheRowsState {
    u32x4_t q[D / 32][NB];  // B operands (bf16, or fp16 times the row's power of two)
    f32x4_t o[D / 16][NB];  // O^T: lane (q, l16): row l16, columns column(j, 4q + i)
    f32x4_t sum[NB];        // 8 bits: the sum of the rounded p s
    float m[NB], l[NB];     // maximum in use (-inf: no key yet), the lane's own keys' sum of p
    float r[NB];            // power of two on p s
    float low[NB][2];       // 4 bits: the lane's own keys' sum of p b
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

// The score operand ks of block kb: lane (q, l16) has eight codes of key l16.
template <int D, int BITS>
__device__ __forceinline__ u32x4_t k_operand(const CacheTile<D, BITS>& t, int kb, int ks) {
    if constexpr (BITS == 16) {
        return u32x4_t{t.k[kb][4 * ks], t.k[kb][4 * ks + 1], t.k[kb][4 * ks + 2], t.k[kb][4 * ks + 3]};
    } else if constexpr (BITS == 8) {
        const uint32_t a = t.k[kb][2 * ks], b = t.k[kb][2 * ks + 1];
        return u32x4_t{perm_b32(0, a, 0x0C010C00u), perm_b32(0, a, 0x0C030C02u), perm_b32(0, b, 0x0C010C00u), perm_b32(0, b, 0x0C030C02u)};
    } else {
        const uint32_t w = t.k[kb][ks], h = w >> 8;  // the second and fourth pair come 16 times too large
        return u32x4_t{w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u};
    }
}

// The value operand j of a tile: lane (q, l16) has column o_column(j, l16) of keys 4q .. of block 0, then of block 1.
// Odd columns of 4-bit codes come 16 times too large.
template <int D, int BITS>
__device__ __forceinline__ u32x4_t v_operand(const CacheTile<D, BITS>& t, int j) {
    u32x4_t a;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int p = 0; p < 2; ++p) {  // keys 2p and 2p + 1
            constexpr int kPiece = CacheFmt<D, BITS>::kPiece;
            uint32_t x;
            if constexpr (BITS == 16) {
                const int at = kPiece / 4 * 2 * p + j / 2;
                x = perm_b32(t.v[kb][at + kPiece / 4], t.v[kb][at], j % 2 ? 0x07060302u : 0x05040100u);
            } else if constexpr (BITS == 8) {
                const int at = kPiece / 4 * 2 * p + j / 4;
                x = perm_b32(t.v[kb][at + kPiece / 4], t.v[kb][at], 0x0C040C00u + 0x00010001u * (j % 4));
            } else if constexpr (kPiece == 4) {
                const int byte = 2 * (j / 4) + j % 4 / 2;
                x = perm_b32(t.v[kb][2 * p + 1], t.v[kb][2 * p], 0x0C040C00u + 0x00010001u * byte) & (j % 2 ? 0x00F000F0u : 0x000F000Fu);
            } else {
                x = (j / 2 ? t.v[kb][p] >> 8 : t.v[kb][p]) & (j % 2 ? 0x00F000F0u : 0x000F000Fu);
            }
            a[2 * kb + p] = x;
        }
    return a;
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

template <int D, int BITS, int NB>
__device__ __forceinline__ void load_queries(CacheRowsState<D, BITS, NB>& w, const CacheAttnArgs& a, const CacheWork& at) {
    const int lane = int(threadIdx.x) & 63, q = lane >> 4, l16 = lane & 15;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int row = at.row0 + 16 * nb + l16;
        const bool in = 16 * nb + l16 < at.rows;
        const int t = in ? row / a.group : 0, g = in ? row - t * a.group : 0;
        const uint16_t* src = a.q + int64_t(at.b) * a.q_batch + int64_t(t) * a.q_token + int64_t(at.hk * a.group + g) * a.q_head;
        u32x4_t raw[D / 32];
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            raw[ks] = u32x4_t{0, 0, 0, 0};
            if (in) raw[ks] = *reinterpret_cast<const u32x4_t*>(src + q_element<BITS>(ks, q));
        }
        w.gain[nb] = a.scale_log2;
        w.start[nb] = w.qsum[nb][0] = w.qsum[nb][1] = 0.f;
        if constexpr (BITS == 16) {
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) w.q[ks][nb] = raw[ks];
        } else {
            float top = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(__builtin_fabsf(bf16_low(raw[ks][e])), __builtin_fabsf(bf16_high(raw[ks][e]))));
            top = row_max(top);
            int up = 14 - (int((__float_as_uint(top) >> 23) & 255u) - 127);  // the largest element comes to lie in [2^14, 2^15)
            up = up > 126 ? 126 : up < -113 ? -113 : up;  // (infinite or NaN: they stay that)
            const float f = power_of_two(up);
            float sum[D / 64];
#pragma unroll
            for (int g64 = 0; g64 < D / 64; ++g64) sum[g64] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = bf16_low(raw[ks][e]) * f, y = bf16_high(raw[ks][e]) * f;
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
        w.m[nb] = kNegInf;
        w.l[nb] = w.low[nb][0] = w.low[nb][1] = 0.f;
        w.r[nb] = kFirstFactor;
        w.sum[nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) w.o[j][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
}

// Where the 16 keys of a block lie: (page * heads + head) * page_size + place of the first in its page; -1: no such page.
__device__ __forceinline__ int64_t block_place(const CacheAttnArgs& a, const CacheWork& at, int key0, int end) {
    if (key0 >= end) return -1;
    const int page = __builtin_amdgcn_readfirstlane(a.table[int64_t(at.b) * a.table_stride + (key0 >> a.cache.page_shift)]);
    if (uint32_t(page) >= uint32_t(a.cache.pages)) return -1;
    return ((int64_t(page) * a.cache.heads + at.hk) << a.cache.page_shift) + (key0 & ((1 << a.cache.page_shift) - 1));
}

template <int D, int BITS>
__device__ __forceinline__ void load_block(CacheTile<D, BITS>& t, const CacheAttnArgs& a, int kb, int64_t place) {
    using F = CacheFmt<D, BITS>;
    const int lane = int(threadIdx.x) & 63, q = lane >> 4, l16 = lane & 15;
    const uint32_t none = place < 0 ? 0u : 1u;  // an empty resource: zeros without a read
    const int64_t p = place < 0 ? 0 : place;
    const auto kr = make_rsrc(a.cache.k + p * F::kRow, none * 16u * F::kRow);
    const auto vr = make_rsrc(a.cache.v + p * F::kRow, none * 16u * F::kRow);
    constexpr int kW = CacheTile<D, BITS>::kWords;
    if constexpr (kW >= 4) {
#pragma unroll
        for (int i = 0; i < kW / 4; ++i) {
            const u32x4_t x = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(kr, uint32_t(l16 * F::kRow + 16 * q) + 64u * i, 0, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) t.k[kb][4 * i + e] = x[e];
        }
        constexpr int kT = F::kBlock;
#pragma unroll
        for (int i = 0; i < kW / 4; ++i) {  // 16 bytes: kBlock keys
            const u32x4_t x = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                              vr, uint32_t(4 * q / kT * (kT * F::kRow) + 16 * l16) + uint32_t(kT * F::kRow * i), 0, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) t.v[kb][4 * i + e] = x[e];
        }
    } else {
        const u32x2_t x = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(kr, uint32_t(l16 * F::kRow + 8 * q), 0, 0));
        const u32x2_t y = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(vr, uint32_t(q * (4 * F::kRow) + 8 * l16), 0, 0));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            t.k[kb][e] = x[e];
            t.v[kb][e] = y[e];
        }
    }
    if constexpr (BITS != 16) {
        constexpr int kS = F::kScaleBytes;
        const auto ksr = make_rsrc(a.cache.k_scales + p * kS, none * 16u * kS);
        const auto vsr = make_rsrc(a.cache.v_scales + p * kS, none * 16u * kS);
        if constexpr (kS == 2) {
            const u32x2_t x = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(ksr, uint32_t(8 * q), 0, 0));
            const u32x2_t y = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(vsr, uint32_t(8 * q), 0, 0));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                t.ks[kb][e] = x[e];
                t.vs[kb][e] = y[e];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kS / 4; ++i) {
                const u32x4_t x = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ksr, uint32_t(4 * kS * q + 16 * i), 0, 0));
                const u32x4_t y = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(vsr, uint32_t(4 * kS * q + 16 * i), 0, 0));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    t.ks[kb][4 * i + e] = x[e];
                    t.vs[kb][4 * i + e] = y[e];
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

__device__ __forceinline__ bool odd_bf16(uint32_t half) { return (half & 0x7F80u) == 0x7F80u; }

// 16-bit values that are an infinity or a NaN, in a tile with keys that some row leaves out (zero in a product does not silence them):
// they are added to the rows that take their keys, and become zeros in the operand.
template <int D, int NB>
__device__ __forceinline__ void set_odd_values_aside(CacheRowsState<D, 16, NB>& w, CacheTile<D, 16>& t, const CacheAttnArgs& a,
                                                     const int64_t (&place)[2], const uint32_t (&allowed)[NB]) {
    using F = CacheFmt<D, 16>;
    constexpr int kW = CacheTile<D, 16>::kWords;
    const int lane = int(threadIdx.x) & 63, q = lane >> 4;
    bool odd = false;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int e = 0; e < kW; ++e) odd = odd || odd_bf16(t.v[kb][e]) || odd_bf16(t.v[kb][e] >> 16);
    if (!__any(odd)) return;
    for (int key = 0; key < kCacheTile; ++key) {
        const int64_t p = key < 16 ? place[0] : place[1];
        bool some = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) some = some || ((allowed[nb] >> key) & 1);
        if (p < 0 || !__any(some)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the lane's columns: pieces 4q + i
            const unsigned char* src = a.cache.v + p * F::kRow + F::v_offset(uint32_t(key & 15), uint32_t(4 * q + i));
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const uint32_t b = reinterpret_cast<const uint16_t*>(src)[j];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    if (odd_bf16(b) && ((allowed[nb] >> key) & 1)) w.o[j][nb][i] += bf16_low(b);
            }
        }
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int e = 0; e < kW; ++e) {
            if (odd_bf16(t.v[kb][e])) t.v[kb][e] &= 0xFFFF0000u;
            if (odd_bf16(t.v[kb][e] >> 16)) t.v[kb][e] &= 0xFFFFu;
        }
}

// One tile.  PARTIAL: some row leaves out some of its keys (bit of `allowed` clear; bit of `live` clear: a key that is not there).
template <bool PARTIAL, int D, int BITS, int NB>
__device__ __forceinline__ void cache_step(CacheRowsState<D, BITS, NB>& w, CacheTile<D, BITS>& t, const CacheAttnArgs& a,
                                           const int64_t (&place)[2], uint32_t live, const uint32_t (&allowed)[NB]) {
    constexpr int kGroups = CacheFmt<D, BITS>::kGroups;
    const int lane = int(threadIdx.x) & 63, q = lane >> 4;
    if constexpr (PARTIAL) {  // what lies where no key is may be anything
        constexpr int kW = CacheTile<D, BITS>::kWords;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!((live >> (16 * kb + 4 * q + i)) & 1)) {
                    if constexpr (BITS == 16) {
#pragma unroll
                        for (int e = 0; e < kW / 4; ++e) t.v[kb][kW / 4 * i + e] = 0;
                    } else if constexpr (BITS == 8) {
                        t.vs[kb][i / 2] &= i % 2 ? 0xFFFFu : 0xFFFF0000u;
                    } else {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) t.vs[kb][i * kGroups + g] = 0;
                    }
                }
        if constexpr (BITS == 16) set_odd_values_aside<D, NB>(w, t, a, place, allowed);
    }
    // scores, in powers of two
    f32x4_t s[2][NB];
    if constexpr (BITS == 4) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            f32x4_t raw[kGroups][NB];
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) raw[g][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                const u32x4_t k = k_operand<D, BITS>(t, kb, ks);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) raw[ks / 2][nb] = cache_mfma<BITS>(k, w.q[ks][nb], raw[ks / 2][nb]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float x = 0.f, y = 0.f;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        x = __builtin_fmaf(raw[g][nb][i], scale_at<D, BITS>(t.ks[kb], i, g), x);
                        y = __builtin_fmaf(w.qsum[nb][g], low_at<D, BITS>(t.ks[kb], i, g), y);
                    }
                    s[kb][nb][i] = __builtin_fmaf(x, w.gain[nb], y);
                }
        }
    } else {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) s[kb][nb] = f32x4_t{w.start[nb], w.start[nb], w.start[nb], w.start[nb]};
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                const u32x4_t k = k_operand<D, BITS>(t, kb, ks);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) s[kb][nb] = cache_mfma<BITS>(k, w.q[ks][nb], s[kb][nb]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    s[kb][nb][i] *= BITS == 16 ? w.gain[nb] : w.gain[nb] * scale_at<D, 8>(t.ks[kb], i, 0);
        }
    }
    bool takes[2][NB][4];
    if constexpr (PARTIAL) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    takes[kb][nb][i] = (allowed[nb] >> (16 * kb + 4 * q + i)) & 1;
                    s[kb][nb][i] = takes[kb][nb][i] ? s[kb][nb][i] : kNegInf;
                }
    }
    // the maximum follows where a score is more than kRise above it
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float top = kNegInf;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s[kb][nb][i]);
        if (__any(top > w.m[nb] + kRise)) {
            top = row_max(top);
            const bool move = top > w.m[nb] + kRise;
            const float f = move ? __builtin_amdgcn_exp2f(w.m[nb] - top) : 1.f;
            w.m[nb] = move ? top : w.m[nb];
            w.l[nb] *= f;
            w.low[nb][0] *= f;
            w.low[nb][1] *= f;
            float fo = f;
            if constexpr (BITS != 16) {  // the values that now count may be far smaller: let p s set the row's factor anew
                const float r = move ? fminf(w.r[nb] * 0x1p30f, kFirstFactor) : w.r[nb];
                fo *= r / w.r[nb];
                w.r[nb] = r;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w.sum[nb][i] *= fo;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) w.o[j][nb][i] *= fo;
        }
    }
    // probabilities, and their products with the values' scales
    u32x4_t p[NB][kGroups];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const float m = w.m[nb] == kNegInf ? 0.f : w.m[nb];  // without a key yet every score is -inf
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[kb][nb][i] = __builtin_amdgcn_exp2f(s[kb][nb][i] - m);
                w.l[nb] += s[kb][nb][i];
            }
        if constexpr (BITS == 16) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 4; i += 2) p[nb][0][2 * kb + i / 2] = pack_bf16(s[kb][nb][i], s[kb][nb][i + 1]);
        } else {
            // a probability times a NaN scale: in the rows that take the key only
            auto weight = [&](int kb, int i, int g) __attribute__((always_inline)) {
                const float x = s[kb][nb][i] * scale_at<D, BITS>(t.vs[kb], i, g);
                return PARTIAL && !takes[kb][nb][i] ? 0.f : x;
            };
            float top = 0.f, x[kGroups][2][4];
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[g][kb][i] = weight(kb, i, g);
                        top = fmaxf(top, x[g][kb][i]);
                        if constexpr (BITS == 4) {
                            const float y = s[kb][nb][i] * low_at<D, BITS>(t.vs[kb], i, g);
                            w.low[nb][g] += PARTIAL && !takes[kb][nb][i] ? 0.f : y;
                        }
                    }
            if (__any(top * w.r[nb] > kMostWeight)) {  // the row's factor: such that the largest of these lies in [1, 2)
                top = row_max(top);
                const bool move = top * w.r[nb] > kMostWeight;
                int up = 127 - int(__float_as_uint(top) >> 23);
                up = up < -126 ? -126 : up > 120 ? 120 : up;
                const float r = move ? power_of_two(up) : w.r[nb], f = r / w.r[nb];
                w.r[nb] = r;
#pragma unroll
                for (int i = 0; i < 4; ++i) w.sum[nb][i] *= f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) w.o[j][nb][i] *= f;
            }
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; i += 2) p[nb][g][2 * kb + i / 2] = pack_f16(x[g][kb][i] * w.r[nb], x[g][kb][i + 1] * w.r[nb]);
        }
    }
    // values
    if constexpr (BITS == 8) {
        const u32x4_t ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) w.sum[nb] = cache_mfma<BITS>(ones, p[nb][0], w.sum[nb]);
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        const u32x4_t v = v_operand<D, BITS>(t, j);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) w.o[j][nb] = cache_mfma<BITS>(v, p[nb][BITS == 4 ? j / 4 : 0], w.o[j][nb]);
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

template <int D, int BITS, int NB>
__global__ __launch_bounds__(256, NB == 4 ? 1 : 2) void cache_attention_kernel(CacheAttnArgs a) {
    constexpr int kWaves = 4, kRows = 16 * NB;
    __shared__ __attribute__((aligned(16))) float lds_o[kWaves][kRows * D];
    __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows];
    __shared__ int last_split;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int q = lane >> 4, l16 = lane & 15;
    // row tiles of one range of keys next to each other on one XCD, then the ranges of one head
    int id = xcd_remap(int(blockIdx.x), int(gridDim.x));
    const int rt = id % a.row_tiles;
    id /= a.row_tiles;
    const int split = id % a.splits;
    id /= a.splits;
    CacheWork at;
    at.hk = id % a.cache.heads;
    at.b = id / a.cache.heads;
    const int group_of = (at.b * a.cache.heads + at.hk) * a.row_tiles + rt;  // of the workgroups that share rows
    int n = a.lens[at.b];
    n = n < 0 ? 0 : n < a.kv_len ? n : a.kv_len;
    int ql = a.q_len;
    if (a.q_lens != nullptr) {
        const int v = a.q_lens[at.b];
        ql = v < 0 ? 0 : v < ql ? v : ql;
    }
    n = __builtin_amdgcn_readfirstlane(n);
    ql = __builtin_amdgcn_readfirstlane(ql);
    at.n = n;
    at.base = n - ql;
    at.row0 = rt * kRows;
    const int64_t left = int64_t(ql) * a.group - at.row0;
    if (left <= 0) return;  // rows past the request's last token: none of this tile's workgroups counts
    at.rows = left < kRows ? int(left) : kRows;

    // keys that some row takes: [0, end); that every row takes: [0, first)
    const bool tree = a.tree != nullptr;
    const int64_t last = tree ? n : int64_t(at.base) + (at.row0 + at.rows - 1) / a.group + 1;
    const int end = last < 0 ? 0 : last < n ? int(last) : n;
    const int64_t first64 = tree ? at.base : int64_t(at.base) + at.row0 / a.group + 1;
    const int first = first64 < 0 ? 0 : first64 < n ? int(first64) : n;
    const int tiles = (end + kCacheTile - 1) / kCacheTile;
    // the ranges share the keys there are, not the keys there could be
    const int t0 = int(int64_t(tiles) * split / a.splits), t1 = int(int64_t(tiles) * (split + 1) / a.splits);

    CacheRowsState<D, BITS, NB> w;
    load_queries(w, a, at);
    int token[NB];
    uint64_t own[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int row = 16 * nb + l16 < at.rows ? at.row0 + 16 * nb + l16 : at.row0;
        token[nb] = row / a.group;
        own[nb] = 0;
        if (tree) own[nb] = a.tree[int64_t(at.b) * a.q_len + token[nb]];
    }

    for (int t = t0 + wave; t < t1; t += kWaves) {
        const int key0 = kCacheTile * t;
        CacheTile<D, BITS> x;
        const int64_t place[2] = {block_place(a, at, key0, end), block_place(a, at, key0 + 16, end)};
        load_block(x, a, 0, place[0]);
        load_block(x, a, 1, place[1]);
        uint32_t live = first_bits(int64_t(n) - key0 - 1);
        live &= (place[0] < 0 ? 0u : 0xFFFFu) | (place[1] < 0 ? 0u : 0xFFFF0000u);
        uint32_t allowed[NB];
        if (live != ~0u || key0 + kCacheTile > first) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) allowed[nb] = live & taken(tree, own[nb], token[nb], at.base, key0);
            cache_step<true>(w, x, a, place, live, allowed);
        } else {
            cache_step<false>(w, x, a, place, live, allowed);
        }
    }

    // ---- the waves' results, as numbers: row by row in LDS ----
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const float l = row_sum(w.l[nb]);
        float low[2] = {0.f, 0.f};
        if constexpr (BITS == 4) {
            low[0] = row_sum(w.low[nb][0]);
            low[1] = row_sum(w.low[nb][1]);
        }
        const float f = BITS == 16 ? 1.f : kCodeUnit / w.r[nb], minus = BITS == 8 ? 128.f / w.r[nb] : 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = w.o[j][nb][i] * (BITS == 4 && j % 2 ? f * 0.0625f : f);
                if constexpr (BITS == 8) v -= minus * w.sum[nb][i];
                if constexpr (BITS == 4) v += low[j / 4];
                lds_o[wave][(16 * nb + l16) * D + o_column<D, BITS>(j, 4 * q + i)] = v;
            }
        if (q == 0) {
            lds_m[wave][16 * nb + l16] = w.m[nb];
            lds_l[wave][16 * nb + l16] = l;
        }
    }
    __syncthreads();
    // O of a row of the tile, columns col .. col + 3, divided by the sum l (0: a row without keys)
    auto store4 = [&](int in_tile, int col, f32x4_t v, float l) {
        const int row = at.row0 + in_tile;
        const int tok = row / a.group, g = row - tok * a.group;
        uint16_t* dst = a.o + int64_t(at.b) * a.o_batch + int64_t(tok) * a.o_token + int64_t(at.hk * a.group + g) * a.o_head + col;
        const float r = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{pack_bf16(v[0] * r, v[1] * r), pack_bf16(v[2] * r, v[3] * r)};
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
            if (lds_m[i][row] == kNegInf) {  // no key (a sum of 0) or a NaN score
                total += lds_l[i][row];
                continue;
            }
            const float f = __builtin_amdgcn_exp2f(lds_m[i][row] - top);
            total += f * lds_l[i][row];
            const f32x4_t u = *reinterpret_cast<const f32x4_t*>(&lds_o[i][row * D + col]);
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
    float* const factors = &lds_o[0][0];  // [rows][splits], then the sums [rows]
    float* const totals = factors + kRows * kMaxCacheSplits;
    for (int row = wave; row < at.rows; row += kWaves) {  // a lane per split
        const uint32_t from = uint32_t(lane * kRows + row) * kPart + 4u * D;
        const bool in = lane < a.splits;
        const float m = in ? __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(part_rs, from, 0, kSc1)) : kNegInf;
        const float l = in ? __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(part_rs, from + 4u, 0, kSc1)) : 0.f;
        float top = m;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
        const float f = m == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m - top);
        float sum = m == kNegInf ? l : f * l;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
        if (in) factors[row * kMaxCacheSplits + lane] = f;
        if (lane == 0) totals[row] = sum;
    }
    __syncthreads();
    constexpr int kAhead = 8;
    for (int item = int(threadIdx.x); item < items; item += 64 * kWaves) {
        const int row = item / (D / 4), col = 4 * (item % (D / 4));
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = 0; s0 < a.splits; s0 += kAhead) {
            f32x4_t u[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)  // a split past the last reads as zeros
                u[i] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                       part_rs, s0 + i < a.splits ? uint32_t((s0 + i) * kRows + row) * kPart + 4u * uint32_t(col) : 0xFFFFFF00u,
                                                       0, kSc1));
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float f = s0 + i < a.splits ? factors[row * kMaxCacheSplits + s0 + i] : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, u[i][e], v[e]);
            }
        }
        store4(row, col, v, totals[row]);
    }
}

template <int D, int BITS>
hipError_t launch_cache_attention_as(const CacheAttnArgs& a, int row_blocks, hipStream_t stream) {
    const unsigned grid = unsigned(a.row_tiles) * unsigned(a.splits) * unsigned(a.cache.heads) * unsigned(a.batch);
    if (row_blocks == 1)
        hipLaunchKernelGGL((cache_attention_kernel<D, BITS, 1>), dim3(grid), dim3(256), 0, stream, a);
    else if (row_blocks == 2)
        hipLaunchKernelGGL((cache_attention_kernel<D, BITS, 2>), dim3(grid), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((cache_attention_kernel<D, BITS, 4>), dim3(grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace lowbit
