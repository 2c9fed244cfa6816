// Writing keys and values of new tokens into a paged cache, quantised on the way, and reading rows back as bf16.
//
//   8 bits: s = up(max|x| * (1/127)) per token and head, code = rint(x / s), stands for s * code;
//   4 bits: per group of 64 elements  b = min x, s = up((max x - b) * (1/15)), code = rint((x - b) / s), stands for s * code + b;
// up(t): the smallest bf16 not below t, so that no code leaves its range and a bf16 scale costs no more than its share
// of the range.  1/127 and 1/15 are fp32 numbers, b is a bf16 already, x / s is a correctly rounded fp32 division and rint goes to
// even: codes depend on the inputs alone.  A group with an infinity or a NaN (or, at 4 bits, a range past fp32) gets a NaN for its scale and reads
// back as NaN: its neighbours are untouched.
//
// Bound by memory (every element read once and written once) or, for a few tokens, by the launch and the two loads that wait for each other (the
// slot, then the row).  8 elements per lane: 16 or 8 lanes hold a token's row of a head.  A wave takes keys and values of its rows together: one
// look at the slot, twice the loads in flight; maxima meet by operand routing within 16 lanes, and codes cost one division a row.  With a wave for
// keys and another for values, exchanges through shared memory and a division an element, 16,510 tokens read from 4 bits and 4,084 of 16 heads of 64
// written in 8 took 21 and 10 us with their data in the last-level cache, where they take 15.3 and 6.4.
// Measured, 8 heads of 128, everything from and to HBM, launch included (us at 16, 8 and 4 bits; with what the last pass left in the caches):
//   61 tokens written 2.0, 2.6, 2.8, read 2.0, 2.1, 2.2;
//   4,084 tokens written 9.9, 8.2, 8.5 (6.4, 6.3, 6.9), read 9.9, 7.9, 7.6 (5.2, 5.4, 6.0);
//   16,510 tokens written 28.3, 24.3, 24.9 (21.2, 20.0, 21.5), read 27.8, 23.1, 21.8 (20.9, 16.8, 15.3): 135, 102 and 87 MB, 4.8, 4.2 and 3.5 TB/s
//   written, 4.9, 4.4 and 4.0 read.
#include "kv_cache.h"
#include "lowbit_device.h"
#include "decode_internal.h"

namespace lowbit {
namespace {

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }
// The smallest bf16 not below f >= 0.
__device__ __forceinline__ uint32_t up_bf16(float f) { return (__float_as_uint(f) + 0xFFFFu) >> 16; }

constexpr uint32_t kNanBf16 = 0x7FC0;
constexpr uint32_t kInfBf16 = 0x7F80;

// A value of another lane of the 16 of a row, by the adders' operand routing: no trip through shared memory.
template <int CONTROL>
__device__ __forceinline__ uint32_t from_lane(uint32_t x) {
    return uint32_t(__builtin_amdgcn_mov_dpp(int(x), CONTROL, 0xF, 0xF, true));
}
constexpr int kOtherEight = 0x128;  // rotation by 8 lanes

// Where a row's token lies: base addresses of its head's page in k (v alike) and in the scales, and its place in the page.
struct Place {
    int64_t page_row;  // (page * heads + head) * page_size
    uint32_t token;
};

// A workgroup's rows: 16 (heads of 128) or 32 tokens of a head after each other, keys and values, a wave takes a quarter of them.  The head counts
// fastest over the workgroups: with 8 heads, or a multiple, a head's pages and scales then stay in one XCD's cache.
template <int D, class F>
__device__ __forceinline__ void for_each_row(const CacheArgs& c, const CacheRows& r, F f) {
    constexpr int kLanes = D / 8, kRows = 64 / kLanes;
    const int lane = int(threadIdx.x) & 63;
    const uint32_t capacity = uint32_t(c.pages) << c.page_shift;
    const uint32_t heads = uint32_t(c.heads), step = gridDim.x / heads, step_heads = gridDim.x % heads;
    int64_t tb = blockIdx.x / heads;
    uint32_t h = blockIdx.x % heads;
    for (;;) {
        const int64_t t = (tb * 4 + (threadIdx.x >> 6)) * kRows + lane / kLanes;
        if (tb * 4 * kRows >= r.tokens) return;
        const uint32_t slot = t < r.tokens ? uint32_t(r.slots[t]) : ~0u;
        const bool in = slot < capacity;  // a negative slot is past it too
        f(t, int(h), in, Place{(int64_t(in ? slot >> c.page_shift : 0u) * c.heads + h) << c.page_shift, slot & ((1u << c.page_shift) - 1)}, lane % kLanes);
        tb += step;
        if ((h += step_heads) >= heads) {
            h -= heads;
            ++tb;
        }
    }
}

// Eight elements of a token's key (value) of a head, the i-th eight of the row.  Lanes without a row go along (the rows' lanes exchange values).
template <int D, int BITS, bool is_v>
__device__ __forceinline__ void write_eight(const CacheArgs& c, u32x4_t raw, bool in, Place at, int i) {
    using F = CacheFmt<D, BITS>;
    unsigned char* const page = (is_v ? c.v : c.k) + at.page_row * F::kRow;
    if constexpr (BITS == 16) {
        if (!in) return;
        if (!is_v || F::kPiece == 16) {
            *reinterpret_cast<u32x4_t*>(page + (is_v ? F::v_offset(at.token, i) : at.token * F::kRow + 16 * i)) = raw;
        } else {
            *reinterpret_cast<u32x2_t*>(page + F::v_offset(at.token, 2 * i)) = u32x2_t{raw[0], raw[1]};
            *reinterpret_cast<u32x2_t*>(page + F::v_offset(at.token, 2 * i + 1)) = u32x2_t{raw[2], raw[3]};
        }
        return;
    }
    float x[8];
    typedef unsigned short pair_t __attribute__((ext_vector_type(2)));
    pair_t bigs = 0;
    float lo = __builtin_inff(), hi = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = e & 1 ? __uint_as_float(raw[e / 2] & 0xFFFF0000u) : bf16_float(raw[e / 2]);
        if (e % 2 == 0) bigs = __builtin_elementwise_max(bigs, __builtin_bit_cast(pair_t, raw[e / 2] & 0x7FFF7FFFu));
        if constexpr (BITS == 4) {
            lo = fminf(lo, x[e]);
            hi = fmaxf(hi, x[e]);
        }
    }
    uint32_t big = max(bigs[0], bigs[1]);  // the largest magnitude's bits; from kInfBf16 on the group is not finite
    constexpr int kShare = BITS == 8 ? D / 8 : kCacheGroup / 8;  // lanes of a group
    auto meet = [&](auto other) __attribute__((always_inline)) {
        big = max(big, other(big));
        if constexpr (BITS == 4) {
            lo = fminf(lo, __uint_as_float(other(__float_as_uint(lo))));
            hi = fmaxf(hi, __uint_as_float(other(__float_as_uint(hi))));
        }
    };
    meet([](uint32_t x) { return from_lane<0xB1>(x); });   // the neighbour
    meet([](uint32_t x) { return from_lane<0x4E>(x); });   // the other pair of a quad
    meet([](uint32_t x) { return from_lane<0x141>(x); });  // the other quad of eight lanes, whose lanes agree by now
    if constexpr (kShare == 16) meet([](uint32_t x) { return from_lane<kOtherEight>(x); });
    const float range = BITS == 8 ? bf16_float(big) : hi - lo;
    const bool fine = big < kInfBf16 && range < __builtin_inff();
    const uint32_t sb = fine ? up_bf16(range * (BITS == 8 ? 1.f / 127.f : 1.f / 15.f)) : kNanBf16;
    float s = bf16_float(sb);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if constexpr (BITS == 4) x[e] -= lo;
    if (s < 0x1p-60f) {  // tiny groups: both sides of the division by a power of two that keeps its intermediates normal
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= 0x1p64f;
        s *= 0x1p64f;
    }
    // t / s rounded once, without a division per element: r is 1 / s rounded, q = t r is within an ulp or so of t / s, t - q s is exact in an fma,
    // and q + (t - q s) r rounds to the fp32 next to t / s.  Adding 1.5 * 2^23 (and 128) rounds that to a whole number, to even, in the low bits.
    const bool any = fine && sb != 0;
    const float r = any ? 1.f / s : 0.f;
    uint32_t code[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = x[e] * r;
        code[e] = __float_as_uint(__builtin_fmaf(__builtin_fmaf(-q, s, x[e]), r, q) + (BITS == 8 ? 12582912.f + 128.f : 12582912.f));
        if constexpr (BITS == 4) code[e] = any ? code[e] & 15u : 0u;
    }
    unsigned char* const scales = (is_v ? c.v_scales : c.k_scales) + (at.page_row + at.token) * F::kScaleBytes;
    if constexpr (BITS == 8) {
        if (!in) return;
        const auto low_bytes = [&](int e) {
            return any ? perm_b32(perm_b32(code[e + 3], code[e + 2], 0x0C0C0400u), perm_b32(code[e + 1], code[e], 0x0C0C0400u), 0x05040100u) : 0x80808080u;
        };
        const u32x2_t w = {low_bytes(0), low_bytes(4)};
        if (!is_v || F::kPiece == 8) {
            *reinterpret_cast<u32x2_t*>(page + (is_v ? F::v_offset(at.token, i) : at.token * F::kRow + 8 * i)) = w;
        } else {
            *reinterpret_cast<uint32_t*>(page + F::v_offset(at.token, 2 * i)) = w[0];
            *reinterpret_cast<uint32_t*>(page + F::v_offset(at.token, 2 * i + 1)) = w[1];
        }
        if (i == 0) *reinterpret_cast<uint16_t*>(scales) = uint16_t(sb);
    } else {
        const int g = i / 8, j = i % 8;  // group, eight elements of it
        if (is_v) {
            // 8 elements: pieces 2j and 2j + 1 of this group, two bytes each
            const uint32_t even = code[0] | code[1] << 4 | code[2] << 8 | code[3] << 12;
            const uint32_t odd = code[4] | code[5] << 4 | code[6] << 8 | code[7] << 12;
            if constexpr (F::kGroups == 2) {  // the other group's two bytes stand beside them: one piece a lane
                const uint32_t other = from_lane<kOtherEight>(g == 0 ? odd : even);
                if (in) *reinterpret_cast<uint32_t*>(page + F::v_offset(at.token, 2 * j + g)) = g == 0 ? even | other << 16 : other | odd << 16;
            } else if (in) {
                *reinterpret_cast<uint16_t*>(page + F::v_offset(at.token, 2 * j)) = uint16_t(even);
                *reinterpret_cast<uint16_t*>(page + F::v_offset(at.token, 2 * j + 1)) = uint16_t(odd);
            }
        } else if (in) {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) w |= code[e] << (4 * (e / 2 + 4 * (e % 2)));
            *reinterpret_cast<uint32_t*>(page + at.token * F::kRow + j / 2 * (8 * F::kGroups) + 8 * g + 4 * (j % 2)) = w;
        }
        if (in && j == 0)  // the smallest value is one of the inputs: a bf16
            *reinterpret_cast<uint32_t*>(scales + 4 * g) = sb | (fine ? __float_as_uint(lo) & 0xFFFF0000u : 0u);
    }
}

template <int D, int BITS>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheArgs c, CacheRows r) {
    for_each_row<D>(c, r, [&](int64_t t, int h, bool in, Place at, int i) __attribute__((always_inline)) {
        u32x4_t k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
        if (in) {
            k = *reinterpret_cast<const u32x4_t*>(r.k + t * r.k_token + int64_t(h) * r.k_head + 8 * i);
            v = *reinterpret_cast<const u32x4_t*>(r.v + t * r.v_token + int64_t(h) * r.v_head + 8 * i);
        }
        write_eight<D, BITS, false>(c, k, in, at, i);
        write_eight<D, BITS, true>(c, v, in, at, i);
    });
}

template <int D, int BITS, bool is_v>
__device__ __forceinline__ u32x4_t read_eight(const CacheArgs& c, Place at, int i) {
    using F = CacheFmt<D, BITS>;
    const unsigned char* const page = (is_v ? c.v : c.k) + at.page_row * F::kRow;
    const unsigned char* const scales = (is_v ? c.v_scales : c.k_scales) + (at.page_row + at.token) * F::kScaleBytes;
    u32x4_t out;
    if constexpr (BITS == 16) {
        if (!is_v || F::kPiece == 16) {
            out = *reinterpret_cast<const u32x4_t*>(page + (is_v ? F::v_offset(at.token, i) : at.token * F::kRow + 16 * i));
        } else {
            const u32x2_t a = *reinterpret_cast<const u32x2_t*>(page + F::v_offset(at.token, 2 * i));
            const u32x2_t b = *reinterpret_cast<const u32x2_t*>(page + F::v_offset(at.token, 2 * i + 1));
            out = u32x4_t{a[0], a[1], b[0], b[1]};
        }
    } else {
        float v[8];
        float s, low = 0.f;
        if constexpr (BITS == 8) {
            u32x2_t w;
            if (!is_v || F::kPiece == 8) {
                w = *reinterpret_cast<const u32x2_t*>(page + (is_v ? F::v_offset(at.token, i) : at.token * F::kRow + 8 * i));
            } else {
                w[0] = *reinterpret_cast<const uint32_t*>(page + F::v_offset(at.token, 2 * i));
                w[1] = *reinterpret_cast<const uint32_t*>(page + F::v_offset(at.token, 2 * i + 1));
            }
            s = bf16_float(*reinterpret_cast<const uint16_t*>(scales));
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = float(int((w[e / 4] >> (8 * (e % 4))) & 255u) - 128);
        } else {
            const int g = i / 8, j = i % 8;
            const uint32_t sw = *reinterpret_cast<const uint32_t*>(scales + 4 * g);
            s = bf16_float(sw & 0xFFFFu);
            low = __uint_as_float(sw & 0xFFFF0000u);
            if (is_v) {
                const uint32_t even = *reinterpret_cast<const uint16_t*>(page + F::v_offset(at.token, 2 * j) + 2 * g);
                const uint32_t odd = *reinterpret_cast<const uint16_t*>(page + F::v_offset(at.token, 2 * j + 1) + 2 * g);
                const uint32_t w = even | odd << 16;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = float((w >> (4 * e)) & 15u);
            } else {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(page + at.token * F::kRow + j / 2 * (8 * F::kGroups) + 8 * g + 4 * (j % 2));
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = float((w >> (4 * (e / 2 + 4 * (e % 2)))) & 15u);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {  // the product is exact, so this is two roundings at 4 bits and one at 8
            const uint32_t a = float_to_bf16_bits(__builtin_fmaf(v[e], s, low)), b = float_to_bf16_bits(__builtin_fmaf(v[e + 1], s, low));
            out[e / 2] = a | b << 16;
        }
    }
    return out;
}

template <int D, int BITS>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheArgs c, CacheRows r) {
    for_each_row<D>(c, r, [&](int64_t t, int h, bool in, Place at, int i) __attribute__((always_inline)) {
        if (!in) return;
        const u32x4_t k = read_eight<D, BITS, false>(c, at, i), v = read_eight<D, BITS, true>(c, at, i);
        *reinterpret_cast<u32x4_t*>(r.k_out + t * r.k_token + int64_t(h) * r.k_head + 8 * i) = k;
        *reinterpret_cast<u32x4_t*>(r.v_out + t * r.v_token + int64_t(h) * r.v_head + 8 * i) = v;
    });
}

template <int D, int BITS>
hipError_t launch_rows(const CacheArgs& c, const CacheRows& r, bool write, hipStream_t stream) {
    const int64_t groups = tiles_of(r.tokens, 4 * 64 / (D / 8)) * c.heads;
    const unsigned grid = unsigned(groups < (1 << 20) ? groups : (1 << 20));  // more rows: several turns of the loop
    if (write)
        hipLaunchKernelGGL((cache_write_kernel<D, BITS>), dim3(grid), dim3(256), 0, stream, c, r);
    else
        hipLaunchKernelGGL((cache_read_kernel<D, BITS>), dim3(grid), dim3(256), 0, stream, c, r);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_rows(const CacheArgs& c, const CacheRows& r, bool write, hipStream_t stream) {
    if (c.head_dim == 64) {
        return c.bits == 16 ? launch_rows<64, 16>(c, r, write, stream)
             : c.bits == 8  ? launch_rows<64, 8>(c, r, write, stream)
                            : launch_rows<64, 4>(c, r, write, stream);
    }
    return c.bits == 16 ? launch_rows<128, 16>(c, r, write, stream)
         : c.bits == 8  ? launch_rows<128, 8>(c, r, write, stream)
                        : launch_rows<128, 4>(c, r, write, stream);
}

}  // namespace lowbit
