// Writing keys and values of new tokens into a paged cache, quantised on the way, and reading rows back as bf16.
//
//   8 bits: s = up(max|x| * (1/127)) per token and head, code = rint(x / s), stands for s * code;
//   4 bits: per group of 64 elements  b = min x, s = up((max x - b) * (1/15)), code = rint((x - b) / s), stands for s * code + b;
// up(t): the smallest bf16 not below t, so that no code leaves its range and a bf16 scale costs no more than its share
// of the range.  1/127 and 1/15 are fp32 numbers, b is a bf16 already, x / s is a correctly rounded fp32 division and rint goes to
// even: codes depend on the inputs alone.  A group with an infinity or a NaN (or, at 4 bits, a range past fp32) gets a NaN for its scale and reads
// back as NaN: its neighbours are untouched.
//
// Bound by memory (every element read once and written once) or, for a few tokens, by the launch.  8 elements per lane: 16
// or 8 lanes hold a token's row of a head, neighbouring rows of a wave are neighbouring tokens of one head, whose codes
// lie in the same lines of the cache.
#include "kv_cache.h"
#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {
namespace {

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }
// The smallest bf16 not below f >= 0.
__device__ __forceinline__ uint32_t up_bf16(float f) { return (__float_as_uint(f) + 0xFFFFu) >> 16; }

constexpr uint32_t kNanBf16 = 0x7FC0;
constexpr uint32_t kInfBf16 = 0x7F80;

// Where a row's token lies: base addresses of its head's page in k (v alike) and in the scales, and its place in the page.
struct Place {
    int64_t page_row;  // (page * heads + head) * page_size
    uint32_t token;
};

// A wave's rows: row `lane / (D / 8)` of them.  Waves go (token block, head, K or V).
template <int D, class F>
__device__ __forceinline__ void for_each_row(const CacheArgs& c, const int32_t* slots, int64_t tokens, F f) {
    constexpr int kLanes = D / 8, kRows = 64 / kLanes;
    const int lane = int(threadIdx.x) & 63;
    const int64_t waves = (tokens + kRows - 1) / kRows * c.heads * 2;
    const uint32_t capacity = uint32_t(c.pages) << c.page_shift;
    for (int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); w < waves; w += int64_t(gridDim.x) * 4) {
        const bool is_v = w & 1;
        const int64_t th = w >> 1;
        const int64_t tb = th / c.heads;
        const int h = int(th - tb * c.heads);
        const int64_t t = tb * kRows + lane / kLanes;
        const uint32_t slot = t < tokens ? uint32_t(slots[t]) : ~0u;
        const bool in = slot < capacity;  // a negative slot is past it too
        const Place at{(int64_t(in ? slot >> c.page_shift : 0u) * c.heads + h) << c.page_shift, slot & ((1u << c.page_shift) - 1)};
        f(is_v, t, h, in, at, lane % kLanes);
    }
}

template <int D, int BITS>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheArgs c, CacheRows r) {
    using F = CacheFmt<D, BITS>;
    for_each_row<D>(c, r.slots, r.tokens, [&](bool is_v, int64_t t, int h, bool in, Place at, int i) __attribute__((always_inline)) {
        // lanes without a row go along (the rows' lanes exchange values) with zeros
        const uint16_t* src = (is_v ? r.v : r.k) + t * (is_v ? r.v_token : r.k_token) + int64_t(h) * (is_v ? r.v_head : r.k_head) + 8 * i;
        u32x4_t raw = {0, 0, 0, 0};
        if (in) raw = *reinterpret_cast<const u32x4_t*>(src);
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
        uint32_t big = 0;  // the largest magnitude's bits; from kInfBf16 on the group is not finite
        float lo = __builtin_inff(), hi = -__builtin_inff();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = e & 1 ? raw[e / 2] >> 16 : raw[e / 2] & 0xFFFFu;
            x[e] = bf16_float(b);
            big = max(big, b & 0x7FFFu);
            if constexpr (BITS == 4) {
                lo = fminf(lo, x[e]);
                hi = fmaxf(hi, x[e]);
            }
        }
        constexpr int kShare = BITS == 8 ? D / 8 : kCacheGroup / 8;  // lanes of a group
#pragma unroll
        for (int d = 1; d < kShare; d *= 2) {
            big = max(big, uint32_t(__shfl_xor(int(big), d)));
            if constexpr (BITS == 4) {
                lo = fminf(lo, __shfl_xor(lo, d));
                hi = fmaxf(hi, __shfl_xor(hi, d));
            }
        }
        const float range = BITS == 8 ? bf16_float(big) : hi - lo;
        const bool fine = big < kInfBf16 && range < __builtin_inff();
        const uint32_t sb = fine ? up_bf16(range * (BITS == 8 ? 1.f / 127.f : 1.f / 15.f)) : kNanBf16;
        const float s = bf16_float(sb);
        uint32_t code[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = fine && sb != 0 ? __builtin_rintf((BITS == 8 ? x[e] : x[e] - lo) / s) : 0.f;
            code[e] = BITS == 8 ? uint32_t(int(v) + 128) : min(uint32_t(v), 15u);
        }
        unsigned char* const scales = (is_v ? c.v_scales : c.k_scales) + (at.page_row + at.token) * F::kScaleBytes;
        if constexpr (BITS == 8) {
            if (!in) return;
            const u32x2_t w = {code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24, code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24};
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
                    const uint32_t other = uint32_t(__shfl_xor(int(g == 0 ? odd : even), 8));
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
    });
}

template <int D, int BITS>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheArgs c, CacheRows r) {
    using F = CacheFmt<D, BITS>;
    for_each_row<D>(c, r.slots, r.tokens, [&](bool is_v, int64_t t, int h, bool in, Place at, int i) __attribute__((always_inline)) {
        if (!in) return;
        uint16_t* const dst = (is_v ? r.v_out : r.k_out) + t * (is_v ? r.v_token : r.k_token) + int64_t(h) * (is_v ? r.v_head : r.k_head) + 8 * i;
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
        *reinterpret_cast<u32x4_t*>(dst) = out;
    });
}

template <int D, int BITS>
hipError_t launch_rows(const CacheArgs& c, const CacheRows& r, bool write, hipStream_t stream) {
    constexpr int kRows = 64 / (D / 8);
    const int64_t groups = (tiles_of(r.tokens, kRows) * c.heads * 2 + 3) / 4;
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
