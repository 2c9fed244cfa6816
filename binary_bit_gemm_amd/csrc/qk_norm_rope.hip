// Norms of queries and keys for each head, with the position rotation in the same pass.
//
// For token t and head h with x = x[t, h, 0:D) (bf16) and weight w[D]:
//     y_d = x_d * r * w_d,   r = 1 / sqrt(sum_d x_d^2 / D + eps)            (y = x without a weight)
//     pair i of the first R = sum(axis_dims) elements turns by  pos[t, a(i)] * freq[i]  radians,
// where a(i) is the axis whose block of axis_dims[a] / 2 pairs holds i.  A pair is (y_2i, y_2i+1)
// (interleaved) or (y_i, y_i+R/2) (halves); elements from R on pass through.
//
// Memory-bound: 4 bytes move per element for about 20 operations.  A lane holds 8 consecutive elements
// (one 16-byte load and store), so a head is D / 8 lanes and a wave instruction moves whole heads;
// a wave takes one token and up to kHeadRounds such groups of heads, whose loads are all issued
// before the first is used.  The norm is a sum over the head's lanes.  Everything is fp32 from the
// load to the one rounding at the store.  Measured: 4608 tokens x 48 heads of 128 with norm and four axes 27.8 us (4.1
// TB/s), 16383 tokens x 32 heads of 64 with three axes 28.0 us (4.8 TB/s, the rate of a large copy).
//
// Angles: the pairs' cosines and sines are computed once per wave, pair i in lane i, and fetched
// from there.  In fp32 the product pos * freq would be off by 2^-24 of the angle, which is
// 5e-4 rad at position 8192; so the product and its reduction to a fraction of a turn are done
// in fp64 (one multiply each, exact to 2^-53 of the angle) and only the fraction is fp32.
#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {
namespace {

constexpr int kHeadRounds = 4;
constexpr int kWaves = 4;

// Sum over the L consecutive lanes of a head, in every lane of it.
template <int L>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int d = 1; d < L; d *= 2) v += __shfl_xor(v, d);
    return v;
}

template <int D, bool PAIRED>
__global__ __launch_bounds__(64 * kWaves) void qk_norm_rope_kernel(QkArgs a) {
    constexpr int L = D / 8;        // lanes per head
    constexpr int HPR = 64 / L;     // heads per round
    constexpr int PW = (D / 2 + 63) / 64;
    const int lane = int(threadIdx.x) & 63;
    const int64_t wave = int64_t(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int64_t t = wave / a.chunks;
    if (t >= a.tokens) return;
    const int chunk = int(wave - t * a.chunks);
    const int j = lane % L;                                            // the lane's elements: 8j .. 8j+7
    const int h0 = chunk * (kHeadRounds * HPR) + lane / L;
    const int heads = a.q_heads + a.k_heads;

    u32x4_t raw[kHeadRounds];
    const uint16_t* src[kHeadRounds];
#pragma unroll
    for (int i = 0; i < kHeadRounds; ++i) {
        const int h = h0 + i * HPR;
        src[i] = h < a.q_heads ? a.q + t * a.q_token + int64_t(h) * a.q_head
                               : a.k + t * a.k_token + int64_t(h - a.q_heads) * a.k_head;
        raw[i] = u32x4_t{0, 0, 0, 0};
        if (h < heads) raw[i] = *reinterpret_cast<const u32x4_t*>(src[i] + 8 * j);
    }

    // cosine and sine of pair 64 c + lane
    const int pairs = a.rot / 2;
    float cs[PW], sn[PW];
#pragma unroll
    for (int c = 0; c < PW; ++c) {
        const int p = 64 * c + lane;
        cs[c] = 1.f;
        sn[c] = 0.f;
        if (p < pairs) {
            int ax = 0;
#pragma unroll
            for (int e = 0; e < 3; ++e) ax += p >= a.axis_end[e] ? 1 : 0;
            const double turns = double(a.positions[t * a.axes + ax]) * (double(a.freqs[p]) * 0.15915494309189533577);
            const float frac = float(turns - __builtin_rint(turns));
            sincospif(2.f * frac, &sn[c], &cs[c]);
        }
    }
    // the lane's factors: interleaved, pairs 4j .. 4j+3; halves, pairs of elements 8j .. 8j+7
    constexpr int NP = PAIRED ? 4 : 8;
    float co[NP], si[NP];
    const bool turned = 8 * j < a.rot;
    const bool upper = !PAIRED && 8 * j >= pairs;  // halves: the lane holds second elements
#pragma unroll
    for (int e = 0; e < NP; ++e) {
        const int p = PAIRED ? 4 * j + e : 8 * j + e - (upper ? pairs : 0);
        const int from = turned ? p : 0;
        co[e] = __shfl(cs[0], from & 63);
        si[e] = __shfl(sn[0], from & 63);
        if constexpr (PW == 2) {
            const float c1 = __shfl(cs[1], from & 63), s1 = __shfl(sn[1], from & 63);
            if (from >= 64) {
                co[e] = c1;
                si[e] = s1;
            }
        }
        if (!turned) {
            co[e] = 1.f;
            si[e] = 0.f;
        }
        if (upper) si[e] = -si[e];
    }
    // halves: the lane with the other element of the pairs
    const int mate = !turned ? lane : upper ? lane - pairs / 8 : lane + pairs / 8;

#pragma unroll
    for (int i = 0; i < kHeadRounds; ++i) {
        const int h = h0 + i * HPR;
        const bool is_q = h < a.q_heads;
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(raw[i][e] << 16);
            x[2 * e + 1] = __uint_as_float(raw[i][e] & 0xFFFF0000u);
        }
        const uint16_t* w = is_q ? a.q_weight : a.k_weight;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(x[e], x[e], ss);
        ss = head_sum<L>(ss);  // by every lane, whether or not its head is normed
        if (w != nullptr) {
            const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
            const u32x4_t wv = *reinterpret_cast<const u32x4_t*>(w + 8 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] *= r * __uint_as_float(wv[e] << 16);
                x[2 * e + 1] *= r * __uint_as_float(wv[e] & 0xFFFF0000u);
            }
        }
        float y[8];
        if constexpr (PAIRED) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[2 * e] = x[2 * e] * co[e] - x[2 * e + 1] * si[e];
                y[2 * e + 1] = x[2 * e] * si[e] + x[2 * e + 1] * co[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float other = __shfl(x[e], mate);
                y[e] = x[e] * co[e] - other * si[e];
            }
        }
        if (!turned) {  // past the rotated elements: unchanged, also where a factor of 0 would make a NaN of an infinity
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e];
        }
        if (h < heads) {
            u32x4_t out;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                out[e] = uint32_t(float_to_bf16_bits(y[2 * e])) | (uint32_t(float_to_bf16_bits(y[2 * e + 1])) << 16);
            uint16_t* dst = is_q ? a.q_out + t * a.qo_token + int64_t(h) * a.qo_head
                                 : a.k_out + t * a.ko_token + int64_t(h - a.q_heads) * a.ko_head;
            *reinterpret_cast<u32x4_t*>(dst + 8 * j) = out;
        }
    }
}

template <int D>
hipError_t launch_d(QkArgs a, bool interleaved, hipStream_t stream) {
    constexpr int kHeads = kHeadRounds * (64 / (D / 8));  // heads of one wave
    a.chunks = (a.q_heads + a.k_heads + kHeads - 1) / kHeads;
    // a launch has at most 2^32 threads: more tokens take several
    const int64_t most = kMaxGrid256 * kWaves / a.chunks;
    auto skip = [&](auto*& ptr, int64_t stride) {
        if (ptr != nullptr) ptr += most * stride;
    };
    for (int64_t left = a.tokens;; left -= most) {
        a.tokens = left < most ? left : most;
        const unsigned grid = unsigned((a.tokens * a.chunks + kWaves - 1) / kWaves);
        if (interleaved)
            hipLaunchKernelGGL((qk_norm_rope_kernel<D, true>), dim3(grid), dim3(64 * kWaves), 0, stream, a);
        else
            hipLaunchKernelGGL((qk_norm_rope_kernel<D, false>), dim3(grid), dim3(64 * kWaves), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || left <= most) return e;
        skip(a.q, a.q_token);
        skip(a.k, a.k_token);
        skip(a.q_out, a.qo_token);
        skip(a.k_out, a.ko_token);
        skip(a.positions, a.axes);
    }
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkArgs& a, int head_dim, bool interleaved, hipStream_t stream) {
    switch (head_dim) {
        case 32: return launch_d<32>(a, interleaved, stream);
        case 64: return launch_d<64>(a, interleaved, stream);
        case 128: return launch_d<128>(a, interleaved, stream);
        case 256: return launch_d<256>(a, interleaved, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace lowbit
