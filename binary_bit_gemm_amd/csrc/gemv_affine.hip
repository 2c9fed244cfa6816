// Matrix-vector products with affine 4-bit weights, up to 16 rows:
//     Y[m, n] = sum_k X[m, k] (S[n, k/g] u[n, k] + B[n, k/g]),   u in 0 .. 15,
// and their forms with a residual, or with gate and up rows and Y = silu(gate) up.
//
// Bound by reading the weights once.  A workgroup owns 16 weight rows (SWIGLU: 16 gate rows and their 16 up rows); its waves
// split K into contiguous runs of 128-element steps, whose fp32 sums are added through LDS in wave order.  A
// 16-byte load brings lane (q, n) chunk q (32 levels) of a step of row n; four lane-row swaps make register c of quarter q word q of
// chunk c, so that one 16x16x32 MFMA takes one chunk, which lies in one group.
//   * Levels become operands by a mask and an OR: 0x4300 | u is the bf16 128 + u, exactly; the pairs come as levels (0, 4), (1, 5),
//     (2, 6), (3, 7) of a word, and X's operand is permuted to that order.  Per group
//         S sum x u + B sum x = S sum x (128 + u) + (B - 128 S) sum x,
//     with sum x from the matrix cores too (a product with ones).  Both sums are fp32, S and B multiply after them: no
//     weight is rounded.
#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {
namespace {

constexpr int kStep = 128;

// RAGGED: K is no multiple of the step: the last one has only its first 64 elements.
template <int G, bool SWIGLU, bool RAGGED, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void gemv_affine_kernel(GemvArgs p) {
    constexpr int NB = SWIGLU ? 2 : 1;  // blocks of 16 weight rows
    constexpr int GPS = kStep / G;      // groups of a step
    __shared__ f32x4_t red[WAVES][NB][64];
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int q = lane >> 4, n = lane & 15;
    const int n0 = xcd_remap(int(blockIdx.x), int(gridDim.x)) * 16;
    const uint32_t row_bytes = uint32_t(p.K) / 2u;
    const uint32_t groups = uint32_t(p.K) / uint32_t(G);
    const int steps = (p.K + kStep - 1) / kStep;
    const int s_begin = int(int64_t(wave) * steps / WAVES), s_end = int(int64_t(wave + 1) * steps / WAVES);

    __amdgpu_buffer_rsrc_t wr[NB], sr[NB], br[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t row = n0 + int64_t(b) * p.N;
        wr[b] = make_rsrc(reinterpret_cast<const unsigned char*>(p.W) + row * row_bytes, 16u * row_bytes);
        sr[b] = make_rsrc(p.S + row * groups, 32u * groups);
        br[b] = make_rsrc(p.B + row * groups, 32u * groups);
    }
    const auto xr = make_rsrc(p.X, uint32_t(p.M) * uint32_t(p.K) * 2u);  // rows past the last read as zeros
    const uint32_t w_off = uint32_t(n) * row_bytes + 16u * uint32_t(q);
    const uint32_t s_off = uint32_t(n) * groups * 2u;
    const uint32_t x_off = (uint32_t(n) * uint32_t(p.K) + 8u * uint32_t(q)) * 2u;
    constexpr uint32_t kNowhere = 0xFFFFFF00u;

    struct Stage {
        u32x4_t w[NB];
        u32x4_t x[4];
        uint32_t s[NB], b[NB];  // G = 64: two fp16, the first group's low
    };
    auto load = [&](Stage& st, int s) __attribute__((always_inline)) {
        const uint32_t k0 = uint32_t(s) * kStep;
        const bool whole = !RAGGED || int(k0) + kStep <= p.K;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            st.w[b] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wr[b], whole || q < 2 ? w_off + k0 / 2 : kNowhere, 0, 0));
            const uint32_t at = s_off + uint32_t(s) * (2u * GPS);
            if constexpr (GPS == 2 && !RAGGED) {
                st.s[b] = __builtin_amdgcn_raw_buffer_load_b32(sr[b], at, 0, 0);
                st.b[b] = __builtin_amdgcn_raw_buffer_load_b32(br[b], at, 0, 0);
            } else {
                st.s[b] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(sr[b], at, 0, 0));
                st.b[b] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(br[b], at, 0, 0));
                if constexpr (GPS == 2) {
                    st.s[b] |= uint32_t(uint16_t(__builtin_amdgcn_raw_buffer_load_b16(sr[b], whole ? at + 2u : kNowhere, 0, 0))) << 16;
                    st.b[b] |= uint32_t(uint16_t(__builtin_amdgcn_raw_buffer_load_b16(br[b], whole ? at + 2u : kNowhere, 0, 0))) << 16;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            st.x[c] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(xr, whole || c < 2 ? x_off + (k0 + 32u * c) * 2u : kNowhere, 0, 0));
    };

    f32x4_t acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    auto compute = [&](Stage& st) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) transpose_words(st.w[b]);
        f32x4_t sum[GPS], part[NB][GPS];
#pragma unroll
        for (int g = 0; g < GPS; ++g) {
            sum[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < NB; ++b) part[b][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int g = c * GPS / 4;
            const u32x4_t v = st.x[c];
            const bf16x8_t x = __builtin_bit_cast(bf16x8_t, u32x4_t{perm_b32(v[2], v[0], 0x05040100u), perm_b32(v[2], v[0], 0x07060302u),
                                                                    perm_b32(v[3], v[1], 0x05040100u), perm_b32(v[3], v[1], 0x07060302u)});
            sum[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, ones, sum[g], 0, 0, 0);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t w = st.w[b][c];
                u32x4_t u;
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = ((w >> (4 * e)) & 0x000F000Fu) | 0x43004300u;
                part[b][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, __builtin_bit_cast(bf16x8_t, u), part[b][g], 0, 0, 0);
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int g = 0; g < GPS; ++g) {
                const float s = half_bits_to_float(uint16_t(st.s[b] >> (16 * g)));
                const float low = __builtin_fmaf(-128.f, s, half_bits_to_float(uint16_t(st.b[b] >> (16 * g))));
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[b][i] = __builtin_fmaf(low, sum[g][i], __builtin_fmaf(s, part[b][g][i], acc[b][i]));
            }
    };

    if (s_begin < s_end) {
        Stage a, b;
        load(a, s_begin);
        int s = s_begin;
        while (true) {
            if (s + 1 < s_end) load(b, s + 1);
            compute(a);
            if (++s >= s_end) break;
            if (s + 1 < s_end) load(a, s + 1);
            compute(b);
            if (++s >= s_end) break;
        }
    }

#pragma unroll
    for (int b = 0; b < NB; ++b) red[wave][b][lane] = acc[b];
    __syncthreads();
    if (wave != 0) return;
    f32x4_t v[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        v[b] = red[0][b][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            const f32x4_t u = red[w][b][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[b][i] += u[i];
        }
    }
    // lane (q, n) holds column n0 + n of rows 4q ..
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = 4 * q + i;
        if (m >= p.M) continue;
        const int64_t at = int64_t(m) * p.N + n0 + n;
        float y = v[0][i];
        if constexpr (SWIGLU) y = y / (1.f + __expf(-y)) * v[1][i];
        if (p.R != nullptr) y += __uint_as_float(uint32_t(p.R[at]) << 16);
        p.Y[at] = float_to_bf16_bits(y);
    }
}

template <int G, bool SWIGLU, bool RAGGED>
hipError_t launch_form(const GemvArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((gemv_affine_kernel<G, SWIGLU, RAGGED, 8>), dim3(unsigned(a.N / 16)), dim3(512), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemv_affine(const GemvArgs& a, int g, bool swiglu, hipStream_t stream) {
    if (g == 128) return swiglu ? launch_form<128, true, false>(a, stream) : launch_form<128, false, false>(a, stream);
    if (a.K % kStep != 0) return swiglu ? launch_form<64, true, true>(a, stream) : launch_form<64, false, true>(a, stream);
    return swiglu ? launch_form<64, true, false>(a, stream) : launch_form<64, false, false>(a, stream);
}

}  // namespace lowbit
