// Matrix-vector products with affine 4-bit weights, up to 16 rows:
//     Y[m, n] = sum_k X[m, k] (S[n, k/g] u[n, k] + B[n, k/g]),   u in 0 .. 15,
// and their forms with a residual, or with gate and up rows and Y = silu(gate) up.
//
// Bound by reading the weights once.  A workgroup owns 16 weight rows (SWIGLU: 16 gate rows and their 16 up rows); its waves
// split K into contiguous runs of 128-element steps, whose fp32 sums are added through LDS in wave order.
//   * What limits a lean kernel here is the vector memory path, which pays per line that neighbouring lanes touch: loads in the matrix cores'
//     order (neighbouring lanes on neighbouring rows) took 400 accesses a step, 8 us of a product of 9 us.  So a wave copies a
//     few steps of weights, activations and scales into its own part of LDS, neighbouring lanes on neighbouring bytes, all copies at once and no
//     barrier between waves, and reads operands from there.
//   * Chunk c of a step's row (16 bytes, 32 levels) lies in one group.  A lane (q, n) reads chunk q of row n; four lane-row swaps make
//     register c of quarter q word q of chunk c, so one 16x16x32 MFMA takes one chunk.
//   * Levels become operands by a mask and an OR: 0x4300 | u is the bf16 128 + u, exactly; the pairs come as levels (0, 4), (1, 5),
//     (2, 6), (3, 7) of a word, and X's operand is permuted to that order.  Per group
//         S sum x u + B sum x = S sum x (128 + u) + (B - 128 S) sum x,
//     with sum x from the matrix cores too (a product with ones).  Both sums are fp32, S and B multiply after them: no
//     weight is rounded.  (With an infinite x the two terms are infinities of opposite signs: NaN.)
// Launch included, us with the weights from HBM (left in the last-level cache by the pass before): 1 x 9728 x 2560 with gate and up rows 11.7 (8.1;
// 28 MB, 2.4 TB/s), 1 x 2560 x 9728 with a residual 8.6 (6.8), 11 x 2560 x 4096 6.5 (5.1).  A wave waits for memory once per turn of kSteps: all
// four waves of the first take a second turn for a single step, twelve of the second's sixteen and two of the third's fifteen do.
// lowbit_gemm_affine's tile kernel, weights from HBM, at 1 as at 16 rows: 19456 x 2560 23.5 (here 10.6 with 1 row, 16.9 with 16), 2560 x 9728 46.5
// (8.3, 12.7), 2560 x 4096 23.0 (5.1, 6.7).
#include <atomic>
#include <cstdio>

#include "decode_device.h"
#include "decode_internal.h"

namespace lowbit {
namespace {

constexpr int kStep = 128;
constexpr int kMaxLds = 160 * 1024;
constexpr uint32_t kNowhere = 0xFFFFFF00u;  // past any resource: zeros without a read

// LDS of a wave: `steps` of weights (1 KB a block), activations (1 KB for four rows), then the scales and biases (16 bytes a
// weight row: the dwords that hold those steps' groups, the first from a whole dword on).
template <int NB, int MQ, int STEPS>
struct GemvLds {
    static constexpr int kX = STEPS * NB * 1024;
    static constexpr int kScales = kX + STEPS * MQ * 1024;
    static constexpr int kBytes = kScales + 2 * NB * 256;
};

// RAGGED: K is no multiple of the step: the last one has only its first 64 elements.  MQ: rows of X in fours.
template <int G, bool SWIGLU, bool RAGGED, int MQ>
struct GemvForm {
    static constexpr int kBlocks = SWIGLU ? 2 : 1;  // of 16 weight rows
    // steps at once: few enough that several workgroups' share a compute unit's LDS (16 rows: two, 11 x 2560 x 4096 4.9 us, with four
    // 5.5), and that with their first group's place in its dword the scales fit 16 bytes (RAGGED)
    static constexpr int kSteps = MQ == 4 ? 2 : MQ == 2 || RAGGED ? 3 : 4;
    using Lds = GemvLds<kBlocks, MQ, kSteps>;
};

template <int G, bool SWIGLU, bool RAGGED, int MQ>
__global__ __launch_bounds__(1024) void gemv_affine_kernel(GemvArgs p) {
    using Form = GemvForm<G, SWIGLU, RAGGED, MQ>;
    using Lds = typename Form::Lds;
    constexpr int NB = Form::kBlocks, kSteps = Form::kSteps;
    constexpr int GPS = kStep / G;  // groups of a step
    extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)), waves = int(blockDim.x) >> 6;
    const int q = lane >> 4, n = lane & 15;
    const int n0 = xcd_remap(int(blockIdx.x), int(gridDim.x)) * 16;
    const uint32_t row_bytes = uint32_t(p.K) / 2u;
    const uint32_t groups = uint32_t(p.K) / uint32_t(G);
    const int steps = (p.K + kStep - 1) / kStep;
    const int s_begin = int(int64_t(wave) * steps / waves), s_end = int(int64_t(wave + 1) * steps / waves);
    unsigned char* const mine = lds + wave * Lds::kBytes;

    __amdgpu_buffer_rsrc_t wr[NB], sr[NB], br[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t row = n0 + int64_t(b) * p.N;
        wr[b] = make_rsrc(reinterpret_cast<const unsigned char*>(p.W) + row * row_bytes, 16u * row_bytes);
        sr[b] = make_rsrc(p.S + row * groups, 32u * groups);
        br[b] = make_rsrc(p.B + row * groups, 32u * groups);
    }
    const auto xr = make_rsrc(p.X, uint32_t(p.M) * uint32_t(p.K) * 2u);  // rows past the last read as zeros
    // copies, neighbouring lanes on neighbouring bytes: 4 lanes a weight row; 16 lanes a row of X, chunk c at position c ^ row of
    // its line, which spreads the rows that an operand read touches over the banks; 4 lanes (dwords) a row of scales
    const uint32_t w_from = uint32_t(lane >> 2) * row_bytes + 16u * uint32_t(lane & 3);
    uint32_t x_from[MQ], x_chunk[MQ];
#pragma unroll
    for (int i = 0; i < MQ; ++i) {
        const uint32_t m = uint32_t(4 * i + (lane >> 4));
        x_chunk[i] = uint32_t(lane & 15) ^ m;
        x_from[i] = m * uint32_t(p.K) * 2u + 16u * x_chunk[i];
    }
    const uint32_t s_row = uint32_t(lane >> 2) * groups;  // first group of the copied row, and of the lane's own
    const uint32_t own_row = uint32_t(n) * groups;

    f32x4_t acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

    for (int s0 = s_begin; s0 < s_end; s0 += kSteps) {
        const int count = s_end - s0 < kSteps ? s_end - s0 : kSteps;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (i >= count) break;
            const uint32_t k0 = uint32_t(s0 + i) * kStep;
            const bool whole = !RAGGED || int(k0) + kStep <= p.K;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                dma16(wr[b], mine + (i * NB + b) * 1024, whole || (lane & 3) < 2 ? w_from + k0 / 2u : kNowhere, 0);
#pragma unroll
            for (int j = 0; j < MQ; ++j)
                dma16(xr, mine + Lds::kX + (i * MQ + j) * 1024, whole || x_chunk[j] < 8u ? x_from[j] + k0 * 2u : kNowhere, 0);
        }
        const uint32_t g0 = uint32_t(s0) * GPS;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t from = ((s_row + g0) >> 1) * 4u + 4u * uint32_t(lane & 3);
            dma4(sr[b], mine + Lds::kScales + (2 * b) * 256, from, 0);
            dma4(br[b], mine + Lds::kScales + (2 * b + 1) * 256, from, 0);
        }
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");
        const unsigned char* const own_scales = mine + Lds::kScales + 16 * n + 2 * ((own_row + g0) & 1u);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (i >= count) break;
            u32x4_t w[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                w[b] = *reinterpret_cast<const u32x4_t*>(mine + (i * NB + b) * 1024 + 64 * n + 16 * q);
                transpose_words(w[b]);
            }
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
                // row m of X in lanes n = m; those past 4 MQ repeat others, for results that nobody stores
                const int m = n & (4 * MQ - 1);
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + Lds::kX + i * (MQ * 1024) + 256 * m + 16 * ((4 * c + q) ^ m));
                const bf16x8_t x = __builtin_bit_cast(bf16x8_t, u32x4_t{perm_b32(v[2], v[0], 0x05040100u), perm_b32(v[2], v[0], 0x07060302u),
                                                                        perm_b32(v[3], v[1], 0x05040100u), perm_b32(v[3], v[1], 0x07060302u)});
                sum[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, ones, sum[g], 0, 0, 0);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    u32x4_t u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[e] = ((w[b][c] >> (4 * e)) & 0x000F000Fu) | 0x43004300u;
                    part[b][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, __builtin_bit_cast(bf16x8_t, u), part[b][g], 0, 0, 0);
                }
            }
#pragma unroll
            for (int g = 0; g < GPS; ++g) {
                if (RAGGED && (s0 + i) * kStep + g * G >= p.K) break;  // no such group: its scale is another row's
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float s = half_bits_to_float(*reinterpret_cast<const uint16_t*>(own_scales + (2 * b) * 256 + 2 * (i * GPS + g)));
                    const float low = half_bits_to_float(*reinterpret_cast<const uint16_t*>(own_scales + (2 * b + 1) * 256 + 2 * (i * GPS + g)));
                    const float rest = __builtin_fmaf(-128.f, s, low);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[b][e] = __builtin_fmaf(rest, sum[g][e], __builtin_fmaf(s, part[b][g][e], acc[b][e]));
                }
            }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the reads are done before the next copies may land
        asm volatile("" ::: "memory");
    }

    // ---- the waves' sums, in wave order ----
    __syncthreads();
    f32x4_t* const red = reinterpret_cast<f32x4_t*>(lds);  // [waves][NB][64]
#pragma unroll
    for (int b = 0; b < NB; ++b) red[(wave * NB + b) * 64 + lane] = acc[b];
    __syncthreads();
    if (wave != 0) return;
    f32x4_t v[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        v[b] = red[b * 64 + lane];
        for (int w = 1; w < waves; ++w) {
            const f32x4_t u = red[(w * NB + b) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[b][e] += u[e];
        }
    }
    // lane (q, n) holds column n0 + n of rows 4q ..
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int m = 4 * q + e;
        if (m >= p.M) continue;
        const int64_t at = int64_t(m) * p.N + n0 + n;
        float y = v[0][e];
        if constexpr (SWIGLU) y = y / (1.f + __expf(-y)) * v[NB - 1][e];
        if (p.R != nullptr) y += __uint_as_float(uint32_t(p.R[at]) << 16);
        p.Y[at] = float_to_bf16_bits(y);
    }
}

// Waves of a workgroup: as many as let all workgroups be on the compute units at once (LDS decides), three at least.  Measured (us, 1
// x 9728 x 2560 SwiGLU, 608 workgroups: three a unit with 4 waves): 3 waves 9.4, 4 8.1, 5 10.2; 1 x 2560 x 9728, one a unit: 4 waves 9.3, 8 7.2,
// 12 6.7; 3 x 151936 x 2560, which take turns: 1 wave 50, 3 44, 5 50.
int gemv_waves(int64_t groups, int64_t chunks, int64_t bytes) {
    const int64_t per_unit = tiles_of(groups, kComputeUnits);
    int64_t waves = kMaxLds / (per_unit * bytes);
    waves = waves < 3 ? 3 : waves < 16 ? waves : 16;
    waves = waves < chunks ? waves : chunks;
    return waves < 1 ? 1 : int(waves);
}

template <int G, bool SWIGLU, bool RAGGED, int MQ>
hipError_t launch_rows(const GemvArgs& a, hipStream_t stream) {
    using Form = GemvForm<G, SWIGLU, RAGGED, MQ>;
    static_assert(16 * Form::Lds::kBytes <= 16 * kMaxLds / 3, "three waves fit");
    const auto kernel = gemv_affine_kernel<G, SWIGLU, RAGGED, MQ>;
    // allow the largest dynamic LDS, once per kernel and device (threads that get here first at the same time may both set it)
    static std::atomic<int> attr_set[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
    if (attr_set[dev].load(std::memory_order_acquire) == 0) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLds);
        if (e != hipSuccess) return e;
        attr_set[dev].store(1, std::memory_order_release);
    }
    int waves = gemv_waves(a.N / 16, tiles_of(tiles_of(a.K, kStep), Form::kSteps), Form::Lds::kBytes);
    const unsigned grid = unsigned(a.N / 16), bytes = unsigned(waves) * Form::Lds::kBytes;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(unsigned(64 * waves)), bytes, stream, a);
    e = hipGetLastError();
    if (e == hipSuccess && trace_enabled())
        std::fprintf(stderr, "lowbit: gemv_affine rows=%d waves=%d g=%d grid=%u block=%d lds=%u problem=%dx%dx%d%s%s\n", 4 * MQ, waves, G, grid,
                     64 * waves, bytes, a.M, a.N, a.K, SWIGLU ? " swiglu" : "", a.R != nullptr ? " residual" : "");
    return e;
}

template <int G, bool SWIGLU, bool RAGGED>
hipError_t launch_form(const GemvArgs& a, hipStream_t stream) {
    return a.M <= 4   ? launch_rows<G, SWIGLU, RAGGED, 1>(a, stream)
           : a.M <= 8 ? launch_rows<G, SWIGLU, RAGGED, 2>(a, stream)
                      : launch_rows<G, SWIGLU, RAGGED, 4>(a, stream);
}

}  // namespace

hipError_t launch_gemv_affine(const GemvArgs& a, int g, bool swiglu, hipStream_t stream) {
    if (g == 128) return swiglu ? launch_form<128, true, false>(a, stream) : launch_form<128, false, false>(a, stream);
    if (a.K % kStep != 0) return swiglu ? launch_form<64, true, true>(a, stream) : launch_form<64, false, true>(a, stream);
    return swiglu ? launch_form<64, true, false>(a, stream) : launch_form<64, false, false>(a, stream);
}

}  // namespace lowbit
