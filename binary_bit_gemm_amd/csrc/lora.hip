// First product of the low-rank adapters beside a packed GEMM: U[m] = alpha_e * A_e X[m] for the adapter e of
// row m, with X [M, K] bf16, A [adapters, rank, K] bf16 and alpha fp32.  The second product (U B_e^T) is where the packed GEMM's
// sums start (lora_device.h).
//
// A workgroup takes 16 rows and one of the adapters among them (the j-th smallest; a workgroup whose j
// is past the last one leaves at once), so rows of many requests cost more workgroups, not a longer one.
// Its waves split K; every wave multiplies 16x16x32 blocks straight from global memory (16
// bytes per lane: 64 consecutive bytes of each of 16 rows of X and of A per instruction), and the waves'
// fp32 sums are added in wave order through LDS, scaled, and stored as hi + lo bf16 pairs.
#include <type_traits>

#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {
namespace {

constexpr int kWaves = 8;

template <int RB>
__global__ __launch_bounds__(64 * kWaves) void lora_shrink_kernel(ShrinkArgs a) {
    __shared__ f32x4_t red[kWaves][RB][64];
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int q = lane >> 4, l16 = lane & 15;
    const int64_t row0 = int64_t(blockIdx.x) * 16;
    const int64_t m = row0 + l16;
    int id = m < a.M ? a.rows[m] : -1;
    id = id >= 0 && id < a.adapters ? id : -1;
    // the blockIdx.y-th adapter of the 16 rows
    int cur = -1;
    for (int j = 0; j <= int(blockIdx.y); ++j) {
        int next = id > cur ? id : 0x7FFFFFFF;
#pragma unroll
        for (int d = 1; d < 16; d *= 2) {
            const int o = __shfl_xor(next, d);
            next = o < next ? o : next;
        }
        next = __builtin_amdgcn_readfirstlane(next);
        if (next == 0x7FFFFFFF) return;  // the same in every wave
        cur = next;
    }
    const int steps = a.K / 32;
    const int s0 = wave * steps / kWaves, s1 = (wave + 1) * steps / kWaves;
    const bool mine = id == cur;
    const uint16_t* x = a.X + (mine ? m : row0) * int64_t(a.K) + 8 * q;
    const uint16_t* w[RB];
    bool live[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int r = 16 * rb + l16;
        live[rb] = r < a.rank;
        w[rb] = a.A + (int64_t(cur) * a.rank + (live[rb] ? r : 0)) * int64_t(a.K) + 8 * q;
    }
    f32x4_t acc[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) acc[rb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // kAhead steps' operands are loaded before the first is used
    constexpr int kAhead = RB >= 8 ? 2 : 4;
    auto steps_of = [&](int s, auto count) __attribute__((always_inline)) {
        constexpr int n = decltype(count)::value;
        bf16x8_t xf[n], wf[n][RB];
#pragma unroll
        for (int j = 0; j < n; ++j) {
            xf[j] = *reinterpret_cast<const bf16x8_t*>(x + 32 * int64_t(s + j));
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) wf[j][rb] = *reinterpret_cast<const bf16x8_t*>(w[rb] + 32 * int64_t(s + j));
        }
#pragma unroll
        for (int j = 0; j < n; ++j)
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) acc[rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j], wf[j][rb], acc[rb], 0, 0, 0);
    };
    int s = s0;
    for (; s + kAhead <= s1; s += kAhead) steps_of(s, std::integral_constant<int, kAhead>{});
    for (; s < s1; ++s) steps_of(s, std::integral_constant<int, 1>{});
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) red[wave][rb][lane] = acc[rb];
    __syncthreads();
    for (int rb = wave; rb < RB; rb += kWaves) {
        f32x4_t v = red[0][rb][lane];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) {
            const f32x4_t o = red[k][rb][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += o[i];
        }
        const int r = 16 * rb + l16;
        const float alpha = a.alpha[cur];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = row0 + 4 * q + i;
            const int owner = __shfl(id, 4 * q + i);
            if (owner == cur && r < a.rank) {
                const float u = v[i] * alpha;
                const __bf16 hi = static_cast<__bf16>(u);
                const float h = static_cast<float>(hi);
                const bool fine = __builtin_fabsf(h) < __builtin_inff();  // an infinity's rest would be a NaN
                uint16_t* dst = a.u + row * (2 * a.rank) + r;
                dst[0] = __builtin_bit_cast(uint16_t, hi);
                dst[a.rank] = fine ? float_to_bf16_bits(u - h) : uint16_t(0);
            }
        }
    }
}

}  // namespace

hipError_t launch_lora_shrink(const ShrinkArgs& a, hipStream_t stream) {
    const dim3 grid(unsigned(tiles_of(a.M, 16)), unsigned(a.adapters < 16 ? a.adapters : 16));
    const int rb = (a.rank + 15) / 16;
    if (rb <= 1)
        hipLaunchKernelGGL(lora_shrink_kernel<1>, grid, dim3(64 * kWaves), 0, stream, a);
    else if (rb <= 2)
        hipLaunchKernelGGL(lora_shrink_kernel<2>, grid, dim3(64 * kWaves), 0, stream, a);
    else if (rb <= 4)
        hipLaunchKernelGGL(lora_shrink_kernel<4>, grid, dim3(64 * kWaves), 0, stream, a);
    else
        hipLaunchKernelGGL(lora_shrink_kernel<8>, grid, dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

}  // namespace lowbit
