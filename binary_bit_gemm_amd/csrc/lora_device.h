// Low-rank adapters inside a packed GEMM (gfx950 only): the fp32 sums of a wave's 16x16 blocks start at
// U B_e^T instead of zero, where U[m] = alpha_e A_e X[m] was laid down by the first kernel (lora.hip) and e is
// row m's adapter.
//
// At the start and not at the end: the loads then overlap the tile's first copies, and the sums are
// only written (added to in loops at the end, they took twice their registers and spilled).
#pragma once

#include <type_traits>

#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {

// acc[mb][nb], in the layout of 16x16 MFMA results (lane (q, l16): column l16, rows 4q + i), becomes GAIN times
// the adapters' term of rows row0 + 16 mb .. and output columns col0 + 16 nb .. (GAIN: the factor that some
// kernels' code operands carry until their epilogue).
//
// U is held as two bf16 halves per number, hi + lo (2^-16 of it is lost), and the product runs over 2 rank
// places, hi then lo, against B's rank columns taken twice: the adapter's term is exact to fp32
// sums of bf16 products, for one more matrix instruction per 16 of rank and block.
//
// Rows of one request (the ordinary case: a wave's rows have one adapter, or none) load all operands of a step
// at once.  Mixed rows go block by block and adapter by adapter.  Requests must not touch each other:
// rows of other adapters are left out of a product by a zero operand and, since zero times
// another request's infinity or NaN is a NaN, by dropping their result as well.
template <int GAIN, int MB, int NB>
__device__ __forceinline__ void lora_init(f32x4_t (&acc)[MB][NB], const LoraArgs& la, int M, int N, int row0, int col0) {
    int lane = int(threadIdx.x) & 63;
    asm volatile("" : "+v"(lane));  // what follows from it is computed here, not held through the main loop
    const int q = lane >> 4, l16 = lane & 15;
    const int have = M - row0 < 16 * MB ? M - row0 : 16 * MB;  // rows of the wave that exist
    const auto id_rs = make_rsrc(la.rows + row0, have > 0 ? uint32_t(have) * 4u : 0u);
    int id[MB];  // adapter of row row0 + 16 mb + l16, -1: none
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int e = int(__builtin_amdgcn_raw_buffer_load_b32(id_rs, uint32_t(l16) * 4u, 64 * mb, 0));
        id[mb] = 16 * mb + l16 < have && e >= 0 && e < la.adapters ? e : -1;
    }
    const int chunks = la.rank / 8;  // 16-byte chunks of a B row and of each half of a U row
    const uint32_t u_row = uint32_t(la.rank) * 4u;
    const auto u_rs = make_rsrc(la.u + int64_t(row0) * (2 * la.rank), have > 0 ? uint32_t(have) * u_row : 0u);
    const int cols = N - col0 < 16 * NB ? N - col0 : 16 * NB;
    constexpr uint32_t kNone = 0xFFF00000u;  // past every range, whatever is added to it here: reads as zero
    auto b_rsrc = [&](int e) __attribute__((always_inline)) {
        return make_rsrc(la.b + (int64_t(e) * N + col0) * la.rank, cols > 0 ? uint32_t(cols) * uint32_t(la.rank) * 2u : 0u);
    };
    auto load = [](__amdgpu_buffer_rsrc_t rs, uint32_t off, int soff) __attribute__((always_inline)) {
        return __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rs, off, soff, 0));
    };
    // byte offsets of the lane's chunk of step ks: place 4 ks + q of the 2 rank / 8
    auto u_off = [&](int ks) __attribute__((always_inline)) {
        const int c = 4 * ks + q;
        return c < 2 * chunks ? uint32_t(l16) * u_row + uint32_t(c) * 16u : kNone;
    };
    auto b_off = [&](int ks) __attribute__((always_inline)) {
        const int c = 4 * ks + q;
        return c < 2 * chunks ? uint32_t(l16 * chunks + (c < chunks ? c : c - chunks)) * 16u : kNone;
    };
    const int b_block = 32 * la.rank;  // bytes of 16 rows of B

    bool one = true;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) one = one && id[mb] == id[0];
    const int first = __builtin_amdgcn_readfirstlane(id[0]);
    const int steps = (2 * chunks + 3) / 4;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (__all(one && id[0] == first)) {
        if (first < 0) return;
        const auto rs = b_rsrc(first);
        auto run = [&](auto count) __attribute__((always_inline)) {
#pragma unroll
            for (int ks = 0; ks < decltype(count)::value; ++ks) {
                bf16x8_t bf[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) bf[nb] = load(rs, b_off(ks), nb * b_block);
                // kAhead row blocks' operands in flight at a time: what the sums leave room for
                constexpr int kAhead = 5;
#pragma unroll
                for (int m0 = 0; m0 < MB; m0 += kAhead) {
                    bf16x8_t uf[kAhead];
#pragma unroll
                    for (int j = 0; j < kAhead; ++j)
                        if (m0 + j < MB) uf[j] = load(u_rs, u_off(ks), (m0 + j) * 16 * int(u_row));
#pragma unroll
                    for (int j = 0; j < kAhead; ++j)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            if (m0 + j < MB)
                                acc[m0 + j][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(uf[j], bf[nb], acc[m0 + j][nb], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        if (steps <= 1)
            run(std::integral_constant<int, 1>{});
        else if (steps <= 2)
            run(std::integral_constant<int, 2>{});
        else if (steps <= 4)
            run(std::integral_constant<int, 4>{});
        else
            run(std::integral_constant<int, 8>{});
    } else {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            f32x4_t sum[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) sum[nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            for (int cur = -1;;) {
                int next = id[mb] > cur ? id[mb] : 0x7FFFFFFF;  // the block's next adapter
#pragma unroll
                for (int d = 1; d < 16; d *= 2) {
                    const int o = __shfl_xor(next, d);
                    next = o < next ? o : next;
                }
                next = __builtin_amdgcn_readfirstlane(next);
                if (next == 0x7FFFFFFF) break;
                cur = next;
                const auto rs = b_rsrc(cur);
                f32x4_t t[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) t[nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                for (int ks = 0; ks < steps; ++ks) {
                    const bf16x8_t uf = load(u_rs, id[mb] == cur ? u_off(ks) : kNone, mb * 16 * int(u_row));
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        t[nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(uf, load(rs, b_off(ks), nb * b_block), t[nb], 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool mine = __shfl(id[mb], 4 * q + i) == cur;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) sum[nb][i] = mine ? t[nb][i] : sum[nb][i];
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = sum[nb];
        }
    }
    if constexpr (GAIN != 1) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mb][nb][i] *= float(GAIN);
    }
}

}  // namespace lowbit
