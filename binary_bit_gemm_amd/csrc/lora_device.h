// Low-rank adapters inside a packed GEMM (gfx950 only): the fp32 sums of a wave's 16x16 blocks start at
// U B_e^T instead of zero, where U[m] = alpha_e A_e X[m] was laid down by the first kernel (lora.hip) and e is
// row m's adapter.
//
// Costs, 4608 x 9216 at K = 3072, ternary, beside lowbit_gemm's 235 us (first product of 13 us included): one adapter of
// rank 32 262 us, three in turn 262, rows of three interleaved 291; of rank 128 352, 368 and 493.
//
// At the start and not at the end: the loads then overlap the tile's first copies, and the sums are
// only written (added to in loops at the end, they took twice their registers and spilled).
#pragma once

#include <type_traits>

#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {

// Smallest of the 16 lanes' values of a lane quarter whose quarters are alike.
__device__ __forceinline__ int min_of_16(int v) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
        const int o = __shfl_xor(v, d);
        v = o < v ? o : v;
    }
    return __builtin_amdgcn_readfirstlane(v);
}

__device__ __forceinline__ uint32_t or_of_16(uint32_t v) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) v |= uint32_t(__shfl_xor(int(v), d));
    return __builtin_amdgcn_readfirstlane(v);
}

__device__ __forceinline__ bool all_finite(u32x4_t v) {
    bool fine = true;
#pragma unroll
    for (int e = 0; e < 4; ++e) fine = fine && (v[e] & 0x7F80u) != 0x7F80u && (v[e] & 0x7F800000u) != 0x7F800000u;
    return fine;
}

// acc[mb][nb], in the layout of 16x16 MFMA results (lane (q, l16): column l16, rows 4q + i), becomes
// the adapters' term of rows row0 + 16 mb .. and output columns col0 + 16 nb ..
//
// U is held as two bf16 halves per number, hi + lo (2^-16 of it is lost), and the product runs over 2 rank
// places, hi then lo, against B's rank columns taken twice: the adapter's term is exact to fp32
// sums of bf16 products, for one more matrix instruction per 16 of rank and block.
//
// Rows of one request (the ordinary case: a wave's rows have one adapter, or none) go straight through.  Mixed rows
// take a turn per adapter, in ascending order, in which rows of others enter as zeros.
//   half: two waves whose sums are added later share the work on mixed rows (0: the first half of the row blocks,
// and all of one request's rows; 1: the second half; -1: a wave by itself).
template <int MB, int NB>
__device__ __forceinline__ void lora_init(f32x4_t (&acc)[MB][NB], const LoraArgs& la, int M, int N, int row0, int col0, int half = -1) {
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

    const int steps = (2 * chunks + 3) / 4;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // One adapter's step ks, the wave's rows all being its own: the products added to the sums.
    // kAhead row blocks' operands in flight at a time: what the sums leave room for
    constexpr int kAhead = 5;
    auto step = [&](__amdgpu_buffer_rsrc_t rs, int ks) __attribute__((always_inline)) {
        bf16x8_t bf[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) bf[nb] = load(rs, b_off(ks), nb * b_block);
        const uint32_t uo = u_off(ks);
#pragma unroll
        for (int m0 = 0; m0 < MB; m0 += kAhead) {
            bf16x8_t uf[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (m0 + j < MB) uf[j] = load(u_rs, uo, (m0 + j) * 16 * int(u_row));
            __builtin_amdgcn_sched_barrier(0);  // or the loads sink to their uses, and each is waited for
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    if (m0 + j < MB)
                        acc[m0 + j][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(uf[j], bf[nb], acc[m0 + j][nb], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr int kHalf = (MB + 1) / 2;
    const int first = __builtin_amdgcn_readfirstlane(id[0]);
    bool one = true;  // rows past the last belong to any request: their operands are zeros, and nothing of them is kept
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) one = one && (id[mb] == first || 16 * mb + l16 >= have);
    if (__all(one)) {  // the ordinary case: one request's rows
        if (first < 0 || half == 1) return;
        const auto rs = b_rsrc(first);
        step(rs, 0);
        if (steps > 1) step(rs, 1);
        if (steps > 2) {
            step(rs, 2);
            step(rs, 3);  // past the rank: zeros
        }
        if (steps > 4) {
            step(rs, 4);
            step(rs, 5);
            step(rs, 6);
            step(rs, 7);
        }
    } else {
        // A turn per adapter.  The rows' U operands are loaded once a step and masked per turn; the adapters of the wave
        // are the bits of a scalar word (64 at a time), and the next turn's part of B is on its way
        // during a turn.  An infinity or a NaN in it makes NaN of the other rows' zeros: it is noticed, and the
        // block-by-block form below, which drops other rows' results, takes over from the start.
        uint32_t odd = 0;
        for (int base = 0;;) {
            int lowest = 0x7FFFFFFF;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) lowest = id[mb] >= base && id[mb] < lowest ? id[mb] : lowest;
            lowest = min_of_16(lowest);
            if (lowest == 0x7FFFFFFF) break;
            base = lowest & ~63;
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                const int d = id[mb] - base;
                lo |= d >= 0 && d < 32 ? 1u << d : 0u;
                hi |= d >= 32 && d < 64 ? 1u << (d - 32) : 0u;
            }
            const uint64_t present = (uint64_t(or_of_16(hi)) << 32) | or_of_16(lo);
#pragma nounroll
            for (int ks = 0; ks < steps; ++ks) {
                const uint32_t uo = u_off(ks), bo = b_off(ks);
                // row blocks in two halves: their operands stay in registers through the turns
#pragma unroll
                for (int m0 = 0; m0 < MB; m0 += kHalf) {
                    if (half >= 0 && half != m0 / kHalf) continue;
                    u32x4_t uf[kHalf];
#pragma unroll
                    for (int j = 0; j < kHalf; ++j)
                        if (m0 + j < MB) uf[j] = __builtin_bit_cast(u32x4_t, load(u_rs, uo, (m0 + j) * 16 * int(u_row)));
                    uint64_t left = present;
                    int cur = base + __builtin_ctzll(left);
                    bf16x8_t bf[NB];
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) bf[nb] = load(b_rsrc(cur), bo, nb * b_block);
#pragma nounroll
                    for (;;) {
                        left &= left - 1;
                        const int next = left != 0 ? base + __builtin_ctzll(left) : cur;
                        bf16x8_t bn[NB];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) bn[nb] = load(b_rsrc(next), bo, nb * b_block);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) odd |= all_finite(__builtin_bit_cast(u32x4_t, bf[nb])) ? 0u : 1u;
#pragma unroll
                        for (int j = 0; j < kHalf; ++j) {
                            if (m0 + j >= MB) continue;
                            u32x4_t mine;
#pragma unroll
                            for (int i = 0; i < 4; ++i) mine[i] = id[m0 + j] == cur ? uf[j][i] : 0u;
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                acc[m0 + j][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, mine), bf[nb],
                                                                                          acc[m0 + j][nb], 0, 0, 0);
                        }
                        if (left == 0) break;
                        cur = next;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) bf[nb] = bn[nb];
                    }
                }
            }
            base += 64;
        }
        if (__any(odd != 0)) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                if (half >= 0 && half != mb / kHalf) continue;
                f32x4_t sum[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) sum[nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                for (int cur = -1;;) {
                    const int next = min_of_16(id[mb] > cur ? id[mb] : 0x7FFFFFFF);  // the block's next adapter
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
    }
}

// The adapters' term of one 16x16 block (rows row0 .., columns col0 .. below N), for the kernels of few rows, where
// each row may well belong to a request of its own.  Mixed rows take a turn each, with the loads of eight
// turns in flight; a turn's product has one row that is not zero, and only that row of the result is
// kept, so requests cannot touch each other.
__device__ __forceinline__ f32x4_t lora_term16(const LoraArgs& la, int M, int N, int row0, int col0) {
    const int lane = int(threadIdx.x) & 63;
    const int q = lane >> 4, l16 = lane & 15;
    const int have = M - row0 < 16 ? M - row0 : 16;
    const int e = l16 < have ? la.rows[row0 + l16] : -1;
    const int id = e >= 0 && e < la.adapters ? e : -1;
    const int chunks = la.rank / 8, steps = (2 * chunks + 3) / 4;
    const uint32_t u_row = uint32_t(la.rank) * 4u;
    const auto u_rs = make_rsrc(la.u + int64_t(row0) * (2 * la.rank), uint32_t(have) * u_row);
    constexpr uint32_t kNone = 0xFFF00000u;  // past every range: reads as zero
    // 16 rows of B of adapter `ad`; none (an empty range) for -1
    auto b_load = [&](int ad, uint32_t off) __attribute__((always_inline)) {
        const auto rs = make_rsrc(la.b + (int64_t(ad < 0 ? 0 : ad) * N + col0) * la.rank, ad < 0 ? 0u : 32u * uint32_t(la.rank));
        return __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
    };
    const int first = __builtin_amdgcn_readfirstlane(id);
    const bool one = __all(id == first || l16 >= have);  // rows past the last belong to any request
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    if (one && first < 0) return sum;
    for (int ks = 0; ks < steps; ++ks) {
        const int c = 4 * ks + q;  // the lane's chunk of the 2 rank places
        const bool in = c < 2 * chunks;
        const u32x4_t uf = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                           u_rs, in && id >= 0 ? uint32_t(l16) * u_row + uint32_t(c) * 16u : kNone, 0, 0));
        const uint32_t b_off = in ? uint32_t(l16 * chunks + (c < chunks ? c : c - chunks)) * 16u : kNone;
        if (one) {
            sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, uf), __builtin_bit_cast(bf16x8_t, b_load(first, b_off)),
                                                          sum, 0, 0, 0);
            continue;
        }
#pragma unroll
        for (int r0 = 0; r0 < 16; r0 += 8) {
            if (r0 >= have) break;
            bf16x8_t bf[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                bf[j] = __builtin_bit_cast(bf16x8_t, b_load(__builtin_amdgcn_readlane(id, r0 + j), b_off));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = r0 + j;
                u32x4_t row;
#pragma unroll
                for (int i = 0; i < 4; ++i) row[i] = l16 == r ? uf[i] : 0u;
                const f32x4_t t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, row), bf[j], f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
                sum[r % 4] += q == r / 4 ? t[r % 4] : 0.f;
            }
        }
    }
    return sum;
}

}  // namespace lowbit
